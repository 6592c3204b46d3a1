// zc_tensor.cuh -- the tensor cores' pieces: matrices read tile by tile through
// tensor maps, block-scaled 8-bit products with sums in tensor memory, waits
// with an end.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "zc_device.cuh"

namespace zc {

// Waits for phase `parity`; false after kWaitLimitNs.  The clock is read only
// where the phase is not complete at once.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done ? true : mbar_wait(bar, parity);
}

// Whether a wait has run out, from a kernel's word of it, which is cleared.
template <class Word>
cudaError_t take_flag(const Word& word, cudaStream_t s, bool* ran_out) {
  const Word zero = 0;
  Word v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, word, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) {
    *ran_out = true;
    e = cudaMemcpyToSymbolAsync(word, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

// ---- pairs of blocks: two blocks of a cluster whose multiprocessors multiply
// together.  The even one leads.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same place of another block's shared memory.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
// Arrives once on a barrier of any block of the cluster.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same without waiting for this thread's earlier stores: for what it has read
// from tensor memory (after tmem_wait_load and tmem_fence_before).
__device__ __forceinline__ void arrive_at_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// As wait_phase, for what blocks of the cluster have arrived on; false after `limit`.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint64_t limit = kWaitLimitNs) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(500000u)
        : "memory");
    if (done) return true;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > limit) return false;
  }
}
// The same for a whole warp, with one answer for its lanes: what follows a wait that
// has run out for some of them only would name lanes that do not come.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit = kWaitLimitNs) {
  return __all_sync(kAll, wait_cluster(bar, parity, limit));
}
// The limit of a wait for `blocks` blocks of a sum: 4 us more for each, ten times what
// one takes at most (one chunk of 900 M rows is 7 M blocks: 2.9 s).
__device__ __forceinline__ uint64_t limit_for(uint32_t blocks) { return kWaitLimitNs + blocks * 4096ull; }

// ---- tensor maps
__device__ __forceinline__ void tma_prefetch(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const void* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// Into this block's memory, announced at a barrier of either block of the pair.
__device__ __forceinline__ void pair_load_2d(void* dst, const void* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* dst, const void* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ---- tensor memory: 128 lanes x 512 columns of 32 bits in each block of a pair;
// both allocate and free
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: a lane's values of 32 consecutive columns.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
        "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]),
        "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(at)
      : "memory");
}

// Arrives once on `bar` of both blocks of the pair when the tensor operations that
// this thread has issued are done.
__device__ __forceinline__ void tensor_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "h"((uint16_t)3)
               : "memory");
}

// 32 columns of 16 lanes, in the order of a matrix instruction's result: of each 8
// columns a lane of the warp has columns 2 (lane % 4) and + 1 of rows lane / 4 and
// lane / 4 + 8.
__device__ __forceinline__ void tmem_load_16x32(uint32_t at, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at)
      : "memory");
}
// Four 8 x 8 matrices of 16-bit values in that order, the other way round: a
// column's 8 values become 16 consecutive bytes.  Lane l has the place of column
// l % 8 of matrix l / 8.
__device__ __forceinline__ void store_turned(uint32_t at, uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(m0), "r"(m1), "r"(m2), "r"(m3) : "memory");
}

// Descriptor of an operand in shared memory: lines of 128 bytes, their 16-byte
// pieces exchanged as a 128-byte swizzled tensor copy leaves them, 8 lines to
// the next 1,024 bytes.  Along the sum: a line holds 128 places of the sum (an
// instruction takes 32, a quarter line further each).  Across it: a line holds
// one place of the sum for the operand's 128 rows (an instruction takes 32 lines).
__device__ __forceinline__ uint64_t operand(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// The same for scales: 512 bytes, plain.
__device__ __forceinline__ uint64_t scale_operand(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | 1ull << 46;
}

// 128 rows' scales into four columns of tensor memory: 32 lanes x 16 bytes, for
// each of the four quarters of its lanes; in each block from its own memory.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t from) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(from) : "memory");
}

// Instruction word of an E4M3 x E4M3 product of 256 x `columns`, E8M0 scales;
// mn_a, mn_b: the operand lies across the sum.
__device__ __forceinline__ uint32_t product_word(uint32_t columns, bool mn_a, bool mn_b) {
  return (uint32_t)mn_a << 15 | (uint32_t)mn_b << 16 | (columns >> 3) << 17 | 1u << 23 | 1u << 28;
}
// The same with byte `i` of the scales' words.
__device__ __forceinline__ uint32_t with_scale(uint32_t word, uint32_t i) { return word | i << 4 | i << 29; }

// 32 places of the sum: tensor memory at d (+)= a x b, in each block its 128 rows of
// a; each has half the rows of b, and the scales of all.
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t word, uint32_t scale_a, uint32_t scale_b,
                                        bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(word), "r"(scale_a), "r"(scale_b), "r"((uint32_t)add)
      : "memory");
}

// ---------------------------------------------------------------- host
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline Encode encoder() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<Encode>(f);
}

// Map of rows of `bytes` bytes, `stride` bytes apart (multiples of 16, as the start
// is), as 64-bit words; a copy takes `words` of `box` rows.
inline bool word_map(CUtensorMap* m, const void* at, uint64_t bytes, uint64_t rows, uint64_t stride, uint32_t words, uint32_t box) {
  const Encode f = encoder();
  const cuuint64_t size[2] = {(bytes + 15) / 16 * 2, rows}, strides[1] = {stride};
  const cuuint32_t boxes[2] = {words, box}, steps[2] = {1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void*>(at), size, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace zc
