// zc_matmul.cu -- products of the experts' chunks with their matrices, operands
// in 8-bit blocks, on the tensor cores.
//
// All three forms are sums over one index of products of codes, times a power of
// two for each 128 places of the index.  The tensor cores take the powers of two
// as they are (one for 32 places of the sum: the same for four instructions), so
// nothing is done between the operands' arrival and the result.
//
// A tile of the result is 256 lanes x up to 256 columns, made by the tensor cores of
// a pair of multiprocessors together: each has 128 of the lanes and loads half of
// the columns' operand, so that a multiprocessor takes 64 bytes from the L2 cache
// for the work of a cycle (alone it would take 96).  The lanes are the matrices'
// rows (outer or inner places), the columns the chunk's rows: a chunk may have any
// number of rows, and the columns of an instruction may be any multiple of 32, so
// that a chunk's end costs at most 31 columns, where the lanes are always full.  In
// the gradient of the weights lanes are the inner places, columns the outer ones, and
// the chunk's rows are summed over.  The result thus lies with its contiguous index
// along the lanes.
//
// Two tiles have room in tensor memory beside the scales but for 32 columns: the
// next tile's first 32 columns are the last 32 of a full one, which are read
// first.
//
// The weights are read along the sum forward and across it backward, from the
// same codes: blocks of 128 x 128 serve both.
//
// Measured: 8,192 rows with one matrix of 14,336 x 4,096, 322 us forward and by
// the rows, 349 by the weights: 2,750 to 2,990 TFLOP/s, where instructions alone run at
// 4,780.  32,768 rows in 64 chunks with matrices of 2,048 x 4,096: 227, 243 and 361;
// the last writes 1.07 GB, which at the rate of writes alone (4,050 GB/s) takes 265.
// Few rows (122 with the same 64): 87 us, 6,100 GB/s of the weights' bytes.
//
// Warps: 0 loads tiles through tensor maps, six stages of 128 places ahead; 1 (of
// the leading block) issues the products; 2 lays the scales out (128 rows x 4
// bytes, four blocks of the sum a time); 3 clears what a chunk's last block of rows
// reads of the next chunk (gradient of the weights); 4 to 11 write results.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "zc_fp8.cuh"
#include "zc_tensor.cuh"
#include "zipccl.h"

namespace zc {

cudaError_t layer_up_waits(cudaStream_t s, bool* ran_out);    // zc_layer_up.cu
cudaError_t layer_down_waits(cudaStream_t s, bool* ran_out);  // zc_layer_down.cu

namespace {

constexpr int kWriters = 8, kThreads = (4 + kWriters) * 32;
constexpr uint32_t kLanes = 256, kOwnLanes = 128;                   // of a tile, and those of a block
constexpr uint32_t kColumns = 256, kOwnColumns = 128, kPlaces = 128;  // columns; places of the sum in a stage
constexpr uint32_t kStages = 6;
constexpr uint32_t kBytesA = kOwnLanes * kPlaces, kBytesB = kOwnColumns * kPlaces, kStageBytes = kBytesA + kBytesB;
constexpr uint32_t kScaleSets = 4, kScaleBytes = 512 * 3;  // four blocks' scales: 128 lanes, 256 columns
// Copies of 16, 32, 64 and 128 rows: as many as half a tile's columns need (with 16 rows
// alone 8,192 rows with 14,336 x 4,096 take 377 us in place of 323, 32,768 with 64
// matrices of 2,048 x 4,096 252 in place of 227).
constexpr uint32_t kBoxRows = 16, kBoxes = 4;
// Tensor memory: sums from columns 0 and 224 on, scales behind them, 16 columns for each of two sets.
constexpr uint32_t kSecond = 224, kScaleColumns = kSecond + kColumns;

__device__ unsigned int g_wait_ran_out;

struct MatmulArgs {
  CUtensorMap a, b[kBoxes];  // (WEIGHTS: b[0] alone)
  const uint8_t *scales_a, *scales_b;
  const int32_t* offsets;
  void* out;
  uint64_t out_stride, out_matrix;       // values between rows and matrices
  uint64_t a_matrix;                     // scales of a matrix of weights
  uint32_t a_lane, a_block;              // bytes from a lane block's scale to the next, from a block of the sum's to the next
  uint32_t lanes, columns, sum;          // of the result and the sum (WEIGHTS: columns; sum unused; else columns unused)
  uint32_t rows, chunks, lane_tiles, column_tiles;
  uint32_t b_blocks;                     // scales of a row
  bool wide;                             // rows of the result start at multiples of 16 bytes
  bool whole_words;                      // scales of a row: whole words of four
};

struct Shared {
  alignas(1024) uint8_t stage[kStages][kStageBytes];
  alignas(128) uint8_t scales[kScaleSets][kScaleBytes];
  alignas(16) uint8_t turned[kWriters][32 * 64];  // 16-bit results of a writing warp, the other way round
  uint64_t full[kStages], empty[kStages], scales_full[kScaleSets], scales_empty[kScaleSets];
  uint64_t ends[kStages], clear[kStages], cleared[kStages];  // a stage with a chunk's last block (gradient of the weights)
  uint64_t done[2], shared_taken[2], taken[2];
  uint32_t tmem;
  uint32_t first[kMaxChunks + 2];  // first row of each chunk; the rows behind the last are one more
  uint32_t tiles[kMaxChunks + 2];  // tiles of rows before each (WEIGHTS: blocks of the scales)
};

struct Tile {
  uint32_t chunk, row, count;   // rows of the tile (WEIGHTS: of the chunk)
  uint32_t lane0, column0, columns, width, blocks;  // lane0: of this block; width: columns of the instructions
};

template <bool kWeights>
__device__ __forceinline__ Tile tile_of(const MatmulArgs& a, const Shared& s, uint32_t t, uint32_t rank) {
  Tile x;
  if constexpr (kWeights) {
    const uint32_t per = a.lane_tiles * a.column_tiles;
    x.chunk = t / per;
    t -= x.chunk * per;
    x.column0 = t / a.lane_tiles * kColumns;
    x.lane0 = t % a.lane_tiles * kLanes;
    x.row = s.first[x.chunk];
    x.count = s.first[x.chunk + 1] - x.row;
    x.columns = min(kColumns, a.columns - x.column0);
    x.blocks = (x.count + kPlaces - 1) / kPlaces;
  } else {
    const uint32_t r = t / a.lane_tiles;
    x.lane0 = (t - r * a.lane_tiles) * kLanes;
    uint32_t lo = 0, hi = a.chunks + 1;  // the chunk whose tiles begin at r or before, the next one's behind it
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (s.tiles[mid] <= r) lo = mid;
      else hi = mid;
    }
    x.chunk = lo;
    const uint32_t all = s.first[lo + 1] - s.first[lo], n = s.tiles[lo + 1] - s.tiles[lo];
    const uint32_t step = ((all + n - 1) / n + 31) / 32 * 32, from = (r - s.tiles[lo]) * step;
    x.row = s.first[lo] + from;
    x.count = from < all ? min(step, all - from) : 0;
    x.column0 = 0;
    x.columns = x.count;
    x.blocks = lo < a.chunks && x.count ? (a.sum + kPlaces - 1) / kPlaces : 0;
  }
  x.lane0 += rank * kOwnLanes;
  x.width = (x.columns + 31) / 32 * 32;
  return x;
}

template <class T>
__device__ __forceinline__ uint32_t pair_of(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Results of 16 bits: 32 columns of a warp's 32 lanes go to shared memory the other
// way round (four instructions; value by value it took 32, and the writing warps
// held the gradient of the weights at twice its time) and from there in 16 bytes a
// lane, 64 consecutive ones of a column: from column c of `count` to out + column *
// stride.  The pieces of a column lie at other places in every second line, so
// that neither access meets itself in a bank.
template <class T>
__device__ __forceinline__ void turn_columns(const uint32_t (&v)[2][16], uint8_t* turned) {
  const uint32_t lane = threadIdx.x % 32, matrix = lane / 8, base = smem_addr(turned);
#pragma unroll
  for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
    for (uint32_t q = 0; q < 2; ++q) {
      const uint32_t line = (2 * q + matrix / 2) * 8 + lane % 8, piece = (2 * h + matrix % 2) ^ (line / 2 % 4);
      const uint32_t(&x)[16] = v[h];
      store_turned(base + line * 64 + piece * 16, pair_of<T>(x[8 * q], x[8 * q + 1]), pair_of<T>(x[8 * q + 2], x[8 * q + 3]),
                   pair_of<T>(x[8 * q + 4], x[8 * q + 5]), pair_of<T>(x[8 * q + 6], x[8 * q + 7]));
    }
  __syncwarp();
}
template <class T>
__device__ __forceinline__ void write_turned(const uint8_t* turned, T* out, uint64_t stride, uint32_t c, uint32_t count) {
  const uint32_t lane = threadIdx.x % 32;
#pragma unroll
  for (uint32_t i = 0; i < 32; i += 8) {
    const uint32_t line = i + lane / 4, piece = lane % 4 ^ (line / 2 % 4);
    const uint4 q = *reinterpret_cast<const uint4*>(turned + line * 64 + piece * 16);
    if (c + line < count) *reinterpret_cast<uint4*>(out + (c + line) * stride + lane % 4 * 8) = q;
  }
  __syncwarp();
}

// Scales of four blocks of the sum from k0 on, as tensor memory takes them: word j
// of a lane is row 32 j + lane of the 128 lanes, then of the 256 columns, a byte for
// each of the blocks.  What lies outside is read from inside: its rows are zeros or
// not written, and no load hangs on a condition, which would make each wait for
// the one before it (one set took 4,800 cycles so, the products of its blocks 2,048).
template <bool kWeights>
__device__ __forceinline__ void read_scales(const MatmulArgs& a, const Shared& s, const Tile& x, uint32_t k0, uint32_t (&w)[12]) {
  const uint32_t lane = threadIdx.x % 32, last = x.blocks - 1;
  if constexpr (kWeights) {
    const uint64_t block = s.tiles[x.chunk];
#pragma unroll
    for (int j = 0; j < 12; ++j) {
      const uint32_t wide = j < 4 ? a.lanes : a.columns;
      const uint32_t at = min(j < 4 ? x.lane0 + 32 * j + lane : x.column0 + 32 * (j - 4) + lane, wide - 1);
      const uint8_t* p = (j < 4 ? a.scales_a : a.scales_b) + block * wide + at;
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __ldg(p + (uint64_t)min(k0 + i, last) * wide);
      w[j] = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    }
  } else {
    // a matrix's block of 128 x 128 has one scale for all lanes
    const uint8_t* p = a.scales_a + x.chunk * a.a_matrix + (uint64_t)(min(x.lane0, a.lanes - 1) / kOwnLanes) * a.a_lane;
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __ldg(p + (uint64_t)min(k0 + i, last) * a.a_block);
    w[0] = w[1] = w[2] = w[3] = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* q = a.scales_b + (uint64_t)(x.row + min(32 * j + lane, x.count - 1)) * a.b_blocks;
      if (a.whole_words) {
        w[4 + j] = __ldg(reinterpret_cast<const unsigned int*>(q + k0));
      } else {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __ldg(q + min(k0 + i, last));
        w[4 + j] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
      }
    }
  }
}

template <class T, int kForm>
__global__ void __launch_bounds__(kThreads, 1) zc_matmul_kernel(const __grid_constant__ MatmulArgs a) {
  constexpr bool kWeights = kForm == ZIPCCL_MATMUL_WEIGHTS;
  constexpr bool kAcrossA = kForm != ZIPCCL_MATMUL_FORWARD, kAcrossB = kWeights;
  extern __shared__ uint8_t s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw + ((1024 - (smem_addr(s_raw) & 1023)) & 1023));
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, rank = cluster_rank();
  const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (threadIdx.x == 0) {
    tma_prefetch(&a.a);
    for (uint32_t i = 0; i < (kWeights ? 1 : kBoxes); ++i) tma_prefetch(&a.b[i]);
    for (uint32_t i = 0; i < kStages; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (uint32_t i = 0; i < kScaleSets; ++i) mbar_init(&s.scales_full[i], 2), mbar_init(&s.scales_empty[i], 1);
    for (uint32_t i = 0; i < kStages; ++i) mbar_init(&s.ends[i], 1), mbar_init(&s.clear[i], 1), mbar_init(&s.cleared[i], 2);
    for (uint32_t i = 0; i < 2; ++i) mbar_init(&s.done[i], 1), mbar_init(&s.shared_taken[i], 2 * kWriters), mbar_init(&s.taken[i], 2 * kWriters);
  }
  if (warp == 1) tmem_alloc(&s.tmem, 512);
  after_previous();
  // the chunks' rows and their tiles
  for (uint32_t i = threadIdx.x; i < a.chunks; i += kThreads)
    s.tiles[i] = a.offsets ? (uint32_t)min(max(a.offsets[i + 1], 0), (int32_t)a.rows) : a.rows;
  __syncthreads();
  if (warp == 0) {
    uint32_t end = 0, tiles = 0;
    for (uint32_t e0 = 0; e0 <= a.chunks; e0 += 32) {  // one more than the chunks: the rows behind them
      const uint32_t e = e0 + lane;
      uint32_t top = max(e < a.chunks ? s.tiles[e] : e == a.chunks ? a.rows : 0u, end);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, top, d);
        if (lane >= d) top = max(top, y);
      }
      uint32_t first = __shfl_up_sync(kAll, top, 1);
      if (lane == 0) first = end;
      const uint32_t per = kWeights ? kPlaces : kColumns;
      const uint32_t n = (top - first + per - 1) / per, upto = tiles + warp_inclusive_sum(n);
      __syncwarp();
      if (e <= a.chunks) {
        s.first[e] = first;
        s.tiles[e] = upto - n;
        if (e == a.chunks) s.first[e + 1] = top, s.tiles[e + 1] = upto;
      }
      __syncwarp();
      end = __shfl_sync(kAll, top, 31);
      tiles = __shfl_sync(kAll, upto, 31);
    }
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers and tensor memory are there
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  const uint32_t total = kWeights ? a.chunks * a.lane_tiles * a.column_tiles : s.tiles[a.chunks + 1] * a.lane_tiles;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t n = 0;  // stages filled
      for (uint32_t t = pair; t < total && ok; t += pairs) {
        const Tile x = tile_of<kWeights>(a, s, t, rank);
        const uint32_t half = x.width / 2, column0 = x.column0 + rank * half;
        const uint32_t bytes = kBytesA + (kWeights ? kBytesB : half * kPlaces);
        for (uint32_t k = 0; k < x.blocks; ++k, ++n) {
          const uint32_t st = n % kStages;
          if (!(ok = wait_cluster(&s.empty[st], (n / kStages & 1) ^ 1))) break;
          uint8_t* to = s.stage[st];
          if (rank == 0) mbar_arrive_expect_tx(&s.full[st], 2 * bytes);
          const uint32_t full = at_rank(&s.full[st], 0);
          const int32_t at = (int32_t)(k * kPlaces);
          if constexpr (kForm == ZIPCCL_MATMUL_FORWARD) pair_load_3d(to, &a.a, at, x.lane0, x.chunk, full);
          else if constexpr (kForm == ZIPCCL_MATMUL_BACKWARD) pair_load_3d(to, &a.a, x.lane0, at, x.chunk, full);
          else pair_load_3d(to, &a.a, x.lane0, x.row + at, 0, full);
          to += kBytesA;
          if constexpr (kWeights) {
            pair_load_2d(to, &a.b[0], column0, x.row + at, full);
            if (rank == 0 && k + 1 == x.blocks && x.count % 32) mbar_arrive(&s.ends[st]);
          } else {
            uint32_t r = 0;
#pragma unroll
            for (int i = kBoxes - 1; i >= 0; --i)
              if (half & kBoxRows << i) {
                pair_load_2d(to + r * kPlaces, &a.b[i], at, x.row + rank * half + r, full);
                r += kBoxRows << i;
              }
          }
        }
      }
      // a block that gives up does not end under copies: the leading one waits for both
      for (uint32_t i = n > kStages ? n - kStages : 0; rank == 0 && !ok && i < n; ++i) wait_cluster(&s.full[i % kStages], i / kStages & 1);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t n = 0, sets = 0, tiles = 0, columns = 0, cleared = 0;  // cleared: a parity for each stage
      for (uint32_t t = pair; t < total && ok; t += pairs) {
        const Tile x = tile_of<kWeights>(a, s, t, rank);
        if (x.blocks == 0) continue;
        const uint32_t buffer = tiles & 1, turn = tiles >> 1;
        if (!(ok = wait_cluster(&s.taken[buffer], (turn & 1) ^ 1))) break;
        // columns that the tile before has in the way
        if (tiles && (buffer ? columns : x.columns) > kSecond &&
            !(ok = wait_cluster(&s.shared_taken[buffer ^ 1], ((tiles - 1) >> 1) & 1)))
          break;
        columns = x.columns;
        tmem_fence_after();
        const uint32_t sums = tmem + buffer * kSecond, word = product_word(x.width, kAcrossA, kAcrossB);
        uint32_t scales = 0;
        for (uint32_t k = 0; k < x.blocks; ++k, ++n) {
          const uint32_t st = n % kStages;
          if (k % 4 == 0) {
            const uint32_t set = sets % kScaleSets;
            if (!(ok = wait_cluster(&s.scales_full[set], sets / kScaleSets & 1))) break;
            tmem_fence_after();
            scales = tmem + kScaleColumns + sets % 2 * 16;
            const uint32_t from = smem_addr(s.scales[set]);
            copy_scales(scales, scale_operand(from));
            copy_scales(scales + 4, scale_operand(from + 512));
            if (x.columns > 128) copy_scales(scales + 8, scale_operand(from + 1024));
            tensor_commit(&s.scales_empty[set]);
            ++sets;
          }
          if (!(ok = wait_cluster(&s.full[st], n / kStages & 1))) break;
          uint32_t steps = 4;
          if (kWeights && k + 1 == x.blocks && x.count % kPlaces) {
            steps = (x.count % kPlaces + 31) / 32;
            if (x.count % 32) {
              if (!(ok = wait_cluster(&s.cleared[st], cleared >> st & 1))) break;
              cleared ^= 1u << st;
            }
          }
          tmem_fence_after();
          const uint32_t at = smem_addr(s.stage[st]);
          for (uint32_t i = 0; i < steps; ++i)
            product(sums, operand(at + i * (kAcrossA ? 4096 : 32)), operand(at + kBytesA + i * (kAcrossB ? 4096 : 32)),
                    with_scale(word, k % 4), scales, scales + 4, k + i > 0);
          tensor_commit(&s.empty[st]);
        }
        if (!ok) break;
        tensor_commit(&s.done[buffer]);
        ++tiles;
      }
    }
  } else if (warp == 2) {
    // a set is read while the one before it waits for its place
    uint32_t sets = 0, t = pair, k0 = 0;
    Tile x;
    const auto next_tile = [&] {  // the next one with a sum, from t on
      for (; t < total; t += pairs) {
        x = tile_of<kWeights>(a, s, t, rank);
        if (x.blocks) return;
      }
    };
    uint32_t w[12], later[12];
    next_tile();
    if (t < total) read_scales<kWeights>(a, s, x, k0, later);
    while (t < total) {
#pragma unroll
      for (int j = 0; j < 12; ++j) w[j] = later[j];
      if ((k0 += 4) >= x.blocks) {
        k0 = 0;
        t += pairs;
        next_tile();
      }
      if (t < total) read_scales<kWeights>(a, s, x, k0, later);
      const uint32_t set = sets % kScaleSets;
      if (!(ok = warp_wait(&s.scales_empty[set], (sets / kScaleSets & 1) ^ 1))) break;
      uint4* to = reinterpret_cast<uint4*>(s.scales[set]) + lane;
#pragma unroll
      for (int j = 0; j < 3; ++j) to[32 * j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_at(at_rank(&s.scales_full[set], 0));
      ++sets;
    }
  } else if (warp == 3) {
    if constexpr (kWeights) {
      // The leading block's loading thread says that a chunk's last block is on its way
      // (so that the barrier of its stage is at that turn), this warp of the leading
      // block sees it arrive and tells the other's; both clear their half, before the
      // products come to it.
      uint32_t n = 0, before = 0, parity = 0;  // before: blocks up to the last wait; parity: a bit for each stage
      for (uint32_t t = pair; t < total && ok; t += pairs) {
        const Tile x = tile_of<kWeights>(a, s, t, rank);
        n += x.blocks;
        if (x.count % 32 == 0) continue;
        const uint32_t st = (n - 1) % kStages, from = x.count % kPlaces, upto = (from + 31) / 32 * 32;
        const uint64_t limit = limit_for(n - before);
        before = n;
        if (rank == 0) {
          if (!(ok = warp_wait(&s.ends[st], parity >> st & 1, limit)) || !(ok = warp_wait(&s.full[st], (n - 1) / kStages & 1))) break;
          if (lane == 0) arrive_at(at_rank(&s.clear[st], 1));
        } else if (!(ok = warp_wait(&s.clear[st], parity >> st & 1, limit))) {
          break;
        }
        parity ^= 1u << st;
        for (uint32_t i = from * 8 + lane; i < upto * 8; i += 32)
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
            reinterpret_cast<uint4*>(s.stage[st] + piece * kBytesA)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_at(at_rank(&s.cleared[st], 0));
      }
    }
  } else {
    // two warps for each quarter of the lanes, every other 32 columns each.  Columns
    // that the next tile's sums will lie in come first: in the first buffer the last
    // 32 of a full tile, in the second the first 32.
    const uint32_t quarter = warp % 4, other = (warp - 4) / 4;
    uint32_t tiles = 0;
    for (uint32_t t = pair; t < total && ok; t += pairs) {
      const Tile x = tile_of<kWeights>(a, s, t, rank);
      const uint32_t place = x.lane0 + quarter * 32, lanes = place < a.lanes ? a.lanes - place : 0;
      const uint32_t buffer = tiles & 1, sums = tmem + buffer * kSecond + (quarter << 21);
      T* out = static_cast<T*>(a.out) + place;
      if constexpr (kWeights) out += x.chunk * a.out_matrix + x.column0 * a.out_stride;
      else out += x.row * a.out_stride;
      if (x.blocks) {
        if (!(ok = warp_wait(&s.done[buffer], (tiles >> 1) & 1, limit_for(x.blocks)))) break;
        tmem_fence_after();
      }
      const uint32_t parts = x.width / 32;
      // (backwards in the first buffer)
      for (uint32_t i = other; i < parts + other; i += 2) {
        const bool mine = i < parts;
        const uint32_t c = (buffer ? i : parts - 1 - i) * 32;
        const auto given_back = [&] {  // tensor memory, before the results are written
          tmem_fence_before();
          __syncwarp();
          if (lane == 0 && i == other) arrive_at_relaxed(at_rank(&s.shared_taken[buffer], 0));
          if (lane == 0 && i + 2 >= parts + other) arrive_at_relaxed(at_rank(&s.taken[buffer], 0));
        };
        if (sizeof(T) == 2 && a.wide && lanes >= 32 && x.blocks) {
          if constexpr (sizeof(T) == 2) {
            uint32_t v[2][16];
            if (mine) {
              tmem_load_16x32(sums + c, v[0]);
              tmem_load_16x32(sums + (16u << 16) + c, v[1]);
              tmem_wait_load();
            }
            given_back();
            if (mine) {
              turn_columns<T>(v, s.turned[warp - 4]);
              write_turned<T>(s.turned[warp - 4], out, a.out_stride, c, x.columns);
            }
          }
        } else {
          uint32_t v[32];
          if (mine && x.blocks) {
            tmem_load32(sums + c, v);
            tmem_wait_load();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0;
          }
          if (x.blocks) given_back();
          if (mine && lane < lanes) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < x.columns) out[(c + j) * a.out_stride + lane] = from_float<T>(__uint_as_float(v[j]));
          }
        }
      }
      tiles += x.blocks != 0;
    }
  }
  if (!ok) atomicOr(&g_wait_ran_out, 1u);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
// Map of codes [matrices][rows][cols]; a copy takes 128 bytes of `box` rows.  Rows
// and columns beyond the matrix read as zeros.
bool code_map(CUtensorMap* m, const zipccl_fp8_blocks* x, uint64_t cols, uint64_t rows, uint64_t matrices, uint32_t dims,
              uint32_t box) {
  const Encode f = encoder();
  const cuuint64_t size[3] = {cols, rows, matrices}, strides[2] = {x->stride, x->stride * rows};
  const cuuint32_t boxes[3] = {kPlaces, box, 1}, steps[3] = {1, 1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<uint8_t*>(x->d_codes), size, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmem = sizeof(Shared) + 1024;

template <class T, int kForm>
cudaError_t matmul_launch(const MatmulArgs& a, uint64_t tiles, cudaStream_t s) {
  static std::atomic<int> multiprocessors[kMaxDevices];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!(sms = multiprocessors[dev].load(std::memory_order_acquire))) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(zc_matmul_kernel<T, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem)) != cudaSuccess)
      return e;
    multiprocessors[dev].store(sms, std::memory_order_release);
  }
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = 2 * (uint32_t)std::min<uint64_t>(tiles, sms / 2), cfg.blockDim = kThreads, cfg.dynamicSmemBytes = kSmem, cfg.stream = s;
  cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, zc_matmul_kernel<T, kForm>, a);
}

template <class T>
cudaError_t matmul_by_form(const MatmulArgs& a, int form, uint64_t tiles, cudaStream_t s) {
  return form == ZIPCCL_MATMUL_FORWARD    ? matmul_launch<T, ZIPCCL_MATMUL_FORWARD>(a, tiles, s)
         : form == ZIPCCL_MATMUL_BACKWARD ? matmul_launch<T, ZIPCCL_MATMUL_BACKWARD>(a, tiles, s)
                                          : matmul_launch<T, ZIPCCL_MATMUL_WEIGHTS>(a, tiles, s);
}

bool good(const zipccl_fp8_blocks* x, uint64_t cols) {
  return x->d_codes && x->d_scales && host_aligned(x->d_codes, 16) && x->stride >= cols && x->stride % 16 == 0 && x->stride < (1ull << 38);
}

}  // namespace
}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_matmul(int form, const zipccl_fp8_blocks* a, const zipccl_fp8_blocks* b, uint64_t rows,
                                uint64_t inner, uint64_t outer, const int32_t* d_offsets, uint32_t experts, void* d_out,
                                int out_type, uint64_t out_stride, void* stream) {
  const uint64_t z = type_bytes(out_type), kMaxCols = 1ull << 22;
  const bool weights = form == ZIPCCL_MATMUL_WEIGHTS;
  if (form < ZIPCCL_MATMUL_FORWARD || form > ZIPCCL_MATMUL_WEIGHTS || z == 0 || !a || !b) return ZIPCCL_ERR_INVALID_ARG;
  if (rows >= (1ull << 31) || inner == 0 || outer == 0 || inner > kMaxCols || outer > kMaxCols || experts == 0 ||
      experts > kMaxChunks || (!d_offsets && experts != 1) || !host_aligned(d_offsets, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  const uint64_t out_cols = form == ZIPCCL_MATMUL_FORWARD ? outer : inner;
  if (out_stride < out_cols || out_stride >= (1ull << 32)) return ZIPCCL_ERR_INVALID_ARG;
  if (rows == 0 && !weights) return ZIPCCL_OK;
  if (!d_out || !host_aligned(d_out, z)) return ZIPCCL_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0)
    return cudaMemset2DAsync(d_out, out_stride * z, 0, inner * z, (size_t)experts * outer, s) == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
  if (!good(a, form == ZIPCCL_MATMUL_FORWARD ? inner : outer) || !good(b, inner)) return ZIPCCL_ERR_INVALID_ARG;
  MatmulArgs m{};
  m.offsets = d_offsets;
  m.out = d_out;
  m.out_stride = out_stride;
  m.out_matrix = out_stride * outer;
  m.rows = (uint32_t)rows;
  m.chunks = experts;
  m.lanes = (uint32_t)out_cols;
  m.lane_tiles = (m.lanes + kLanes - 1) / kLanes;
  m.wide = host_aligned(d_out, 16) && out_stride * z % 16 == 0;
  uint64_t tiles;
  bool mapped;
  if (weights) {
    m.scales_a = b->d_scales;
    m.scales_b = a->d_scales;
    m.columns = (uint32_t)outer;
    m.column_tiles = (m.columns + kColumns - 1) / kColumns;
    mapped = code_map(&m.a, b, inner, rows, 1, 3, kPlaces) && code_map(&m.b[0], a, outer, rows, 1, 2, kPlaces);
    tiles = (uint64_t)experts * m.lane_tiles * m.column_tiles;
  } else {
    const uint32_t high = (uint32_t)((outer + kFp8Block - 1) / kFp8Block), wide = (uint32_t)((inner + kFp8Block - 1) / kFp8Block);
    const bool forward = form == ZIPCCL_MATMUL_FORWARD;
    m.scales_a = b->d_scales;
    m.scales_b = a->d_scales;
    m.a_matrix = (uint64_t)high * wide;
    m.a_lane = forward ? wide : 1;
    m.a_block = forward ? 1 : wide;
    m.sum = (uint32_t)(forward ? inner : outer);
    m.b_blocks = forward ? wide : high;
    m.whole_words = m.b_blocks % 4 == 0 && host_aligned(a->d_scales, 4);
    mapped = code_map(&m.a, b, inner, outer, experts, 3, kOwnLanes);
    for (uint32_t i = 0; i < kBoxes; ++i) mapped = mapped && code_map(&m.b[i], a, m.sum, rows, 1, 2, kBoxRows << i);
    tiles = (rows / kColumns + experts + 1) * m.lane_tiles;  // at most
  }
  if (!mapped) return ZIPCCL_ERR_CUDA;
  if (tiles >= (1ull << 32)) return ZIPCCL_ERR_INVALID_ARG;
  const cudaError_t e = out_type == ZIPCCL_TYPE_F32    ? matmul_by_form<float>(m, form, tiles, s)
                        : out_type == ZIPCCL_TYPE_BF16 ? matmul_by_form<__nv_bfloat16>(m, form, tiles, s)
                                                       : matmul_by_form<__half>(m, form, tiles, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

zipccl_status zipccl_moe_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool ran_out = false;
  if (take_flag(g_wait_ran_out, s, &ran_out) != cudaSuccess || layer_up_waits(s, &ran_out) != cudaSuccess ||
      layer_down_waits(s, &ran_out) != cudaSuccess) return ZIPCCL_ERR_CUDA;
  return ran_out ? ZIPCCL_ERR_TIMEOUT : ZIPCCL_OK;
}

}  // extern "C"
