// zc_layer.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   logits = router x;  weights, ids = choice of experts (zc_route.cuh)
//   h = weight * act(gate x) * (up x)  for each token and expert of it   (first kernel)
//   y = residual + sum over a token's experts of down h                  (second kernel)
//
// Such a layer reads every chosen expert's matrices once and is bound by that: a
// token of two experts of 3 x 4,096 x 14,336 bfloat16 values reads 705 MB for 0.7
// GFLOP.  The tokens are the narrow side: a warp takes 16 rows of a matrix and
// up to 8 of the expert's tokens to a tensor instruction (m16n8k8, both operands
// as 32-bit floats of which the top 19 bits count), which costs no more than one
// token and less than their sums in ordinary instructions.  16-bit and 8-bit
// values are exact in 19 bits; a 32-bit one is the sum of two such parts (21 bits
// at least), and of products of parts only the two least ones' is left out.
//
// Everything that depends on where a place of the sum lies in an instruction is
// the same for both operands, so a lane reads 16 consecutive bytes of a row and
// hands them to the instructions in its own order.
//
// Rows that start at multiples of 16 bytes come through shared memory in pieces of
// 2,048 bytes of 16 rows, two or three stages ahead; 8 warps take 128 bytes of each
// row at a time, and in turn fill a stage again that all have left.  Others are read
// value by value.  The tokens' own values come from global memory, a chunk ahead.
//
// The choice of experts is made by every cluster of 8 blocks for itself: each block
// takes an eighth of the hidden places for all experts and tokens, the partial
// logits are summed over the cluster's shared memory in one order, and each block
// chooses for its share of the tokens.  A separate kernel would cost a launch, a
// grid-wide wait about the same.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "zc_fp8.cuh"
#include "zc_route.cuh"
#include "zc_tensor.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr uint32_t kCluster = 8, kMaxTokens = ZIPCCL_LAYER_MAX_TOKENS;
constexpr uint32_t kPiece = 2048, kChunk = 128;  // bytes of a row in a stage, and those that a warp takes at a time
constexpr uint32_t kChunks = kPiece / kChunk / kWarps;  // of a warp in a stage
constexpr uint32_t kStageBytes = 16 * kPiece;
// stages of a block: what two blocks of a multiprocessor have room for
template <int G>
constexpr uint32_t kStagesOf = G == 1 ? 3 : 2;
constexpr uint32_t kMaxStages = 3;

__device__ unsigned int g_layer_wait_ran_out;

struct LayerArgs {
  CUtensorMap up_map, down_map;  // 8 rows x 256 words of 8 bytes
  const void *x, *router, *up, *down, *residual;
  const uint8_t *up_scales, *down_scales;
  void* y;
  float* weights;
  int32_t* ids;
  void* h;  // parts of each pair's inner places, rows of h_stride values
  uint64_t x_stride, up_stride, down_stride, h_stride;  // in values
  uint32_t tokens, hidden, inner, experts, top_k;
  int activation;
  bool gated, router_float, wide_x, wide_router, wide_up, wide_down;
  RouteArgs route;
};

__device__ __forceinline__ float load_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ---- values
struct F8 {
  uint8_t bits;
};
template <class W>
constexpr int kPer16 = 16 / sizeof(W);

// 16 bytes of values from p on, `left` of which are the row's; zeros behind them.
template <class W>
__device__ __forceinline__ uint4 load16(const W* p, int left, bool wide) {
  constexpr int V = kPer16<W>;
  if (left >= V && wide) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i >= left) continue;
    if constexpr (sizeof(W) == 4) w[i] = __ldg(reinterpret_cast<const unsigned int*>(p) + i);
    else if constexpr (sizeof(W) == 2) w[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i % 2));
    else w[i / 4] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(p) + i) << (8 * (i % 4));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Values 2 j and 2 j + 1 of 16 bytes, exact.
template <class W>
__device__ __forceinline__ float2 two_of(const uint4& q, int j) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(W) == 4) return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  else if constexpr (std::is_same<W, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  else if constexpr (std::is_same<W, __half>::value)
    return make_float2(__half2float(__ushort_as_half((unsigned short)w[j])), __half2float(__ushort_as_half((unsigned short)(w[j] >> 16))));
  else {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j % 2))), __NV_E4M3);
    return make_float2(__half2float(__ushort_as_half(h.x)), __half2float(__ushort_as_half(h.y)));
  }
}

// A float as two of 11 bits: the nearest (or, where that is out of range, the top
// bits), and the nearest to what it leaves; infinity and NaN leave nothing.
__device__ __forceinline__ void parts(float v, float& hi, float& lo) {
  const uint32_t b = __float_as_uint(v), m = b & 0x7FFFFFFFu;
  if (m >= 0x7F800000u) {
    hi = v, lo = 0.0f;
    if (m > 0x7F800000u) hi = __uint_as_float(0x7FC00000u);  // NaN stays NaN without its low bits
  } else {
    hi = __uint_as_float((m < 0x7F7FF000u ? b + 0x1000u : b) & 0xFFFFE000u);
    lo = __uint_as_float(__float_as_uint(v - hi) + 0x1000u);  // (the instruction drops the low 13 bits)
  }
}

__device__ __forceinline__ void multiply(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// 2^e of a scale's byte (255: NaN).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// The same of 16-bit values, in pairs: m16n8k16.
template <class T>
__device__ __forceinline__ void multiply16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Places of the sum that a warp takes in a step (4 lanes, 16 bytes of weights
// each), in a chunk (two steps) and in a piece.
template <class W>
constexpr uint32_t kStep = 4 * kPer16<W>;
template <class W>
constexpr uint32_t kPlacesOfChunk = kChunk / sizeof(W);
template <class W>
constexpr uint32_t kPlacesOfPiece = kPiece / sizeof(W);

// Zeros behind the first `left` of 16 bytes of values.
template <class W>
__device__ __forceinline__ uint4 keep(uint4 q, int left) {
  if (left >= kPer16<W>) return q;
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bytes = left * (int)sizeof(W) - 4 * i;
    if (bytes <= 0) w[i] = 0;
    else if (bytes < 4) w[i] &= (1u << (8 * bytes)) - 1;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// h as the second kernel takes it, each part in an array of its own: with bfloat16
// weights three bfloat16 values (24 bits), with others two floats of 11 bits.
struct ThreeParts {
  using Value = __nv_bfloat16;
  static constexpr int kParts = 3;
};
struct TwoParts {
  using Value = float;
  static constexpr int kParts = 2;
};
template <class W>
using PartsFor = std::conditional_t<std::is_same<W, __nv_bfloat16>::value, ThreeParts, TwoParts>;
template <class X>
struct PartsOf {  // of a plain vector: itself
  using Value = X;
  static constexpr int kParts = 1;
};
template <>
struct PartsOf<ThreeParts> : ThreeParts {};
template <>
struct PartsOf<TwoParts> : TwoParts {};

__device__ __forceinline__ float bf16_part(float v) {
  float p = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(p) && !isinf(v)) p = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return p;
}
// Writes the parts of v to at[0], at[apart], ...
__device__ __forceinline__ void store_parts(__nv_bfloat16* at, uint64_t apart, float v) {
  const float p = bf16_part(v), r = isfinite(v) ? v - p : 0.0f, q = bf16_part(r);
  at[0] = __float2bfloat16_rn(p);
  at[apart] = __float2bfloat16_rn(q);
  at[2 * apart] = __float2bfloat16_rn(r - q);
}
__device__ __forceinline__ void store_parts(float* at, uint64_t apart, float v) {
  float hi, lo;
  parts(v, hi, lo);
  at[0] = hi;
  at[apart] = lo;
}

// The part of a vector that belongs to a lane's 16 bytes of weights; p: null for none.
template <class W, class X>
struct Share {
  using Value = typename PartsOf<X>::Value;
  static constexpr int P = PartsOf<X>::kParts, V = kPer16<W>, N = kPer16<Value>, kLoads = V > N ? V / N : 1;
  uint4 q[P][kLoads];
  __device__ __forceinline__ void load(const Value* p, uint64_t apart) {  // all of it there, in 16-byte loads
    static_assert(N <= V, "a lane's share is whole loads");
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) q[i][j] = __ldg(reinterpret_cast<const uint4*>(p + i * apart + j * N));
  }
  __device__ __forceinline__ void load(const Value* p, uint64_t apart, int left, bool wide) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        q[i][j] = p ? load16<Value>(p + i * apart + j * N, min(left - j * N, V), wide && N <= V) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float2 two(int part, int j) const { return two_of<Value>(q[part][j / (N / 2)], j % (N / 2)); }
};

// t += 16 rows x 8 vectors over a step: w0 and w1 are 16 bytes of rows gid and
// gid + 8.  16-bit operands of one type go to m16n8k16 as they are; others become
// floats.  The least parts come first.
template <class W, class X>
__device__ __forceinline__ void step_products(float (&t)[4], const uint4& w0, const uint4& w1, const Share<W, X>& x) {
  using Value = typename PartsOf<X>::Value;
  constexpr int P = PartsOf<X>::kParts;
  if constexpr (sizeof(W) == 2 && std::is_same<W, Value>::value) {
#pragma unroll
    for (int i = P - 1; i >= 0; --i) {
      multiply16<W>(t, w0.x, w1.x, w0.y, w1.y, x.q[i][0].x, x.q[i][0].y);
      multiply16<W>(t, w0.z, w1.z, w0.w, w1.w, x.q[i][0].z, x.q[i][0].w);
    }
  } else {
    constexpr bool kPartsW = std::is_same<W, float>::value, kSplitX = std::is_same<X, float>::value;
#pragma unroll
    for (int j = 0; j < kPer16<W> / 2; ++j) {
      float2 p = two_of<W>(w0, j), q = two_of<W>(w1, j), pl, ql;
      if constexpr (kPartsW) {
        const float2 u = p, v = q;
        parts(u.x, p.x, pl.x), parts(u.y, p.y, pl.y), parts(v.x, q.x, ql.x), parts(v.y, q.y, ql.y);
      }
      float2 b = x.two(0, j);
      if constexpr (kSplitX) {
        float2 l;
        const float2 u = b;
        parts(u.x, b.x, l.x), parts(u.y, b.y, l.y);
        multiply(t, p.x, q.x, p.y, q.y, l.x, l.y);
      }
      if constexpr (P == 2) {
        const float2 l = x.two(1, j);
        multiply(t, p.x, q.x, p.y, q.y, l.x, l.y);
      }
      if constexpr (kPartsW) multiply(t, pl.x, ql.x, pl.y, ql.y, b.x, b.y);
      multiply(t, p.x, q.x, p.y, q.y, b.x, b.y);
    }
  }
}

// Where the vectors of a product's columns lie: v[g], that of column gid of group
// g, or null.
template <class X, int G>
struct Vectors {
  const typename PartsOf<X>::Value* v[G];
  uint64_t apart;  // to a vector's next part
  uint32_t groups;
  bool wide;
};

// What a warp reads of the matrices: rows gid and gid + 8 of 16, and their scales.
template <class W>
struct Rows {
  const W *row0, *row1;           // read in place where stages are not used
  const uint8_t *scale0, *scale1;
};

// The first group's vectors for a chunk, or for one step of it where a lane's share
// of two would take too many registers.
template <class W, class X>
struct Chunk {
  static constexpr bool kBothSteps = 2 * sizeof(Share<W, X>) <= 128;
  Share<W, X> x[kBothSteps ? 2 : 1];
};

// Vectors p of step u of the chunk at place k0 of n.  kFast: chunks are whole and
// lie in 16-byte pieces, and p is never null (a column without a token reads
// another's): nothing between a load and its use waits for it.
template <bool kFast, class W, class X>
__device__ __forceinline__ void load_step(Share<W, X>& to, const typename PartsOf<X>::Value* p, uint64_t apart, bool wide, uint32_t k0,
                                          uint32_t u, uint32_t n) {
  const uint32_t k = k0 + u * kStep<W> + threadIdx.x % 4 * kPer16<W>;
  if constexpr (kFast) to.load(p + k, apart);
  else to.load(p ? p + k : nullptr, apart, (int)n - (int)k, wide);
}
template <bool kFast, class W, class X>
__device__ __forceinline__ void load_chunk(Chunk<W, X>& to, const typename PartsOf<X>::Value* p, uint64_t apart, bool wide, uint32_t k0,
                                           uint32_t n) {
  if (kFast) k0 = min(k0, n - kPlacesOfChunk<W>);
  load_step<kFast, W, X>(to.x[0], p, apart, wide, k0, 0, n);
  if constexpr (Chunk<W, X>::kBothSteps) load_step<kFast, W, X>(to.x[1], p, apart, wide, k0, 1, n);
}

// A warp's chunk of 16 rows at place k0 of n, times G groups of 8 vectors; `first`:
// the first group's.  stage: the lane's share of the chunk in shared memory (row
// gid, its first 16 bytes), or null (not kFast): the rows are read in place.  The instructions
// add to sums that begin at 0 and are added to c here: the tensor cores cut what
// they add off, which would tell in long sums.  8-bit weights: the places of a
// chunk are a block.
template <bool kFast, class W, class X, int G>
__device__ __forceinline__ void take_chunk(float (&c)[G][4], const uint8_t* stage, const Rows<W>& rows, const Vectors<X, G>& x,
                                           Chunk<W, X>& first, uint32_t k0, uint32_t n) {
  constexpr uint32_t S = kStep<W>;
  float f0 = 1.0f, f1 = 1.0f;
  if constexpr (std::is_same<W, F8>::value) {
    f0 = scale_value(__ldg(rows.scale0 + k0 / kFp8Block));
    f1 = scale_value(__ldg(rows.scale1 + k0 / kFp8Block));
  }
  uint4 w0[2], w1[2];
  if (kFast) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      w0[u] = *reinterpret_cast<const uint4*>(stage + u * 64);
      w1[u] = *reinterpret_cast<const uint4*>(stage + u * 64 + 8 * kPiece);
    }
  } else {
    const uint32_t k = k0 + threadIdx.x % 4 * kPer16<W>;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int left = (int)n - (int)(k + u * S);
      if (stage) {
        w0[u] = keep<W>(*reinterpret_cast<const uint4*>(stage + u * 64), left);
        w1[u] = keep<W>(*reinterpret_cast<const uint4*>(stage + u * 64 + 8 * kPiece), left);
      } else {
        w0[u] = load16<W>(rows.row0 + k + u * S, left, false);
        w1[u] = load16<W>(rows.row1 + k + u * S, left, false);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (g >= (int)x.groups) break;
    if (g) load_chunk<kFast, W, X>(first, x.v[g], x.apart, x.wide, k0, n);
    float t[4] = {};
    step_products<W, X>(t, w0[0], w1[0], first.x[0]);
    if constexpr (Chunk<W, X>::kBothSteps) {
      step_products<W, X>(t, w0[1], w1[1], first.x[1]);
    } else {
      load_step<kFast, W, X>(first.x[0], x.v[g], x.apart, x.wide, k0, 1, n);
      step_products<W, X>(t, w0[1], w1[1], first.x[0]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same<W, F8>::value) t[j] *= j < 2 ? f0 : f1;
      c[g][j] += t[j];
    }
  }
}

// ---- the stages of a block
struct Ring {
  uint64_t full[kMaxStages], empty[kMaxStages];
};
__device__ __forceinline__ void ring_init(Ring& r) {
  if (threadIdx.x == 0)
    for (uint32_t i = 0; i < kMaxStages; ++i) mbar_init(&r.full[i], 1), mbar_init(&r.empty[i], kWarps);
}

// A warp's way through the stages.  Fill says what comes next: more(), x (in words
// of the map), row0, row1, and advance() to what follows; every warp keeps it, and
// the one whose turn it is asks for it: 8 rows from row0 and 8 from row1 on.  What
// lies outside the map becomes zeros.
template <uint32_t kStages, class Fill>
struct Stages {  // (used: false where the rows are read in place)
  Ring& ring;
  uint8_t* memory;
  const CUtensorMap* map;
  Fill& fill;
  uint32_t warp, stage = 0, parity = 0, number = 0;
  bool used, ok = true;

  __device__ __forceinline__ void ask(uint32_t st) {
    mbar_arrive_expect_tx(&ring.full[st], kStageBytes);
    tma_load_2d(memory + st * kStageBytes, map, (int32_t)fill.x, (int32_t)fill.row0, &ring.full[st]);
    tma_load_2d(memory + st * kStageBytes + 8 * kPiece, map, (int32_t)fill.x, (int32_t)fill.row1, &ring.full[st]);
  }
  __device__ __forceinline__ Stages(Ring& r, uint8_t* m, const CUtensorMap* t, Fill& f, bool in_use)
      : ring(r), memory(m), map(t), fill(f), warp(threadIdx.x / 32), used(in_use) {
    if (!used) return;
    for (uint32_t i = 0; i < kStages; ++i) {
      if (!fill.more()) break;
      if (threadIdx.x == 0) ask(i);
      fill.advance();
    }
  }
  // The lane's share of the stage (row gid, its 16 bytes of the warp's first chunk).
  __device__ __forceinline__ const uint8_t* take() {
    if (!used) return nullptr;
    if (ok) ok = wait_phase(&ring.full[stage], parity);
    const uint32_t lane = threadIdx.x % 32;
    return memory + stage * kStageBytes + lane / 4 * kPiece + warp * kChunk + lane % 4 * 16;
  }
  __device__ __forceinline__ void leave() {
    if (!used) return;
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&ring.empty[stage]);
    if (fill.more()) {
      if (number % kWarps == warp && ok) {
        ok = wait_phase(&ring.empty[stage], parity);
        if (ok && threadIdx.x % 32 == 0) ask(stage);
        __syncwarp();
      }
      fill.advance();
    }
    ++number;
    next();
  }
  __device__ __forceinline__ void next() {
    if (++stage == kStages) stage = 0, parity ^= 1;
  }
  // A block that gives up does not end under its own copies.
  __device__ __forceinline__ void end() {
    if (ok) return;
    atomicOr(&g_layer_wait_ran_out, 1u);
    for (uint32_t i = 0; i < kStages; ++i, next()) wait_phase(&ring.full[stage], parity);
  }
};
// Barriers of the working warps: all wait, or a warp arrives and goes on.
__device__ __forceinline__ void warps_sync(uint32_t id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void warps_arrive(uint32_t id) { asm volatile("bar.arrive %0, 256;" ::"r"(id) : "memory"); }

// ---- what both kernels know of the pairs: the active experts in order, their
// tokens, where each one's pairs begin, each pair's token and weight
template <int G>
struct Pairs {
  static constexpr uint32_t N = 8 * G * kMaxTopK;
  uint32_t count;  // active experts
  union {
    uint32_t tokens[N];  // second kernel: a bit for each token of an active expert
    float weight[N];     // first kernel: of each pair
  };
  uint16_t expert[N];
  uint16_t begin[N + 1];
  uint8_t token[N];
};
// Where the pairs come from: ids and weights [tokens][top_k], the tokens of each
// expert and where its pairs begin.
struct PairSource {
  uint32_t ids[kMaxTokens * kMaxTopK];
  float weights[kMaxTokens * kMaxTopK];
  uint32_t mask[kMaxExperts];
  uint16_t place[kMaxExperts];
};

// Ids outside the experts take no part.  All threads call it, after a barrier that
// covers ids and weights.  Afterwards the source's memory may be given to copies.
template <bool kWeights, int G>
__device__ __forceinline__ void gather_pairs(Pairs<G>& p, PairSource& s, uint32_t tokens, uint32_t top_k, uint32_t experts) {
  const uint32_t lane = threadIdx.x % 32, pairs = tokens * top_k;
  for (uint32_t e = threadIdx.x; e < experts; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < pairs; i += kThreads)
    if (s.ids[i] < experts) atomicOr(&s.mask[s.ids[i]], 1u << (i / top_k));
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t active = 0, begin = 0;
    for (uint32_t e0 = 0; e0 < experts; e0 += 32) {
      const uint32_t e = e0 + lane, mask = e < experts ? s.mask[e] : 0, n = __popc(mask);
      const uint32_t upto = begin + warp_inclusive_sum(n), who = __ballot_sync(kAll, n > 0);
      if (e < experts) s.place[e] = (uint16_t)(upto - n);
      if (n) {
        const uint32_t a = active + __popc(who & ((1u << lane) - 1));
        p.expert[a] = (uint16_t)e;
        if constexpr (!kWeights) p.tokens[a] = mask;
        p.begin[a] = (uint16_t)(upto - n);
      }
      active += __popc(who);
      begin = __shfl_sync(kAll, upto, 31);
    }
    if (lane == 0) p.count = active, p.begin[active] = (uint16_t)begin;
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < pairs; i += kThreads) {
    const uint32_t e = s.ids[i], t = i / top_k;
    if (e >= experts) continue;
    const uint32_t at = s.place[e] + __popc(s.mask[e] & ((1u << t) - 1));
    p.token[at] = (uint8_t)t;
    if constexpr (kWeights) p.weight[at] = s.weights[i];
  }
  fence_proxy_async_smem();
  __syncthreads();
}

__device__ __noinline__ Choice choose_any(const RouteArgs& a, const float* row, bool live, uint32_t lane, float* keys) {
  if (a.experts <= 64) return choose<float, 32, 2>(a, row, live, lane, keys);
  if (a.experts <= 128) return choose<float, 32, 4>(a, row, live, lane, keys);
  if (a.experts <= 256) return choose<float, 32, 8>(a, row, live, lane, keys);
  if (a.experts <= 512) return choose<float, 32, 16>(a, row, live, lane, keys);
  return choose<float, 32, 32>(a, row, live, lane, keys);
}
// experts that a lane of choose_any holds
uint32_t held_by_lane(uint32_t experts) {
  return experts <= 64 ? 2 : experts <= 128 ? 4 : experts <= 256 ? 8 : experts <= 512 ? 16 : 32;
}

__device__ __forceinline__ float activate(int activation, float v) {
  if (activation == ZIPCCL_ACTIVATION_SILU) return v / (1.0f + expf(-v));
  if (activation == ZIPCCL_ACTIVATION_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  return v > 0.0f || isnan(v) ? v : 0.0f;
}

__host__ __device__ __forceinline__ uint32_t router_splits(uint32_t experts) {  // warps that share 16 experts' places
  return experts <= 16 ? 8 : experts <= 32 ? 4 : experts <= 64 ? 2 : 1;
}
constexpr uint32_t kShare = kMaxTokens / kCluster;  // tokens that a block chooses for

template <class R, class T, int G>
__device__ __forceinline__ void router_logits(const LayerArgs& a, float* partial, uint32_t rank) {
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t splits = router_splits(a.experts), tiles = (a.experts + 15) / 16, groups = (a.tokens + 7) / 8;
  const uint32_t steps = (a.hidden + kStep<R> - 1) / kStep<R>, all = kCluster * splits;
  const T* v[G];
#pragma unroll
  for (int g = 0; g < G; ++g) v[g] = g * 8 + gid < a.tokens ? static_cast<const T*>(a.x) + (uint64_t)(g * 8 + gid) * a.x_stride : nullptr;
  for (uint32_t tile = warp / splits; tile < tiles; tile += kWarps / splits) {
    const uint32_t part = rank * splits + warp % splits;
    float c[G][4] = {};
    const R* row = static_cast<const R*>(a.router);
    const uint32_t r0 = min(tile * 16 + gid, a.experts - 1), r1 = min(tile * 16 + gid + 8, a.experts - 1);
    const R *row0 = row + (uint64_t)r0 * a.hidden, *row1 = row + (uint64_t)r1 * a.hidden;
    constexpr int kAhead = G == 1 ? 4 : 2;
    for (uint32_t s = steps * part / all, end = steps * (part + 1) / all; s < end; s += kAhead) {
      uint4 w0[kAhead], w1[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
        const int left = s + u < end ? (int)a.hidden - (int)k : 0;
        w0[u] = load16<R>(row0 + k, left, a.wide_router);
        w1[u] = load16<R>(row1 + k, left, a.wide_router);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= (int)groups) break;
        float t[4] = {};
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
          Share<R, T> x;
          x.load(v[g] ? v[g] + k : nullptr, 0, s + u < end ? (int)a.hidden - (int)k : 0, a.wide_x);
          step_products<R, T>(t, w0[u], w1[u], x);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) c[g][i] += t[i];
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = tile * 16 + gid + (i / 2) * 8, t = g * 8 + quad * 2 + i % 2;
        if (e < a.experts && t < a.tokens) partial[(warp % splits * a.tokens + t) * a.experts + e] = c[g][i];
      }
  }
}

// The first kernel's work once the experts are chosen.
template <bool kFast, class T, class W, int G>
__device__ __forceinline__ void layer_up(const LayerArgs& a, const Pairs<G>& pairs, Ring& ring, uint8_t* memory) {
  constexpr uint32_t kStages = kStagesOf<G>;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  // 16 rows of an expert at a time: 8 of the gate's and 8 of the other's, so that
  // both of a place come to the same lane; or 16 of the only matrix
  const uint32_t high = a.gated ? 8 : 16, tiles = (a.inner + high - 1) / high, rows = a.gated ? 2 * a.inner : a.inner;
  const uint32_t pieces = (a.hidden + kPlacesOfPiece<W> - 1) / kPlacesOfPiece<W>, units = pairs.count * tiles;
  struct Fill {
    const LayerArgs& a;
    const Pairs<G>& pairs;
    uint32_t u, units, tiles, pieces, rows, high;
    uint32_t p = 0, x = 0, row0 = 0, row1 = 0;
    __device__ __forceinline__ bool more() const { return u < units; }
    __device__ __forceinline__ void place() {
      if (u >= units) return;
      const uint32_t n = u / tiles;
      row0 = pairs.expert[n] * rows + (u - n * tiles) * high;
      row1 = a.gated ? row0 + a.inner : row0 + 8;
    }
    __device__ __forceinline__ void advance() {
      x += kPiece / 8;
      if (++p < pieces) return;
      p = x = 0;
      u += gridDim.x;
      place();
    }
  } fill{a, pairs, blockIdx.x, units, tiles, pieces, rows, high};
  fill.place();
  Stages<kStages, Fill> stages(ring, memory, &a.up_map, fill, a.wide_up);
  float4* sums = reinterpret_cast<float4*>(memory + kStages * kStageBytes);
  const uint64_t apart = (uint64_t)(a.tokens * a.top_k + 1) * a.h_stride;
  const uint32_t k0 = warp * kPlacesOfChunk<W>;
  const auto vector = [&](uint32_t n, uint32_t col) -> const T* {  // of the column of active expert n
    uint32_t at = pairs.begin[n] + col;
    if (at >= pairs.begin[n + 1]) {
      if (!kFast) return nullptr;
      at = pairs.begin[n];
    }
    return static_cast<const T*>(a.x) + (uint64_t)pairs.token[at] * a.x_stride;
  };
  Chunk<W, T> x[2];
  if (blockIdx.x < units) load_chunk<kFast, W, T>(x[0], vector(blockIdx.x / tiles, gid), 0, a.wide_x, k0, a.hidden);
  uint32_t done = 0;
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++done) {
    const uint32_t n = u / tiles, i0 = (u - n * tiles) * high, e = pairs.expert[n];
    const uint32_t begin = pairs.begin[n], tokens = pairs.begin[n + 1] - begin, groups = (tokens + 7) / 8;
    const uint32_t r0 = min(i0 + gid, a.inner - 1), r1 = a.gated ? a.inner + r0 : min(i0 + gid + 8, a.inner - 1);
    Vectors<T, G> v;
    v.apart = 0, v.groups = groups, v.wide = a.wide_x;
#pragma unroll
    for (int g = 0; g < G; ++g) v.v[g] = vector(n, g * 8 + gid);
    const T* after = u + gridDim.x < units ? vector((u + gridDim.x) / tiles, gid) : v.v[0];  // the next unit's
    float c[G][4] = {};
    const W* at = static_cast<const W*>(a.up) + (uint64_t)e * rows * a.up_stride;
    const uint32_t across = (a.hidden + kFp8Block - 1) / kFp8Block;
    const uint8_t* scales = a.up_scales + (uint64_t)e * ((rows + kFp8Block - 1) / kFp8Block) * across;
    const Rows<W> its = {at + r0 * a.up_stride, at + r1 * a.up_stride, scales + r0 / kFp8Block * across, scales + r1 / kFp8Block * across};
    uint32_t k = k0;
    for (uint32_t p = 0; p < pieces; ++p) {
      const uint8_t* stage = stages.take();
#pragma unroll
      for (int i = 0; i < 2; ++i, k += kWarps * kPlacesOfChunk<W>) {
        const bool last = i && p + 1 == pieces;
        load_chunk<kFast, W, T>(x[i ^ 1], last ? after : v.v[0], 0, a.wide_x, last ? k0 : k + kWarps * kPlacesOfChunk<W>, a.hidden);
        if (k < a.hidden) take_chunk<kFast, W, T, G>(c, stage ? stage + i * kWarps * kChunk : nullptr, its, v, x[i], k, a.hidden);
      }
      stages.leave();
    }
    // The warps add up in turn, while the others go on: each arrives where its sums
    // are written, one waits for all, and before the memory is written again, two
    // units on, all wait for that one.
    const uint32_t half = done % 2;
    float4* mine = sums + half * kWarps * G * 32;
    if (done >= 2) {
      if (warp == (done - 2) % kWarps) warps_arrive(3 + half);
      else warps_sync(3 + half);
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < (int)groups) mine[(warp * G + g) * 32 + lane] = make_float4(c[g][0], c[g][1], c[g][2], c[g][3]);
    if (warp != done % kWarps) {
      warps_arrive(1 + half);
      continue;
    }
    warps_sync(1 + half);
    for (uint32_t g = 0; g < groups; ++g) {
      float4 all = mine[g * 32 + lane];
      for (int w = 1; w < kWarps; ++w) {
        const float4 q = mine[(w * G + g) * 32 + lane];
        all.x += q.x, all.y += q.y, all.z += q.z, all.w += q.w;
      }
      const float v4[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t col = g * 8 + quad * 2 + i;
        if (col >= tokens) continue;
        const float w = pairs.weight[begin + col];
        auto* h = static_cast<typename PartsFor<W>::Value*>(a.h) + (uint64_t)(begin + col) * a.h_stride + i0 + gid;
        if (a.gated) {
          if (i0 + gid < a.inner) store_parts(h, apart, w * (activate(a.activation, v4[i]) * v4[2 + i]));
        } else {
          if (i0 + gid < a.inner) store_parts(h, apart, w * activate(a.activation, v4[i]));
          if (i0 + gid + 8 < a.inner) store_parts(h + 8, apart, w * activate(a.activation, v4[2 + i]));
        }
      }
    }
  }
  stages.end();
}

// Dynamic shared memory of the first kernel: the stages, the working warps' sums.
// Before these: partial logits, rows and keys of the block's tokens, the pairs'
// source.
template <class T, class W, int G>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_up_kernel(const __grid_constant__ LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t s_dyn[];
  __shared__ Pairs<G> s_pairs;
  __shared__ Ring s_ring;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t rank = cluster_rank(), splits = router_splits(a.experts);
  ring_init(s_ring);
  PairSource& source = *reinterpret_cast<PairSource*>(s_dyn);
  float* partial = reinterpret_cast<float*>(s_dyn + sizeof(PairSource));
  {
    if (a.router_float) router_logits<float, T, G>(a, partial, rank);
    else router_logits<T, T, G>(a, partial, rank);
  }
  cluster_sync();
  {
    const uint32_t held = (a.experts + 3) / 4 * 4;
    float* rows = partial + (splits * a.tokens * a.experts + 3) / 4 * 4;
    for (uint32_t i = warp; i < kShare; i += kThreads / 32) {
      const uint32_t t = rank + i * kCluster;
      if (t >= a.tokens) break;
      float *row = rows + i * (held + 1024), *keys = row + held;
      for (uint32_t e = lane; e < a.experts; e += 32) {
        float sum = 0.0f;
        for (uint32_t r = 0; r < kCluster; ++r)
          for (uint32_t p = 0; p < splits; ++p) sum += load_cluster(at_rank(partial + (p * a.tokens + t) * a.experts + e, r));
        row[e] = sum;
      }
      __syncwarp();
      const Choice c = choose_any(a.route, row, !a.route.mask || a.route.mask[t], lane, keys);
      if (lane < a.top_k) {
        const float w = c.weight * a.route.scale;
        for (uint32_t r = 0; r < kCluster; ++r) {
          store_cluster(at_rank(source.ids + t * a.top_k + lane, r), (uint32_t)c.id);
          store_cluster(at_rank(source.weights + t * a.top_k + lane, r), __float_as_uint(w));
        }
        if (blockIdx.x < kCluster) {
          a.ids[t * a.top_k + lane] = c.id;
          a.weights[t * a.top_k + lane] = w;
        }
      }
    }
  }
  cluster_sync();  // also: nobody reads this block's shared memory any more
  gather_pairs<true>(s_pairs, source, a.tokens, a.top_k, a.experts);
  // the rows of h that columns without a token read in the second kernel
  if (blockIdx.x == 0) {
    auto* zero = static_cast<typename PartsFor<W>::Value*>(a.h) + (uint64_t)a.tokens * a.top_k * a.h_stride;
    const uint64_t apart = (uint64_t)(a.tokens * a.top_k + 1) * a.h_stride;
    for (uint32_t i = threadIdx.x; i < a.inner; i += kThreads) store_parts(zero + i, apart, 0.0f);
  }
  const bool fast = a.wide_up && a.wide_x && a.hidden % kPlacesOfChunk<W> == 0;
  if (fast) layer_up<true, T, W, G>(a, s_pairs, s_ring, s_dyn);
  else layer_up<false, T, W, G>(a, s_pairs, s_ring, s_dyn);
}

// 16 hidden places at a time; the pieces of the active experts' rows, one expert
// after the other, are dealt out in equal runs to 1, 2, 4 or 8 blocks of a cluster:
// whichever leaves the fewest pieces to the block that has most.  With one group of
// tokens the columns are the tokens themselves, so that a tile's sums stay in
// registers over all experts; with more, a warp adds what an expert gives to its
// tokens' sums in shared memory.  A block adds its warps', and after 8 tiles the
// blocks that share them each all blocks' of some of them.
template <bool kFast, class T, class W, int G>
__device__ __forceinline__ void layer_down(const LayerArgs& a, const Pairs<G>& pairs, Ring& ring, uint8_t* memory) {
  constexpr uint32_t kStages = kStagesOf<G>, kRound = kCluster;  // tiles before the blocks' sums are added
  using X = PartsFor<W>;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t rank = cluster_rank(), cluster = blockIdx.x / kCluster, clusters = gridDim.x / kCluster;
  const uint32_t size = a.tokens * 16;  // of a tile: [token][place]
  float* warps = reinterpret_cast<float*>(memory + kStages * kStageBytes);
  float* own = warps + warp * size;        // a warp's sums
  float* block = warps + kWarps * size;    // a block's, of a round's tiles
  const auto* h = static_cast<const typename X::Value*>(a.h);
  const uint64_t apart = (uint64_t)(a.tokens * a.top_k + 1) * a.h_stride;
  const uint32_t pieces = (a.inner + kPlacesOfPiece<W> - 1) / kPlacesOfPiece<W>, all = pieces * pairs.count;
  const uint32_t tiles = (a.hidden + 15) / 16, across = (a.inner + kFp8Block - 1) / kFp8Block;
  uint32_t split = 1, fewest = 0xFFFFFFFFu;
  for (uint32_t s = 1; s <= kCluster; s *= 2) {
    const uint32_t most = (tiles * s + clusters * kCluster - 1) / (clusters * kCluster) * ((all + s - 1) / s);
    if (most < fewest) fewest = most, split = s;
  }
  // blocks first .. first + split - 1 of the cluster share tiles t0, t0 + apart_tiles, ...
  const uint32_t part = rank % split, first = rank - part, stride = clusters * (kCluster / split);
  const uint32_t t0 = cluster * (kCluster / split) + rank / split;
  const uint32_t from = (uint32_t)((uint64_t)all * part / split), upto = (uint32_t)((uint64_t)all * (part + 1) / split);
  struct Fill {
    const LayerArgs& a;
    const Pairs<G>& pairs;
    uint32_t tile, tiles, stride, s, from, upto, pieces;
    uint32_t x = 0, row0 = 0, row1 = 0;
    __device__ __forceinline__ bool more() const { return tile < tiles && s < upto; }
    __device__ __forceinline__ void place() {
      if (!more()) return;
      const uint32_t n = s / pieces;
      x = (s - n * pieces) * (kPiece / 8);
      row0 = pairs.expert[n] * a.hidden + tile * 16;
      row1 = row0 + 8;
    }
    __device__ __forceinline__ void advance() {
      if (++s == upto) s = from, tile += stride;
      place();
    }
  } fill{a, pairs, t0, tiles, stride, from, from, upto, pieces};
  fill.place();
  Stages<kStages, Fill> stages(ring, memory, &a.down_map, fill, a.wide_down);
  const uint32_t k0 = warp * kPlacesOfChunk<W>;
  const auto vector = [&](uint32_t n, uint32_t col) -> const typename X::Value* {  // of a column of active expert n
    uint32_t at = pairs.begin[n] + col;
    if constexpr (G == 1) {
      const uint32_t mask = pairs.tokens[n];
      at = mask >> col & 1 ? pairs.begin[n] + __popc(mask & ((1u << col) - 1)) : a.tokens * a.top_k;
    } else if (at >= pairs.begin[n + 1]) {
      at = a.tokens * a.top_k;
    }
    return h + (uint64_t)at * a.h_stride;
  };
  Chunk<W, X> x[2];
  if (from < upto) load_chunk<kFast, W, X>(x[0], vector(from / pieces, gid), apart, true, from % pieces * kPlacesOfPiece<W> + k0, a.inner);
  const uint32_t rounds = (tiles + stride * kRound - 1) / (stride * kRound);  // the same for all blocks
  for (uint32_t round = 0; round < rounds; ++round) {
    for (uint32_t j = 0; j < kRound; ++j) {
      const uint32_t tile = t0 + (round * kRound + j) * stride;
      if (tile >= tiles) break;
      const uint32_t r0 = min(tile * 16 + gid, a.hidden - 1), r1 = min(tile * 16 + gid + 8, a.hidden - 1);
      float c[G][4] = {};
      if constexpr (G > 1) {
        for (uint32_t i = lane; i < size; i += 32) own[i] = 0.0f;
        __syncwarp();
      }
      uint32_t n = from / pieces, p = from - n * pieces;
      for (uint32_t s = from; s < upto;) {  // an expert's pieces of the run
        const uint32_t begin = pairs.begin[n], tokens = pairs.begin[n + 1] - begin;
        Vectors<X, G> v;
        v.apart = apart, v.groups = G == 1 ? 1 : (tokens + 7) / 8, v.wide = true;
#pragma unroll
        for (int g = 0; g < G; ++g) v.v[g] = vector(n, g * 8 + gid);
        const W* at = static_cast<const W*>(a.down) + (uint64_t)pairs.expert[n] * a.hidden * a.down_stride;
        const uint8_t* scales = a.down_scales + (uint64_t)pairs.expert[n] * ((a.hidden + kFp8Block - 1) / kFp8Block) * across;
        const Rows<W> its = {at + r0 * a.down_stride, at + r1 * a.down_stride, scales + r0 / kFp8Block * across, scales + r1 / kFp8Block * across};
        const uint32_t last = min(pieces, p + (upto - s));
        s += last - p;
        // what follows: the next expert's first piece, or the run's again
        const bool again = s == upto;
        const auto* after = vector(again ? from / pieces : n + 1, gid);
        const uint32_t after_k = (again ? from % pieces : 0) * kPlacesOfPiece<W> + k0;
        uint32_t k = p * kPlacesOfPiece<W> + k0;
        for (; p < last; ++p) {
          const uint8_t* stage = stages.take();
#pragma unroll
          for (int i = 0; i < 2; ++i, k += kWarps * kPlacesOfChunk<W>) {
            const bool leaves = i && p + 1 == last;
            load_chunk<kFast, W, X>(x[i ^ 1], leaves ? after : v.v[0], apart, true, leaves ? after_k : k + kWarps * kPlacesOfChunk<W>, a.inner);
            if (k < a.inner) take_chunk<kFast, W, X, G>(c, stage ? stage + i * kWarps * kChunk : nullptr, its, v, x[i], k, a.inner);
          }
          stages.leave();
        }
        p = 0, ++n;
        if constexpr (G > 1) {
#pragma unroll
          for (int g = 0; g < G; ++g) {
            if (g >= (int)v.groups) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t col = g * 8 + quad * 2 + i % 2;
              if (col < tokens) own[pairs.token[begin + col] * 16 + gid + (i / 2) * 8] += c[g][i];
              c[g][i] = 0.0f;
            }
          }
          __syncwarp();
        }
      }
      if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (quad * 2 + i % 2 < a.tokens) own[(quad * 2 + i % 2) * 16 + gid + (i / 2) * 8] = c[0][i];
      }
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
        float sum = warps[i];
        for (int w = 1; w < kWarps; ++w) sum += warps[w * size + i];
        block[j * size + i] = sum;
      }
      __syncthreads();
    }
    cluster_sync();
    for (uint32_t j = part; j < kRound; j += split) {
      const uint32_t tile = t0 + (round * kRound + j) * stride;
      if (tile >= tiles) break;
      for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
        const uint32_t t = i / 16, place = tile * 16 + i % 16;
        if (place >= a.hidden) continue;
        float sum = a.residual ? to_float(static_cast<const T*>(a.residual)[(uint64_t)t * a.hidden + place]) : 0.0f;
        for (uint32_t r = first; r < first + split; ++r) sum += load_cluster(at_rank(block + j * size + i, r));
        static_cast<T*>(a.y)[(uint64_t)t * a.hidden + place] = from_float<T>(sum);
      }
    }
    cluster_sync();
  }
  stages.end();
}

template <class T, class W, int G>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_down_kernel(const __grid_constant__ LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t s_dyn[];
  __shared__ Pairs<G> s_pairs;
  __shared__ Ring s_ring;
  PairSource& source = *reinterpret_cast<PairSource*>(s_dyn);
  ring_init(s_ring);
  for (uint32_t i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads) source.ids[i] = (uint32_t)a.ids[i];
  __syncthreads();
  gather_pairs<false>(s_pairs, source, a.tokens, a.top_k, a.experts);
  const bool fast = a.wide_down && a.inner % kPlacesOfChunk<W> == 0;
  if (fast) layer_down<true, T, W, G>(a, s_pairs, s_ring, s_dyn);
  else layer_down<false, T, W, G>(a, s_pairs, s_ring, s_dyn);
}

// ---------------------------------------------------------------- host
// Clusters of a kernel that run at the same time, found once for each device.  The
// kernel's limit of shared memory is set to the largest that any call asks for.
template <class... P>
cudaError_t clusters_at_once(void (*kernel)(P...), std::atomic<int>* known, size_t smem, size_t most, int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!(*out = known[dev].load(std::memory_order_acquire))) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kCluster, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = kCluster, cfg.blockDim = kThreads, cfg.dynamicSmemBytes = smem;
    cfg.attrs = &at, cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(out, kernel, &cfg)) != cudaSuccess) return e;
    *out = std::max(*out, 1);
    known[dev].store(*out, std::memory_order_release);
  }
  return cudaSuccess;
}

// Not set up beside the end of the kernel before: clusters would take the places
// that come free first, unevenly (one token of two experts of 3 x 4,096 x 14,336:
// 175 us with an early start, 142 without).
template <class... P, class... A>
cudaError_t launch_clusters(void (*kernel)(P...), uint32_t clusters, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kCluster, at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = clusters * kCluster, cfg.blockDim = kThreads, cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cfg.attrs = &at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int G>
size_t up_smem(uint32_t tokens, uint32_t experts) {
  const size_t choice = sizeof(PairSource) + 4ull * (router_splits(experts) * tokens * experts + 3 + kShare * ((experts + 3) / 4 * 4 + 1024));
  return std::max<size_t>(choice, kStagesOf<G> * kStageBytes + 2ull * kWarps * G * 512);
}
template <int G>
size_t down_smem(uint32_t tokens) { return kStagesOf<G> * kStageBytes + 4ull * (kWarps + kCluster) * tokens * 16; }

template <class T, class W, int G>
cudaError_t layer_launch(const LayerArgs& a, cudaStream_t s) {
  static std::atomic<int> up_known[kMaxDevices], down_known[kMaxDevices];
  constexpr uint32_t most = G == 1 ? 8 : kMaxTokens;
  const size_t up = up_smem<G>(a.tokens, a.experts), down = down_smem<G>(a.tokens);
  int up_clusters = 0, down_clusters = 0;
  cudaError_t e = clusters_at_once(zc_layer_up_kernel<T, W, G>, up_known, up_smem<G>(1, 1), up_smem<G>(most, kMaxExperts), &up_clusters);
  if (e == cudaSuccess) e = clusters_at_once(zc_layer_down_kernel<T, W, G>, down_known, down_smem<G>(most), down_smem<G>(most), &down_clusters);
  if (e == cudaSuccess) e = launch_clusters(zc_layer_up_kernel<T, W, G>, up_clusters, up, s, a);
  const uint32_t tiles = (a.hidden + 15) / 16;
  if (e == cudaSuccess) e = launch_clusters(zc_layer_down_kernel<T, W, G>, std::min<uint32_t>(down_clusters, tiles), down, s, a);
  return e;
}

template <class T>
cudaError_t layer_by_weights(const LayerArgs& a, bool blocks, cudaStream_t s) {
  // up to 8 tokens have one group each way; the other form serves any number
  if (blocks) return a.tokens <= 8 ? layer_launch<T, F8, 1>(a, s) : layer_launch<T, F8, 4>(a, s);
  return a.tokens <= 8 ? layer_launch<T, T, 1>(a, s) : layer_launch<T, T, 4>(a, s);
}

}  // namespace

cudaError_t layer_waits(cudaStream_t s, bool* ran_out) { return take_flag(g_layer_wait_ran_out, s, ran_out); }

}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_layer_workspace_bytes(uint64_t tokens, uint32_t top_k, uint64_t inner, uint64_t* out_bytes) {
  if (!out_bytes || tokens > kMaxTokens || top_k == 0 || top_k > kMaxTopK || inner >= (1ull << 22)) return ZIPCCL_ERR_INVALID_ARG;
  // a row for each pair and one of zeros, two floats or three bfloat16 a value
  *out_bytes = ((tokens * top_k + 1) * ((inner + 7) / 8 * 8) * 8 + 255) / 256 * 256;
  return ZIPCCL_OK;
}

zipccl_status zipccl_moe_layer(const zipccl_moe_layer_args* l, const zipccl_route_options* o, void* d_ws, uint64_t ws_bytes, void* stream) {
  if (!l || !o) return ZIPCCL_ERR_INVALID_ARG;
  const uint64_t z = type_bytes(l->type);
  const bool blocks = l->weight_bits == 8;
  if (z == 0 || (l->weight_bits != 8 && l->weight_bits != 8 * z)) return ZIPCCL_ERR_INVALID_ARG;
  if (l->router_type != l->type && l->router_type != ZIPCCL_TYPE_F32) return ZIPCCL_ERR_INVALID_ARG;
  const uint32_t experts = l->experts;
  if (experts == 0 || experts > kMaxExperts || l->tokens > kMaxTokens || l->hidden == 0 || l->inner == 0 || l->hidden >= (1ull << 22) ||
      l->inner >= (1ull << 22) || (l->x_stride < l->hidden && l->tokens > 1))
    return ZIPCCL_ERR_INVALID_ARG;
  if (o->top_k == 0 || o->top_k > kMaxTopK || o->top_k > experts) return ZIPCCL_ERR_INVALID_ARG;
  if (o->score != ZIPCCL_SCORE_SOFTMAX && o->score != ZIPCCL_SCORE_SIGMOID) return ZIPCCL_ERR_INVALID_ARG;
  if (o->group_score != ZIPCCL_GROUP_MAX && o->group_score != ZIPCCL_GROUP_TOP2) return ZIPCCL_ERR_INVALID_ARG;
  if (o->groups == 0 || o->groups > kMaxGroups || experts % o->groups || o->groups_kept == 0 || o->groups_kept > o->groups ||
      o->top_k > o->groups_kept * (experts / o->groups) || !isfinite(o->scale))
    return ZIPCCL_ERR_INVALID_ARG;
  if (l->activation < ZIPCCL_ACTIVATION_SILU || l->activation > ZIPCCL_ACTIVATION_RELU) return ZIPCCL_ERR_INVALID_ARG;
  if (l->tokens == 0) return ZIPCCL_OK;
  const uint64_t wz = blocks ? 1 : z;
  if (!l->d_x || !l->d_router || !l->d_up || !l->d_down || !l->d_y || !l->d_weights || !l->d_ids) return ZIPCCL_ERR_INVALID_ARG;
  if (!host_aligned(l->d_x, z) || !host_aligned(l->d_router, type_bytes(l->router_type)) || !host_aligned(l->d_up, wz) ||
      !host_aligned(l->d_down, wz) || !host_aligned(l->d_y, z) || !host_aligned(l->d_weights, 4) || !host_aligned(l->d_ids, 4) ||
      !host_aligned(l->d_residual, z) || !host_aligned(l->d_bias, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  if (l->up_stride < l->hidden || l->down_stride < l->inner) return ZIPCCL_ERR_INVALID_ARG;
  if (blocks && (!l->d_up_scales || !l->d_down_scales || !host_aligned(l->d_up, 16) || !host_aligned(l->d_down, 16) ||
                 l->up_stride % 16 || l->down_stride % 16))
    return ZIPCCL_ERR_INVALID_ARG;
  uint64_t need = 0;
  const zipccl_status st = zipccl_moe_layer_workspace_bytes(l->tokens, o->top_k, l->inner, &need);
  if (st != ZIPCCL_OK) return st;
  if (!d_ws || !host_aligned(d_ws, 256)) return ZIPCCL_ERR_INVALID_ARG;
  if (ws_bytes < need) return ZIPCCL_ERR_CAPACITY;
  LayerArgs a{};
  a.x = l->d_x;
  a.router = l->d_router;
  a.up = l->d_up;
  a.down = l->d_down;
  a.residual = l->d_residual;
  a.up_scales = l->d_up_scales;
  a.down_scales = l->d_down_scales;
  a.y = l->d_y;
  a.weights = l->d_weights;
  a.ids = l->d_ids;
  a.h = d_ws;
  a.h_stride = (l->inner + 7) / 8 * 8;
  a.x_stride = l->x_stride;
  a.up_stride = l->up_stride;
  a.down_stride = l->down_stride;
  a.tokens = (uint32_t)l->tokens;
  a.hidden = (uint32_t)l->hidden;
  a.inner = (uint32_t)l->inner;
  a.experts = experts;
  a.top_k = o->top_k;
  a.activation = l->activation;
  a.gated = l->gated != 0;
  const uint64_t rz = type_bytes(l->router_type);
  a.router_float = l->router_type != l->type;
  a.wide_x = host_aligned(l->d_x, 16) && l->x_stride * z % 16 == 0;
  a.wide_router = host_aligned(l->d_router, 16) && l->hidden * rz % 16 == 0;
  a.wide_up = host_aligned(l->d_up, 16) && l->up_stride * wz % 16 == 0;
  a.wide_down = host_aligned(l->d_down, 16) && l->down_stride * wz % 16 == 0;
  // (row numbers of a map are whole numbers of 32 bits)
  const uint64_t up_rows = (l->gated ? 2 : 1) * l->inner;
  if (experts * up_rows >= (1ull << 31) || experts * l->hidden >= (1ull << 31)) return ZIPCCL_ERR_INVALID_ARG;
  if ((a.wide_up && !word_map(&a.up_map, l->d_up, l->hidden * wz, experts * up_rows, l->up_stride * wz, kPiece / 8, 8)) ||
      (a.wide_down && !word_map(&a.down_map, l->d_down, l->inner * wz, experts * l->hidden, l->down_stride * wz, kPiece / 8, 8)))
    return ZIPCCL_ERR_CUDA;
  RouteArgs& r = a.route;
  const uint32_t V = held_by_lane(experts), B = V < 4 ? V : 4;
  r.bias = l->d_bias;
  r.mask = l->d_mask;
  r.experts = experts;
  r.top_k = o->top_k;
  r.groups = o->groups;
  r.kept = o->groups_kept;
  r.group_size = experts / o->groups;
  r.scale = o->scale;
  const uint32_t lanes = r.group_size % V ? 0 : r.group_size / V;
  r.group_lanes = lanes & (lanes - 1) || r.groups > 32 ? 0 : lanes;
  r.softmax = o->score == ZIPCCL_SCORE_SOFTMAX;
  r.renormalize = o->renormalize != 0;
  r.top2 = o->group_score == ZIPCCL_GROUP_TOP2;
  r.wide = experts % B == 0;
  r.wide_bias = host_aligned(l->d_bias, B * sizeof(float)) && experts % B == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = l->type == ZIPCCL_TYPE_F32    ? layer_by_weights<float>(a, blocks, s)
                        : l->type == ZIPCCL_TYPE_BF16 ? layer_by_weights<__nv_bfloat16>(a, blocks, s)
                                                      : layer_by_weights<__half>(a, blocks, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // extern "C"
