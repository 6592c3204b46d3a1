// zc_layer.cuh -- a whole mixture-of-experts layer for a few tokens: what its two
// kernels share.
//
//   logits = router x;  weights, ids = choice of experts (zc_route.cuh)
//   h = weight * act(gate x) * (up x)  for each token and expert of it   (first kernel)
//   y = residual + sum over a token's experts of down h                  (second kernel)
//
// Such a layer reads every chosen expert's matrices once and is bound by that: a
// token of two experts of 3 x 4,096 x 14,336 bfloat16 values reads 705 MB for 0.7
// GFLOP.  The tokens are the narrow side: a warp takes 16 rows of a matrix and
// up to 8 of the expert's tokens to a tensor instruction, which costs no more than one
// token and less than their sums in ordinary instructions.  16-bit operands of one
// type go to it as they are (m16n8k16): x with weights of its type, and h, in parts,
// with bfloat16 weights; others as 32-bit floats of which the top 19 bits count
// (m16n8k8): 16-bit and 8-bit values are exact in these, a 32-bit one is the sum of
// two such parts (21 bits at least), and of products of parts only the two least
// ones' is left out.
//
// Everything that depends on where a place of the sum lies in an instruction is
// the same for both operands, so a lane reads 16 consecutive bytes of a row and
// hands them to the instructions in its own order.
//
// The matrices come through shared memory in pieces of 2,048 bytes of 16 rows, two
// or three stages ahead; 8 warps take 128 bytes of each row at a time, and in turn
// fill a stage again that all have left.  Rows that start at multiples of 16 bytes
// are copied by a tensor map, others one by one from the last multiple before, and
// a lane shifts what it reads.  What is left of a row behind the last whole 128
// bytes is read in place by one warp.  The tokens' own values come from global
// memory, a chunk ahead; nothing between such a load and its use may hang on a
// condition, or the load is waited for at once (142 us instead of 199 for the one
// token).
//
// Measured, both kernels and the choice: that token 134 us, 79% of the copy rate;
// 32 tokens, 8 of 128 experts of 3 x 2,048 x 768 244 us, 65%; 7 tokens, 2 of 64 of
// 3 x 4,096 x 2,048: 128 us in 16 bits, 75%, 121 in 8, 40%: there turning codes into
// floats takes half of the issue slots, and each warp waits for its own; 373 in 32,
// 51%, for six instructions in place of one.  Rows that start anywhere cost 1.3 to
// 1.7 times that.
#pragma once
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

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr uint32_t kCluster = 8, kMaxTokens = ZIPCCL_LAYER_MAX_TOKENS;
constexpr uint32_t kPiece = 2048, kChunk = 128;  // bytes of a row in a stage, and those that a warp takes at a time
constexpr uint32_t kChunks = kPiece / kChunk / kWarps;  // of a warp in a stage
// Rows that start anywhere: the bytes from the last multiple of 16 on, 64 bytes more
// for each row, which also keep two rows out of each other's banks.
template <bool kShift>
constexpr uint32_t kPitch = kPiece + (kShift ? 64 : 0);
template <bool kShift>
constexpr uint32_t kStageBytes = 16 * kPitch<kShift>;
constexpr uint32_t kMaxStages = 3;
// Shared memory that leaves room for two blocks of a multiprocessor, without what
// the kernels declare themselves.
constexpr size_t kRoomForTwo = 114000;
constexpr uint32_t kTokens = 8;  // columns of an instruction: tokens of an expert taken together

struct LayerArgs {
  CUtensorMap up_map, down_map;  // 8 rows x 256 words of 8 bytes
  const void *x, *router, *up, *down, *residual;
  const uint8_t *up_scales, *down_scales;
  void* y;
  float* weights;
  int32_t* ids;
  void* h;  // parts of each pair's inner places, rows of h_stride values
  uint64_t x_stride, up_stride, down_stride, h_stride;  // in values
  uint32_t tokens, hidden, inner, experts, top_k, stages;
  int activation;
  bool gated, router_float;
  bool shift_up, shift_down;  // rows start anywhere (up: of up, x or router)
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

// Sum over blocks first .. first + count - 1 of the cluster of one place of their shared memory, in order;
// all are asked for before the first is used (one after the other they take a
// quarter of a microsecond each).
__device__ __forceinline__ float cluster_sum(const float* p, uint32_t first, uint32_t count) {
  float v[kCluster], sum = 0.0f;
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r) v[r] = load_cluster(at_rank(p, first + min(r, count - 1)));
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r)
    if (r < count) sum += v[r];
  return sum;
}

// ---- values
struct F8 {
  uint8_t bits;
};

// 16 bytes of a row that starts anywhere, from byte `off` on (a multiple of 16 from the row's start) of `bytes`.  What
// lies behind the row is read from its last 16 bytes: no access leaves the 16 that
// hold one of its values.
template <bool kShift>
__device__ __forceinline__ Raw raw16(const void* row, uint32_t off, uint32_t bytes) {
  Raw r;
  if constexpr (kShift) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row), base = at & ~uintptr_t(15);
    const uint32_t last = ((uint32_t)(at & 15) + bytes - 1) & ~15u;
    r.a = __ldg(reinterpret_cast<const uint4*>(base + min(off, last)));
    r.b = __ldg(reinterpret_cast<const uint4*>(base + min(off + 16, last)));
  } else {
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + min(off, (bytes - 1) & ~15u)));
  }
  return r;
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

// h as the second kernel takes it, each part in an array of its own: with bfloat16
// weights three bfloat16 values, 24 bits.  With others in a layer of 16 bits the
// float itself: the instruction drops its low 13 bits, and what they hold is the
// second part, of which it takes 11 bits (h is 2^-21 off at most, and a part costs
// no more than to unpack).  For 32-bit layers two floats of 11 bits, made once.
// (16 bits of h in two bfloat16 values made ten times as many results differ from
// the rounded sum as 24 do: 0.3% of bfloat16 ones, 0.8% of float16 ones.)
struct ThreeSmall {
  using Value = __nv_bfloat16;
  static constexpr int kParts = 3;
};
struct Whole {
  using Value = float;
  static constexpr int kParts = 1;
};
struct TwoParts {
  using Value = float;
  static constexpr int kParts = 2;
};
template <class T, class W>
using PartsFor = std::conditional_t<sizeof(T) == 4, TwoParts, std::conditional_t<std::is_same<W, __nv_bfloat16>::value, ThreeSmall, Whole>>;
template <class X>
struct PartsOf {  // of a plain vector: itself
  using Value = X;
  static constexpr int kParts = 1;
};
template <>
struct PartsOf<ThreeSmall> : ThreeSmall {};
template <>
struct PartsOf<Whole> : Whole {};
template <>
struct PartsOf<TwoParts> : TwoParts {};

__device__ __forceinline__ float bf16_part(float v) {
  float p = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(p) && !isinf(v)) p = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return p;
}
// Writes the parts of v to at[0], at[apart], ...
template <class X>
__device__ __forceinline__ void store_parts(typename X::Value* at, uint64_t apart, float v) {
  if constexpr (X::kParts == 1) {
    at[0] = v;
  } else if constexpr (X::kParts == 2) {
    float hi, lo;
    parts(v, hi, lo);
    at[0] = hi;
    at[apart] = lo;
  } else {
    const float p = bf16_part(v), r = isfinite(v) ? v - p : 0.0f, q = bf16_part(r);
    at[0] = __float2bfloat16_rn(p);
    at[apart] = __float2bfloat16_rn(q);
    at[2 * apart] = __float2bfloat16_rn(r - q);
  }
}

// The part of a vector that belongs to a lane's 16 bytes of weights, as it is read
// and as it is used.
template <class W, class X>
struct Share {
  using Value = typename PartsOf<X>::Value;
  static constexpr int P = PartsOf<X>::kParts, V = kPer16<W>, N = kPer16<Value>, kLoads = V > N ? V / N : 1;
  uint4 q[P][kLoads];
  __device__ __forceinline__ float2 two(int part, int j) const { return two_of<Value>(q[part][j / (N / 2)], j % (N / 2)); }
};
template <class W, class X, bool kShift>
struct RawShare {
  using S = Share<W, X>;
  using Value = typename S::Value;
  static constexpr int kVectors = S::kLoads + (kShift || S::N > S::V ? 1 : 0);
  uint4 q[S::P][kVectors];
  // Places k .. of n of the vector at p, parts `apart` values from each other.
  __device__ __forceinline__ void load(const Value* p, uint64_t apart, uint32_t k, uint32_t n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), base = at & ~uintptr_t(15);
    const uint32_t off = k * (uint32_t)sizeof(Value), last = ((uint32_t)(at & 15) + n * (uint32_t)sizeof(Value) - 1) & ~15u;
    const uint32_t first = S::N > S::V ? ((uint32_t)(at & 15) + off) & ~15u : off;  // (fewer than 16 bytes: they may begin within 16)
#pragma unroll
    for (int i = 0; i < S::P; ++i)
#pragma unroll
      for (int j = 0; j < kVectors; ++j)
        q[i][j] = __ldg(reinterpret_cast<const uint4*>(base + i * apart * sizeof(Value) + min(first + 16 * j, last)));
  }
  __device__ __forceinline__ S used(const Value* p, uint32_t k, uint32_t n, bool whole) const {
    S s;
    const uint32_t shift = S::N > S::V ? ((uint32_t)(reinterpret_cast<uintptr_t>(p) & 15) + k * (uint32_t)sizeof(Value)) & 15 : shift_of(p);
#pragma unroll
    for (int i = 0; i < S::P; ++i)
#pragma unroll
      for (int j = 0; j < S::kLoads; ++j) {
        if constexpr (kVectors > S::kLoads) s.q[i][j] = settle<true>({q[i][j], q[i][j + 1]}, shift);
        else s.q[i][j] = q[i][j];
        if (!whole) s.q[i][j] = keep<Value>(s.q[i][j], (int)n - (int)k - j * S::N);
      }
    return s;
  }
};

// t = 16 rows x 8 vectors over a step: w0 and w1 are 16 bytes of rows gid and
// gid + 8.  16-bit operands of one type go to m16n8k16 as they are; others become
// floats.  The instructions cut what lies below a sum's last place: in floats, sums
// of large and small parts are kept apart, and of four instructions at most; 16-bit
// operands make one chain of a chunk's instructions, 12 with three parts, the least
// parts first in each step (2^-20 of the chunk's sum at most, where a result of 16
// bits has 2^-8 or 2^-11).
// kLogits: a value that is not finite meets no second part, whose sign or 0 would
// make infinity a NaN (a token's choice hangs on it; what the experts make of such a
// value may be either).
template <class W, class X, bool kLogits = false>
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
    constexpr bool kPartsW = std::is_same<W, float>::value, kSplitX = std::is_same<X, float>::value, kWholeX = std::is_same<X, Whole>::value;
    constexpr bool kSmall = kPartsW || kSplitX || kWholeX || P == 2;
    constexpr int J = kPer16<W> / 2;
    const auto finite = [](float v) { return kLogits && (__float_as_uint(v) & 0x7FFFFFFFu) >= 0x7F800000u ? 0.0f : v; };
#pragma unroll
    for (int j0 = 0; j0 < J; j0 += 4) {
      float large[4] = {}, small[4] = {};
#pragma unroll
      for (int j = j0; j < (J < j0 + 4 ? J : j0 + 4); ++j) {
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
          multiply(small, finite(p.x), finite(q.x), finite(p.y), finite(q.y), l.x, l.y);
        }
        if constexpr (kWholeX) {
          const auto low = [](float v) { return v - __uint_as_float(__float_as_uint(v) & 0xFFFFE000u); };
          multiply(small, p.x, q.x, p.y, q.y, low(b.x), low(b.y));
        }
        if constexpr (P == 2) {
          const float2 l = x.two(1, j);
          multiply(small, p.x, q.x, p.y, q.y, l.x, l.y);
        }
        if constexpr (kPartsW) multiply(small, pl.x, ql.x, pl.y, ql.y, finite(b.x), finite(b.y));
        multiply(large, p.x, q.x, p.y, q.y, b.x, b.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] += kSmall ? large[i] + small[i] : large[i];
    }
  }
}

// Where the vector of a lane's column lies (gid's; a column without a token has
// another's, and its sums are not used), and its next part.
template <class X>
struct Vector {
  const typename PartsOf<X>::Value* at;
  uint64_t apart;
};

// What a warp reads of the matrices: rows gid and gid + 8 of 16, and their scales.
template <class W>
struct Rows {
  const W *row0, *row1;
  const uint8_t *scale0, *scale1;
};

// The vectors for a chunk, or for one step of it where a lane's share
// of two would take too many registers.
template <class W, class X, bool kShift>
struct Chunk {
  using R = RawShare<W, X, kShift>;
  static constexpr bool kBothSteps = 2 * sizeof(R) <= (R::S::P == 3 ? 96 : 64);
  R x[kBothSteps ? 2 : 1];
  __device__ __forceinline__ void load(const typename R::Value* p, uint64_t apart, uint32_t k0, uint32_t n) {
    const uint32_t k = k0 + threadIdx.x % 4 * kPer16<W>;
    x[0].load(p, apart, k, n);
    if constexpr (kBothSteps) x[1].load(p, apart, k + kStep<W>, n);
  }
};

// A warp's chunk of 16 rows at place k0 of n, times 8 vectors, those in `mine`.
// stage: the lane's share of the chunk in shared memory (row gid, its first 16
// bytes); kTail: the chunk is not whole, and read in place.  The sums of a chunk
// begin at 0 and are added to c here.  8-bit weights: the places of a chunk are a
// block.  kShiftW, kShiftX: rows, vectors may start anywhere.
template <bool kTail, bool kShiftW, bool kShiftX, class W, class X>
__device__ __forceinline__ void take_chunk(float (&c)[4], const uint8_t* stage, const Rows<W>& rows, const Vector<X>& x,
                                           Chunk<W, X, kShiftX>& mine, uint32_t k0, uint32_t n) {
  constexpr uint32_t S = kStep<W>;
  using C = Chunk<W, X, kShiftX>;
  const uint32_t k = k0 + threadIdx.x % 4 * kPer16<W>;
  float f0 = 1.0f, f1 = 1.0f;
  if constexpr (std::is_same<W, F8>::value) {
    f0 = scale_value(__ldg(rows.scale0 + k0 / kFp8Block));
    f1 = scale_value(__ldg(rows.scale1 + k0 / kFp8Block));
  }
  uint4 w0[2], w1[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    Raw a, b;
    if constexpr (kTail) {
      const uint32_t off = (k + u * S) * (uint32_t)sizeof(W), bytes = n * (uint32_t)sizeof(W);
      a = raw16<kShiftW>(rows.row0, off, bytes), b = raw16<kShiftW>(rows.row1, off, bytes);
    } else {
      a.a = *reinterpret_cast<const uint4*>(stage + u * 64);
      b.a = *reinterpret_cast<const uint4*>(stage + u * 64 + 8 * kPitch<kShiftW>);
      if constexpr (kShiftW) {
        a.b = *reinterpret_cast<const uint4*>(stage + u * 64 + 16);
        b.b = *reinterpret_cast<const uint4*>(stage + u * 64 + 16 + 8 * kPitch<kShiftW>);
      }
    }
    w0[u] = settle<kShiftW>(a, shift_of(rows.row0)), w1[u] = settle<kShiftW>(b, shift_of(rows.row1));
    if constexpr (kTail) {
      const int left = (int)n - (int)(k + u * S);
      w0[u] = keep<W>(w0[u], left), w1[u] = keep<W>(w1[u], left);
    }
  }
  float t[4] = {};
  step_products<W, X>(t, w0[0], w1[0], mine.x[0].used(x.at, k, n, !kTail));
  if constexpr (!C::kBothSteps) mine.x[0].load(x.at, x.apart, k + S, n);
  step_products<W, X>(t, w0[1], w1[1], mine.x[C::kBothSteps ? 1 : 0].used(x.at, k + S, n, !kTail));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (std::is_same<W, F8>::value) t[j] *= j < 2 ? f0 : f1;
    c[j] += t[j];
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

// A warp's way through the stages.  Fill says what comes next: more(), piece, row0
// and row1 (their numbers), and advance() to what follows; every warp keeps it, and
// the one whose turn it is asks for it: 8 rows from row0 and 8 from row1 on, or, where
// rows start anywhere, what each holds of the piece, in multiples of 16 bytes.  What
// lies outside the map becomes zeros.
struct Matrix {
  const CUtensorMap* map;
  const uint8_t* at;
  uint64_t rows, stride;  // stride: bytes
  uint32_t bytes;         // of a row
};
template <bool kShift, class Fill>
struct Stages {
  Ring& ring;
  uint8_t* memory;
  const Matrix& matrix;
  Fill& fill;
  uint32_t count, warp, stage = 0, parity = 0, number = 0;  // count: of the stages
  bool ok = true;
  unsigned int* ran_out;

  __device__ __forceinline__ void ask(uint32_t st) {  // a whole warp
    const uint32_t lane = threadIdx.x % 32;
    uint8_t* to = memory + st * kStageBytes<kShift>;
    if constexpr (kShift) {
      const uint64_t row = min((uint64_t)(lane < 8 ? fill.row0 + lane : fill.row1 + lane % 8), matrix.rows - 1);
      const uint8_t* p = matrix.at + row * matrix.stride;
      const uint32_t shift = shift_of(p), from = fill.piece * kPiece;
      const uint32_t bytes = lane < 16 ? min(kPiece + 16, (shift + matrix.bytes + 15) / 16 * 16 - from) : 0;
      const uint32_t all = __reduce_add_sync(kAll, bytes);
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[st], all);
      __syncwarp();
      if (lane < 16) bulk_copy_g2s(to + lane * kPitch<kShift>, p - shift + from, bytes, &ring.full[st]);
    } else if (lane == 0) {
      mbar_arrive_expect_tx(&ring.full[st], kStageBytes<kShift>);
      tma_load_2d(to, matrix.map, (int32_t)(fill.piece * (kPiece / 8)), (int32_t)fill.row0, &ring.full[st]);
      tma_load_2d(to + 8 * kPiece, matrix.map, (int32_t)(fill.piece * (kPiece / 8)), (int32_t)fill.row1, &ring.full[st]);
    }
  }
  __device__ __forceinline__ Stages(Ring& r, uint8_t* m, const Matrix& x, Fill& f, uint32_t n, unsigned int* flag)
      : ring(r), memory(m), matrix(x), fill(f), count(n), warp(threadIdx.x / 32), ran_out(flag) {
    for (uint32_t i = 0; i < count; ++i) {
      if (!fill.more()) break;
      if (warp == 0) ask(i);
      fill.advance();
    }
  }
  // The lane's share of the stage (row gid, its 16 bytes of the warp's first chunk).
  __device__ __forceinline__ const uint8_t* take() {
    if (ok) ok = wait_phase(&ring.full[stage], parity);
    const uint32_t lane = threadIdx.x % 32;
    return memory + stage * kStageBytes<kShift> + lane / 4 * kPitch<kShift> + warp * kChunk + lane % 4 * 16;
  }
  __device__ __forceinline__ void leave() {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&ring.empty[stage]);
    if (fill.more()) {
      if (number % kWarps == warp) {  // one answer for the warp: ask() names all its lanes
        ok = __all_sync(kAll, ok && wait_phase(&ring.empty[stage], parity));
        if (ok) ask(stage);
        __syncwarp();
      }
      fill.advance();
    }
    ++number;
    next();
  }
  __device__ __forceinline__ void next() {
    if (++stage == count) stage = 0, parity ^= 1;
  }
  // A block that gives up does not end under its own copies.
  __device__ __forceinline__ void end() {
    if (ok) return;
    atomicOr(ran_out, 1u);
    for (uint32_t i = 0; i < count; ++i, next()) wait_phase(&ring.full[stage], parity);
  }
};
// Barriers of the working warps: all wait, or a warp arrives and goes on.
__device__ __forceinline__ void warps_sync(uint32_t id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void warps_arrive(uint32_t id) { asm volatile("bar.arrive %0, 256;" ::"r"(id) : "memory"); }

// ---- what both kernels know of the pairs: the active experts in order, one with
// more than 8 tokens several times, where the pairs of each entry begin (8 at most),
// each pair's token and weight.  An entry beyond the first reads its matrices again,
// from the L2 cache as a rule: neighbouring blocks take it at the same time.  (All
// of an expert's tokens in one entry, four times 8 sums: the registers did not hold
// what 8-bit weights become, 515 us where 16-bit ones took 258; 32 tokens, 8 of 128
// experts.)
struct Pairs {
  uint32_t* count;
  float* weight;  // of each pair (first kernel)
  uint16_t *expert, *begin;
  uint8_t* token;
  __host__ __device__ static constexpr size_t bytes(uint32_t pairs) { return (16 + 9ull * pairs + 2 + 15) / 16 * 16; }
  __device__ __forceinline__ Pairs(uint8_t* memory, uint32_t pairs) {
    count = reinterpret_cast<uint32_t*>(memory);
    weight = reinterpret_cast<float*>(memory + 16);
    begin = reinterpret_cast<uint16_t*>(weight + pairs);
    expert = begin + pairs + 1;
    token = reinterpret_cast<uint8_t*>(expert + pairs);
  }
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
template <bool kWeights>
__device__ __forceinline__ void gather_pairs(const Pairs& p, PairSource& s, uint32_t tokens, uint32_t top_k, uint32_t experts) {
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
      const uint32_t entries = (n + kTokens - 1) / kTokens;
      const uint32_t upto = begin + warp_inclusive_sum(n), last = active + warp_inclusive_sum(entries);
      if (e < experts) s.place[e] = (uint16_t)(upto - n);
      for (uint32_t i = 0; i < entries; ++i) {
        p.expert[last - entries + i] = (uint16_t)e;
        p.begin[last - entries + i] = (uint16_t)(upto - n + i * kTokens);
      }
      active = __shfl_sync(kAll, last, 31);
      begin = __shfl_sync(kAll, upto, 31);
    }
    if (lane == 0) *p.count = active, p.begin[active] = (uint16_t)begin;
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

// Set up beside the last blocks of the kernel before, which lets the next one start
// only when it ends: clusters that start in its middle take the places that come
// free first, unevenly (one token of two experts of 3 x 4,096 x 14,336: 175 us with
// an early start, 142 without any, 131 so; 3 tokens of small experts 19 without, 15
// so).
template <class... P, class... A>
cudaError_t launch_clusters(void (*kernel)(P...), uint32_t clusters, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = clusters * kCluster, cfg.blockDim = kThreads, cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// zc_layer_up.cu, zc_layer_down.cu
cudaError_t layer_up_launch(const LayerArgs& a, int type, bool blocks, cudaStream_t s);
cudaError_t layer_down_launch(const LayerArgs& a, int type, bool blocks, cudaStream_t s);
cudaError_t layer_up_waits(cudaStream_t s, bool* ran_out);
cudaError_t layer_down_waits(cudaStream_t s, bool* ran_out);

}  // namespace zc
