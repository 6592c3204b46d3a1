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
// The choice of experts is made by every cluster of 8 blocks for itself: each block
// takes an eighth of the hidden places for all experts and tokens, the partial
// logits are summed over the cluster's shared memory in one order, and each block
// chooses for its share of the tokens.  A separate kernel would cost a launch, a
// grid-wide wait about the same.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "zc_fp8.cuh"
#include "zc_route.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kCluster = 8, kMaxTokens = ZIPCCL_LAYER_MAX_TOKENS;

struct LayerArgs {
  const void *x, *router, *up, *down, *residual;
  const uint8_t *up_scales, *down_scales;
  void* y;
  float* weights;
  int32_t* ids;
  float* h;
  uint64_t x_stride, up_stride, down_stride;  // in values
  uint32_t tokens, hidden, inner, experts, top_k;
  int activation;
  bool gated, router_float, wide_x, wide_router, wide_up, wide_down, wide_h;
  RouteArgs route;
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The same place of another block's shared memory.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
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

// A float as two of 19 bits: the top ones, and what they leave (0 for infinity and NaN).
__device__ __forceinline__ void parts(float v, float& hi, float& lo) {
  const uint32_t b = __float_as_uint(v);
  hi = __uint_as_float((b & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : b & 0xFFFFE000u);
  lo = (b & 0x7F800000u) == 0x7F800000u ? 0.0f : v - hi;
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

// Places of the sum that a warp takes in a step: 4 lanes, 16 bytes of weights each.
template <class W>
constexpr uint32_t kStep = 4 * kPer16<W>;

// One warp: two rows a lane (gid and gid + 8 of 16) times G groups of 8 vectors,
// over steps s0 .. s1-1 of a sum of n places.  v[j]: the vector of column gid of
// group j, or null.  scale0, scale1: the rows' scales, a byte for 128 places.
// kAhead steps' weights are asked for before the first is used.
template <class W, class X, int G>
__device__ __forceinline__ void accumulate(float (&c)[G][4], const W* row0, const W* row1, const uint8_t* scale0, const uint8_t* scale1,
                                           const X* const (&v)[G], uint32_t groups, uint32_t s0, uint32_t s1, uint32_t n, bool wide_w,
                                           bool wide_x) {
  constexpr int V = kPer16<W>, kAhead = 4;
  constexpr bool kPartsW = std::is_same<W, float>::value, kPartsX = std::is_same<X, float>::value;
  const uint32_t quad = threadIdx.x % 4;
  for (uint32_t s = s0; s < s1; s += kAhead) {
    uint4 w0[kAhead], w1[kAhead];
    float f0[kAhead], f1[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t k = (s + u) * kStep<W> + quad * V;
      const int left = s + u < s1 ? (int)n - (int)k : 0;
      w0[u] = load16<W>(row0 + k, left, wide_w);
      w1[u] = load16<W>(row1 + k, left, wide_w);
      if constexpr (std::is_same<W, F8>::value) {
        f0[u] = left > 0 ? scale_value(__ldg(scale0 + k / kFp8Block)) : 1.0f;
        f1[u] = left > 0 ? scale_value(__ldg(scale1 + k / kFp8Block)) : 1.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u >= s1) break;
      const uint32_t k = (s + u) * kStep<W> + quad * V;
      const int left = (int)n - (int)k;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= (int)groups) break;
        constexpr int N = kPer16<X>;  // the vector's values, 16 bytes at a time
#pragma unroll
        for (int i = 0; i < V; i += N) {
          // (a 16-byte load where the lane's share of the vector has as many)
          const uint4 x = v[g] ? load16<X>(v[g] + k + i, min(left - i, V), wide_x && N <= V) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < (N < V ? N : V) / 2; ++j) {
            float2 p = two_of<W>(w0[u], i / 2 + j), q = two_of<W>(w1[u], i / 2 + j);
            if constexpr (std::is_same<W, F8>::value) {
              p.x *= f0[u], p.y *= f0[u];
              q.x *= f1[u], q.y *= f1[u];
            }
            const float2 b = two_of<X>(x, j);
            float bh0 = b.x, bh1 = b.y, bl0, bl1;
            if constexpr (kPartsX) parts(b.x, bh0, bl0), parts(b.y, bh1, bl1);
            if constexpr (kPartsW) {
              float2 ph, qh, pl, ql;
              parts(p.x, ph.x, pl.x), parts(p.y, ph.y, pl.y), parts(q.x, qh.x, ql.x), parts(q.y, qh.y, ql.y);
              multiply(c[g], pl.x, ql.x, pl.y, ql.y, bh0, bh1);
              p = ph, q = qh;
            }
            if constexpr (kPartsX) multiply(c[g], p.x, q.x, p.y, q.y, bl0, bl1);
            multiply(c[g], p.x, q.x, p.y, q.y, bh0, bh1);
          }
        }
      }
    }
  }
}

// ---- what both kernels know of the pairs: the active experts in order, where each
// one's pairs begin, and each pair's token
struct Pairs {
  uint32_t count;  // active experts
  uint32_t expert[kMaxTokens * kMaxTopK];
  uint32_t begin[kMaxTokens * kMaxTopK + 1];
  uint8_t token[kMaxTokens * kMaxTopK];
  float weight[kMaxTokens * kMaxTopK];
  uint32_t mask[kMaxExperts];   // tokens of each expert
  uint32_t place[kMaxExperts];  // where its pairs begin
};

// From ids and weights [tokens][top_k] in shared memory; ids outside the experts
// take no part.  All threads call it, after a barrier that covers both.
__device__ __forceinline__ void gather_pairs(Pairs& p, const uint32_t* ids, const float* weights, uint32_t tokens, uint32_t top_k,
                                             uint32_t experts) {
  const uint32_t lane = threadIdx.x % 32, pairs = tokens * top_k;
  for (uint32_t e = threadIdx.x; e < experts; e += kThreads) p.mask[e] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < pairs; i += kThreads)
    if (ids[i] < experts) atomicOr(&p.mask[ids[i]], 1u << (i / top_k));
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t active = 0, begin = 0;
    for (uint32_t e0 = 0; e0 < experts; e0 += 32) {
      const uint32_t e = e0 + lane, n = e < experts ? __popc(p.mask[e]) : 0;
      const uint32_t upto = begin + warp_inclusive_sum(n), who = __ballot_sync(kAll, n > 0);
      if (e < experts) p.place[e] = upto - n;
      if (n) {
        const uint32_t a = active + __popc(who & ((1u << lane) - 1));
        p.expert[a] = e;
        p.begin[a] = upto - n;
      }
      active += __popc(who);
      begin = __shfl_sync(kAll, upto, 31);
    }
    if (lane == 0) p.count = active, p.begin[active] = begin;
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < pairs; i += kThreads) {
    const uint32_t e = ids[i], t = i / top_k;
    if (e >= experts) continue;
    const uint32_t at = p.place[e] + __popc(p.mask[e] & ((1u << t) - 1));
    p.token[at] = (uint8_t)t;
    if (weights) p.weight[at] = weights[i];
  }
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

// Dynamic shared memory of the first kernel: partial logits, then rows and keys of
// the block's tokens, then the warps' sums (which may lie over the former).
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
    accumulate<R, T, G>(c, row + (uint64_t)r0 * a.hidden, row + (uint64_t)r1 * a.hidden, nullptr, nullptr, v, groups,
                        steps * part / all, steps * (part + 1) / all, a.hidden, a.wide_router, a.wide_x);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = tile * 16 + gid + (i / 2) * 8, t = g * 8 + quad * 2 + i % 2;
        if (e < a.experts && t < a.tokens) partial[(warp % splits * a.tokens + t) * a.experts + e] = c[g][i];
      }
  }
}

template <class T, class W, int G>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_up_kernel(const __grid_constant__ LayerArgs a) {
  after_previous();
  extern __shared__ __align__(16) float s_dyn[];
  __shared__ Pairs s_pairs;
  __shared__ uint32_t s_ids[kMaxTokens * kMaxTopK];
  __shared__ float s_weights[kMaxTokens * kMaxTopK];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t rank = cluster_rank(), splits = router_splits(a.experts);
  float* partial = s_dyn;
  if (a.router_float) router_logits<float, T, G>(a, partial, rank);
  else router_logits<T, T, G>(a, partial, rank);
  cluster_sync();
  {
    const uint32_t held = (a.experts + 31) / 32 * 32 * 2;
    float* rows = s_dyn + splits * a.tokens * a.experts;
    rows += (4 - (splits * a.tokens * a.experts) % 4) % 4;
    for (uint32_t i = warp; i < kShare; i += kWarps) {
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
          store_cluster(at_rank(s_ids + t * a.top_k + lane, r), (uint32_t)c.id);
          store_cluster(at_rank(s_weights + t * a.top_k + lane, r), __float_as_uint(w));
        }
        if (blockIdx.x < kCluster) {
          a.ids[t * a.top_k + lane] = c.id;
          a.weights[t * a.top_k + lane] = w;
        }
      }
    }
  }
  cluster_sync();  // also: nobody reads this block's shared memory any more
  gather_pairs(s_pairs, s_ids, s_weights, a.tokens, a.top_k, a.experts);
  // 16 rows of an expert at a time: 8 of the gate's and 8 of the other's, so that
  // both of a place come to the same lane; or 16 of the only matrix
  const uint32_t high = a.gated ? 8 : 16, tiles = (a.inner + high - 1) / high, rows = a.gated ? 2 * a.inner : a.inner;
  const uint32_t steps = (a.hidden + kStep<W> - 1) / kStep<W>;
  float4* sums = reinterpret_cast<float4*>(s_dyn);
  uint32_t turn = 0;
  for (uint32_t u = blockIdx.x; u < s_pairs.count * tiles; u += gridDim.x, ++turn) {
    const uint32_t n = u / tiles, i0 = (u - n * tiles) * high, e = s_pairs.expert[n];
    const uint32_t begin = s_pairs.begin[n], tokens = s_pairs.begin[n + 1] - begin, groups = (tokens + 7) / 8;
    const uint32_t r0 = min(i0 + gid, a.inner - 1), r1 = a.gated ? a.inner + r0 : min(i0 + gid + 8, a.inner - 1);
    const T* v[G];
#pragma unroll
    for (int g = 0; g < G; ++g)
      v[g] = g * 8 + gid < tokens ? static_cast<const T*>(a.x) + (uint64_t)s_pairs.token[begin + g * 8 + gid] * a.x_stride : nullptr;
    float c[G][4] = {};
    const W* at = static_cast<const W*>(a.up) + (uint64_t)e * rows * a.up_stride;
    const uint32_t across = (a.hidden + kFp8Block - 1) / kFp8Block;
    const uint8_t* scales = a.up_scales + (uint64_t)e * ((rows + kFp8Block - 1) / kFp8Block) * across;
    accumulate<W, T, G>(c, at + r0 * a.up_stride, at + r1 * a.up_stride, scales + r0 / kFp8Block * across,
                        scales + r1 / kFp8Block * across, v, groups, steps * warp / kWarps, steps * (warp + 1) / kWarps, a.hidden,
                        a.wide_up, a.wide_x);
    float4* mine = sums + (turn % 2 * kWarps) * G * 32;
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < (int)groups) mine[(warp * G + g) * 32 + lane] = make_float4(c[g][0], c[g][1], c[g][2], c[g][3]);
    __syncthreads();
    // the warps add up in turn, while the others go on
    if (warp == turn % kWarps) {
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
          const float w = s_pairs.weight[begin + col];
          float* h = a.h + (uint64_t)(begin + col) * a.inner + i0 + gid;
          if (a.gated) {
            if (i0 + gid < a.inner) h[0] = w * (activate(a.activation, v4[i]) * v4[2 + i]);
          } else {
            if (i0 + gid < a.inner) h[0] = w * activate(a.activation, v4[i]);
            if (i0 + gid + 8 < a.inner) h[8] = w * activate(a.activation, v4[2 + i]);
          }
        }
      }
    }
  }
}

// 16 hidden places at a time; the active experts' inner places, one expert after
// the other, are dealt out to the cluster's 64 warps in equal runs.  A warp adds
// what an expert gives to its tokens' sums in shared memory; a block adds its
// warps', and after 8 tiles each block of the cluster all blocks' of one of them.
template <class T, class W, int G>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_down_kernel(const __grid_constant__ LayerArgs a) {
  after_previous();
  extern __shared__ __align__(16) float s_dyn[];
  __shared__ Pairs s_pairs;
  __shared__ uint32_t s_ids[kMaxTokens * kMaxTopK];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t rank = cluster_rank(), cluster = blockIdx.x / kCluster, clusters = gridDim.x / kCluster;
  for (uint32_t i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads) s_ids[i] = (uint32_t)a.ids[i];
  __syncthreads();
  gather_pairs(s_pairs, s_ids, nullptr, a.tokens, a.top_k, a.experts);
  const uint32_t size = a.tokens * 16;        // of a tile: [token][place]
  float* own = s_dyn + warp * size;           // a warp's sums
  float* block = s_dyn + kWarps * size;       // a block's, of up to 8 tiles
  const uint32_t steps = (a.inner + kStep<W> - 1) / kStep<W>, part = rank * kWarps + warp;
  const uint64_t all = (uint64_t)steps * s_pairs.count;
  const uint64_t from = all * part / (kCluster * kWarps), upto = all * (part + 1) / (kCluster * kWarps);
  const uint32_t tiles = (a.hidden + 15) / 16, across = (a.inner + kFp8Block - 1) / kFp8Block;
  for (uint32_t t0 = cluster; t0 < tiles; t0 += clusters * kCluster) {
    for (uint32_t j = 0; j < kCluster; ++j) {
      const uint32_t tile = t0 + j * clusters;
      if (tile >= tiles) break;
      for (uint32_t i = lane; i < size; i += 32) own[i] = 0.0f;
      __syncwarp();
      const uint32_t r0 = min(tile * 16 + gid, a.hidden - 1), r1 = min(tile * 16 + gid + 8, a.hidden - 1);
      for (uint64_t s = from; s < upto;) {
        const uint32_t n = (uint32_t)(s / steps), first = (uint32_t)(s - (uint64_t)n * steps);
        const uint32_t last = (uint32_t)min((uint64_t)steps, first + (upto - s));
        s += last - first;
        const uint32_t begin = s_pairs.begin[n], tokens = s_pairs.begin[n + 1] - begin, groups = (tokens + 7) / 8;
        const float* v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) v[g] = g * 8 + gid < tokens ? a.h + (uint64_t)(begin + g * 8 + gid) * a.inner : nullptr;
        float c[G][4] = {};
        const W* at = static_cast<const W*>(a.down) + (uint64_t)s_pairs.expert[n] * a.hidden * a.down_stride;
        const uint8_t* scales = a.down_scales + (uint64_t)s_pairs.expert[n] * ((a.hidden + kFp8Block - 1) / kFp8Block) * across;
        accumulate<W, float, G>(c, at + r0 * a.down_stride, at + r1 * a.down_stride, scales + r0 / kFp8Block * across,
                                scales + r1 / kFp8Block * across, v, groups, first, last, a.inner, a.wide_down, a.wide_h);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t col = g * 8 + quad * 2 + i % 2;
            if (col < tokens) own[s_pairs.token[begin + col] * 16 + gid + (i / 2) * 8] += c[g][i];
          }
        __syncwarp();
      }
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
        float sum = s_dyn[i];
        for (int w = 1; w < kWarps; ++w) sum += s_dyn[w * size + i];
        block[j * size + i] = sum;
      }
      __syncthreads();
    }
    cluster_sync();
    const uint32_t tile = t0 + rank * clusters;
    if (tile < tiles)
      for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
        const uint32_t t = i / 16, place = tile * 16 + i % 16;
        if (place >= a.hidden) continue;
        float sum = a.residual ? to_float(static_cast<const T*>(a.residual)[(uint64_t)t * a.hidden + place]) : 0.0f;
        for (uint32_t r = 0; r < kCluster; ++r) sum += load_cluster(at_rank(block + rank * size + i, r));
        static_cast<T*>(a.y)[(uint64_t)t * a.hidden + place] = from_float<T>(sum);
      }
    cluster_sync();
  }
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

template <class... P, class... A>
cudaError_t launch_clusters(void (*kernel)(P...), uint32_t clusters, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kCluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = clusters * kCluster, cfg.blockDim = kThreads, cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

size_t up_smem(uint32_t tokens, uint32_t experts, int groups) {
  const size_t logits = 4ull * (router_splits(experts) * tokens * experts + 4 + kShare * ((experts + 31) / 32 * 64 + 1024));
  return std::max<size_t>(logits, 2ull * kWarps * groups * 512);
}
size_t down_smem(uint32_t tokens) { return 4ull * (kWarps + kCluster) * tokens * 16; }

template <class T, class W, int G>
cudaError_t layer_launch(const LayerArgs& a, cudaStream_t s) {
  static std::atomic<int> up_known[kMaxDevices], down_known[kMaxDevices];
  const size_t up = up_smem(a.tokens, a.experts, G), down = down_smem(a.tokens);
  int up_clusters = 0, down_clusters = 0;
  cudaError_t e = clusters_at_once(zc_layer_up_kernel<T, W, G>, up_known, 2 * kWarps * G * 512, up_smem(kMaxTokens, kMaxExperts, G), &up_clusters);
  if (e == cudaSuccess) e = clusters_at_once(zc_layer_down_kernel<T, W, G>, down_known, down_smem(8 * G), down_smem(kMaxTokens), &down_clusters);
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
}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_layer_workspace_bytes(uint64_t tokens, uint32_t top_k, uint64_t inner, uint64_t* out_bytes) {
  if (!out_bytes || tokens > kMaxTokens || top_k == 0 || top_k > kMaxTopK || inner >= (1ull << 22)) return ZIPCCL_ERR_INVALID_ARG;
  *out_bytes = (tokens * top_k * inner * 4 + 255) / 256 * 256;
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
  a.h = static_cast<float*>(d_ws);
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
  a.wide_h = l->inner % 4 == 0;
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
