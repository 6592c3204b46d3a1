// zc_route.cu -- routing of tokens to experts, its gradient, and the plan of
// the experts' chunks (counts, offsets and the row of every token-expert
// pair).
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopK = 32;
constexpr uint32_t kMaxGroups = 32;
constexpr int kRouteThreads = 256;

struct RouteArgs {
  const void* logits;
  const float* bias;     // nullable
  const uint8_t* mask;   // nullable: 0 leaves the token out
  const float* grad;     // backward: gradient of the weights
  float* weights;
  int32_t* ids;          // written forward, read backward
  void* grad_logits;
  uint64_t stride;       // values between rows
  uint32_t tokens, experts, top_k, groups, kept, group_size;
  float scale;
  uint32_t group_lanes;  // lanes of a group where groups are whole lanes, a power of two of them; else 0
  bool softmax, renormalize, top2, wide, wide_out, wide_bias;
};

// Over the L lanes of a token, which are consecutive in a warp.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (L == 32) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
  } else {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// The first of the token's lanes that the condition holds for; one does.
template <int L>
__device__ __forceinline__ uint32_t first_lane(bool x) {
  uint32_t who = __ballot_sync(kAll, x);
  if constexpr (L < 32) who = who >> ((threadIdx.x & 31) / L * L) & ((1u << L) - 1);
  return __ffs(who) - 1;
}

// Reciprocal of a number from 1 to 2: the hardware's approximation (1 ulp) and a
// step of Newton's iteration, y + y (1 - x y), which squares its error: half a
// unit in the last place is left.  Four instructions; an IEEE division has 10
// for the cases that do not come up here (8,192 tokens of 256 sigmoids: 8.7 us
// with it, 8.1 like this, 7.9 with the approximation alone).
__device__ __forceinline__ float rcp_1_to_2(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return fmaf(y, fmaf(-x, y, 1.0f), y);
}
// 1 / (1 + e^-l), below 0 as e^l / (1 + e^l): neither overflows, so scores keep
// their value and order down to the smallest float (l = -103).
__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l));
  return (l < 0.0f ? e : 1.0f) * rcp_1_to_2(1.0f + e);
}

// V values of a row from place e0 on; -inf where the row has ended.  `wide`:
// every row starts and ends at a multiple of 16 bytes.
template <class T, int V>
__device__ __forceinline__ void load_logits(const T* row, uint32_t e0, uint32_t experts, bool wide, float (&l)[V]) {
  constexpr int N = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
#pragma unroll
  for (int j = 0; j < V; j += N) {
    if (wide) {
      Pack<T, N> p;
      const bool in = e0 + j < experts;
      if (in) p = *reinterpret_cast<const Pack<T, N>*>(row + e0 + j);
#pragma unroll
      for (int i = 0; i < N; ++i) l[j + i] = in ? to_float(p.v[i]) : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) l[j + i] = e0 + j + i < experts ? to_float(row[e0 + j + i]) : -INFINITY;
    }
  }
}

// Scores of V logits: the softmax over the whole row, or sigmoids.  A logit
// that is -inf or NaN becomes -inf and takes no part, +inf the largest float.
template <int V>
__device__ __forceinline__ void settle(float (&l)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = fminf(fmaxf(l[j], -INFINITY), FLT_MAX);  // a maximum leaves NaN out
}
template <int L, int V>
__device__ __forceinline__ void softmax(const float (&l)[V], float (&s)[V], float* top, float* sum) {
  float m = l[0], z = 0.0f;
#pragma unroll
  for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
  m = lanes_max<L>(m);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    s[j] = l[j] > -INFINITY ? expf(l[j] - m) : 0.0f;
    z += s[j];
  }
  z = lanes_sum<L>(z);
  const float inv = z > 0.0f ? 1.0f / z : 0.0f;  // 0: no eligible expert
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] *= inv;
  *top = m;
  *sum = inv;
}

// Leaves the choice scores of a token's kept groups and makes the others
// -inf.  Groups are 2^n whole lanes, or of any size through shared memory: a
// lane then scans a group alone (8,192 tokens of 160 experts in 8 groups of 20:
// 10.0 us, 998 instructions a token; 128 in 8 of 16: 7.1 and 622).
template <int L, int V>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, float (&c)[V], float* shared, uint32_t lane) {
  float hi = -INFINITY, lo = -INFINITY;
  const uint32_t stride = a.group_lanes ? a.group_lanes : 1;  // lanes from a group's score to the next's
  if (a.group_lanes) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      lo = fmaxf(lo, fminf(hi, c[j]));
      hi = fmaxf(hi, c[j]);
    }
    for (uint32_t o = 1; o < stride; o <<= 1) {
      const float h = __shfl_xor_sync(kAll, hi, o), l = __shfl_xor_sync(kAll, lo, o);
      lo = fmaxf(fminf(hi, h), fmaxf(lo, l));
      hi = fmaxf(hi, h);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) shared[lane * V + j] = c[j];
    __syncwarp();
    if (lane < a.groups)
      for (uint32_t i = 0; i < a.group_size; ++i) {
        const float x = shared[lane * a.group_size + i];
        lo = fmaxf(lo, fminf(hi, x));
        hi = fmaxf(hi, x);
      }
    __syncwarp();
  }
  // a group is kept if fewer than `kept` groups come before it; equal: the
  // lower first.  The lanes of a group share the others
  const float mine = (a.top2 && lo > -INFINITY ? hi + lo : hi) + 0.0f;
  const uint32_t g = lane / stride;
  uint32_t before = 0;
  for (uint32_t h0 = 0; h0 < a.groups; h0 += stride) {
    const uint32_t h = h0 + lane % stride;
    const float y = __shfl_sync(kAll, mine, min(h * stride, (uint32_t)L - 1), L);
    before += h < a.groups && (y > mine || (y == mine && h < g));
  }
  for (uint32_t o = 1; o < stride; o <<= 1) before += __shfl_xor_sync(kAll, before, o);
  const bool kept = g < a.groups && before < a.kept;
  if (a.group_lanes) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (!kept) c[j] = -INFINITY;
    return;
  }
  const uint32_t keep = __ballot_sync(kAll, kept) >> ((threadIdx.x & 31) / L * L);
  uint32_t e = lane * V / a.group_size, r = lane * V - e * a.group_size;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (e < a.groups && !(keep >> e & 1)) c[j] = -INFINITY;
    if (++r == a.group_size) r = 0, ++e;
  }
}

// L lanes take a token, V consecutive experts each.  The choice scores lie in
// shared memory; each lane knows the best of its own, and top_k times the
// lanes find the best of these, its place among the V of its lane (the lowest
// place of the lowest lane is the lowest expert among equals), and what is
// then best in that lane: no step is one lane's alone, but for the scan of
// groups that are not whole lanes.
// For few tokens it takes a launch (2.4 us); for many its instructions bound
// it: of 256 experts in 8 groups, 8 chosen, a token takes 795, 29 of them for
// each chosen expert, about 145 each for the groups and the sigmoids (8,192
// tokens: 8.1 us).
template <class T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) zc_route_kernel(RouteArgs a) {
  static_assert(V <= L, "a lane's experts are scanned by one lane each");
  after_previous();
  constexpr uint32_t kTok = kRouteThreads / L;
  __shared__ __align__(16) float s_key[kTok][L * V];
  const uint32_t lane = threadIdx.x % L;
  const uint32_t tok = blockIdx.x * kTok + threadIdx.x / L;
  const bool in = tok < a.tokens;
  const T* row = static_cast<const T*>(a.logits) + (in ? tok : 0) * a.stride;
  const uint32_t e0 = lane * V;
  float* keys = s_key[threadIdx.x / L];
  float top = 0.0f, inv = 0.0f;
  int32_t id = -1;  // of pair `lane`
  float l[V], c[V];
  load_logits<T, V>(row, e0, a.experts, a.wide, l);
  if (!in || (a.mask && !a.mask[tok])) {
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = -INFINITY;
  }
  settle(l);
  // either score grows with the logit: where nothing is added to it, the logits
  // choose, and two that score alike in 32 bits (sigmoids are 1 from 17 on) are told apart
  const bool by_logit = !a.bias && (a.groups == 1 || !a.top2);
  if (a.softmax && (!by_logit || !a.renormalize)) softmax<L, V>(l, c, &top, &inv);
  if (!a.softmax && !by_logit) {
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = sigmoid(l[j]);
  }
  if (by_logit) {
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = l[j];
  } else {
    if (a.bias) {
      float b[V];
      load_logits<float, V>(a.bias, e0, a.experts, a.wide_bias, b);
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] += b[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      c[j] = l[j] > -INFINITY ? fmaxf(c[j], -INFINITY) : -INFINITY;
  }
  if (a.groups > 1) keep_groups<L, V>(a, c, keys, lane);
  float best = c[0];
#pragma unroll
  for (int j = 1; j < V; ++j) best = fmaxf(best, c[j]);
  constexpr int K = V < 4 ? V : 4;  // stored four at a time: single ones would meet in the same banks
#pragma unroll
  for (int j = 0; j < V; j += K) {
    Pack<float, K> p;
#pragma unroll
    for (int i = 0; i < K; ++i) p.v[i] = c[j + i];
    *reinterpret_cast<Pack<float, K>*>(keys + e0 + j) = p;
  }
  for (uint32_t k = 0; k < a.top_k; ++k) {
    __syncwarp();
    const float m = lanes_max<L>(best);
    const uint32_t from = first_lane<L>(best == m);
    const float x = lane < V ? keys[from * V + lane] : -INFINITY;
    const uint32_t j = first_lane<L>(lane < V && x == m);
    if (lane == j) keys[from * V + j] = -INFINITY;
    const float left = lanes_max<L>(lane == j ? -INFINITY : x);
    if (lane == from) best = left;
    if (lane == k && m > -INFINITY) id = from * V + j;
  }
  // lane k has pair k
  float s = 0.0f;
  if (id >= 0) {
    s = fminf(to_float(row[id]), FLT_MAX);
    if (!a.softmax) s = sigmoid(s);
  }
  if (a.softmax) {
    if (a.renormalize) top = lanes_max<L>(id >= 0 ? s : -INFINITY);
    s = id >= 0 ? expf(s - top) : 0.0f;
  }
  if (a.renormalize) {  // a division: a single pair's weight is 1 where its score is not 0, and its gradient 0
    const float all = lanes_sum<L>(s);
    s = all > 0.0f ? s / all : 0.0f;
  } else if (a.softmax) {
    s *= inv;
  }
  if (in && lane < a.top_k) {
    a.weights[(uint64_t)tok * a.top_k + lane] = s * a.scale;
    a.ids[(uint64_t)tok * a.top_k + lane] = id;
  }
}

// Gradient of the weights carried to the logits.  With w the weights before
// the scale and d the incoming gradient times the scale, s_k dw/ds_k sums to
// u_k = w_k (d_k - sum_j w_j d_j) when renormalised and u_k = s_k d_k when
// not; then dl_e = u_e - s_e sum u (softmax; the sum is 0 when renormalised)
// or u_e (1 - s_e) (sigmoid).  Only the softmax without renormalisation has
// to read the whole row again.  A lane has a pair first, then V experts.
template <class T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) zc_route_backward_kernel(RouteArgs a) {
  after_previous();
  constexpr uint32_t kTok = kRouteThreads / L;
  __shared__ __align__(16) float s_row[kTok][L * V];
  const uint32_t lane = threadIdx.x % L;
  const uint32_t tok = blockIdx.x * kTok + threadIdx.x / L;
  const bool in = tok < a.tokens;
  const T* row = static_cast<const T*>(a.logits) + (in ? tok : 0) * a.stride;
  float* grads = s_row[threadIdx.x / L];
  const uint32_t e0 = lane * V;
  const bool whole = a.softmax && !a.renormalize;
  int32_t id = in && lane < a.top_k ? a.ids[(uint64_t)tok * a.top_k + lane] : -1;
  if ((uint32_t)id >= a.experts) id = -1;
  float d = 0.0f, s = 0.0f;
  if (id >= 0) {
    d = a.grad[(uint64_t)tok * a.top_k + lane] * a.scale;
    s = fminf(to_float(row[id]), FLT_MAX);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) grads[e0 + j] = 0.0f;
  float p[V], top = 0.0f, inv = 0.0f;
  if (whole) {
    float l[V];
    load_logits<T, V>(row, e0, a.experts, a.wide, l);
    settle(l);
    softmax<L, V>(l, p, &top, &inv);
  }
  if (a.softmax) {
    if (a.renormalize) top = lanes_max<L>(id >= 0 ? s : -INFINITY);
    s = id >= 0 ? expf(s - top) : 0.0f;
    if (whole) s *= inv;
  } else if (id >= 0) {
    s = sigmoid(s);
  }
  float u = s * d;
  if (a.renormalize) {
    const float all = lanes_sum<L>(s), w = all > 0.0f ? s / all : 0.0f;
    u = w * (d - lanes_sum<L>(w * d));
  }
  const float total = whole ? lanes_sum<L>(u) : 0.0f;
  if (!a.softmax) u *= 1.0f - s;
  __syncwarp();
  if (id >= 0) atomicAdd(&grads[id], u);  // a token's ids are distinct: one add each
  __syncwarp();
  if (!in) return;
  T* out = static_cast<T*>(a.grad_logits) + (uint64_t)tok * a.experts;
  constexpr int N = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
#pragma unroll
  for (int j = 0; j < V; j += N) {
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      g[i] = grads[e0 + j + i];
      if (whole) g[i] -= p[j + i] * total;
    }
    if (a.wide_out) {
      if (e0 + j < a.experts) *reinterpret_cast<Pack<T, N>*>(out + e0 + j) = rounded<T, N>(g);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + j + i < a.experts) out[e0 + j + i] = from_float<T>(g[i]);
    }
  }
}

template <class T, int L, int V>
cudaError_t route_launch(RouteArgs a, bool backward, cudaStream_t s) {
  constexpr uint32_t kTok = kRouteThreads / L, N = 16 / sizeof(T) < V ? 16 / sizeof(T) : V, B = V < 4 ? V : 4;
  // accesses of N values: rows of a multiple of N, from an aligned start
  a.wide = host_aligned(a.logits, N * sizeof(T)) && a.stride % N == 0 && a.experts % N == 0;
  a.wide_out = host_aligned(a.grad_logits, N * sizeof(T)) && a.experts % N == 0;
  a.wide_bias = host_aligned(a.bias, B * sizeof(float)) && a.experts % B == 0;
  const uint32_t lanes = a.group_size % V ? 0 : a.group_size / V;
  a.group_lanes = lanes & (lanes - 1) || a.groups > L ? 0 : lanes;
  const uint32_t grid = (a.tokens + kTok - 1) / kTok;
  return launch(backward ? zc_route_backward_kernel<T, L, V> : zc_route_kernel<T, L, V>, grid, kRouteThreads, 0, s, a);
}

// A warp takes a token; 8 lanes do where they hold its experts, 8 each, its
// pairs and its groups: 16,384 tokens of 64 experts, two chosen, 3.4 us against
// 5.6 with 32 lanes, one token 2.6 against 2.3.  (Between 65 and 128 experts 16
// lanes made no difference, nor did they up to 256.)
template <class T>
cudaError_t route_by_experts(const RouteArgs& a, bool backward, cudaStream_t s) {
  const uint32_t e = a.experts;
  if (e <= 64 && a.top_k <= 8 && a.groups <= 8) return route_launch<T, 8, 8>(a, backward, s);
  if (e <= 64) return route_launch<T, 32, 2>(a, backward, s);
  if (e <= 128) return route_launch<T, 32, 4>(a, backward, s);
  if (e <= 256) return route_launch<T, 32, 8>(a, backward, s);
  if (e <= 512) return route_launch<T, 32, 16>(a, backward, s);
  return route_launch<T, 32, 32>(a, backward, s);
}

zipccl_status route(RouteArgs& a, int type, const zipccl_route_options* o, uint64_t tokens, uint32_t experts,
                    bool backward, void* stream) {
  const uint32_t z = type_bytes(type);
  if (!o || z == 0 || experts == 0 || experts > kMaxExperts || a.stride < experts) return ZIPCCL_ERR_INVALID_ARG;
  if (o->top_k == 0 || o->top_k > kMaxTopK || o->top_k > experts) return ZIPCCL_ERR_INVALID_ARG;
  if (o->score != ZIPCCL_SCORE_SOFTMAX && o->score != ZIPCCL_SCORE_SIGMOID) return ZIPCCL_ERR_INVALID_ARG;
  if (o->group_score != ZIPCCL_GROUP_MAX && o->group_score != ZIPCCL_GROUP_TOP2) return ZIPCCL_ERR_INVALID_ARG;
  if (o->groups == 0 || o->groups > kMaxGroups || experts % o->groups || o->groups_kept == 0 ||
      o->groups_kept > o->groups || o->top_k > o->groups_kept * (experts / o->groups) || !isfinite(o->scale))
    return ZIPCCL_ERR_INVALID_ARG;
  if (tokens >= (1ull << 31) || tokens * o->top_k >= (1ull << 31)) return ZIPCCL_ERR_INVALID_ARG;
  if (tokens == 0) return ZIPCCL_OK;
  if (!a.logits || !a.ids || !host_aligned(a.logits, z) || !host_aligned(a.ids, 4) || !host_aligned(a.bias, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  if (backward ? !a.grad || !a.grad_logits || !host_aligned(a.grad, 4) || !host_aligned(a.grad_logits, z)
               : !a.weights || !host_aligned(a.weights, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  a.tokens = (uint32_t)tokens;
  a.experts = experts;
  a.top_k = o->top_k;
  a.groups = o->groups;
  a.kept = o->groups_kept;
  a.group_size = experts / o->groups;
  a.scale = o->scale;
  a.softmax = o->score == ZIPCCL_SCORE_SOFTMAX;
  a.renormalize = o->renormalize != 0;
  a.top2 = o->group_score == ZIPCCL_GROUP_TOP2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == ZIPCCL_TYPE_F32    ? route_by_experts<float>(a, backward, s)
                        : type == ZIPCCL_TYPE_BF16 ? route_by_experts<__nv_bfloat16>(a, backward, s)
                                                   : route_by_experts<__half>(a, backward, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

// ------------------------------------------------------------------ plan
// A stable counting sort of the pairs by expert.  A block takes a run of
// consecutive pairs, a warp of it a run of these.  With more than one block a
// first kernel leaves the counts of every kPlanGroup blocks in the workspace;
// the second starts beside it, counts its warps' runs and those of the blocks
// before it in its group meanwhile, and then adds up, for each bucket, the
// pairs of the groups before and of all.  524,288 pairs of 256 experts: 9.5 us
// for both, most of it the chain launch, count, read, place (24 us with a row
// of counts for every block, of which each block read 131 KB).
constexpr uint32_t kPlanRun = 2048;    // pairs of a block, or more where that makes
constexpr uint32_t kPlanBlocks = 128;  // more blocks than this
constexpr uint32_t kPlanGroup = 4;
constexpr int kCountThreads = 1024;
constexpr int kPlaceThreads = 1024;

struct PlanArgs {
  const int32_t* ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* slots;
  uint32_t* group_counts;  // [groups][experts + 1]
  uint32_t pairs, experts, blocks, run;
};

// A pair that is not routed (id outside 0..experts-1) counts for one more
// bucket after the experts.
__device__ __forceinline__ uint32_t plan_key(int32_t id, uint32_t experts) { return min((uint32_t)id, experts); }

__global__ void __launch_bounds__(kCountThreads) zc_plan_count_kernel(PlanArgs a) {
  __shared__ uint32_t h[kMaxExperts + 1];
  after_previous();  // from here on the placing kernel may start: it waits for this one where it needs the counts
  for (uint32_t e = threadIdx.x; e <= a.experts; e += kCountThreads) h[e] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * kPlanGroup * a.run, hi = min(lo + kPlanGroup * a.run, a.pairs);
#pragma unroll 8
  for (uint32_t i = lo + threadIdx.x; i < hi; i += kCountThreads) atomicAdd(&h[plan_key(a.ids[i], a.experts)], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= a.experts; e += kCountThreads)
    a.group_counts[blockIdx.x * (a.experts + 1) + e] = h[e];
}

__global__ void __launch_bounds__(kPlaceThreads) zc_plan_place_kernel(PlanArgs a) {
  constexpr int kThreads = kPlaceThreads, kWarps = kThreads / 32;
  if (a.blocks == 1) after_previous();
  extern __shared__ uint32_t h[];  // [kWarps][nb] counts, then places, by warp; [nb] totals, then starts; [nb] places
  const uint32_t nb = a.experts + 1;
  uint32_t *start = h + kWarps * nb, *base = start + nb;
  __shared__ uint32_t s_scan[kWarps];
  const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (uint32_t i = threadIdx.x; i < (kWarps + 2) * nb; i += kThreads) h[i] = 0;
  __syncthreads();
  const uint32_t per = a.run / kWarps;  // a multiple of 32
  const uint32_t lo = blockIdx.x * a.run + w * per;
  const uint32_t hi = max(lo, min(lo + per, min((blockIdx.x + 1) * a.run, a.pairs)));
  uint32_t* mine = h + w * nb;
#pragma unroll 2
  for (uint32_t i = lo + lane; i < hi; i += 32) atomicAdd(&mine[plan_key(a.ids[i], a.experts)], 1u);
  if (a.blocks > 1) {
    const uint32_t group = blockIdx.x / kPlanGroup;
#pragma unroll 4
    for (uint32_t i = group * kPlanGroup * a.run + threadIdx.x; i < blockIdx.x * a.run; i += kThreads)
      atomicAdd(&base[plan_key(a.ids[i], a.experts)], 1u);
    after_previous();  // the counting kernel; what came before it had ended when it let this one start
    // the threads of a bucket share the groups
    const uint32_t groups = (a.blocks + kPlanGroup - 1) / kPlanGroup;
    const uint32_t wide = (nb + 31) / 32 * 32, parts = max(1u, (uint32_t)kThreads / wide), part = threadIdx.x / wide;
    for (uint32_t e = threadIdx.x - part * wide; e < nb && part < parts; e += kThreads) {
      const uint32_t* c = a.group_counts + e;
      uint32_t before = 0, all = 0;
#pragma unroll 8
      for (uint32_t b = part; b < groups; b += parts) {
        const uint32_t n = c[b * nb];
        all += n;
        if (b < group) before += n;
      }
      atomicAdd(&start[e], all);
      atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < nb; e += kThreads) {
    uint32_t n[kWarps], at = base[e];
#pragma unroll
    for (int v = 0; v < kWarps; ++v) n[v] = h[v * nb + e];
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      h[v * nb + e] = at;
      at += n[v];
    }
    if (a.blocks == 1) start[e] = at;
  }
  __syncthreads();
  // starts: exclusive scan of the totals, kThreads buckets at a time
  uint32_t carry = 0;
  for (uint32_t e0 = 0; e0 < nb; e0 += kThreads) {
    const uint32_t e = e0 + threadIdx.x;
    const uint32_t n = e < nb ? start[e] : 0;
    uint32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[w] = x;
    __syncthreads();
    const uint32_t part = lane < kWarps ? s_scan[lane] : 0;
    const uint32_t first = carry + __reduce_add_sync(kAll, lane < w ? part : 0) + x - n;
    if (e < nb) {
      start[e] = first;
      if (blockIdx.x == 0) {
        a.offsets[e] = (int32_t)first;
        if (e < a.experts) a.counts[e] = (int32_t)n;
      }
    }
    carry += __reduce_add_sync(kAll, part);
    __syncthreads();
  }
  // places in order: 32 pairs at a time, equal buckets ranked by lane.  Lanes
  // of the same bucket are found bit by bit of its number
  const uint32_t bits = 32 - __clz(nb);
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    const uint32_t key = i < hi ? plan_key(a.ids[i], a.experts) : nb;
    uint32_t same = kAll;
#pragma unroll 4
    for (uint32_t b = 0; b < bits; ++b) {
      const uint32_t one = 0u - (key >> b & 1);
      same &= __ballot_sync(kAll, one) ^ ~one;
    }
    const uint32_t rank = __popc(same & ((1u << lane) - 1));
    uint32_t at = 0;
    if (key < nb) at = start[key] + mine[key] + rank;
    __syncwarp();
    if (key < nb && rank == 0) mine[key] += __popc(same);
    __syncwarp();
    if (i < hi) a.slots[i] = key < a.experts ? (int32_t)at : ~(int32_t)at;
  }
}

// Blocks and their runs: whole warps of 32 pairs for 32 warps.
void plan_split(uint64_t pairs, uint32_t* blocks, uint32_t* run) {
  uint64_t r = (pairs + kPlanBlocks - 1) / kPlanBlocks;
  r = r < kPlanRun ? kPlanRun : (r + 1023) / 1024 * 1024;
  *run = (uint32_t)r;
  *blocks = pairs ? (uint32_t)((pairs + r - 1) / r) : 1;
}

size_t plan_smem(uint32_t experts) { return (kPlaceThreads / 32 + 2) * (experts + 1) * sizeof(uint32_t); }

// Allows the placing kernel the 139 KB that 1,024 experts take, once for each
// device: the limit is the kernel's, shared by every thread's calls, so no call
// sets it to its own need, nor finds it below that.
cudaError_t plan_allow_smem() {
  static std::atomic<bool> allowed[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(zc_plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kMaxExperts));
  if (e == cudaSuccess) allowed[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace
}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_route(const void* d_logits, int type, uint64_t row_stride, uint64_t tokens, uint32_t experts,
                               const zipccl_route_options* options, const float* d_bias, const uint8_t* d_mask,
                               float* d_weights, int32_t* d_ids, void* stream) {
  RouteArgs a{};
  a.logits = d_logits;
  a.stride = row_stride;
  a.bias = d_bias;
  a.mask = d_mask;
  a.weights = d_weights;
  a.ids = d_ids;
  return route(a, type, options, tokens, experts, false, stream);
}

zipccl_status zipccl_moe_route_backward(const float* d_grad_weights, const void* d_logits, int type,
                                        uint64_t row_stride, uint64_t tokens, uint32_t experts,
                                        const zipccl_route_options* options, const int32_t* d_ids,
                                        void* d_grad_logits, void* stream) {
  RouteArgs a{};
  a.logits = d_logits;
  a.stride = row_stride;
  a.grad = d_grad_weights;
  a.ids = const_cast<int32_t*>(d_ids);
  a.grad_logits = d_grad_logits;
  return route(a, type, options, tokens, experts, true, stream);
}

zipccl_status zipccl_moe_plan_workspace_bytes(uint64_t pairs, uint32_t experts, uint64_t* out_bytes) {
  if (!out_bytes || pairs >= (1ull << 31) || experts == 0 || experts > kMaxExperts) return ZIPCCL_ERR_INVALID_ARG;
  uint32_t blocks, run;
  plan_split(pairs, &blocks, &run);
  *out_bytes = blocks > 1 ? 4ull * ((blocks + kPlanGroup - 1) / kPlanGroup) * (experts + 1) : 0;
  return ZIPCCL_OK;
}

zipccl_status zipccl_moe_plan(const int32_t* d_ids, uint64_t pairs, uint32_t experts, int32_t* d_counts,
                              int32_t* d_offsets, int32_t* d_slots, void* d_ws, uint64_t ws_bytes, void* stream) {
  uint64_t need = 0;
  const zipccl_status st = zipccl_moe_plan_workspace_bytes(pairs, experts, &need);
  if (st != ZIPCCL_OK) return st;
  if (!d_counts || !d_offsets || !host_aligned(d_counts, 4) || !host_aligned(d_offsets, 4)) return ZIPCCL_ERR_INVALID_ARG;
  if (pairs && (!d_ids || !d_slots || !host_aligned(d_ids, 4) || !host_aligned(d_slots, 4)))
    return ZIPCCL_ERR_INVALID_ARG;
  if (need && (!d_ws || !host_aligned(d_ws, 256))) return ZIPCCL_ERR_INVALID_ARG;
  if (ws_bytes < need) return ZIPCCL_ERR_CAPACITY;
  PlanArgs a;
  a.ids = d_ids;
  a.counts = d_counts;
  a.offsets = d_offsets;
  a.slots = d_slots;
  a.group_counts = static_cast<uint32_t*>(d_ws);
  a.pairs = (uint32_t)pairs;
  a.experts = experts;
  plan_split(pairs, &a.blocks, &a.run);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = plan_smem(experts);
  cudaError_t e = smem > 48000 ? plan_allow_smem() : cudaSuccess;
  if (e == cudaSuccess && a.blocks > 1)
    e = launch(zc_plan_count_kernel, (a.blocks + kPlanGroup - 1) / kPlanGroup, kCountThreads, 0, s, a);
  if (e == cudaSuccess) e = launch(zc_plan_place_kernel, a.blocks, kPlaceThreads, smem, s, a);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // extern "C"
