// zc_route.cu -- routing of tokens to experts, its gradient, and the plan of
// the experts' chunks (counts, offsets and the row of every token-expert
// pair).
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopK = 32;
constexpr uint32_t kMaxGroups = 32;
constexpr int kRouteThreads = 128;

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
  bool softmax, renormalize, top2;
};

// Order-preserving bits of a choice score; 0 stands for "cannot be chosen"
// (-inf and NaN map to it).  -0 counts as +0, so that the two tie.
__device__ __forceinline__ uint32_t order_bits(float c) {
  if (!(c > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(c + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int L>
__device__ __forceinline__ float seg_max(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t seg_max_bits(uint32_t v) {
  if (L == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// L lanes hold a token, V consecutive experts each.
template <class T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) zc_route_kernel(RouteArgs a) {
  constexpr int kTok = kRouteThreads / L;
  __shared__ float s_val[kTok][L * V + 1];  // choice scores, for the groups
  __shared__ float s_group[kTok][kMaxGroups];
  __shared__ float s_pick[kTok][kMaxTopK];
  __shared__ int32_t s_id[kTok][kMaxTopK];
  const int lane = threadIdx.x % L, t = threadIdx.x / L;
  const uint64_t tok = (uint64_t)blockIdx.x * kTok + t;
  const bool live = tok < a.tokens && (!a.mask || a.mask[tok]);
  const T* row = static_cast<const T*>(a.logits) + (tok < a.tokens ? tok : 0) * a.stride;
  const uint32_t e0 = lane * V;

  float l[V];
  uint32_t fit = 0;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = live && e0 + j < a.experts ? to_float(row[e0 + j]) : -INFINITY;
    if (x > -INFINITY) fit |= 1u << j;
    l[j] = x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY;
    top = fmaxf(top, l[j]);
  }
  const bool by_logit = a.softmax && !a.bias && (a.groups == 1 || !a.top2);
  float s[V];
  if (a.softmax) {
    if (!by_logit || !a.renormalize) {
      top = seg_max<L>(top);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = (fit >> j & 1) ? expf(l[j] - top) : 0.0f;
        sum += s[j];
      }
      sum = seg_sum<L>(sum);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = s[j] / sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 1.0f / (1.0f + expf(-l[j]));
  }
  float c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    c[j] = by_logit ? l[j] : s[j];
    if (a.bias && e0 + j < a.experts) c[j] += a.bias[e0 + j];
    if (!(fit >> j & 1) || !(c[j] > -INFINITY)) c[j] = -INFINITY;
  }
  if (a.groups > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) s_val[t][e0 + j] = c[j];
    __syncwarp();
    for (uint32_t g = lane; g < a.groups; g += L) {
      float hi = -INFINITY, lo = -INFINITY;
      for (uint32_t i = 0; i < a.group_size; ++i) {
        const float x = s_val[t][g * a.group_size + i];
        lo = fmaxf(lo, fminf(hi, x));
        hi = fmaxf(hi, x);
      }
      s_group[t][g] = (a.top2 && lo > -INFINITY ? hi + lo : hi) + 0.0f;
    }
    __syncwarp();
    // a group is kept if fewer than `kept` groups come before it
    uint32_t keep = 0;
    for (uint32_t g = lane; g < a.groups; g += L) {
      uint32_t before = 0;
      const float x = s_group[t][g];
      for (uint32_t h = 0; h < a.groups; ++h) {
        const float y = s_group[t][h];
        before += y > x || (y == x && h < g);
      }
      if (before < a.kept) keep |= 1u << g;
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) keep |= __shfl_xor_sync(kAll, keep, o);
    uint32_t g = e0 / a.group_size, r = e0 % a.group_size;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (e0 + j < a.experts && !(keep >> g & 1)) c[j] = -INFINITY;
      if (++r == a.group_size) r = 0, ++g;
    }
  }

  // top_k times the best that is left: the lowest lane and, there, the lowest
  // place among equals is the lowest expert
  uint32_t key[V], best = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    key[j] = order_bits(c[j]);
    best = max(best, key[j]);
  }
  const unsigned base = (threadIdx.x & 31) / L * L;
  for (uint32_t k = 0; k < a.top_k; ++k) {
    const uint32_t m = seg_max_bits<L>(best);
    const unsigned who = __ballot_sync(kAll, best == m) >> base;
    if (m == 0) {
      if (lane == 0) s_id[t][k] = -1, s_pick[t][k] = -INFINITY;
    } else if (lane == __ffs(who) - 1) {
      best = 0;
      bool found = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!found && key[j] == m) {
          found = true;
          key[j] = 0;
          s_id[t][k] = e0 + j;
          s_pick[t][k] = a.softmax && a.renormalize ? l[j] : s[j];
        }
        best = max(best, key[j]);
      }
    }
  }
  __syncwarp();
  float norm = 1.0f, high = 0.0f;
  if (a.renormalize) {
    if (a.softmax) {
      high = -INFINITY;
      for (uint32_t k = lane; k < a.top_k; k += L) high = fmaxf(high, s_pick[t][k]);
      high = seg_max<L>(high);
    }
    norm = 0.0f;
    for (uint32_t k = lane; k < a.top_k; k += L)
      if (s_id[t][k] >= 0) norm += a.softmax ? expf(s_pick[t][k] - high) : s_pick[t][k];
    norm = seg_sum<L>(norm);
  }
  if (tok >= a.tokens) return;
  for (uint32_t k = lane; k < a.top_k; k += L) {
    const int32_t id = s_id[t][k];
    float w = 0.0f;
    if (id >= 0) {
      w = s_pick[t][k];
      if (a.softmax && a.renormalize) w = expf(w - high);
      if (a.renormalize) w = norm > 0.0f ? w / norm : 0.0f;
    }
    a.weights[tok * a.top_k + k] = w * a.scale;
    a.ids[tok * a.top_k + k] = id;
  }
}

// Gradient of the weights carried to the logits.  With w the weights before
// the scale and d the incoming gradient times the scale, s_k dw/ds_k sums to
// u_k = w_k (d_k - sum_j w_j d_j) when renormalised and u_k = s_k d_k when
// not; then dl_e = u_e - s_e sum u (softmax; the sum is 0 when renormalised)
// or u_e (1 - s_e) (sigmoid).  Only the softmax without renormalisation has
// to read the whole row again.
template <class T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) zc_route_backward_kernel(RouteArgs a) {
  constexpr int kTok = kRouteThreads / L;
  __shared__ float s_row[kTok][L * V + 1];
  const int lane = threadIdx.x % L, t = threadIdx.x / L;
  const uint64_t tok = (uint64_t)blockIdx.x * kTok + t;
  const bool in = tok < a.tokens;
  const T* row = static_cast<const T*>(a.logits) + (in ? tok : 0) * a.stride;
  const uint32_t e0 = lane * V;
#pragma unroll
  for (int j = 0; j < V; ++j) s_row[t][e0 + j] = 0.0f;

  float l[V], top = -INFINITY, sum = 1.0f;
  const bool whole = a.softmax && !a.renormalize;
  if (whole) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = in && e0 + j < a.experts ? to_float(row[e0 + j]) : -INFINITY;
      l[j] = x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY;
      top = fmaxf(top, l[j]);
    }
    top = seg_max<L>(top);
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = l[j] > -INFINITY ? expf(l[j] - top) : 0.0f;
      sum += l[j];
    }
    sum = seg_sum<L>(sum);
  }
  constexpr int R = kMaxTopK / L;  // pairs a lane may hold
  int32_t id[R];
  float w[R], d[R], own[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t k = lane + r * L;
    id[r] = -1;
    w[r] = d[r] = own[r] = 0.0f;
    if (in && k < a.top_k) {
      id[r] = a.ids[tok * a.top_k + k];
      if (id[r] < 0 || (uint32_t)id[r] >= a.experts) id[r] = -1;
    }
    if (id[r] >= 0) {
      d[r] = a.grad[tok * a.top_k + k] * a.scale;
      own[r] = fminf(to_float(row[id[r]]), FLT_MAX);
    }
  }
  float high = -INFINITY, norm = 0.0f, mean = 0.0f;
  if (a.softmax) {
    if (a.renormalize) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (id[r] >= 0) high = fmaxf(high, own[r]);
      high = seg_max<L>(high);
    } else {
      high = top;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (id[r] >= 0) {
      own[r] = a.softmax ? expf(own[r] - high) : 1.0f / (1.0f + expf(-own[r]));
      if (whole) own[r] = own[r] / sum;
      norm += own[r];
    }
  if (a.renormalize) {
    norm = seg_sum<L>(norm);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[r] = norm > 0.0f ? own[r] / norm : 0.0f;
      mean += w[r] * d[r];
    }
    mean = seg_sum<L>(mean);
  }
  __syncwarp();
  float all = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (id[r] >= 0) {
      float u = a.renormalize ? w[r] * (d[r] - mean) : own[r] * d[r];
      all += u;
      if (!a.softmax) u *= 1.0f - own[r];
      atomicAdd(&s_row[t][id[r]], u);  // ids of a token are distinct: one add each
    }
  if (whole) all = seg_sum<L>(all);
  __syncwarp();
  if (!in) return;
  T* out = static_cast<T*>(a.grad_logits) + tok * a.experts;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (e0 + j < a.experts) {
      float g = s_row[t][e0 + j];
      if (whole && sum > 0.0f) g -= l[j] / sum * all;  // 0: no eligible expert
      out[e0 + j] = from_float<T>(g);
    }
}

template <class T, int L, int V>
cudaError_t route_launch(const RouteArgs& a, bool backward, cudaStream_t s) {
  constexpr uint32_t kTok = kRouteThreads / L;
  const uint32_t grid = (uint32_t)(((uint64_t)a.tokens + kTok - 1) / kTok);
  if (backward)
    zc_route_backward_kernel<T, L, V><<<grid, kRouteThreads, 0, s>>>(a);
  else
    zc_route_kernel<T, L, V><<<grid, kRouteThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t route_by_experts(const RouteArgs& a, bool backward, cudaStream_t s) {
  if (a.experts <= 64) return route_launch<T, 8, 8>(a, backward, s);
  if (a.experts <= 128) return route_launch<T, 16, 8>(a, backward, s);
  if (a.experts <= 256) return route_launch<T, 32, 8>(a, backward, s);
  if (a.experts <= 512) return route_launch<T, 32, 16>(a, backward, s);
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
// A stable counting sort of the pairs by expert.  One block takes kPlanChunk
// consecutive pairs; with more than one block a first kernel leaves every
// block's counts in the workspace.
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr uint32_t kPlanChunk = 4096;

struct PlanArgs {
  const int32_t* ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* slots;
  uint32_t* block_counts;  // [blocks][experts + 1]
  uint32_t pairs, experts, blocks;
};

// A pair that is not routed (id outside 0..experts-1) counts for one more
// bucket after the experts.
__device__ __forceinline__ uint32_t plan_key(int32_t id, uint32_t experts) { return min((uint32_t)id, experts); }

__global__ void __launch_bounds__(kPlanThreads) zc_plan_count_kernel(PlanArgs a) {
  __shared__ uint32_t h[kMaxExperts + 1];
  for (uint32_t e = threadIdx.x; e <= a.experts; e += kPlanThreads) h[e] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * kPlanChunk, hi = min(lo + kPlanChunk, a.pairs);
  for (uint32_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) atomicAdd(&h[plan_key(a.ids[i], a.experts)], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= a.experts; e += kPlanThreads)
    a.block_counts[(uint64_t)blockIdx.x * (a.experts + 1) + e] = h[e];
}

__global__ void __launch_bounds__(kPlanThreads) zc_plan_place_kernel(PlanArgs a) {
  extern __shared__ uint32_t h[];  // [kPlanWarps][buckets], then the totals and the scan's carry
  const uint32_t nb = a.experts + 1;
  uint32_t* total = h + kPlanWarps * nb;
  __shared__ uint32_t s_scan[kPlanWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (uint32_t i = threadIdx.x; i < kPlanWarps * nb; i += kPlanThreads) h[i] = 0;
  __syncthreads();
  // this block's pairs, one run of consecutive pairs for each warp
  const uint32_t per = kPlanChunk / kPlanWarps;
  const uint32_t lo = blockIdx.x * kPlanChunk + w * per, hi = min(lo + per, a.pairs);
  for (uint32_t i = lo + lane; i < hi; i += 32) atomicAdd(&h[w * nb + plan_key(a.ids[i], a.experts)], 1u);
  __syncthreads();
  // per bucket: pairs of earlier blocks, and of all
  for (uint32_t e = threadIdx.x; e < nb; e += kPlanThreads) {
    uint32_t before = 0, all = 0;
    if (a.blocks == 1) {
      for (int v = 0; v < kPlanWarps; ++v) all += h[v * nb + e];
    } else {
      for (uint32_t b = 0; b < a.blocks; ++b) {
        const uint32_t n = a.block_counts[(uint64_t)b * nb + e];
        if (b < blockIdx.x) before += n;
        all += n;
      }
    }
    total[e] = all;
    // the warps' counts become where each warp's first pair goes, less the
    // bucket's start
    for (int v = 0; v < kPlanWarps; ++v) {
      const uint32_t n = h[v * nb + e];
      h[v * nb + e] = before;
      before += n;
    }
  }
  __syncthreads();
  // exclusive scan of the totals, kPlanThreads buckets at a time
  uint32_t carry = 0;
  for (uint32_t e0 = 0; e0 < nb; e0 += kPlanThreads) {
    const uint32_t e = e0 + threadIdx.x;
    const uint32_t n = e < nb ? total[e] : 0;
    uint32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[w] = x;
    __syncthreads();
    uint32_t front = carry, sum = 0;
    for (int v = 0; v < kPlanWarps; ++v) {
      if (v < w) front += s_scan[v];
      sum += s_scan[v];
    }
    const uint32_t start = front + x - n;
    if (e < nb) {
      for (int v = 0; v < kPlanWarps; ++v) h[v * nb + e] += start;
      if (blockIdx.x == 0) {
        a.offsets[e] = (int32_t)start;
        if (e < a.experts) a.counts[e] = (int32_t)n;
      }
    }
    carry += sum;
    __syncthreads();
  }
  // places in order: 32 pairs at a time, equal buckets ranked by lane
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    const uint32_t key = i < hi ? plan_key(a.ids[i], a.experts) : nb;
    const unsigned same = __match_any_sync(kAll, key);
    const uint32_t rank = __popc(same & ((1u << lane) - 1));
    uint32_t at = 0;
    if (key < nb) at = h[w * nb + key] + rank;
    __syncwarp();
    if (key < nb && rank == 0) h[w * nb + key] += __popc(same);
    __syncwarp();
    if (i < hi) a.slots[i] = key < a.experts ? (int32_t)at : ~(int32_t)at;
  }
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
  const uint64_t blocks = (pairs + kPlanChunk - 1) / kPlanChunk;
  *out_bytes = blocks > 1 ? 4 * blocks * (experts + 1) : 0;
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
  a.block_counts = static_cast<uint32_t*>(d_ws);
  a.pairs = (uint32_t)pairs;
  a.experts = experts;
  a.blocks = pairs ? (uint32_t)((pairs + kPlanChunk - 1) / kPlanChunk) : 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.blocks > 1) zc_plan_count_kernel<<<a.blocks, kPlanThreads, 0, s>>>(a);
  zc_plan_place_kernel<<<a.blocks, kPlanThreads, (kPlanWarps + 1) * (experts + 1) * 4, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // extern "C"
