// zc_route.cu -- routing of tokens to experts, its gradient, and the plan of
// the experts' chunks (counts, offsets and the row of every token-expert
// pair).
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "zc_ops.cuh"
#include "zc_route.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kRouteThreads = 256;

// A token's pairs (choose).  For few tokens it takes a launch (2.4 us); for many its instructions bound
// it: of 256 experts in 8 groups, 8 chosen, a token takes 795, 29 of them for
// each chosen expert, about 145 each for the groups and the sigmoids (8,192
// tokens: 8.1 us).
template <class T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) zc_route_kernel(RouteArgs a) {
  after_previous();
  constexpr uint32_t kTok = kRouteThreads / L;
  __shared__ __align__(16) float s_key[kTok][L * V];
  const uint32_t lane = threadIdx.x % L;
  const uint32_t tok = blockIdx.x * kTok + threadIdx.x / L;
  const bool in = tok < a.tokens;
  const T* row = static_cast<const T*>(a.logits) + (in ? tok : 0) * a.stride;
  const Choice c = choose<T, L, V>(a, row, in && (!a.mask || a.mask[tok]), lane, s_key[threadIdx.x / L]);
  if (in && lane < a.top_k) {
    a.weights[(uint64_t)tok * a.top_k + lane] = c.weight * a.scale;
    a.ids[(uint64_t)tok * a.top_k + lane] = c.id;
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

template <class T>
cudaError_t route_by_experts(const RouteArgs& a, bool backward, cudaStream_t s) {
  const uint32_t lanes = lanes_of_token(a.experts, a.top_k, a.groups);
  if (lanes == 8) return route_launch<T, 8, 8>(a, backward, s);
  switch (experts_of_lane(a.experts, lanes)) {
    case 2: return route_launch<T, 32, 2>(a, backward, s);
    case 4: return route_launch<T, 32, 4>(a, backward, s);
    case 8: return route_launch<T, 32, 8>(a, backward, s);
    case 16: return route_launch<T, 32, 16>(a, backward, s);
    default: return route_launch<T, 32, 32>(a, backward, s);
  }
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
