// zc_route.cuh -- the choice of a token's experts and their weights: shared by the
// routing call and the layer for a few tokens.
#pragma once
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {

constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopK = 32;
constexpr uint32_t kMaxGroups = 32;

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

// Lanes that take a token, and experts that a lane holds: the sums over a token go by
// both, so that every call that chooses asks here.  A warp takes a token; 8 lanes do
// where they hold its experts, 8 each, its pairs and its groups: 16,384 tokens of 64
// experts, two chosen, 3.4 us against 5.6 with 32 lanes, one token 2.6 against 2.3.
// (Between 65 and 128 experts 16 lanes made no difference, nor did they up to 256.)
__host__ __device__ __forceinline__ uint32_t lanes_of_token(uint32_t experts, uint32_t top_k, uint32_t groups) {
  return experts <= 64 && top_k <= 8 && groups <= 8 ? 8 : 32;
}
__host__ __device__ __forceinline__ uint32_t experts_of_lane(uint32_t experts, uint32_t lanes) {
  return lanes == 8 ? 8 : experts <= 64 ? 2 : experts <= 128 ? 4 : experts <= 256 ? 8 : experts <= 512 ? 16 : 32;
}

// A pair of a token: the expert (-1: none) and its weight before the scale.
struct Choice {
  int32_t id;
  float weight;
};

// L lanes take a token, V consecutive experts each.  The choice scores lie in
// shared memory (`keys`, L * V floats); each lane knows the best of its own, and
// top_k times the lanes find the best of these, its place among the V of its lane
// (the lowest place of the lowest lane is the lowest expert among equals), and
// what is then best in that lane: no step is one lane's alone, but for the scan of
// groups that are not whole lanes.  Lane k gets pair k.  A token that is not
// `live` has no pairs.
template <class T, int L, int V>
__device__ __forceinline__ Choice choose(const RouteArgs& a, const T* row, bool live, uint32_t lane, float* keys) {
  static_assert(V <= L, "a lane's experts are scanned by one lane each");
  const uint32_t e0 = lane * V;
  float top = 0.0f, inv = 0.0f;
  int32_t id = -1;  // of pair `lane`
  float l[V], c[V];
  load_logits<T, V>(row, e0, a.experts, a.wide, l);
  if (!live) {
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
  return {id, s};
}

}  // namespace zc
