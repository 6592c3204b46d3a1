// zc_layer_up.cu -- the first kernel of the layer for a few tokens: the choice of
// experts, and what the chosen ones make of the tokens up to the activation.
//
// The choice of experts is made by every cluster of 8 blocks for itself: each block
// takes an eighth of the hidden places for all experts and tokens, the partial
// logits are summed over the cluster's shared memory in one order, and each block
// chooses for its share of the tokens.  A separate kernel would cost a launch, a
// grid-wide wait about the same.
#include "zc_layer.cuh"

namespace zc {
namespace {

__device__ unsigned int g_layer_up_ran_out;

// As the routing call chooses, in the same order.  A warp has one token: where 8 lanes
// take it, the others have none.
__device__ __noinline__ Choice choose_any(const RouteArgs& a, const float* row, bool live, uint32_t lane, float* keys) {
  const uint32_t lanes = lanes_of_token(a.experts, a.top_k, a.groups);
  if (lanes == 8) return choose<float, 8, 8>(a, row, live && lane < 8, lane % 8, keys + lane / 8 * 64);
  switch (experts_of_lane(a.experts, lanes)) {
    case 2: return choose<float, 32, 2>(a, row, live, lane, keys);
    case 4: return choose<float, 32, 4>(a, row, live, lane, keys);
    case 8: return choose<float, 32, 8>(a, row, live, lane, keys);
    case 16: return choose<float, 32, 16>(a, row, live, lane, keys);
    default: return choose<float, 32, 32>(a, row, live, lane, keys);
  }
}
// (SiLU: e^-v overflows from v = -88.8 on, where the result is still a normal float;
// GELU by the complement: 1 + erf cancels for v < 0 and is 0 from -5.5 on, where
// v (1 + erf) / 2 is still -1e-7.)
__device__ __forceinline__ float activate(int activation, float v) {
  if (activation == ZIPCCL_ACTIVATION_SILU) return v * sigmoid(v);
  if (activation == ZIPCCL_ACTIVATION_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  return v > 0.0f || isnan(v) ? v : 0.0f;
}

__host__ __device__ __forceinline__ uint32_t router_splits(uint32_t experts) {  // warps that share 16 experts' places
  return experts <= 16 ? 8 : experts <= 32 ? 4 : experts <= 64 ? 2 : 1;
}
constexpr uint32_t kShare = kMaxTokens / kCluster;  // tokens that a block chooses for

// The block's share of all logits, as partial sums: an eighth of the hidden places.
template <class R, class T, bool kShift>
__device__ __forceinline__ void router_logits(const LayerArgs& a, float* partial, uint32_t rank) {
  constexpr int kAhead = 2;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t splits = router_splits(a.experts), tiles = (a.experts + 15) / 16, groups = (a.tokens + 7) / 8;
  const uint32_t steps = (a.hidden + kStep<R> - 1) / kStep<R>, all = kCluster * splits, bytes = a.hidden * (uint32_t)sizeof(R);
  const R* row = static_cast<const R*>(a.router);
  for (uint32_t i = warp / splits; i < tiles * groups; i += kWarps / splits) {  // 16 experts, 8 tokens
    const uint32_t tile = i / groups, g = i - tile * groups, part = rank * splits + warp % splits;
    float c[4] = {};
    const T* v = static_cast<const T*>(a.x) + (uint64_t)min(g * 8 + gid, a.tokens - 1) * a.x_stride;
    const R *row0 = row + (uint64_t)min(tile * 16 + gid, a.experts - 1) * a.hidden;
    const R *row1 = row + (uint64_t)min(tile * 16 + gid + 8, a.experts - 1) * a.hidden;
    // the next steps' values are asked for before the products of these
    Raw w0[2][kAhead], w1[2][kAhead];
    RawShare<R, T, kShift> x[2][kAhead];
    const auto load = [&](int to, uint32_t s) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
        w0[to][u] = raw16<kShift>(row0, k * (uint32_t)sizeof(R), bytes);
        w1[to][u] = raw16<kShift>(row1, k * (uint32_t)sizeof(R), bytes);
        x[to][u].load(v, 0, k, a.hidden);
      }
    };
    const uint32_t begin = steps * part / all, end = steps * (part + 1) / all;
    const auto take = [&](int from, uint32_t s) {
      float t[4] = {};
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
        const int left = s + u < end ? (int)a.hidden - (int)k : 0;
        // (both zeros behind the warp's share: an infinite value of the next one's would make 0 a NaN)
        step_products<R, T, true>(t, keep<R>(settle<kShift>(w0[from][u], shift_of(row0)), left),
                                  keep<R>(settle<kShift>(w1[from][u], shift_of(row1)), left), x[from][u].used(v, k, min(a.hidden, end * kStep<R>), false));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] += t[j];
    };
    if (begin < end) load(0, begin);
    for (uint32_t s = begin; s < end; s += 2 * kAhead) {
      load(1, s + kAhead);
      take(0, s);
      if (s + kAhead >= end) break;
      load(0, s + 2 * kAhead);
      take(1, s + kAhead);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e = tile * 16 + gid + (j / 2) * 8, t = g * 8 + quad * 2 + j % 2;
      if (e < a.experts && t < a.tokens) partial[(warp % splits * a.tokens + t) * a.experts + e] = c[j];
    }
  }
}

// Dynamic shared memory: the stages and the working warps' sums, or, before these,
// the pairs' source, partial logits, rows and keys of the block's tokens.  Behind
// either the pairs.
template <bool kShiftW>
__host__ __device__ __forceinline__ size_t up_memory(uint32_t tokens, uint32_t experts, uint32_t stages) {
  const size_t choice = sizeof(PairSource) + 4ull * (router_splits(experts) * tokens * experts + 3 + kShare * ((experts + 3) / 4 * 4 + 1024));
  const size_t work = stages * kStageBytes<kShiftW> + 2ull * kWarps * 512;
  return ((choice > work ? choice : work) + 15) / 16 * 16;
}

// The first kernel's work once the experts are chosen.
template <bool kShift, class T, class W>
__device__ __forceinline__ void layer_up(const LayerArgs& a, const Pairs& pairs, Ring& ring, uint8_t* memory) {
  constexpr bool kShiftW = kShift && !std::is_same<W, F8>::value;  // rows of codes start at multiples of 16
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  // 16 rows of an expert at a time: 8 of the gate's and 8 of the other's, so that
  // both of a place come to the same lane; or 16 of the only matrix
  const uint32_t high = a.gated ? 8 : 16, tiles = (a.inner + high - 1) / high, rows = a.gated ? 2 * a.inner : a.inner;
  // whole chunks of a row, and their pieces; what is left is one warp's
  const uint32_t body = a.hidden / kPlacesOfChunk<W> * kPlacesOfChunk<W>, pieces = (body + kPlacesOfPiece<W> - 1) / kPlacesOfPiece<W>;
  const uint32_t units = *pairs.count * tiles;
  struct Fill {
    const LayerArgs& a;
    const Pairs& pairs;
    uint32_t u, units, tiles, pieces, rows, high;
    uint32_t piece = 0, row0 = 0, row1 = 0;
    __device__ __forceinline__ bool more() const { return u < units && pieces; }
    __device__ __forceinline__ void place() {
      if (u >= units) return;
      const uint32_t n = u / tiles;
      row0 = pairs.expert[n] * rows + (u - n * tiles) * high;
      row1 = a.gated ? row0 + a.inner : row0 + 8;
    }
    __device__ __forceinline__ void advance() {
      if (++piece < pieces) return;
      piece = 0;
      u += gridDim.x;
      place();
    }
  } fill{a, pairs, blockIdx.x, units, tiles, pieces, rows, high};
  fill.place();
  const Matrix matrix = {&a.up_map, static_cast<const uint8_t*>(a.up), (uint64_t)a.experts * rows, a.up_stride * sizeof(W), a.hidden * (uint32_t)sizeof(W)};
  Stages<kShiftW, Fill> stages(ring, memory, matrix, fill, a.stages, &g_layer_up_ran_out);
  float4* sums = reinterpret_cast<float4*>(memory + a.stages * kStageBytes<kShiftW>);
  using X = PartsFor<T, W>;
  const uint64_t apart = (uint64_t)a.tokens * a.top_k * a.h_stride;
  const uint32_t k0 = warp * kPlacesOfChunk<W>;
  const auto vector = [&](uint32_t n, uint32_t col) -> const T* {  // of the column of active expert n
    uint32_t at = pairs.begin[n] + col;
    if (at >= pairs.begin[n + 1]) at = pairs.begin[n];
    return static_cast<const T*>(a.x) + (uint64_t)pairs.token[at] * a.x_stride;
  };
  Chunk<W, T, kShift> x[2];
  if (blockIdx.x < units) x[0].load(vector(blockIdx.x / tiles, gid), 0, min(k0, body), a.hidden);
  uint32_t done = 0;
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++done) {
    const uint32_t n = u / tiles, i0 = (u - n * tiles) * high, e = pairs.expert[n];
    const uint32_t begin = pairs.begin[n], tokens = pairs.begin[n + 1] - begin;
    const uint32_t r0 = min(i0 + gid, a.inner - 1), r1 = a.gated ? a.inner + r0 : min(i0 + gid + 8, a.inner - 1);
    const Vector<T> v = {vector(n, gid), 0};
    const T* after = u + gridDim.x < units ? vector((u + gridDim.x) / tiles, gid) : v.at;  // the next unit's
    float c[4] = {};
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
        x[i ^ 1].load(last ? after : v.at, 0, last ? k0 : k + kWarps * kPlacesOfChunk<W>, a.hidden);
        if (k < body) take_chunk<false, kShiftW, kShift, W, T>(c, stage + i * kWarps * kChunk, its, v, x[i], k, a.hidden);
      }
      stages.leave();
    }
    if (body < a.hidden && warp == done % kWarps) {
      x[1].load(v.at, 0, body, a.hidden);
      take_chunk<true, kShiftW, kShift, W, T>(c, nullptr, its, v, x[1], body, a.hidden);
    }
    // The warps add up in turn, while the others go on: each arrives where its sums
    // are written, one waits for all, and before the memory is written again, two
    // units on, all wait for that one.
    const uint32_t half = done % 2;
    float4* mine = sums + half * kWarps * 32;
    if (done >= 2) {
      if (warp == (done - 2) % kWarps) warps_arrive(3 + half);
      else warps_sync(3 + half);
    }
    mine[warp * 32 + lane] = make_float4(c[0], c[1], c[2], c[3]);
    if (warp != done % kWarps) {
      warps_arrive(1 + half);
      continue;
    }
    warps_sync(1 + half);
    float4 all = mine[lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 q = mine[w * 32 + lane];
      all.x += q.x, all.y += q.y, all.z += q.z, all.w += q.w;
    }
    const float v4[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t col = quad * 2 + i;
      if (col >= tokens) continue;
      const float w = pairs.weight[begin + col];
      auto* h = static_cast<typename X::Value*>(a.h) + (uint64_t)(begin + col) * a.h_stride + i0 + gid;
      if (a.gated) {
        if (i0 + gid < a.inner) store_parts<X>(h, apart, w * (activate(a.activation, v4[i]) * v4[2 + i]));
      } else {
        if (i0 + gid < a.inner) store_parts<X>(h, apart, w * activate(a.activation, v4[i]));
        if (i0 + gid + 8 < a.inner) store_parts<X>(h + 8, apart, w * activate(a.activation, v4[2 + i]));
      }
    }
  }
  stages.end();
}

template <bool kShift, class T, class W>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_up_kernel(const __grid_constant__ LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t s_dyn[];
  __shared__ Ring s_ring;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t rank = cluster_rank(), splits = router_splits(a.experts);
  ring_init(s_ring);
  pdl_wait();
  PairSource& source = *reinterpret_cast<PairSource*>(s_dyn);
  float* partial = reinterpret_cast<float*>(s_dyn + sizeof(PairSource));
  if (a.router_float) router_logits<float, T, kShift>(a, partial, rank);
  else router_logits<T, T, kShift>(a, partial, rank);
  __syncthreads();
  if (splits > 1) {  // one partial sum of each block
    const uint32_t all = a.tokens * a.experts;
    for (uint32_t i = threadIdx.x; i < all; i += kThreads) {
      float sum = partial[i];
      for (uint32_t p = 1; p < splits; ++p) sum += partial[p * all + i];
      partial[i] = sum;
    }
  }
  cluster_sync();
  {
    const uint32_t held = (a.experts + 3) / 4 * 4;
    float* rows = partial + (splits * a.tokens * a.experts + 3) / 4 * 4;
    for (uint32_t i = warp; i < kShare; i += kThreads / 32) {
      const uint32_t t = rank + i * kCluster;
      if (t >= a.tokens) break;
      float *row = rows + i * (held + 1024), *keys = row + held;
      for (uint32_t e = lane; e < a.experts; e += 32) row[e] = cluster_sum(partial + t * a.experts + e, 0, kCluster);
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
  const Pairs pairs(s_dyn + up_memory<kShift && !std::is_same<W, F8>::value>(a.tokens, a.experts, a.stages), a.tokens * a.top_k);
  gather_pairs<true>(pairs, source, a.tokens, a.top_k, a.experts);
  layer_up<kShift, T, W>(a, pairs, s_ring, s_dyn);
  pdl_trigger();
}

template <bool kShift, class T, class W>
cudaError_t up_launch(LayerArgs a, cudaStream_t s) {
  constexpr bool kShiftW = kShift && !std::is_same<W, F8>::value;
  static std::atomic<int> known[kMaxDevices];
  const auto kernel = zc_layer_up_kernel<kShift, T, W>;
  const uint32_t pairs = a.tokens * a.top_k;
  a.stages = kMaxStages;
  while (a.stages > 2 && up_memory<kShiftW>(a.tokens, a.experts, a.stages) + Pairs::bytes(pairs) > kRoomForTwo) --a.stages;
  int clusters = 0;
  const cudaError_t e = clusters_at_once(kernel, known, kRoomForTwo, up_memory<kShiftW>(kMaxTokens, kMaxExperts, kMaxStages) + Pairs::bytes(kMaxTokens * kMaxTopK), &clusters);
  return e != cudaSuccess ? e : launch_clusters(kernel, clusters, up_memory<kShiftW>(a.tokens, a.experts, a.stages) + Pairs::bytes(pairs), s, a);
}

template <class T>
cudaError_t up_by_weights(const LayerArgs& a, bool blocks, cudaStream_t s) {
  if (blocks) return a.shift_up ? up_launch<true, T, F8>(a, s) : up_launch<false, T, F8>(a, s);
  return a.shift_up ? up_launch<true, T, T>(a, s) : up_launch<false, T, T>(a, s);
}

}  // namespace

cudaError_t layer_up_launch(const LayerArgs& a, int type, bool blocks, cudaStream_t s) {
  return type == ZIPCCL_TYPE_F32    ? up_by_weights<float>(a, blocks, s)
         : type == ZIPCCL_TYPE_BF16 ? up_by_weights<__nv_bfloat16>(a, blocks, s)
                                    : up_by_weights<__half>(a, blocks, s);
}
cudaError_t layer_up_waits(cudaStream_t s, bool* ran_out) { return take_flag(g_layer_up_ran_out, s, ran_out); }

}  // namespace zc
