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

__device__ __noinline__ Choice choose_any(const RouteArgs& a, const float* row, bool live, uint32_t lane, float* keys) {
  if (a.experts <= 64) return choose<float, 32, 2>(a, row, live, lane, keys);
  if (a.experts <= 128) return choose<float, 32, 4>(a, row, live, lane, keys);
  if (a.experts <= 256) return choose<float, 32, 8>(a, row, live, lane, keys);
  if (a.experts <= 512) return choose<float, 32, 16>(a, row, live, lane, keys);
  return choose<float, 32, 32>(a, row, live, lane, keys);
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

// The block's share of all logits, as partial sums: an eighth of the hidden places.
template <class R, class T, int G, bool kShift>
__device__ __forceinline__ void router_logits(const LayerArgs& a, float* partial, uint32_t rank) {
  constexpr int kAhead = G == 1 && !kShift ? 4 : 2;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t splits = router_splits(a.experts), tiles = (a.experts + 15) / 16, groups = (a.tokens + 7) / 8;
  const uint32_t steps = (a.hidden + kStep<R> - 1) / kStep<R>, all = kCluster * splits, bytes = a.hidden * (uint32_t)sizeof(R);
  const T* v[G];
#pragma unroll
  for (int g = 0; g < G; ++g) v[g] = static_cast<const T*>(a.x) + (uint64_t)min(g * 8 + gid, a.tokens - 1) * a.x_stride;
  for (uint32_t tile = warp / splits; tile < tiles; tile += kWarps / splits) {
    const uint32_t part = rank * splits + warp % splits;
    float c[G][4] = {};
    const R* row = static_cast<const R*>(a.router);
    const R *row0 = row + (uint64_t)min(tile * 16 + gid, a.experts - 1) * a.hidden;
    const R *row1 = row + (uint64_t)min(tile * 16 + gid + 8, a.experts - 1) * a.hidden;
    for (uint32_t s = steps * part / all, end = steps * (part + 1) / all; s < end; s += kAhead) {
      Raw w0[kAhead], w1[kAhead];
      RawShare<R, T, kShift> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
        w0[u] = raw16<kShift>(row0, k * (uint32_t)sizeof(R), bytes);
        w1[u] = raw16<kShift>(row1, k * (uint32_t)sizeof(R), bytes);
        x[u].load(v[0], 0, k, a.hidden);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= (int)groups) break;
        float t[4] = {};
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const uint32_t k = (s + u) * kStep<R> + quad * kPer16<R>;
          const int left = s + u < end ? (int)a.hidden - (int)k : 0;
          if (g) x[u].load(v[g], 0, k, a.hidden);
          step_products<R, T>(t, keep<R>(settle<kShift>(w0[u], shift_of(row0)), left), keep<R>(settle<kShift>(w1[u], shift_of(row1)), left),
                              x[u].used(v[g], k, a.hidden, false));
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
template <bool kShift, class T, class W, int G>
__device__ __forceinline__ void layer_up(const LayerArgs& a, const Pairs<G>& pairs, Ring& ring, uint8_t* memory) {
  constexpr uint32_t kStages = kStagesOf<G>;
  constexpr bool kShiftW = kShift && !std::is_same<W, F8>::value;  // rows of codes start at multiples of 16
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  // 16 rows of an expert at a time: 8 of the gate's and 8 of the other's, so that
  // both of a place come to the same lane; or 16 of the only matrix
  const uint32_t high = a.gated ? 8 : 16, tiles = (a.inner + high - 1) / high, rows = a.gated ? 2 * a.inner : a.inner;
  // whole chunks of a row, and their pieces; what is left is one warp's
  const uint32_t body = a.hidden / kPlacesOfChunk<W> * kPlacesOfChunk<W>, pieces = (body + kPlacesOfPiece<W> - 1) / kPlacesOfPiece<W>;
  const uint32_t units = pairs.count * tiles;
  struct Fill {
    const LayerArgs& a;
    const Pairs<G>& pairs;
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
  Stages<kStages, kShiftW, Fill> stages(ring, memory, matrix, fill, &g_layer_up_ran_out);
  float4* sums = reinterpret_cast<float4*>(memory + kStages * kStageBytes<kShiftW>);
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
    const uint32_t begin = pairs.begin[n], tokens = pairs.begin[n + 1] - begin, groups = (tokens + 7) / 8;
    const uint32_t r0 = min(i0 + gid, a.inner - 1), r1 = a.gated ? a.inner + r0 : min(i0 + gid + 8, a.inner - 1);
    Vectors<T, G> v;
    v.apart = 0, v.groups = groups;
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
        x[i ^ 1].load(last ? after : v.v[0], 0, last ? k0 : k + kWarps * kPlacesOfChunk<W>, a.hidden);
        if (k < body) take_chunk<false, kShiftW, kShift, W, T, G>(c, stage + i * kWarps * kChunk, its, v, x[i], k, a.hidden);
      }
      stages.leave();
    }
    if (body < a.hidden && warp == done % kWarps) {
      x[1].load(v.v[0], 0, body, a.hidden);
      take_chunk<true, kShiftW, kShift, W, T, G>(c, nullptr, its, v, x[1], body, a.hidden);
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
template <bool kShift, class T, class W, int G>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_up_kernel(const __grid_constant__ LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t s_dyn[];
  __shared__ Pairs<G> s_pairs;
  __shared__ Ring s_ring;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t rank = cluster_rank(), splits = router_splits(a.experts);
  ring_init(s_ring);
  PairSource& source = *reinterpret_cast<PairSource*>(s_dyn);
  float* partial = reinterpret_cast<float*>(s_dyn + sizeof(PairSource));
  if (a.router_float) router_logits<float, T, G, kShift>(a, partial, rank);
  else router_logits<T, T, G, kShift>(a, partial, rank);
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
  layer_up<kShift, T, W, G>(a, s_pairs, s_ring, s_dyn);
}

template <int G>
size_t up_smem(uint32_t tokens, uint32_t experts, bool shift) {
  const size_t choice = sizeof(PairSource) + 4ull * (router_splits(experts) * tokens * experts + 3 + kShare * ((experts + 3) / 4 * 4 + 1024));
  return std::max<size_t>(choice, kStagesOf<G> * (shift ? kStageBytes<true> : kStageBytes<false>) + 2ull * kWarps * G * 512);
}

template <bool kShift, class T, class W, int G>
cudaError_t up_launch(const LayerArgs& a, cudaStream_t s) {
  static std::atomic<int> known[kMaxDevices];
  constexpr uint32_t most = G == 1 ? 8 : kMaxTokens;
  const auto kernel = zc_layer_up_kernel<kShift, T, W, G>;
  int clusters = 0;
  const cudaError_t e = clusters_at_once(kernel, known, up_smem<G>(1, 1, kShift), up_smem<G>(most, kMaxExperts, kShift), &clusters);
  return e != cudaSuccess ? e : launch_clusters(kernel, clusters, up_smem<G>(a.tokens, a.experts, kShift), s, a);
}

template <class T, class W>
cudaError_t up_by_tokens(const LayerArgs& a, cudaStream_t s) {
  // up to 8 tokens have one group each way; the other form serves any number
  if (a.shift_up) return a.tokens <= 8 ? up_launch<true, T, W, 1>(a, s) : up_launch<true, T, W, 4>(a, s);
  return a.tokens <= 8 ? up_launch<false, T, W, 1>(a, s) : up_launch<false, T, W, 4>(a, s);
}

template <class T>
cudaError_t up_by_weights(const LayerArgs& a, bool blocks, cudaStream_t s) {
  return blocks ? up_by_tokens<T, F8>(a, s) : up_by_tokens<T, T>(a, s);
}

}  // namespace

cudaError_t layer_up_launch(const LayerArgs& a, int type, bool blocks, cudaStream_t s) {
  return type == ZIPCCL_TYPE_F32    ? up_by_weights<float>(a, blocks, s)
         : type == ZIPCCL_TYPE_BF16 ? up_by_weights<__nv_bfloat16>(a, blocks, s)
                                    : up_by_weights<__half>(a, blocks, s);
}
cudaError_t layer_up_waits(cudaStream_t s, bool* ran_out) { return take_flag(g_layer_up_ran_out, s, ran_out); }

}  // namespace zc
