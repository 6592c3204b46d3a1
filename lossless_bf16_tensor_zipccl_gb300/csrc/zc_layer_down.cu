// zc_layer_down.cu -- the second kernel of the layer for a few tokens: the chosen
// experts' rows back to the hidden size, added up for each token.  And the call.
#include "zc_layer.cuh"

namespace zc {
namespace {

__device__ unsigned int g_layer_down_ran_out;

// Dynamic shared memory: the stages (before them the pairs' source), the warps'
// sums and a round's; behind them the pairs.
template <bool kShift>
__host__ __device__ __forceinline__ size_t down_memory(uint32_t tokens, uint32_t stages) {
  return stages * kStageBytes<kShift> + 4ull * (kWarps + kCluster) * tokens * 16;
}

// 16 hidden places at a time; the pieces of the active experts' rows, one expert
// after the other, are dealt out in equal runs to 1, 2, 4 or 8 blocks of a cluster:
// whichever leaves the fewest pieces to the block that has most.  A warp adds what an
// expert gives to its tokens' sums in shared memory: an expert's columns are its own
// tokens only, so that nothing of it reaches another's.  A block adds its warps', and after 8 tiles the
// blocks that share them each all blocks' of some of them.
template <bool kShift, class T, class W>
__device__ __forceinline__ void layer_down(const LayerArgs& a, const Pairs& pairs, Ring& ring, uint8_t* memory) {
  constexpr uint32_t kRound = kCluster;  // tiles before the blocks' sums are added
  using X = PartsFor<T, W>;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, gid = lane / 4, quad = lane % 4;
  const uint32_t rank = cluster_rank(), cluster = blockIdx.x / kCluster, clusters = gridDim.x / kCluster;
  const uint32_t size = a.tokens * 16;  // of a tile: [token][place]
  float* warps = reinterpret_cast<float*>(memory + a.stages * kStageBytes<kShift>);
  float* own = warps + warp * size;        // a warp's sums
  float* block = warps + kWarps * size;    // a block's, of a round's tiles
  const auto* h = static_cast<const typename X::Value*>(a.h);
  const uint64_t apart = (uint64_t)a.tokens * a.top_k * a.h_stride;
  // whole chunks of a row, and their pieces (one at least); what is left is a warp's of the block that has a row's last
  const uint32_t body = a.inner / kPlacesOfChunk<W> * kPlacesOfChunk<W>, pieces = max((body + kPlacesOfPiece<W> - 1) / kPlacesOfPiece<W>, 1u);
  const uint32_t all = pieces * *pairs.count;
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
    const Pairs& pairs;
    uint32_t tile, tiles, stride, s, from, upto, pieces;
    bool any;
    uint32_t piece = 0, row0 = 0, row1 = 0;
    __device__ __forceinline__ bool more() const { return tile < tiles && s < upto && any; }
    __device__ __forceinline__ void place() {
      if (!more()) return;
      const uint32_t n = s / pieces;
      piece = s - n * pieces;
      row0 = pairs.expert[n] * a.hidden + tile * 16;
      row1 = row0 + 8;
    }
    __device__ __forceinline__ void advance() {
      if (++s == upto) s = from, tile += stride;
      place();
    }
  } fill{a, pairs, t0, tiles, stride, from, from, upto, pieces, body > 0};
  fill.place();
  const Matrix matrix = {&a.down_map, static_cast<const uint8_t*>(a.down), (uint64_t)a.experts * a.hidden, a.down_stride * sizeof(W), a.inner * (uint32_t)sizeof(W)};
  Stages<kShift, Fill> stages(ring, memory, matrix, fill, a.stages, &g_layer_down_ran_out);
  const uint32_t k0 = warp * kPlacesOfChunk<W>;
  const auto vector = [&](uint32_t n, uint32_t col) -> const typename X::Value* {  // of a column of active expert n
    uint32_t at = pairs.begin[n] + col;
    if (at >= pairs.begin[n + 1]) at = pairs.begin[n];  // (not used)
    return h + (uint64_t)at * a.h_stride;
  };
  Chunk<W, X, false> x[2];
  if (from < upto) x[0].load(vector(from / pieces, gid), apart, from % pieces * kPlacesOfPiece<W> + k0, a.inner);
  const uint32_t rounds = (tiles + stride * kRound - 1) / (stride * kRound);  // the same for all blocks
  for (uint32_t round = 0; round < rounds; ++round) {
    for (uint32_t j = 0; j < kRound; ++j) {
      const uint32_t tile = t0 + (round * kRound + j) * stride;
      if (tile >= tiles) break;
      const uint32_t r0 = min(tile * 16 + gid, a.hidden - 1), r1 = min(tile * 16 + gid + 8, a.hidden - 1);
      float c[4] = {};
      for (uint32_t i = lane; i < size; i += 32) own[i] = 0.0f;
      __syncwarp();
      uint32_t n = from / pieces, p = from - n * pieces;
      for (uint32_t s = from; s < upto;) {  // an expert's pieces of the run
        const uint32_t begin = pairs.begin[n], tokens = pairs.begin[n + 1] - begin;
        const Vector<X> v = {vector(n, gid), apart};
        const W* at = static_cast<const W*>(a.down) + (uint64_t)pairs.expert[n] * a.hidden * a.down_stride;
        const uint8_t* scales = a.down_scales + (uint64_t)pairs.expert[n] * ((a.hidden + kFp8Block - 1) / kFp8Block) * across;
        const Rows<W> its = {at + r0 * a.down_stride, at + r1 * a.down_stride, scales + r0 / kFp8Block * across, scales + r1 / kFp8Block * across};
        const uint32_t last = min(pieces, p + (upto - s));
        s += last - p;
        // what follows: the next expert's first piece, or the run's again
        const bool again = s == upto;
        const auto* after = vector(again ? from / pieces : n + 1, gid);
        const uint32_t after_k = (again ? from % pieces : 0) * kPlacesOfPiece<W> + k0;
        const bool to_end = last == pieces;
        uint32_t k = p * kPlacesOfPiece<W> + k0;
        for (; p < last; ++p) {
          const uint8_t* stage = body ? stages.take() : nullptr;
#pragma unroll
          for (int i = 0; i < 2; ++i, k += kWarps * kPlacesOfChunk<W>) {
            const bool leaves = i && p + 1 == last;
            x[i ^ 1].load(leaves ? after : v.at, apart, leaves ? after_k : k + kWarps * kPlacesOfChunk<W>, a.inner);
            if (k < body) take_chunk<false, kShift, false, W, X>(c, stage + i * kWarps * kChunk, its, v, x[i], k, a.inner);
          }
          if (body) stages.leave();
        }
        if (to_end && body < a.inner && warp == n % kWarps) {
          x[1].load(v.at, apart, body, a.inner);
          take_chunk<true, kShift, false, W, X>(c, nullptr, its, v, x[1], body, a.inner);
        }
        p = 0, ++n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t col = quad * 2 + i % 2;
          if (col < tokens) own[pairs.token[begin + col] * 16 + gid + (i / 2) * 8] += c[i];
          c[i] = 0.0f;
        }
        __syncwarp();
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
        sum += cluster_sum(block + j * size + i, first, split);
        static_cast<T*>(a.y)[(uint64_t)t * a.hidden + place] = from_float<T>(sum);
      }
    }
    cluster_sync();
  }
  stages.end();
}

template <bool kShift, class T, class W>
__global__ void __launch_bounds__(kThreads, 2) zc_layer_down_kernel(const __grid_constant__ LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t s_dyn[];
  __shared__ Ring s_ring;
  PairSource& source = *reinterpret_cast<PairSource*>(s_dyn);
  ring_init(s_ring);
  pdl_wait();
  for (uint32_t i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads) source.ids[i] = (uint32_t)a.ids[i];
  __syncthreads();
  const Pairs pairs(s_dyn + down_memory<kShift>(a.tokens, a.stages), a.tokens * a.top_k);
  gather_pairs<false>(pairs, source, a.tokens, a.top_k, a.experts);
  layer_down<kShift, T, W>(a, pairs, s_ring, s_dyn);
  pdl_trigger();
}

template <bool kShift, class T, class W>
cudaError_t down_launch(LayerArgs a, cudaStream_t s) {
  static std::atomic<int> known[kMaxDevices];
  const auto kernel = zc_layer_down_kernel<kShift, T, W>;
  const uint32_t pairs = a.tokens * a.top_k, tiles = (a.hidden + 15) / 16;
  a.stages = kMaxStages;
  while (a.stages > 2 && down_memory<kShift>(a.tokens, a.stages) + Pairs::bytes(pairs) > kRoomForTwo) --a.stages;
  int clusters = 0;
  const cudaError_t e = clusters_at_once(kernel, known, kRoomForTwo, down_memory<kShift>(kMaxTokens, kMaxStages) + Pairs::bytes(kMaxTokens * kMaxTopK), &clusters);
  return e != cudaSuccess ? e : launch_clusters(kernel, std::min<uint32_t>(clusters, tiles), down_memory<kShift>(a.tokens, a.stages) + Pairs::bytes(pairs), s, a);
}

template <class T>
cudaError_t down_by_weights(const LayerArgs& a, bool blocks, cudaStream_t s) {
  if (blocks) return down_launch<false, T, F8>(a, s);  // rows of codes start at multiples of 16
  return a.shift_down ? down_launch<true, T, T>(a, s) : down_launch<false, T, T>(a, s);
}

}  // namespace

cudaError_t layer_down_launch(const LayerArgs& a, int type, bool blocks, cudaStream_t s) {
  return type == ZIPCCL_TYPE_F32    ? down_by_weights<float>(a, blocks, s)
         : type == ZIPCCL_TYPE_BF16 ? down_by_weights<__nv_bfloat16>(a, blocks, s)
                                    : down_by_weights<__half>(a, blocks, s);
}
cudaError_t layer_down_waits(cudaStream_t s, bool* ran_out) { return take_flag(g_layer_down_ran_out, s, ran_out); }

}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_layer_workspace_bytes(uint64_t tokens, uint32_t top_k, uint64_t inner, uint64_t* out_bytes) {
  if (!out_bytes || tokens > kMaxTokens || top_k == 0 || top_k > kMaxTopK || inner >= (1ull << 22)) return ZIPCCL_ERR_INVALID_ARG;
  *out_bytes = (tokens * top_k * ((inner + 7) / 8 * 8) * 8 + 255) / 256 * 256;  // two floats a value at most
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
      l->inner >= (1ull << 22) || (l->x_stride < l->hidden && l->x_stride != 0 && l->tokens > 1))
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
  const auto shifts = [](const void* p, uint64_t stride) { return !host_aligned(p, 16) || stride % 16 != 0; };
  const bool shift_x = shifts(l->d_x, l->x_stride * z);
  a.shift_up = shift_x || shifts(l->d_router, l->hidden * rz) || shifts(l->d_up, l->up_stride * wz);
  a.shift_down = shifts(l->d_down, l->down_stride * wz);
  // (row numbers of a map are whole numbers of 32 bits)
  const uint64_t up_rows = (l->gated ? 2 : 1) * l->inner;
  if (experts * up_rows >= (1ull << 31) || experts * l->hidden >= (1ull << 31)) return ZIPCCL_ERR_INVALID_ARG;
  if (((!a.shift_up || blocks) && !word_map(&a.up_map, l->d_up, l->hidden * wz, experts * up_rows, l->up_stride * wz, kPiece / 8, 8)) ||
      (!a.shift_down && !word_map(&a.down_map, l->d_down, l->inner * wz, experts * l->hidden, l->down_stride * wz, kPiece / 8, 8)))
    return ZIPCCL_ERR_CUDA;
  RouteArgs& r = a.route;
  const uint32_t L = lanes_of_token(experts, o->top_k, o->groups), V = experts_of_lane(experts, L), B = V < 4 ? V : 4;
  r.bias = l->d_bias;
  r.mask = l->d_mask;
  r.experts = experts;
  r.top_k = o->top_k;
  r.groups = o->groups;
  r.kept = o->groups_kept;
  r.group_size = experts / o->groups;
  r.scale = o->scale;
  const uint32_t lanes = r.group_size % V ? 0 : r.group_size / V;
  r.group_lanes = lanes & (lanes - 1) || r.groups > L ? 0 : lanes;
  r.softmax = o->score == ZIPCCL_SCORE_SOFTMAX;
  r.renormalize = o->renormalize != 0;
  r.top2 = o->group_score == ZIPCCL_GROUP_TOP2;
  r.wide = experts % B == 0;
  r.wide_bias = host_aligned(l->d_bias, B * sizeof(float)) && experts % B == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = layer_up_launch(a, l->type, blocks, s);
  if (e == cudaSuccess) e = layer_down_launch(a, l->type, blocks, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // extern "C"
