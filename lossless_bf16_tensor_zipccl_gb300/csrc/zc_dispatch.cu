// zc_dispatch.cu -- tokens' rows to the experts' chunks and back: dispatch,
// combine and their gradients.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr uint32_t kMaxTopK = 32;
constexpr int kRowThreads = 256;
constexpr uint32_t kPipeSmemMax = 110 << 10;

struct RowArgs {
  const void* src;        // dispatch: x;  combine: rows;  combine backward: rows
  const void* side;       // combine: residual (nullable);  combine backward: gradient of y
  const float* weights;   // nullable: 1
  const int32_t* slots;
  void* dst;              // dispatch: rows;  combine: y;  combine backward: gradient of rows
  float* grad_weights;
  uint64_t stride;        // dispatch: values between rows of x
  uint64_t hidden;
  uint32_t tokens, top_k;
  uint64_t rows;          // tokens * top_k
  uint32_t lead;          // dispatch of rows without a common alignment: x starts `lead` bytes after src
};

// Two forms of the kernels.
//  - Plain: blockDim.x threads share a token, blockDim.y tokens a block, so
//    that narrow rows fill it too.  Dispatch of rows that are multiples of 16
//    bytes takes it, a vector at a time: it only stores what it has loaded
//    once, and stores wait for nothing (16,384 x 4,096 bf16, two pairs: 61 us,
//    99% of the measured copy rate).  Elsewhere it goes value by value: where
//    results or the experts' rows do not start at a multiple of 16 bytes (the
//    same size, combine: 277 us against 61).
//  - Piped: combine and its gradient gather rows, so a warp that loads, sums
//    and stores waits for a slot and then for a row each time, and more loads
//    in registers cost warps (the same size: 73 and 124 us at best).  Here
//    each warp keeps a ring of row pieces in shared memory, filled by
//    asynchronous copies two stages ahead of what it sums, over all its rows
//    in turn: 61 and 105 us, 99 and 96% of the copy rate.  For a few tokens it is
//    0.3 us slower than the plain form by vectors, which is not kept for that.
// Rows whose size is no multiple of 16 bytes start at any place within 16.
// The piped form (and dispatch) then works on the vectors of the row that is
// written, and takes the other rows' bytes from the aligned pieces that cover
// them, shifted.

// rows[slot] = x[token] for each of the token's pairs; a dropped pair's row
// (slot -1 - row) is zeros.  A slot outside the buffer is skipped.  Values are
// moved as they are: W is any type of a vector's size.
template <class W>
__global__ void __launch_bounds__(kRowThreads) zc_dispatch_kernel(RowArgs a, uint64_t stride, uint64_t nv) {
  after_previous();
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.tokens) return;
  const int32_t* slots = a.slots + t * a.top_k;
  const W* x = static_cast<const W*>(a.src) + t * stride;
  W* dst = static_cast<W*>(a.dst);
  for (uint64_t v = threadIdx.x; v < nv; v += blockDim.x) {
    const W p = x[v];
    for (uint32_t k = 0; k < a.top_k; ++k) {
      const int32_t s = slots[k];
      const uint64_t row = (uint64_t)(s < 0 ? ~s : s);
      if (row < a.rows) dst[row * nv + v] = s < 0 ? W{} : p;
    }
  }
}

// y[token] = residual + sum over its pairs of weight * rows[slot], in pair
// order, held in 32 bits and rounded once.
template <class T>
__global__ void __launch_bounds__(kRowThreads) zc_combine_kernel(RowArgs a) {
  after_previous();
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.tokens) return;
  const int32_t* slots = a.slots + t * a.top_k;
  const T* src = static_cast<const T*>(a.src);
  for (uint64_t i = threadIdx.x; i < a.hidden; i += blockDim.x) {
    float y = 0.0f;
    for (uint32_t k = 0; k < a.top_k; ++k) {
      const int32_t s = slots[k];
      if (s < 0 || (uint64_t)s >= a.rows) continue;
      const float w = a.weights ? a.weights[t * a.top_k + k] : 1.0f;
      y = fmaf(w, to_float(src[(uint64_t)s * a.hidden + i]), y);
    }
    if (a.side) y += to_float(static_cast<const T*>(a.side)[t * a.hidden + i]);
    static_cast<T*>(a.dst)[t * a.hidden + i] = from_float<T>(y);
  }
}

// grad_rows[slot] = weight * grad[token], grad_weight = <grad[token], rows[slot]>.
// The products are summed along a fixed tree: a thread's, lanes, warps.
template <class T>
__global__ void __launch_bounds__(kRowThreads) zc_combine_backward_kernel(RowArgs a) {
  after_previous();
  __shared__ float s_dot[kRowThreads / 32];
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < a.tokens;
  const uint32_t width = min(blockDim.x, 32u);
  const uint32_t warp = (threadIdx.y * blockDim.x + threadIdx.x) / 32, warps = blockDim.x / 32;
  const T* g = static_cast<const T*>(a.side) + t * a.hidden;
  for (uint32_t k = 0; k < a.top_k; ++k) {
    const int32_t s = live ? a.slots[t * a.top_k + k] : INT32_MIN;
    const uint64_t row = (uint64_t)(s < 0 ? ~s : s);
    const bool in = row < a.rows;
    const float w = !in || s < 0 ? 0.0f : a.weights ? a.weights[t * a.top_k + k] : 1.0f;
    const T* r = static_cast<const T*>(a.src) + row * a.hidden;
    T* out = static_cast<T*>(a.dst) + row * a.hidden;
    float dot = 0.0f;
    if (in)
      for (uint64_t i = threadIdx.x; i < a.hidden; i += blockDim.x) {
        const float x = s < 0 ? 0.0f : to_float(g[i]);
        if (s >= 0) dot = fmaf(x, to_float(r[i]), dot);
        out[i] = from_float<T>(s < 0 ? 0.0f : w * x);
      }
    if (!a.grad_weights) continue;
    for (uint32_t o = width / 2; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
    if (blockDim.x <= 32) {
      if (live && threadIdx.x == 0) a.grad_weights[t * a.top_k + k] = dot;
      continue;
    }
    if (threadIdx.x % 32 == 0) s_dot[warp] = dot;
    __syncthreads();
    if (live && threadIdx.x == 0) {
      float sum = 0.0f;
      for (uint32_t i = 0; i < warps; ++i) sum += s_dot[warp + i];
      a.grad_weights[t * a.top_k + k] = sum;
    }
    __syncthreads();
  }
}

// ---- piped form
constexpr int kPipeThreads = 256, kPipeWarps = kPipeThreads / 32;
constexpr uint32_t kOpenRows = 12;  // rows of two pieces or more that two turns of a block's warps touch, and one more
constexpr int kStages = 3;   // of a lane's ring
constexpr int kStageVec = 4; // vectors of 16 bytes a lane has in a stage: V of each of kStageVec / V rows

// 16 bytes global -> shared, asynchronously; `bytes` < 16 reads only these and
// fills up with zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 shared8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

// The 16 bytes at a shared address that is a multiple of 2; up to 24 bytes
// from the multiple of 8 below it are read.
__device__ __forceinline__ uint4 shared16_shifted(uint32_t at) {
  const uint32_t from = at & ~7u;
  const uint2 p = shared8(from), q = shared8(from + 8), r = shared8(from + 16);
  const bool word = at & 4;
  const uint32_t bits = (at & 2) * 8;
  const uint32_t w0 = word ? p.y : p.x, w1 = word ? q.x : p.y, w2 = word ? q.y : q.x, w3 = word ? r.x : q.y,
                 w4 = word ? r.y : r.x;
  uint4 v;
  v.x = __funnelshift_r(w0, w1, bits);
  v.y = __funnelshift_r(w1, w2, bits);
  v.z = __funnelshift_r(w2, w3, bits);
  v.w = __funnelshift_r(w3, w4, bits);
  return v;
}

// The same where it is known which words and halves of words are wanted.
template <int kWord, int kHalf>
__device__ __forceinline__ uint4 shared16_at(uint32_t from) {
  const uint2 p = shared8(from), q = shared8(from + 8);
  if constexpr (!kWord && !kHalf) return make_uint4(p.x, p.y, q.x, q.y);
  const uint2 r = shared8(from + 16);
  const uint32_t w[6] = {p.x, p.y, q.x, q.y, r.x, r.y};
  if constexpr (!kHalf) return make_uint4(w[1], w[2], w[3], w[4]);
  return make_uint4(__funnelshift_r(w[kWord], w[kWord + 1], 16), __funnelshift_r(w[kWord + 1], w[kWord + 2], 16),
                    __funnelshift_r(w[kWord + 2], w[kWord + 3], 16), __funnelshift_r(w[kWord + 3], w[kWord + 4], 16));
}

// Calls f(h, the 16 bytes at shared address at + h * step) for h < V; `at` is a
// multiple of 2, and its place within 8 the same for a whole warp if kWarp
// (one branch then takes the place of selecting every word).
template <int V, bool kWarp, class F>
__device__ __forceinline__ void each_shifted(uint32_t at, uint32_t step, F f) {
  if constexpr (!kWarp) {
#pragma unroll
    for (int h = 0; h < V; ++h) f(h, shared16_shifted(at + h * step));
  } else {
    const uint32_t from = at & ~7u;
    switch (at >> 1 & 3) {
      case 0:
#pragma unroll
        for (int h = 0; h < V; ++h) f(h, shared16_at<0, 0>(from + h * step));
        break;
      case 1:
#pragma unroll
        for (int h = 0; h < V; ++h) f(h, shared16_at<0, 1>(from + h * step));
        break;
      case 2:
#pragma unroll
        for (int h = 0; h < V; ++h) f(h, shared16_at<1, 0>(from + h * step));
        break;
      default:
#pragma unroll
        for (int h = 0; h < V; ++h) f(h, shared16_at<1, 1>(from + h * step));
    }
  }
}

template <class T>
using Vec = Pack<T, 16 / sizeof(T)>;

template <class T>
__device__ __forceinline__ Vec<T> as_vec(uint4 v) {
  union { uint4 u; Vec<T> p; } x;
  x.u = v;
  return x.p;
}

// A vector of a row of `hidden` values whose first value has place `first`.  Its
// values outside the row are not written: that is a function of its own, for
// the code around each vector to stay small.
template <class T>
__device__ __noinline__ void put_edge(T* row, uint4 v, int32_t first, int32_t hidden) {
  constexpr int N = 16 / sizeof(T);
  const Vec<T> o = as_vec<T>(v);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (first + i >= 0 && first + i < hidden) row[first + i] = o.v[i];
}
template <class T>
__device__ __forceinline__ uint4 as_words(const Vec<T>& v) {
  union { Vec<T> p; uint4 u; } x;
  x.p = v;
  return x.u;
}
template <class T, bool kOdd>
__device__ __forceinline__ void put(T* row, const Vec<T>& o, int32_t first, int32_t hidden) {
  constexpr int N = 16 / sizeof(T);
  if (!kOdd || (first >= 0 && first + N <= hidden))
    *reinterpret_cast<Vec<T>*>(row + first) = o;
  else
    put_edge<T>(row, as_words<T>(o), first, hidden);
}

// The gradient's row and the product's part of such a vector.
template <class T>
__device__ __noinline__ float take_edge(T* row, uint4 grad, uint4 value, float w, int32_t first, int32_t hidden) {
  constexpr int N = 16 / sizeof(T);
  const Vec<T> g = as_vec<T>(grad), p = as_vec<T>(value);
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (first + i >= 0 && first + i < hidden) {
      dot = fmaf(to_float(g.v[i]), to_float(p.v[i]), dot);
      row[first + i] = from_float<T>(w * to_float(g.v[i]));
    }
  return dot;
}

// What the piped kernels work with: groups of `lanes` lanes take pieces of
// lanes * V vectors of a row.
struct Pipe {
  uint32_t log_lanes;  // lanes of a group: 4 to 32
  uint32_t pieces;     // of a row
  uint32_t bytes;      // of a row
};

// Copies the aligned 16-byte units that cover a piece of a row without common
// alignment; the piece starts at byte `at` (of `total`) of the buffer, `at`
// mod 16 into the stage.  Lane's units lane, lane + lanes, ... of
// V * lanes + kExtra, those below `count`, exist; units outside the buffer are
// left out, one that passes its end is cut there, and of one that starts
// before its first byte (`lead` after a multiple of 16) the rest is read singly.
template <int V, int kExtra>
__device__ __forceinline__ void copy_cover(uint32_t stage, const void* buffer, int64_t at, int64_t total, uint32_t lane,
                                           uint32_t lanes, int32_t count, uint32_t lead = 0) {
  const int64_t at0 = (at & ~int64_t(15)) + 16 * lane;
  const bool inside = (at & ~int64_t(15)) >= (int64_t)lead && (at & ~int64_t(15)) + 16 * (int64_t)(V * lanes + kExtra) <= total;
  const uint8_t* from = static_cast<const uint8_t*>(buffer) + at0;
  uint32_t to = stage + 16 * lane;
#pragma unroll
  for (int i = 0; i <= V; ++i) {
    if (i == V && (int)lane >= kExtra) break;
    if ((int32_t)(i * lanes + lane) < count) {
      const int64_t b = at0 + 16 * (int64_t)(i * lanes);
      if (inside) copy16(to + 16 * i * lanes, from + 16 * i * lanes);
      else if (b >= (int64_t)lead && b < total) copy16(to + 16 * i * lanes, from + 16 * i * lanes, (uint32_t)min(total - b, (int64_t)16));
      else if (b == 0 && lead) {
        for (uint32_t j = lead; j < 16 && j < total; j += 2)
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 16 * i * lanes + j),
                       "h"(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(buffer) + j))
                       : "memory");
      }
    }
  }
}

template <class T, int V, bool kOdd>
__global__ void __launch_bounds__(kPipeThreads) zc_combine_pipe_kernel(RowArgs a, Pipe q) {
  constexpr int N = 16 / sizeof(T), R = kStageVec / V;  // rows of a stage
  extern __shared__ __align__(16) uint8_t ring[];
  const uint32_t lanes = V > 1 ? 32 : 1u << q.log_lanes, lane = threadIdx.x & (lanes - 1);
  const uint32_t row_stage = (lanes * V + (kOdd ? 1 : 0)) * 16, group_stage = row_stage * R;
  const uint32_t groups = gridDim.x * kPipeThreads >> q.log_lanes;
  const uint32_t group = (blockIdx.x * kPipeThreads + threadIdx.x) >> q.log_lanes;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + (threadIdx.x >> q.log_lanes) * group_stage * kStages;
  const uint32_t items = a.tokens * q.pieces, turns = (items + groups - 1) / groups;
  const uint32_t rows = (uint32_t)a.rows, top_k = a.top_k;
  const uint32_t loads = top_k + (a.side ? 1 : 0);  // rows of an item, the residual's last
  const int32_t hidden = (int32_t)a.hidden;
  const uint8_t* src = static_cast<const uint8_t*>(a.src);
  const uint8_t* side = static_cast<const uint8_t*>(a.side);

  // the item whose rows are being copied, ahead of the one that is summed
  uint32_t c_item = group, c_k = 0, c_to = mine, c_t = 0;
  int32_t c_rel = 0, c_count = 0;  // first byte within the row; vectors or units from there on
  const int32_t* c_slots = nullptr;
  auto open = [&]() {
    uint32_t piece = 0;
    c_t = c_item;
    if (q.pieces > 1) c_t = c_item / q.pieces, piece = c_item - c_t * q.pieces;
    const uint32_t shift = kOdd ? c_t * q.bytes & 15 : 0;
    c_rel = (int32_t)(16 * piece * lanes * V) - (int32_t)shift;
    c_count = (int32_t)((q.bytes + shift + 15) / 16 - piece * lanes * V) + (kOdd ? 1 : 0);
    c_slots = a.slots + (uint64_t)c_t * top_k;
  };
  if (c_item < items) open();
  auto copy_next = [&]() {
    if (c_item < items) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t k = c_k + j, to = c_to + j * row_stage;
        if (k >= loads) break;
        uint32_t row = c_t;
        bool ok = true;
        const uint8_t* from = side;
        if (k < top_k) {
          row = (uint32_t)c_slots[k];
          ok = row < rows;
          from = src;
        }
        if (!ok) continue;
        if (kOdd) {
          copy_cover<V, 1>(to, from, (int64_t)((uint64_t)row * q.bytes) + c_rel,
                           (int64_t)((uint64_t)(k < top_k ? rows : a.tokens) * q.bytes), lane, lanes, c_count);
        } else {
          const uint8_t* at = from + (uint64_t)row * q.bytes + (c_rel + 16 * lane);
#pragma unroll
          for (int h = 0; h < V; ++h)
            if ((int32_t)(h * lanes + lane) < c_count) copy16(to + 16 * (h * lanes + lane), at + 16 * h * lanes);
        }
      }
      if ((c_k += R) >= loads) {
        c_k = 0;
        if ((c_item += groups) < items) open();
      }
    }
    copy_commit();
    if ((c_to += group_stage) == mine + kStages * group_stage) c_to = mine;
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_next();

  uint32_t stage = mine;
  for (uint32_t turn = 0; turn < turns; ++turn) {
    const uint32_t item = group + turn * groups;
    const bool live = item < items;
    uint32_t t = live ? item : 0, piece = 0;
    if (q.pieces > 1) piece = t, t /= q.pieces, piece -= t * q.pieces;
    const uint32_t shift = kOdd ? t * q.bytes & 15 : 0;
    const int32_t* slots = a.slots + (uint64_t)t * top_k;
    const float* weights = a.weights ? a.weights + (uint64_t)t * top_k : nullptr;
    float y[V][N];
#pragma unroll
    for (int h = 0; h < V; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) y[h][i] = 0.0f;
    for (uint32_t k0 = 0; k0 < loads; k0 += R) {
      uint32_t row[R];
      float w[R];
      bool ok[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t k = k0 + j;
        row[j] = k < top_k ? (uint32_t)slots[k] : t;
        ok[j] = live && k < loads && (k >= top_k || row[j] < rows);
        w[j] = weights && k < top_k ? weights[k] : 1.0f;
      }
      copy_wait<kStages - 2>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!ok[j]) continue;
        const uint32_t at = stage + j * row_stage + 16 * lane + (kOdd ? (row[j] * q.bytes - shift) & 15 : 0);
        auto add = [&](int h, uint4 v) {
          const Vec<T> p = as_vec<T>(v);
#pragma unroll
          for (int i = 0; i < N; ++i) y[h][i] = fmaf(w[j], to_float(p.v[i]), y[h][i]);
        };
        if constexpr (kOdd) {
          each_shifted<V, (V > 1)>(at, 16 * lanes, add);
        } else {
#pragma unroll
          for (int h = 0; h < V; ++h) add(h, shared16(at + 16 * h * lanes));
        }
      }
      copy_next();
      if ((stage += group_stage) == mine + kStages * group_stage) stage = mine;
    }
    if (!live) continue;
    T* out = static_cast<T*>(a.dst) + (uint64_t)t * a.hidden;
#pragma unroll
    for (int h = 0; h < V; ++h) {
      const int32_t e = (int32_t)((piece * lanes * V + h * lanes + lane) * N) - (int32_t)(shift / sizeof(T));
      if (e >= hidden) break;
      put<T, kOdd>(out, rounded<T, N>(y[h]), e, hidden);
    }
  }
}

// As zc_combine_pipe_kernel; of each piece the token's gradient is copied
// first, then the pairs' rows.  A row of one piece belongs to a group, which
// has its products' sums.  A row of more belongs to a block, whose warps take
// its pieces in turn (tokens are too large a share: 16,384 of them over 3,648
// warps leave a tenth of the time to the last turn) and leave their sums in
// shared memory; they are added after the round of pieces that ends the row.
template <class T, int V, bool kOdd>
__global__ void __launch_bounds__(kPipeThreads) zc_combine_backward_pipe_kernel(RowArgs a, Pipe q) {
  constexpr int N = 16 / sizeof(T), R = kStageVec / V;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float s_sum[kOpenRows][kPipeWarps][kMaxTopK];
  const uint32_t lanes = V > 1 ? 32 : 1u << q.log_lanes, lane = threadIdx.x & (lanes - 1);
  const uint32_t row_stage = (lanes * V + (kOdd ? 2 : 0)) * 16, group_stage = row_stage * R;
  const uint32_t groups = gridDim.x * kPipeThreads >> q.log_lanes;
  const uint32_t group = (blockIdx.x * kPipeThreads + threadIdx.x) >> q.log_lanes;
  // where rows have no common alignment the gradient's piece stays in a place
  // of its own, in front of the ring, for every pair to read at its own shift
  const uint32_t kept = (uint32_t)__cvta_generic_to_shared(ring) +
                        (threadIdx.x >> q.log_lanes) * (group_stage * kStages + (kOdd ? row_stage + 32 : 0));
  const uint32_t mine = kept + (kOdd ? row_stage + 32 : 0);
  const uint32_t rows = (uint32_t)a.rows, top_k = a.top_k;
  const int32_t hidden = (int32_t)a.hidden;
  const uint8_t* src = static_cast<const uint8_t*>(a.src);
  const uint8_t* side = static_cast<const uint8_t*>(a.side);

  // the pieces of this group or warp: it starts with one and goes on by one
  // turn of all groups, or of the block's warps
  const bool split = q.pieces > 1;
  const uint32_t warp = threadIdx.x / 32;
  const uint32_t my_tokens = a.tokens > blockIdx.x ? (a.tokens - blockIdx.x - 1) / gridDim.x + 1 : 0;  // split: the block's
  const uint32_t turns = split ? (my_tokens * q.pieces + kPipeWarps - 1) / kPipeWarps : (a.tokens + groups - 1) / groups;
  struct At { uint32_t n, piece, t; };  // split: the n-th token of the block
  auto norm = [&](At& p) {
    if (split) {
      while (p.piece >= q.pieces) p.piece -= q.pieces, ++p.n;
      p.t = p.n < my_tokens ? blockIdx.x + p.n * gridDim.x : a.tokens;
    }
  };
  auto next = [&](At& p) {
    if (split) {
      p.piece += kPipeWarps;
      norm(p);
    } else {
      p.t += groups;
    }
  };
  At c = {0, split ? warp : 0, group}, at = c;
  norm(c);
  norm(at);

  uint32_t c_to = mine;
  int32_t c_k = -1;  // -1: the token's gradient
  auto copy_next = [&]() {
    if (c.t < a.tokens) {
      const uint32_t c_first = c.piece * lanes * V;
      if (c_k < 0) {
        const uint8_t* from = side + 16 * (uint64_t)lane;
        if (kOdd) {
          // from the first value any pair may want: 15 bytes before the piece
          copy_cover<V, 2>(c_to, side, (int64_t)((uint64_t)c.t * q.bytes + 16 * c_first) - (c_first ? 15 : 0),
                           (int64_t)((uint64_t)a.tokens * q.bytes), lane, lanes, (int32_t)((q.bytes + 15) / 16 - c_first) + 2);
        } else {
          from += (uint64_t)c.t * q.bytes + 16 * c_first;
#pragma unroll
          for (int h = 0; h < V; ++h)
            if (c_first + h * lanes + lane < q.bytes / 16) copy16(c_to + 16 * (h * lanes + lane), from + 16 * h * lanes);
        }
        c_k = 0;
      } else {
        const int32_t* c_slots = a.slots + (uint64_t)c.t * top_k;
#pragma unroll
        for (int j = 0; j < R; ++j) {
          if (c_k + j >= (int32_t)top_k) break;
          const uint32_t row = (uint32_t)c_slots[c_k + j], to = c_to + j * row_stage;
          if (row >= rows) continue;
          // the row's own vectors: aligned, from the multiple of 16 it starts at or after
          const uint64_t at = (uint64_t)row * q.bytes & ~uint64_t(15);
          const uint32_t count = kOdd ? (uint32_t)(((uint32_t)(row * q.bytes & 15) + q.bytes + 15) / 16) : q.bytes / 16;
          const uint64_t total = (uint64_t)rows * q.bytes;
          const bool inside = at + 16 * (uint64_t)count <= total;
          const uint8_t* from = src + at + 16 * (uint64_t)(c_first + lane);
#pragma unroll
          for (int h = 0; h < V; ++h) {
            const uint32_t u = c_first + h * lanes + lane;
            if (u >= count) break;
            const uint32_t dst = to + 16 * (h * lanes + lane);
            if (!kOdd || inside) {
              copy16(dst, from + 16 * h * lanes);
            } else {
              copy16(dst, from + 16 * h * lanes, (uint32_t)min(total - (at + 16 * (uint64_t)u), (uint64_t)16));
            }
          }
        }
        c_k += R;
      }
      if (c_k >= (int32_t)top_k) {
        c_k = -1;
        next(c);
      }
    }
    copy_commit();
    if ((c_to += group_stage) == mine + kStages * group_stage) c_to = mine;
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_next();

  uint32_t stage = mine;
  float sum = 0.0f;  // split: of pair `lane`, over this warp's pieces of a row
  for (uint32_t turn = 0; turn < turns; ++turn, next(at)) {
    const uint32_t t = at.t, first = at.piece * lanes * V;
    const bool live = t < a.tokens;
    const int32_t* slots = a.slots + (uint64_t)(live ? t : 0) * top_k;
    const float* weights = a.weights ? a.weights + (uint64_t)(live ? t : 0) * top_k : nullptr;
    float* grads = a.grad_weights ? a.grad_weights + (uint64_t)t * top_k : nullptr;
    {
      float x[V][N];
      copy_wait<kStages - 2>();
      __syncwarp();
      if (kOdd) {
#pragma unroll
        for (int h = 0; h <= V; ++h) {
          if (h == V && lane >= 2) break;
          const uint4 v = shared16(stage + 16 * (h * lanes + lane));
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(kept + 16 + 16 * (h * lanes + lane)), "r"(v.x),
                       "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int h = 0; h < V; ++h) {
          const Vec<T> p = as_vec<T>(shared16(stage + 16 * (h * lanes + lane)));
#pragma unroll
          for (int i = 0; i < N; ++i) x[h][i] = to_float(p.v[i]);
        }
      }
      copy_next();
      if ((stage += group_stage) == mine + kStages * group_stage) stage = mine;
      // shared address of the token's row, as kept
      const uint32_t row_at = kept + 16 + (kOdd ? (uint32_t)((t * q.bytes + (first ? 16 * first - 15 : 0)) & 15) + (first ? 15 : 0) - 16 * first : 0);
      for (uint32_t k0 = 0; k0 < top_k; k0 += R) {
        int32_t s[R];
        float w[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const uint32_t k = k0 + j;
          s[j] = live && k < top_k ? slots[k] : INT32_MIN;
          w[j] = weights && k < top_k ? weights[k] : 1.0f;
        }
        copy_wait<kStages - 2>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < R; ++j) {
          if (k0 + j >= top_k) break;
          const uint32_t row = (uint32_t)(s[j] < 0 ? ~s[j] : s[j]);
          float dot = 0.0f;
          if (row < rows) {
            const uint32_t shift = kOdd ? row * q.bytes & 15 : 0;
            const uint32_t own = stage + j * row_stage + 16 * lane;
            T* out = static_cast<T*>(a.dst) + (uint64_t)row * a.hidden;
            const int32_t e0 = (int32_t)((first + lane) * N) - (int32_t)(shift / sizeof(T)), step = (int32_t)lanes * N;
            if (s[j] < 0) {
#pragma unroll
              for (int h = 0; h < V; ++h)
                if (e0 + h * step < hidden) put<T, kOdd>(out, as_vec<T>(make_uint4(0, 0, 0, 0)), e0 + h * step, hidden);
            } else {
              auto take = [&](int h, uint4 g16) {
                const int32_t e = e0 + h * step;
                if (e >= hidden) return;
                const uint4 p16 = shared16(own + 16 * h * lanes);
                if (kOdd && (e < 0 || e + N > hidden)) {
                  dot += take_edge<T>(out, g16, p16, w[j], e, hidden);
                  return;
                }
                if constexpr (kOdd) {
                  const Vec<T> g = as_vec<T>(g16);
#pragma unroll
                  for (int i = 0; i < N; ++i) x[h][i] = to_float(g.v[i]);
                }
                const Vec<T> p = as_vec<T>(p16);
                float z[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                  dot = fmaf(x[h][i], to_float(p.v[i]), dot);
                  z[i] = w[j] * x[h][i];
                }
                *reinterpret_cast<Vec<T>*>(out + e) = rounded<T, N>(z);
              };
              if constexpr (kOdd) {
                each_shifted<V, (V > 1)>(row_at + e0 * (int32_t)sizeof(T), 16 * lanes, take);
              } else {
#pragma unroll
                for (int h = 0; h < V; ++h) take(h, uint4{});
              }
            }
          }
          if (grads) {
            for (uint32_t o = lanes / 2; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
            if (!split) {
              if (live && lane == 0) grads[k0 + j] = dot;
            } else if (lane == k0 + j) {
              sum += dot;
            }
          }
        }
        copy_next();
        if ((stage += group_stage) == mine + kStages * group_stage) stage = mine;
      }
    }
    if (!split || !a.grad_weights) continue;
    if (at.piece + kPipeWarps >= q.pieces) {  // this warp's last of the row
      s_sum[at.n % kOpenRows][warp][lane] = sum;
      sum = 0.0f;
    }
    __syncthreads();
    // rows that end in this turn; the sums of the next turn's go elsewhere
    const uint32_t done = turn * kPipeWarps / q.pieces, until = min((turn + 1) * kPipeWarps / q.pieces, my_tokens);
    for (uint32_t i = threadIdx.x; i < (until - done) * top_k && done < until; i += kPipeThreads) {
      const uint32_t n = done + i / top_k, k = i % top_k;
      float dot = 0.0f;
      for (uint32_t p = 0; p < min(q.pieces, (uint32_t)kPipeWarps); ++p) dot += s_sum[n % kOpenRows][(n * q.pieces + p) % kPipeWarps][k];
      a.grad_weights[(uint64_t)(blockIdx.x + n * gridDim.x) * top_k + k] = dot;
    }
  }
}

// Dispatch of rows without a common alignment: a group takes a piece of a
// token's row, whose aligned cover it copies to shared memory one item ahead,
// and writes it to each pair's row in that row's vectors.
template <class T, int V>
__global__ void __launch_bounds__(kPipeThreads) zc_dispatch_odd_kernel(RowArgs a, Pipe q) {
  constexpr int N = 16 / sizeof(T), S = 2;
  extern __shared__ __align__(16) uint8_t ring[];
  const uint32_t lanes = V > 1 ? 32 : 1u << q.log_lanes, lane = threadIdx.x & (lanes - 1);
  const uint32_t group_stage = (lanes * V + 4) * 16;  // a unit in front: reads of a row's first vector start there
  const uint32_t groups = gridDim.x * kPipeThreads >> q.log_lanes;
  const uint32_t group = (blockIdx.x * kPipeThreads + threadIdx.x) >> q.log_lanes;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + (threadIdx.x >> q.log_lanes) * group_stage * S;
  const uint32_t items = a.tokens * q.pieces;
  const uint32_t turns = (items + groups - 1) / groups;
  const int64_t hidden = a.hidden, step = a.stride * sizeof(T);

  auto copy = [&](uint32_t item, uint32_t stage) {
    if (item < items) {
      const uint32_t t = item / q.pieces, piece = item - t * q.pieces;
      const int64_t first = (int64_t)piece * lanes * V, row = (int64_t)t * step + a.lead;
      copy_cover<V, 2>(mine + stage * group_stage + 16, a.src, row + 16 * first - (first ? 15 : 0), row + (int64_t)q.bytes,
                       lane, lanes, (int32_t)((q.bytes + 15) / 16 - first) + 2, a.lead);
    }
    copy_commit();
  };
  copy(group, 0);
  for (uint32_t turn = 0; turn < turns; ++turn) {
    const uint32_t item = group + turn * groups;
    copy(item + groups, (turn + 1) & 1);
    copy_wait<1>();
    __syncwarp();
    if (item < items) {
      const uint32_t t = item / q.pieces, piece = item - t * q.pieces;
      const int64_t first = (int64_t)piece * lanes * V, row_at = (int64_t)t * step + a.lead;
      const int64_t kept0 = ((row_at + 16 * first - (first ? 15 : 0)) & ~int64_t(15)) - row_at;
      const uint32_t from = mine + (turn & 1) * group_stage + 16;
      for (uint32_t k = 0; k < a.top_k; ++k) {
        const int32_t s = a.slots[(uint64_t)t * a.top_k + k];
        const int64_t row = s < 0 ? ~s : s;
        if ((uint64_t)row >= a.rows) continue;
        const int64_t shift = (int64_t)((uint64_t)row * q.bytes & 15);
        T* out = static_cast<T*>(a.dst) + row * hidden;
        const int32_t e0 = (int32_t)((first + lane) * N - shift / (int64_t)sizeof(T)), step = (int32_t)lanes * N;
        auto give = [&](int h, uint4 v) {
          if (e0 + h * step < (int32_t)hidden) put<T, true>(out, as_vec<T>(v), e0 + h * step, (int32_t)hidden);
        };
        if (s < 0) {
#pragma unroll
          for (int h = 0; h < V; ++h) give(h, make_uint4(0, 0, 0, 0));
        } else {
          each_shifted<V, (V > 1)>((uint32_t)((int64_t)from + e0 * (int64_t)sizeof(T) - kept0), 16 * lanes, give);
        }
      }
    }
    __syncwarp();
  }
}

enum class RowOp { kDispatch, kCombine, kCombineBackward };

// Plain form: threads that share a token, 4 to 256.
dim3 row_block(uint64_t nv) {
  uint32_t x = 4;
  while (x < kRowThreads && x < nv) x *= 2;
  return dim3(x, kRowThreads / x);
}

// Plain form, kN values at a time for dispatch and one otherwise.
template <class T, int kN>
cudaError_t plain_launch(RowOp op, const RowArgs& a, cudaStream_t s) {
  const dim3 block = row_block(a.hidden / kN);
  const uint32_t grid = (a.tokens + block.y - 1) / block.y;
  if (op == RowOp::kDispatch)
    return launch(zc_dispatch_kernel<Pack<T, kN>>, grid, block, 0, s, a, a.stride / kN, a.hidden / kN);
  return launch(op == RowOp::kCombine ? zc_combine_kernel<T> : zc_combine_backward_kernel<T>, grid, block, 0, s, a);
}

// A persistent launch: as many blocks as the device holds at once (looked up
// once for each kernel, device and group width), or as the items need.
template <void (*kKernel)(RowArgs, Pipe)>
cudaError_t pipe_launch(const RowArgs& a, const Pipe& q, uint64_t items, uint32_t smem, cudaStream_t s) {
  static std::atomic<int> resident[kMaxDevices][6];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int blocks = resident[dev][q.log_lanes].load(std::memory_order_acquire);
  if (!blocks) {
    int sms = 0, per = 0;
    if ((e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPipeSmemMax)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kKernel, kPipeThreads, smem)) != cudaSuccess)
      return e;
    if ((blocks = sms * per) == 0) return cudaErrorInvalidConfiguration;
    resident[dev][q.log_lanes].store(blocks, std::memory_order_release);
  }
  // as few blocks as take no more turns: all have the same number of items
  const uint64_t groups = kPipeThreads >> q.log_lanes, want = (items + groups - 1) / groups;
  const uint64_t turns = (want + blocks - 1) / blocks;
  // not through launch(): blocks that start where room first appears lie
  // unevenly, and a persistent block stays where it started (200 us for combine
  // and its gradient, 165 like this)
  kKernel<<<(uint32_t)((want + turns - 1) / turns), kPipeThreads, smem, s>>>(a, q);
  return cudaGetLastError();
}

template <class T, int V, bool kOdd>
cudaError_t pipe_form(RowOp op, const RowArgs& a, uint32_t log_lanes, uint64_t vectors, cudaStream_t s) {
  const uint32_t lanes = 1u << log_lanes, groups = kPipeThreads / lanes;
  Pipe q;
  q.log_lanes = log_lanes;
  q.bytes = (uint32_t)(a.hidden * sizeof(T));
  q.pieces = (uint32_t)((vectors + lanes * V - 1) / (lanes * V));
  const uint64_t items = (uint64_t)a.tokens * q.pieces;
  if (op == RowOp::kCombine)
    return pipe_launch<zc_combine_pipe_kernel<T, V, kOdd>>(a, q, items,
                       groups * (lanes * V + (kOdd ? 1 : 0)) * 16 * (kStageVec / V) * kStages + (kOdd ? 16 : 0), s);
  if (op == RowOp::kCombineBackward) {
    const uint32_t stage = (lanes * V + (kOdd ? 2 : 0)) * 16;
    return pipe_launch<zc_combine_backward_pipe_kernel<T, V, kOdd>>(
        a, q, q.pieces > 1 ? (uint64_t)a.tokens * groups : a.tokens, groups * (stage * (kStageVec / V * kStages) + (kOdd ? stage + 32 : 0)), s);
  }
  if constexpr (kOdd) return pipe_launch<zc_dispatch_odd_kernel<T, V>>(a, q, items, groups * (lanes * V + 4) * 16 * 2, s);
  return cudaErrorInvalidValue;
}

template <class T, bool kOdd>
cudaError_t pipe_by_width(RowOp op, const RowArgs& a, cudaStream_t s) {
  // vectors of a row: one more where it may start within one
  const uint64_t vectors = (a.hidden * sizeof(T) + 15) / 16 + (kOdd ? 1 : 0);
  if (vectors > 32) {
    // vectors of a lane, 4 to 2: those that leave the fewest places of a row's pieces empty
    const auto places = [&](uint64_t v) { return (vectors + 32 * v - 1) / (32 * v) * v; };
    if (places(4) <= places(3) && places(4) <= places(2)) return pipe_form<T, 4, kOdd>(op, a, 5, vectors, s);
    if (places(3) <= places(2)) return pipe_form<T, 3, kOdd>(op, a, 5, vectors, s);
    return pipe_form<T, 2, kOdd>(op, a, 5, vectors, s);
  }
  uint32_t log_lanes = 2;
  while ((1u << log_lanes) < vectors) ++log_lanes;
  return pipe_form<T, 1, kOdd>(op, a, log_lanes, vectors, s);
}

template <class T>
cudaError_t row_form(RowOp op, RowArgs& a, cudaStream_t s) {
  constexpr uint32_t z = sizeof(T), N = 16 / z;
  // pieces are counted in 32 bits; buffers start at multiples of 16 bytes, but
  // for the x of dispatch
  const bool pipe = host_aligned(a.side, 16) && host_aligned(a.dst, 16) && a.hidden && a.hidden * z < (1ull << 30) &&
                    (uint64_t)a.tokens * ((a.hidden + 511) / 512 + 1) < (1ull << 31) &&
                    (op == RowOp::kDispatch || host_aligned(a.src, 16));
  if (!pipe) return plain_launch<T, 1>(op, a, s);
  if (op != RowOp::kDispatch) return a.hidden % N ? pipe_by_width<T, true>(op, a, s) : pipe_by_width<T, false>(op, a, s);
  if (host_aligned(a.src, 16) && a.hidden % N == 0 && a.stride % N == 0) return plain_launch<T, N>(op, a, s);
  a.lead = (uint32_t)(reinterpret_cast<uintptr_t>(a.src) & 15);
  a.src = static_cast<const uint8_t*>(a.src) - a.lead;
  return pipe_by_width<T, true>(op, a, s);
}

zipccl_status rows(RowOp op, RowArgs& a, int type, uint64_t tokens, uint32_t top_k, uint64_t hidden, void* stream) {
  const uint32_t z = type_bytes(type);
  if (z == 0 || top_k == 0 || top_k > kMaxTopK || tokens * top_k >= (1ull << 31) || tokens >= (1ull << 31) ||
      hidden >= (1ull << 31))
    return ZIPCCL_ERR_INVALID_ARG;
  if (tokens == 0) return ZIPCCL_OK;
  if (!a.slots || !host_aligned(a.slots, 4) || !host_aligned(a.weights, 4) || !host_aligned(a.grad_weights, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  if (hidden && (!a.src || !a.dst || !host_aligned(a.src, z) || !host_aligned(a.dst, z) || !host_aligned(a.side, z)))
    return ZIPCCL_ERR_INVALID_ARG;
  if (hidden && op == RowOp::kCombineBackward && !a.side) return ZIPCCL_ERR_INVALID_ARG;
  if (hidden == 0 && !a.grad_weights) return ZIPCCL_OK;
  a.tokens = (uint32_t)tokens;
  a.top_k = top_k;
  a.hidden = hidden;
  a.rows = tokens * top_k;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == ZIPCCL_TYPE_F32    ? row_form<float>(op, a, s)
                        : type == ZIPCCL_TYPE_BF16 ? row_form<__nv_bfloat16>(op, a, s)
                                                   : row_form<__half>(op, a, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // namespace
}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_dispatch(const void* d_x, int type, uint64_t row_stride, uint64_t tokens, uint32_t top_k,
                                  uint64_t hidden, const int32_t* d_slots, void* d_rows, void* stream) {
  if (hidden >= (1ull << 31) || (tokens > 1 && row_stride < hidden && row_stride != 0)) return ZIPCCL_ERR_INVALID_ARG;
  RowArgs a{};
  a.src = d_x;
  a.stride = row_stride;
  a.slots = d_slots;
  a.dst = d_rows;
  return rows(RowOp::kDispatch, a, type, tokens, top_k, hidden, stream);
}

zipccl_status zipccl_moe_dispatch_backward(const void* d_grad_rows, int type, uint64_t tokens, uint32_t top_k,
                                           uint64_t hidden, const int32_t* d_slots, void* d_grad_x, void* stream) {
  RowArgs a{};
  a.src = d_grad_rows;
  a.slots = d_slots;
  a.dst = d_grad_x;
  return rows(RowOp::kCombine, a, type, tokens, top_k, hidden, stream);
}

zipccl_status zipccl_moe_combine(const void* d_rows, int type, uint64_t tokens, uint32_t top_k, uint64_t hidden,
                                 const int32_t* d_slots, const float* d_weights, const void* d_residual, void* d_y,
                                 void* stream) {
  RowArgs a{};
  a.src = d_rows;
  a.side = d_residual;
  a.weights = d_weights;
  a.slots = d_slots;
  a.dst = d_y;
  return rows(RowOp::kCombine, a, type, tokens, top_k, hidden, stream);
}

zipccl_status zipccl_moe_combine_backward(const void* d_grad_y, const void* d_rows, int type, uint64_t tokens,
                                          uint32_t top_k, uint64_t hidden, const int32_t* d_slots,
                                          const float* d_weights, void* d_grad_rows, float* d_grad_weights,
                                          void* stream) {
  RowArgs a{};
  a.src = d_rows;
  a.side = d_grad_y;
  a.weights = d_weights;
  a.slots = d_slots;
  a.dst = d_grad_rows;
  a.grad_weights = d_grad_weights;
  return rows(RowOp::kCombineBackward, a, type, tokens, top_k, hidden, stream);
}

}  // extern "C"
