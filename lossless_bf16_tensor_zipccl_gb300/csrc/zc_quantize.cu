// zc_quantize.cu -- rows and weights as 8-bit floating point with a power of two
// for each block of 128 values: along a row, down a column within its chunk, or
// 128 x 128 of a matrix.
//
// code = E4M3(x * 2^-e), scale = 2^e: the scaling is exact, so the one rounding
// is the code's.  e is the smallest exponent that leaves nothing above 448.
// Every form reads its input once: a value takes its own bytes, one for each code,
// and 1/128 for each scale.  32,768 x 4,096 bfloat16 values take 62.5 us by rows (96%
// of the copy rate), 84 by columns and 133 both ways (61%: a tile's columns need
// three barriers, and 18 instructions a value for two codes leave room for few
// warps); 268 M weights 126 us (95%).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zc_fp8.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kThreads = 256;
constexpr uint64_t kMaxCols = 1ull << 22;  // tiles of a row fit a grid's second dimension
constexpr uint32_t kInf = 0x7F800000u;

// 16 consecutive values of a row as they lie in memory.
template <class T>
struct Sixteen {
  static constexpr int kWords = 4 * sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {  // p: 16-byte aligned
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
  // Places col .. of a row of `cols` that starts anywhere (kShift) or at a multiple of
  // 16 bytes; zeros behind it.  No access leaves the 16 bytes that hold one of its values.
  template <bool kShift>
  __device__ __forceinline__ void load(const T* row, uint32_t col, uint32_t cols) {
    if constexpr (kShift) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(row), base = at & ~uintptr_t(15);
      const uint32_t shift = (uint32_t)(at & 15);
      const uint64_t off = (uint64_t)col * sizeof(T), last = (shift + (uint64_t)cols * sizeof(T) - 1) & ~uint64_t(15);
      uint4 v[kWords / 4 + 1];
#pragma unroll
      for (int i = 0; i <= kWords / 4; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(base + min(off + 16 * i, last)));
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) put(i, settle<true>({v[i], v[i + 1]}, shift));
    } else if (col + 16 <= cols) {
      load(row + col);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        put(i, __ldg(reinterpret_cast<const uint4*>(row + min(col + i * kPer16<T>, (cols - 1) / kPer16<T> * kPer16<T>))));
    }
    if (col + 16 > cols) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) put(i / 4, keep<T>(make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]), (int)cols - (int)col - i / 4 * kPer16<T>));
    }
  }
  __device__ __forceinline__ void put(int i, const uint4& v) { w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w; }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return __half2float(__ushort_as_half((unsigned short)(i % 2 ? w[i / 2] >> 16 : w[i / 2])));
  }
};

// Magnitudes, compared as whole numbers: a pair in a word for 16-bit types, the
// infinite ones and NaN above all others.
template <class T>
struct Magnitude {
  static constexpr bool kPair = sizeof(T) == 2;
  static __device__ __forceinline__ uint32_t of(uint32_t w) { return w & (kPair ? 0x7FFF7FFFu : 0x7FFFFFFFu); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return max(a, b, b);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b, uint32_t c) {  // one instruction
    if constexpr (kPair) return __vimax3_u16x2(a, b, c);
    else return __vimax3_u32(a, b, c);
  }
  // the same without what is not finite
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    constexpr uint32_t inf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    w = of(w);
    if constexpr (!kPair) return w >= kInf ? 0 : w;
    else return ((w & 0xFFFFu) >= inf ? 0 : w & 0xFFFFu) | ((w >> 16) >= inf ? 0 : w & 0xFFFF0000u);
  }
  // bits of one of them as a float
  static __device__ __forceinline__ uint32_t as_float(uint32_t m) {
    if constexpr (!kPair) return m;
    else if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    else return m << 16;
  }
  // the larger of a word's two, or the word itself
  static __device__ __forceinline__ uint32_t fold(uint32_t m) {
    if constexpr (kPair) return ::max(m & 0xFFFFu, m >> 16);
    else return m;
  }
};

// Largest magnitude of a thread's 16 values, as the bits of a float.
template <class T, bool kFinite>
__device__ __forceinline__ uint32_t top_of(const Sixteen<T>& x) {
  using M = Magnitude<T>;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < Sixteen<T>::kWords; i += 2) {
    if constexpr (kFinite) m = M::max(m, M::finite(x.w[i]), M::finite(x.w[i + 1]));
    else m = M::max(m, M::of(x.w[i]), M::of(x.w[i + 1]));
  }
  return M::as_float(M::fold(m));
}

// 16 codes.  kOdd: what is infinite becomes NaN (saturation would make it 448).
template <class T, bool kOdd>
__device__ __forceinline__ uint4 sixteen_codes(const Sixteen<T>& x, const float (&by)[16]) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = x.get(i);
    y[i] = v * by[i];
    if constexpr (kOdd) {
      if ((__float_as_uint(v) & 0x7FFFFFFFu) >= kInf) y[i] = __uint_as_float(0x7FC00000u);
    }
  }
  return make_uint4(codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7]), codes4(y[8], y[9], y[10], y[11]),
                    codes4(y[12], y[13], y[14], y[15]));
}
template <class T, bool kOdd>
__device__ __forceinline__ uint4 sixteen_codes(const Sixteen<T>& x, float by) {
  float all[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) all[i] = by;
  return sixteen_codes<T, kOdd>(x, all);
}

// Codes of 16 places of a row from `at` on, `left` of which are the row's.
__device__ __forceinline__ void store_codes(uint8_t* at, uint4 c, uint32_t left) {
  if (left >= 16) {
    *reinterpret_cast<uint4*>(at) = c;
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) at[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

struct RowArgs {
  const void* x;
  uint8_t *codes, *scales;
  uint64_t stride, code_stride, groups;  // groups: rows * blocks
  uint32_t cols, blocks;                 // blocks of a row
};

// Along the rows: 8 lanes take a block, 16 values each, in 16-byte loads and one
// 16-byte store.
template <class T, bool kShift>
__global__ void __launch_bounds__(kThreads) zc_quantize_rows_kernel(RowArgs a) {
  after_previous();
  const uint32_t part = threadIdx.x % 8;
  const uint64_t per_grid = (uint64_t)gridDim.x * (kThreads / 8);
  // every lane of a warp takes the same turns: the shuffles name all of them
  for (uint64_t g0 = (uint64_t)blockIdx.x * (kThreads / 8); g0 < a.groups; g0 += per_grid) {
    const uint64_t g = g0 + threadIdx.x / 8;
    const bool in = g < a.groups;
    const uint64_t row = in ? (a.groups >> 32 ? g / a.blocks : (uint32_t)g / a.blocks) : 0;
    const uint32_t block = in ? (uint32_t)(g - row * a.blocks) : 0;
    const uint32_t col = block * kFp8Block + part * 16;
    Sixteen<T> x;
    x.clear();
    if (in && col < a.cols) x.template load<kShift>(static_cast<const T*>(a.x) + row * a.stride, col, a.cols);
    uint32_t m = top_of<T, false>(x);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    const bool odd = m >= kInf;
    if (__any_sync(kAll, odd)) {
      m = top_of<T, true>(x);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    }
    const uint32_t s = scale_byte(m);
    if (!in) continue;
    if (part == 0) a.scales[g] = (uint8_t)s;
    if (col < a.cols) {
      const float by = scale_inverse(s);
      store_codes(a.codes + row * a.code_stride + col, odd ? sixteen_codes<T, true>(x, by) : sixteen_codes<T, false>(x, by),
                  a.cols - col);
    }
  }
}

// Down the columns, and 128 x 128 blocks: a block of the grid takes tiles of
// 128 rows x 128 columns.  A thread holds 16 columns of 4 rows (32 apart).
enum Form { kColumns, kBoth, kWeights };

struct TileArgs {
  const void* x;
  const int32_t* offsets;  // nullable: one chunk
  uint8_t *codes, *scales, *row_codes, *row_scales;
  uint64_t stride, code_stride, row_code_stride;
  uint32_t rows, cols, chunks;  // weights: rows of a matrix, and the matrices
  uint32_t scale_rows;          // columns: rows of the scales
  uint32_t tiles, turn;         // tiles along a row; how many of them a block of the grid takes
};

constexpr int kTileRows = 128;

template <class T, int kForm, bool kShift>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? (kShift || kForm == kBoth ? 3 : 4) : 2) zc_quantize_tiles_kernel(TileArgs a) {
  using M = Magnitude<T>;
  constexpr int W = Sixteen<T>::kWords;
  after_previous();
  __shared__ __align__(16) uint32_t s_top[8][4 * W * 2];
  __shared__ __align__(16) float s_by[kTileRows];
  const uint32_t part = threadIdx.x % 8, line = threadIdx.x / 8, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Span span;
  bool inside = true;
  uint64_t matrix = 0;
  if constexpr (kForm == kWeights) {
    const uint32_t high = (a.rows + kTileRows - 1) / kTileRows;
    matrix = blockIdx.x / high;
    const uint32_t r = (uint32_t)(blockIdx.x - matrix * high) * kTileRows;
    span = {r, min((uint32_t)kTileRows, a.rows - r)};
  } else {
    // the block's rows: each warp walks over the chunks for itself
    const uint32_t want = blockIdx.x;
    uint32_t end = 0, before = 0;
    bool found = false;
    for (uint32_t e0 = 0; e0 < a.chunks && !found; e0 += 32) {
      const Span c = chunk_step(a.offsets, a.chunks, a.rows, e0, &end);
      const uint32_t n = (c.count + kTileRows - 1) / kTileRows, upto = before + warp_inclusive_sum(n);
      const uint32_t who = __ballot_sync(kAll, want < upto);
      if (who) {
        const int l = __ffs(who) - 1;
        const uint32_t in = (want - (__shfl_sync(kAll, upto, l) - __shfl_sync(kAll, n, l))) * kTileRows;
        span.first = __shfl_sync(kAll, c.first, l) + in;
        span.count = min((uint32_t)kTileRows, __shfl_sync(kAll, c.count, l) - in);
        found = true;
      }
      before = __shfl_sync(kAll, upto, 31);
    }
    if (!found) {  // rows behind the last chunk: no blocks of columns, codes of zero
      inside = false;
      const uint64_t first = end + (uint64_t)(want - before) * kTileRows;
      span.first = (uint32_t)min(first, (uint64_t)a.rows);
      span.count = min((uint32_t)kTileRows, a.rows - span.first);
    }
  }
  const uint32_t t0 = blockIdx.y * a.turn, t1 = min(t0 + a.turn, a.tiles);
  for (uint32_t tile = t0; tile < t1; ++tile) {
    const uint32_t col0 = tile * kFp8Block, col = col0 + part * 16;
    const T* base = static_cast<const T*>(a.x) + (matrix * a.rows + span.first) * a.stride;
    Sixteen<T> x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j].clear();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (line + 32 * j < span.count && col < a.cols) x[j].template load<kShift>(base + (uint64_t)(line + 32 * j) * a.stride, col, a.cols);
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) all = max(all, top_of<T, false>(x[j]));
    // (also: the last turn's shared memory has been read)
    const bool odd = __syncthreads_or(all >= kInf) != 0;
    if constexpr (kForm == kBoth) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t r = line + 32 * j;
        uint32_t m = odd ? top_of<T, true>(x[j]) : top_of<T, false>(x[j]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
        if (r >= span.count) continue;
        const uint32_t s = scale_byte(m);
        const uint64_t row = span.first + r;
        if (part == 0) a.row_scales[row * a.tiles + tile] = (uint8_t)s;
        if (col < a.cols) {
          const float by = scale_inverse(s);
          store_codes(a.row_codes + row * a.row_code_stride + col, odd ? sixteen_codes<T, true>(x[j], by) : sixteen_codes<T, false>(x[j], by), a.cols - col);
        }
      }
    }
    if constexpr (kForm == kWeights) {
      if (odd) {
        all = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) all = max(all, top_of<T, true>(x[j]));
      }
      all = __reduce_max_sync(kAll, all);
      if (lane == 0) s_top[0][warp] = all;
      __syncthreads();
      uint32_t m = s_top[0][0];
#pragma unroll
      for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_top[0][i]);
      const uint32_t s = scale_byte(m);
      const float by = scale_inverse(s);
      if (threadIdx.x == 0) a.scales[(uint64_t)blockIdx.x * a.tiles + tile] = (uint8_t)s;
      if (col < a.cols)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (line + 32 * j < span.count)
            store_codes(a.codes + (matrix * a.rows + span.first + line + 32 * j) * a.code_stride + col,
                        odd ? sixteen_codes<T, true>(x[j], by) : sixteen_codes<T, false>(x[j], by), a.cols - col);
    } else {
      // a column's largest: over the thread's rows, the warp's, the block's
      uint32_t m[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (odd) m[i] = M::max(M::max(M::finite(x[0].w[i]), M::finite(x[1].w[i])), M::finite(x[2].w[i]), M::finite(x[3].w[i]));
        else m[i] = M::max(M::max(M::of(x[0].w[i]), M::of(x[1].w[i])), M::of(x[2].w[i]), M::of(x[3].w[i]));
        m[i] = M::max(m[i], __shfl_xor_sync(kAll, m[i], 8));
        m[i] = M::max(m[i], __shfl_xor_sync(kAll, m[i], 16));
      }
      if (lane < 8)
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<uint4*>(&s_top[warp][part * W + i]) = make_uint4(m[i], m[i + 1], m[i + 2], m[i + 3]);
      __syncthreads();
      if (threadIdx.x < 8 * W) {
        uint32_t c = s_top[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) c = M::max(c, s_top[i][threadIdx.x]);
        constexpr int N = M::kPair ? 2 : 1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t place = threadIdx.x * N + i;
          const uint32_t s = inside ? scale_byte(M::as_float(N == 2 ? (c >> (16 * i)) & 0xFFFFu : c)) : 0;
          s_by[place] = scale_inverse(s);
          if (blockIdx.x < a.scale_rows && col0 + place < a.cols) a.scales[(uint64_t)blockIdx.x * a.cols + col0 + place] = (uint8_t)s;
        }
      }
      __syncthreads();
      if (col < a.cols) {
        float by[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&s_by[part * 16 + i]);
          by[i] = v.x, by[i + 1] = v.y, by[i + 2] = v.z, by[i + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (line + 32 * j < span.count) {
            uint4 c = odd ? sixteen_codes<T, true>(x[j], by) : sixteen_codes<T, false>(x[j], by);
            if (!inside) c = make_uint4(0, 0, 0, 0);
            store_codes(a.codes + (uint64_t)(span.first + line + 32 * j) * a.code_stride + col, c, a.cols - col);
          }
      }
    }
  }
}

bool good_codes(const void* codes, uint64_t stride, uint64_t cols) {
  return codes && host_aligned(codes, 16) && stride >= cols && stride % 16 == 0;
}

template <class T>
cudaError_t rows_by_type(const RowArgs& a, bool shift, cudaStream_t s) {
  const uint32_t grid = (uint32_t)std::min<uint64_t>((a.groups + kThreads / 8 - 1) / (kThreads / 8), 152 * 32);
  return launch(shift ? zc_quantize_rows_kernel<T, true> : zc_quantize_rows_kernel<T, false>, grid, kThreads, 0, s, a);
}

template <class T, int kForm>
cudaError_t tiles_launch(const TileArgs& a, uint64_t high, bool shift, cudaStream_t s) {
  const dim3 grid((uint32_t)high, (a.tiles + a.turn - 1) / a.turn);
  return launch(shift ? zc_quantize_tiles_kernel<T, kForm, true> : zc_quantize_tiles_kernel<T, kForm, false>, grid, kThreads, 0, s, a);
}

template <class T>
cudaError_t tiles_by_form(const TileArgs& a, int form, uint64_t high, bool shift, cudaStream_t s) {
  return form == kWeights ? tiles_launch<T, kWeights>(a, high, shift, s)
         : form == kBoth  ? tiles_launch<T, kBoth>(a, high, shift, s)
                          : tiles_launch<T, kColumns>(a, high, shift, s);
}

cudaError_t tiles_by_type(TileArgs& a, int type, int form, uint64_t high, cudaStream_t s) {
  const uint64_t z = type_bytes(type);
  const bool shift = !host_aligned(a.x, 16) || a.stride * z % 16 != 0;
  a.tiles = (a.cols + kFp8Block - 1) / kFp8Block;
  // a block of the grid takes two tiles of its rows where enough blocks are left:
  // finding the rows among the chunks is paid once (32,768 x 4,096 both ways: 135 us
  // with one, 133 with two, 137 with eight)
  a.turn = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(high * a.tiles / (152 * 6), 1), 2);
  return type == ZIPCCL_TYPE_F32    ? tiles_by_form<float>(a, form, high, shift, s)
         : type == ZIPCCL_TYPE_BF16 ? tiles_by_form<__nv_bfloat16>(a, form, high, shift, s)
                                    : tiles_by_form<__half>(a, form, high, shift, s);
}

}  // namespace
}  // namespace zc

using namespace zc;

extern "C" {

zipccl_status zipccl_moe_quantize(const void* d_x, int type, uint64_t row_stride, uint64_t rows, uint64_t cols,
                                  uint8_t* d_codes, uint64_t code_stride, uint8_t* d_scales, void* stream) {
  const uint64_t z = type_bytes(type);
  if (z == 0 || rows >= (1ull << 31) || cols > kMaxCols) return ZIPCCL_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return ZIPCCL_OK;
  if (!d_x || !host_aligned(d_x, z) || !d_scales || !good_codes(d_codes, code_stride, cols)) return ZIPCCL_ERR_INVALID_ARG;
  RowArgs a{};
  a.x = d_x;
  a.codes = d_codes;
  a.scales = d_scales;
  a.stride = row_stride;
  a.code_stride = code_stride;
  a.cols = (uint32_t)cols;
  a.blocks = (uint32_t)((cols + kFp8Block - 1) / kFp8Block);
  a.groups = rows * a.blocks;
  const bool shift = !host_aligned(d_x, 16) || row_stride * z % 16 != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == ZIPCCL_TYPE_F32    ? rows_by_type<float>(a, shift, s)
                        : type == ZIPCCL_TYPE_BF16 ? rows_by_type<__nv_bfloat16>(a, shift, s)
                                                   : rows_by_type<__half>(a, shift, s);
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

zipccl_status zipccl_moe_quantize_columns(const void* d_x, int type, uint64_t row_stride, uint64_t rows, uint64_t cols,
                                          const int32_t* d_offsets, uint32_t experts, uint8_t* d_codes,
                                          uint64_t code_stride, uint8_t* d_scales, uint8_t* d_row_codes,
                                          uint64_t row_code_stride, uint8_t* d_row_scales, void* stream) {
  const uint64_t z = type_bytes(type);
  if (z == 0 || rows >= (1ull << 31) || cols > kMaxCols || experts == 0 || experts > kMaxChunks || (!d_offsets && experts != 1))
    return ZIPCCL_ERR_INVALID_ARG;
  if (cols == 0) return ZIPCCL_OK;
  if (!host_aligned(d_offsets, 4) || !d_scales) return ZIPCCL_ERR_INVALID_ARG;
  if (rows && (!d_x || !host_aligned(d_x, z) || !good_codes(d_codes, code_stride, cols))) return ZIPCCL_ERR_INVALID_ARG;
  if (rows && d_row_codes && (!d_row_scales || !good_codes(d_row_codes, row_code_stride, cols))) return ZIPCCL_ERR_INVALID_ARG;
  TileArgs a{};
  a.x = d_x;
  a.offsets = d_offsets;
  a.codes = d_codes;
  a.scales = d_scales;
  a.row_codes = d_row_codes;
  a.row_scales = d_row_scales;
  a.stride = row_stride;
  a.code_stride = code_stride;
  a.row_code_stride = row_code_stride;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.chunks = experts;
  a.scale_rows = (uint32_t)(rows / kFp8Block + experts);
  // one more than the blocks of all chunks: rows behind the last start anew
  const cudaError_t e = tiles_by_type(a, type, d_row_codes ? kBoth : kColumns, a.scale_rows + 1, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

zipccl_status zipccl_moe_quantize_weights(const void* d_w, int type, uint32_t experts, uint64_t rows, uint64_t cols,
                                          uint8_t* d_codes, uint64_t code_stride, uint8_t* d_scales, void* stream) {
  const uint64_t z = type_bytes(type);
  const uint64_t high = (rows + kTileRows - 1) / kTileRows * experts;
  if (z == 0 || rows >= (1ull << 31) || cols > kMaxCols || high >= (1ull << 31)) return ZIPCCL_ERR_INVALID_ARG;
  if (experts == 0 || rows == 0 || cols == 0) return ZIPCCL_OK;
  if (!d_w || !host_aligned(d_w, z) || !d_scales || !good_codes(d_codes, code_stride, cols)) return ZIPCCL_ERR_INVALID_ARG;
  TileArgs a{};
  a.x = d_w;
  a.codes = d_codes;
  a.scales = d_scales;
  a.stride = cols;
  a.code_stride = code_stride;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.chunks = experts;
  const cudaError_t e = tiles_by_type(a, type, kWeights, high, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
}

}  // extern "C"
