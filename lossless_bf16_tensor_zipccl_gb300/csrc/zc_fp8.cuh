// zc_fp8.cuh -- 8-bit blocks: E4M3 codes with a power of two for each block of
// 128 values, and the chunks of rows that blocks of columns lie in.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zc_ops.cuh"

namespace zc {

constexpr uint32_t kFp8Block = ZIPCCL_FP8_BLOCK;
constexpr uint32_t kMaxChunks = 1024;  // experts of a call

// Byte of the scale 2^e, e the smallest exponent from -127 on with
// amax <= 448 * 2^e; the byte is e + 127.  448 = 1.75 * 2^8: a finite float
// 1.m * 2^a needs e = a - 8, one more where 1.m > 1.75.  In the float's bits:
// adding 0x1FFFFF (the mantissa's distance from above 1.75 to the next
// exponent) carries into the exponent exactly then.  Subnormals have a below
// -126, so e = -127 does for them.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t a = (amax_bits + 0x1FFFFFu) >> 23;  // a + 127, one more above 1.75
  return a > 8 ? a - 8 : 0;
}
// 2^-e of a scale's byte: what values are multiplied with, exact.  The byte is at
// most 247 (the largest float: 2^120).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four values as E4M3, nearest even; a magnitude above 448 does not come up, NaN stays NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Rows of a chunk, or of a block of one: `count` rows from `first` on.
struct Span {
  uint32_t first, count;
};

// Offsets of chunks as the kernels take them: from 0 on, never falling, within
// the rows, whatever the memory holds (none: one chunk of all rows).
// One step of a warp's walk over them, 32 chunks from e0 on: each lane gets its
// chunk's rows, `end` is carried from step to step (0 before the first).
__device__ __forceinline__ Span chunk_step(const int32_t* offsets, uint32_t experts, uint32_t rows, uint32_t e0, uint32_t* end) {
  const uint32_t lane = threadIdx.x & 31, e = e0 + lane;
  uint32_t o = 0;
  if (e < experts) o = offsets ? (uint32_t)min(max(offsets[e + 1], 0), (int32_t)rows) : rows;
  uint32_t top = max(o, *end);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kAll, top, d);
    if (lane >= d) top = max(top, y);
  }
  uint32_t first = __shfl_up_sync(kAll, top, 1);
  if (lane == 0) first = *end;
  *end = __shfl_sync(kAll, top, 31);
  return {first, top - first};
}

__device__ __forceinline__ uint32_t warp_inclusive_sum(uint32_t v) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += y;
  }
  return v;
}

}  // namespace zc
