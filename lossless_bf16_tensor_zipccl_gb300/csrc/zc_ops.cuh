// zc_ops.cuh -- shared by the operators around the exchange (routing, plan,
// dispatch, combine, optimizer step): value types, 16-byte vectors of them,
// streaming loads and stores.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zipccl.h"

namespace zc {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMaxDevices = 64;  // devices of a process that what is looked up once is kept for

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// kN values moved as one 16-byte access, or a single value where rows or
// pointers are not 16-byte aligned.
template <class T, int kN>
struct alignas(sizeof(T) * kN) Pack {
  T v[kN];
};

// kN values rounded to T, in pairs where T has 16 bits.
template <class T, int kN>
__device__ __forceinline__ Pack<T, kN> rounded(const float (&x)[kN]) {
  Pack<T, kN> p;
#pragma unroll
  for (int i = 0; i < kN; ++i) p.v[i] = from_float<T>(x[i]);
  return p;
}
template <>
__device__ __forceinline__ Pack<__nv_bfloat16, 8> rounded<__nv_bfloat16, 8>(const float (&x)[8]) {
  Pack<__nv_bfloat16, 8> p;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[i], x[i + 1]);
    p.v[i] = y.x;
    p.v[i + 1] = y.y;
  }
  return p;
}
template <>
__device__ __forceinline__ Pack<__half, 8> rounded<__half, 8>(const float (&x)[8]) {
  Pack<__half, 8> p;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const __half2 y = __floats2half2_rn(x[i], x[i + 1]);
    p.v[i] = y.x;
    p.v[i + 1] = y.y;
  }
  return p;
}

// ---- rows that start anywhere, in aligned accesses
template <class W>
constexpr int kPer16 = 16 / sizeof(W);  // values in 16 bytes

// 16 bytes of a row that starts anywhere: the two multiples of 16 that they lie in.
struct Raw {
  uint4 a, b;
};
// The 16 bytes from byte `shift` on.
template <bool kShift>
__device__ __forceinline__ uint4 settle(const Raw& r, uint32_t shift) {
  if constexpr (!kShift) return r.a;
  uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
  const uint32_t bits = shift % 4 * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}
__device__ __forceinline__ uint32_t shift_of(const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15); }

// Zeros behind the first `left` of 16 bytes of values.
template <class W>
__device__ __forceinline__ uint4 keep(uint4 q, int left) {
  if (left >= kPer16<W>) return q;
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bytes = left * (int)sizeof(W) - 4 * i;
    if (bytes <= 0) w[i] = 0;
    else if (bytes < 4) w[i] &= (1u << (8 * bytes)) - 1;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A kernel that is launched by launch() begins with after_previous(): it may be
// set up while the kernel before it in the stream still runs.  Its blocks start
// as that one's last blocks leave room and wait here, before they touch memory,
// until it has ended and its writes are visible.  Calls back to back lose 1 to
// 2 us less between them.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool host_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uint32_t type_bytes(int type) {
  return type == ZIPCCL_TYPE_F32 ? 4u : (type == ZIPCCL_TYPE_BF16 || type == ZIPCCL_TYPE_F16) ? 2u : 0u;
}

}  // namespace zc
