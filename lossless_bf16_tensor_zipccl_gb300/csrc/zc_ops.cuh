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
