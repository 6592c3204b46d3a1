// zc_adamw.cu -- one AdamW step over many tensors, with the states in 32 or
// in 8 bits.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kStepThreads = 256;
// Blocks an SM holds at least.  8-bit states need the warps to cover the loads
// (109 M values: 6 blocks 262 us, 5 264, 4 275); with 32-bit states 2 to 5 are
// the same there (432 us) and more than 3 cost a small call 2 us.
template <bool k8>
constexpr int kStepBlocks = k8 ? 6 : 3;
constexpr uint32_t kBlock = ZIPCCL_ADAMW_BLOCK;  // values of one 8-bit scale: 8 for each lane of a warp
constexpr uint32_t kTileValues = 8 * kStepThreads;
constexpr uint32_t kStepTensors = 384;  // tensors of one launch: their records are kernel parameters
constexpr float kF8Min = 0x1p-9f, kScaleMin = 0x1p-126f;

struct StepTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  __nv_bfloat16* copy;
  float* ms;
  float* vs;
  uint64_t n;  // values, times 2; the lowest bit: every part is aligned for eight values at a time
};

struct StepArgs {
  float b1, b1c, b2, b2c, decay, rate, root, eps;
  const float* grad_scale;
  uint32_t count;
  uint32_t tile[kStepTensors + 1];  // first tile of each tensor
  StepTensor t[kStepTensors];
};
static_assert(sizeof(StepArgs) < 32000, "kernel parameters are limited to 32,764 bytes");

__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// Reciprocal of a number that is not negative by the hardware's approximation
// (1 ulp at most): the quotient it enters changes the parameter far above its
// last bits, and no state.  An IEEE division costs 10% where instructions bound
// the kernel, 65 a value with 8-bit states (109 M values: 288 us against 262).
// Below the smallest normal float it is that of the smallest normal float; of
// NaN (a second moment that is not a number) it is NaN.
__device__ __forceinline__ float quick_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(max_nan(x, 0x1p-126f)));
  return y;
}

// The step itself.  What is kept as a state is rounded operation by operation
// (no fused multiply-add, IEEE square root): an 8-bit code is then a function
// of the formula alone, where a last bit off would now and then be a whole
// step of the code, and a percent of the next change.
__device__ __forceinline__ void step_value(const StepArgs& a, float g, float& p, float& m, float& v, float& r) {
  m = a.b1 * m + a.b1c * g;
  v = a.b2 * v + a.b2c * (g * g);
  r = sqrtf(v);
  p = fmaf(p, a.decay, -(a.rate * m) * quick_rcp(fmaf(r, a.root, a.eps)));
}

// Eight consecutive values as one access of 32, 16 or 8 bytes.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const Pack<__nv_bfloat16, 8> v = *reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __bfloat162float(v.v[j]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  Pack<__nv_bfloat162, 4> v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v.v[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
  *reinterpret_cast<Pack<__nv_bfloat162, 4>*>(p) = v;
}

// E4M3 codes, two at a time; what is not finite becomes NaN (0x7F).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 values2(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
}
__device__ __forceinline__ void load8(const uint8_t* p, float (&x)[8]) {
  const uint2 c = *reinterpret_cast<const uint2*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = values2((j < 2 ? c.x : c.y) >> (16 * (j & 1)) & 0xFFFFu);
    x[2 * j] = v.x;
    x[2 * j + 1] = v.y;
  }
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&x)[8]) {
  uint2 c;
  c.x = codes2(x[0], x[1]) | codes2(x[2], x[3]) << 16;
  c.y = codes2(x[4], x[5]) | codes2(x[6], x[7]) << 16;
  *reinterpret_cast<uint2*>(p) = c;
}
__device__ __forceinline__ float load1(const uint8_t* p) { return values2(*p).x; }
template <class T>
__device__ __forceinline__ float load1(const T* p) { return to_float(*p); }
__device__ __forceinline__ void store1(uint8_t* p, float x) { *p = (uint8_t)codes2(x, 0.0f); }
template <class T>
__device__ __forceinline__ void store1(T* p, float x) { *p = from_float<T>(x); }

// Where a lane's eight values of the warp's 256 are: next to each other, for
// one wide access, or, where the tensor's parts are not aligned or the tensor
// ends within the 256, 32 apart for eight narrow ones.
template <bool kWide, class T>
__device__ __forceinline__ void load(const T* p, uint32_t lane, uint32_t left, float (&x)[8]) {
  if constexpr (kWide) {
    load8(p + 8 * lane, x);
  } else {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) x[j] = 32 * j + lane < left ? load1(p + 32 * j + lane) : 0.0f;
  }
}
template <bool kWide, class T>
__device__ __forceinline__ void store(T* p, uint32_t lane, uint32_t left, const float (&x)[8]) {
  if constexpr (kWide) {
    store8(p + 8 * lane, x);
  } else {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (32 * j + lane < left) store1(p + 32 * j + lane, x[j]);
  }
}

// Scales a block of 256 values held by a warp, 8 a lane, to E4M3's range: the
// largest finite magnitude over 448.  What is not finite becomes NaN, a
// positive root too small for the format its smallest value.
template <bool kRoot>
__device__ __forceinline__ float scale_block(float (&x)[8]) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) top = max_nan(top, fabsf(x[j]));
  uint32_t bits = __reduce_max_sync(kAll, __float_as_uint(top));  // magnitudes order like their bits, NaN on top
  const bool odd = bits >= 0x7F800000u;
  if (odd) {  // one is not finite: the largest of the others
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = __float_as_uint(x[j]) & 0x7FFFFFFFu;
      if (u < 0x7F800000u) mine = max(mine, u); else x[j] = NAN;
    }
    bits = __reduce_max_sync(kAll, mine);
  }
  const float scale = fmaxf(__uint_as_float(bits) * (float)(1.0 / 448.0), kScaleMin);
  const float inv = 1.0f / scale;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool some = kRoot && x[j] > 0.0f;
    x[j] *= inv;
    if (some) x[j] = fmaxf(x[j], kF8Min);
  }
  return scale;
}

// One warp's 256 values, `left` of which exist.
template <class P, class G, bool k8, bool kWide>
__device__ __forceinline__ void step_block(const StepArgs& a, const StepTensor& t, uint64_t first, uint32_t left) {
  using S = typename std::conditional<k8, uint8_t, float>::type;
  const uint32_t lane = threadIdx.x & 31;
  P* pp = static_cast<P*>(t.p) + first;
  S* pm = static_cast<S*>(t.m) + first;
  S* pv = static_cast<S*>(t.v) + first;
  float p[8], g[8], m[8], v[8], r[8];
  load<kWide>(pp, lane, left, p);
  load<kWide>(static_cast<const G*>(t.g) + first, lane, left, g);
  load<kWide>(pm, lane, left, m);
  load<kWide>(pv, lane, left, v);
  if (a.grad_scale) {
    const float gs = *a.grad_scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= gs;
  }
  const uint64_t block = first / kBlock;
  if (k8) {
    const float ms = t.ms[block], vs = t.vs[block];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] *= ms;
      v[j] *= vs;
      v[j] *= v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) step_value(a, g[j], p[j], m[j], v[j], r[j]);
  store<kWide>(pp, lane, left, p);
  if (t.copy) store<kWide>(t.copy + first, lane, left, p);
  if (!k8) {
    store<kWide>(pm, lane, left, m);
    store<kWide>(pv, lane, left, v);
    return;
  }
  if (!kWide) {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (32 * j + lane >= left) m[j] = r[j] = 0.0f;  // places past the tensor's end
  }
  const float ms = scale_block<false>(m), vs = scale_block<true>(r);
  store<kWide>(pm, lane, left, m);
  store<kWide>(pv, lane, left, r);
  if (lane == 0) {
    t.ms[block] = ms;
    t.vs[block] = vs;
  }
}

template <class P, class G, bool k8>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks<k8>) zc_adamw_kernel(const __grid_constant__ StepArgs a) {
  after_previous();
  // the tensor of this tile
  uint32_t lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (a.tile[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const StepTensor& t = a.t[lo];
  const uint64_t n = t.n >> 1;
  const uint64_t first = (uint64_t)(blockIdx.x - a.tile[lo]) * kTileValues + (threadIdx.x >> 5) * kBlock;
  if (first >= n) return;
  if ((t.n & 1) && n - first >= kBlock)
    step_block<P, G, k8, true>(a, t, first, kBlock);
  else
    step_block<P, G, k8, false>(a, t, first, (uint32_t)min(n - first, (uint64_t)kBlock));
}

template <class P, class G>
cudaError_t step_launch(const StepArgs& a, bool k8, cudaStream_t s) {
  const uint32_t tiles = a.tile[a.count];
  return launch(k8 ? zc_adamw_kernel<P, G, true> : zc_adamw_kernel<P, G, false>, tiles, kStepThreads, 0, s, a);
}

}  // namespace
}  // namespace zc

using namespace zc;

extern "C" zipccl_status zipccl_adamw_step(const zipccl_adamw_tensor* tensors, uint32_t n_tensors, int param_type,
                                           int grad_type, int state_bits, const zipccl_adamw_options* o,
                                           const float* d_grad_scale, void* stream) {
  const bool pf = param_type == ZIPCCL_TYPE_F32, gf = grad_type == ZIPCCL_TYPE_F32;
  if (!o || (n_tensors && !tensors) || (!pf && param_type != ZIPCCL_TYPE_BF16) ||
      (!gf && grad_type != ZIPCCL_TYPE_BF16) || (state_bits != 32 && state_bits != 8))
    return ZIPCCL_ERR_INVALID_ARG;
  if (!(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0) || !(o->eps >= 0.0) ||
      !(o->lr >= 0.0) || !(o->weight_decay >= 0.0) || o->step == 0 || !isfinite(o->lr) || !isfinite(o->eps) ||
      !isfinite(o->weight_decay) || !host_aligned(d_grad_scale, 4))
    return ZIPCCL_ERR_INVALID_ARG;
  const bool k8 = state_bits == 8;
  const uintptr_t pz = pf ? 4 : 2, gz = gf ? 4 : 2, sz = k8 ? 1 : 4;
  for (uint32_t i = 0; i < n_tensors; ++i) {
    const zipccl_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!t.d_param || !t.d_grad || !t.d_exp_avg || !t.d_exp_avg_sq || (k8 && (!t.d_avg_scale || !t.d_sq_scale)))
      return ZIPCCL_ERR_INVALID_ARG;
    if (!host_aligned(t.d_param, pz) || !host_aligned(t.d_grad, gz) || !host_aligned(t.d_exp_avg, sz) ||
        !host_aligned(t.d_exp_avg_sq, sz) || !host_aligned(t.d_copy, 2) || !host_aligned(t.d_avg_scale, 4) ||
        !host_aligned(t.d_sq_scale, 4) || t.n > (1ull << 40))
      return ZIPCCL_ERR_INVALID_ARG;
  }
  const double c1 = 1.0 - pow(o->beta1, (double)o->step), c2 = 1.0 - pow(o->beta2, (double)o->step);
  StepArgs a;
  a.b1 = (float)o->beta1;
  a.b1c = (float)(1.0 - o->beta1);
  a.b2 = (float)o->beta2;
  a.b2c = (float)(1.0 - o->beta2);
  a.decay = (float)(1.0 - o->lr * o->weight_decay);
  a.rate = (float)(o->lr / c1);
  a.root = (float)(1.0 / sqrt(c2));
  a.eps = (float)o->eps;
  a.grad_scale = d_grad_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (uint32_t i = 0; i < n_tensors;) {
    a.count = 0;
    uint64_t tiles = 0;
    for (; i < n_tensors && a.count < kStepTensors; ++i) {
      const zipccl_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      const uint64_t more = (t.n + kTileValues - 1) / kTileValues;
      if (tiles && tiles + more >= (1ull << 31)) break;
      const bool wide = host_aligned(t.d_param, 8 * pz) && host_aligned(t.d_grad, 8 * gz) &&
                        host_aligned(t.d_exp_avg, 8 * sz) && host_aligned(t.d_exp_avg_sq, 8 * sz) &&
                        host_aligned(t.d_copy, 16);
      a.t[a.count] = {t.d_param, t.d_grad, t.d_exp_avg, t.d_exp_avg_sq, static_cast<__nv_bfloat16*>(t.d_copy),
                      t.d_avg_scale, t.d_sq_scale, t.n << 1 | (wide ? 1 : 0)};
      a.tile[a.count++] = (uint32_t)tiles;
      tiles += more;
    }
    if (a.count == 0) break;
    a.tile[a.count] = (uint32_t)tiles;
    const cudaError_t e = pf ? gf ? step_launch<float, float>(a, k8, s) : step_launch<float, __nv_bfloat16>(a, k8, s)
                             : gf ? step_launch<__nv_bfloat16, float>(a, k8, s)
                                  : step_launch<__nv_bfloat16, __nv_bfloat16>(a, k8, s);
    if (e != cudaSuccess) return ZIPCCL_ERR_CUDA;
  }
  return ZIPCCL_OK;
}
