// zc_adamw.cu -- one AdamW step over many tensors, with the states in 32 or
// in 8 bits.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr int kStepThreads = 256;
constexpr uint32_t kBlock = ZIPCCL_ADAMW_BLOCK;  // values of one 8-bit scale: 8 for each lane of a warp
constexpr uint32_t kTileValues = 8 * kStepThreads;
constexpr uint32_t kStepTensors = 384;  // tensors of one launch: their records are kernel parameters
constexpr float kF8Max = 448.0f, kF8Min = 0x1p-9f, kScaleMin = 0x1p-126f;

struct StepTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  __nv_bfloat16* copy;
  float* ms;
  float* vs;
  uint64_t n;
};

struct StepArgs {
  float b1, b1c, b2, b2c, decay, rate, root, eps;
  const float* grad_scale;
  uint32_t count;
  uint32_t tile[kStepTensors + 1];  // first tile of each tensor
  StepTensor t[kStepTensors];
};
static_assert(sizeof(StepArgs) < 32000, "kernel parameters are limited to 32,764 bytes");

// The step itself; every product and sum is rounded by itself (no fused
// multiply-add), so that the result does not depend on the launch's form.
__device__ __forceinline__ void step_value(const StepArgs& a, float g, float& p, float& m, float& v, float& r) {
  m = a.b1 * m + a.b1c * g;
  v = a.b2 * v + a.b2c * (g * g);
  r = sqrtf(v);
  p = p * a.decay - m / (r * a.root + a.eps) * a.rate;
}

// Scale of a block of 256 values held by a warp, 8 a lane: the largest finite
// magnitude over 448.  Values that are not finite are stored as NaN.
__device__ __forceinline__ float block_scale(const float (&x)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fabsf(x[i]);
    if (y < INFINITY) top = fmaxf(top, y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  return fmaxf(top * (float)(1.0 / 448.0), kScaleMin);
}

__device__ __forceinline__ uint8_t code8(float x, float inv, bool root) {
  float y = x * inv;
  if (root && x > 0.0f) y = fmaxf(y, kF8Min);
  const uint8_t c = __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  return fabsf(x) < INFINITY ? c : 0x7F;
}

__device__ __forceinline__ float value8(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <class P, class G, bool k8>
__global__ void __launch_bounds__(kStepThreads) zc_adamw_kernel(const __grid_constant__ StepArgs a) {
  // the tensor of this tile
  uint32_t lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (a.tile[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const StepTensor& t = a.t[lo];
  const uint64_t tile = (uint64_t)(blockIdx.x - a.tile[lo]) * kTileValues;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  P* p = static_cast<P*>(t.p);
  const G* g = static_cast<const G*>(t.g);
  if (!k8) {
    float* m = static_cast<float*>(t.m);
    float* v = static_cast<float*>(t.v);
    for (uint32_t j = 0; j < 8; ++j) {
      const uint64_t i = tile + j * kStepThreads + threadIdx.x;
      if (i >= t.n) break;
      float x = to_float(p[i]), mm = m[i], vv = v[i], r, gg = to_float(g[i]);
      if (a.grad_scale) gg *= gs;
      step_value(a, gg, x, mm, vv, r);
      p[i] = from_float<P>(x);
      m[i] = mm;
      v[i] = vv;
      if (t.copy) t.copy[i] = __float2bfloat16_rn(x);
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const uint64_t i0 = tile + (uint64_t)(threadIdx.x >> 5) * kBlock + lane;
  const uint64_t block = i0 / kBlock;
  if (block * kBlock >= t.n) return;
  uint8_t* m = static_cast<uint8_t*>(t.m);
  uint8_t* v = static_cast<uint8_t*>(t.v);
  const float ms = t.ms[block], vs = t.vs[block];
  float mm[8], rr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t i = i0 + 32 * j;
    mm[j] = rr[j] = 0.0f;
    if (i < t.n) {
      float x = to_float(p[i]), gg = to_float(g[i]);
      if (a.grad_scale) gg *= gs;
      mm[j] = value8(m[i]) * ms;
      const float r = value8(v[i]) * vs;
      float vv = r * r;
      step_value(a, gg, x, mm[j], vv, rr[j]);
      p[i] = from_float<P>(x);
      if (t.copy) t.copy[i] = __float2bfloat16_rn(x);
    }
  }
  const float nms = block_scale(mm), nvs = block_scale(rr);
  const float im = 1.0f / nms, iv = 1.0f / nvs;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t i = i0 + 32 * j;
    if (i < t.n) {
      m[i] = code8(mm[j], im, false);
      v[i] = code8(rr[j], iv, true);
    }
  }
  if (lane == 0) {
    t.ms[block] = nms;
    t.vs[block] = nvs;
  }
}

template <class P, class G>
void step_launch(const StepArgs& a, bool k8, cudaStream_t s) {
  const uint32_t tiles = a.tile[a.count];
  if (k8)
    zc_adamw_kernel<P, G, true><<<tiles, kStepThreads, 0, s>>>(a);
  else
    zc_adamw_kernel<P, G, false><<<tiles, kStepThreads, 0, s>>>(a);
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
      a.t[a.count] = {t.d_param, t.d_grad, t.d_exp_avg, t.d_exp_avg_sq, static_cast<__nv_bfloat16*>(t.d_copy),
                      t.d_avg_scale, t.d_sq_scale, t.n};
      a.tile[a.count++] = (uint32_t)tiles;
      tiles += more;
    }
    if (a.count == 0) break;
    a.tile[a.count] = (uint32_t)tiles;
    if (pf && gf) step_launch<float, float>(a, k8, s);
    else if (pf) step_launch<float, __nv_bfloat16>(a, k8, s);
    else if (gf) step_launch<__nv_bfloat16, float>(a, k8, s);
    else step_launch<__nv_bfloat16, __nv_bfloat16>(a, k8, s);
    if (cudaGetLastError() != cudaSuccess) return ZIPCCL_ERR_CUDA;
  }
  return ZIPCCL_OK;
}
