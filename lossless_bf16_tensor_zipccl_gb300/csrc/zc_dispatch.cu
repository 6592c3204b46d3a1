// zc_dispatch.cu -- tokens' rows to the experts' chunks and back: dispatch,
// combine and their gradients.
#include <cuda_runtime.h>
#include <stdint.h>

#include "zc_ops.cuh"
#include "zipccl.h"

namespace zc {
namespace {

constexpr uint32_t kMaxTopK = 32;
constexpr int kRowThreads = 256;

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
};

// rows[slot] = x[token] for each of the token's pairs; a dropped pair's row
// (slot -1 - row) is zeros.  A slot outside the buffer is skipped.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads) zc_dispatch_kernel(RowArgs a) {
  using P = Pack<T, N>;
  const uint64_t t = blockIdx.x, nv = a.hidden / N;
  const int32_t* slots = a.slots + t * a.top_k;
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(a.src) + t * a.stride);
  P zero;
#pragma unroll
  for (int i = 0; i < N; ++i) zero.v[i] = from_float<T>(0.0f);
  for (uint64_t v = (uint64_t)blockIdx.y * kRowThreads + threadIdx.x; v < nv; v += (uint64_t)gridDim.y * kRowThreads) {
    const P p = x[v];
    for (uint32_t k = 0; k < a.top_k; ++k) {
      const int32_t s = slots[k];
      const uint64_t row = (uint64_t)(s < 0 ? ~s : s);
      if (row < a.rows) reinterpret_cast<P*>(static_cast<T*>(a.dst) + row * a.hidden)[v] = s < 0 ? zero : p;
    }
  }
}

// y[token] = residual + sum over its pairs of weight * rows[slot], in pair
// order, held in 32 bits and rounded once.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads) zc_combine_kernel(RowArgs a) {
  using P = Pack<T, N>;
  const uint64_t t = blockIdx.x, nv = a.hidden / N;
  const int32_t* slots = a.slots + t * a.top_k;
  for (uint64_t v = (uint64_t)blockIdx.y * kRowThreads + threadIdx.x; v < nv; v += (uint64_t)gridDim.y * kRowThreads) {
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = 0.0f;
    for (uint32_t k = 0; k < a.top_k; ++k) {
      const int32_t s = slots[k];
      if (s < 0 || (uint64_t)s >= a.rows) continue;
      const float w = a.weights ? a.weights[t * a.top_k + k] : 1.0f;
      const P p = reinterpret_cast<const P*>(static_cast<const T*>(a.src) + (uint64_t)s * a.hidden)[v];
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = fmaf(w, to_float(p.v[i]), y[i]);
    }
    if (a.side) {
      const P p = reinterpret_cast<const P*>(static_cast<const T*>(a.side) + t * a.hidden)[v];
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] += to_float(p.v[i]);
    }
    P out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.v[i] = from_float<T>(y[i]);
    reinterpret_cast<P*>(static_cast<T*>(a.dst) + t * a.hidden)[v] = out;
  }
}

// grad_rows[slot] = weight * grad[token], grad_weight = <grad[token], rows[slot]>
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads) zc_combine_backward_kernel(RowArgs a) {
  using P = Pack<T, N>;
  __shared__ float s_part[kRowThreads / 32];
  const uint64_t t = blockIdx.x, nv = a.hidden / N;
  const P* g = reinterpret_cast<const P*>(static_cast<const T*>(a.side) + t * a.hidden);
  for (uint32_t k = 0; k < a.top_k; ++k) {
    const int32_t s = a.slots[t * a.top_k + k];
    const uint64_t row = (uint64_t)(s < 0 ? ~s : s);
    const bool in = row < a.rows;
    const float w = s < 0 ? 0.0f : a.weights ? a.weights[t * a.top_k + k] : 1.0f;
    const P* r = reinterpret_cast<const P*>(static_cast<const T*>(a.src) + (in ? row : 0) * a.hidden);
    P* out = reinterpret_cast<P*>(static_cast<T*>(a.dst) + (in ? row : 0) * a.hidden);
    float dot = 0.0f;
    if (in) {
      for (uint64_t v = threadIdx.x; v < nv; v += kRowThreads) {
        P o;
        if (s < 0) {
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = from_float<T>(0.0f);
        } else {
          const P p = g[v], q = r[v];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float x = to_float(p.v[i]);
            dot = fmaf(x, to_float(q.v[i]), dot);
            o.v[i] = from_float<T>(w * x);
          }
        }
        out[v] = o;
      }
    }
    if (a.grad_weights) {
#pragma unroll
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (int i = 0; i < kRowThreads / 32; ++i) sum += s_part[i];
        a.grad_weights[t * a.top_k + k] = sum;
      }
      __syncthreads();
    }
  }
}

enum class RowOp { kDispatch, kCombine, kCombineBackward };

template <class T, int N>
void row_launch(RowOp op, const RowArgs& a, cudaStream_t s) {
  const uint64_t nv = a.hidden / N;
  const uint32_t parts = (uint32_t)((nv + kRowThreads - 1) / kRowThreads);
  const dim3 grid(a.tokens, parts < 1 ? 1 : parts > 64 ? 64 : parts);
  if (op == RowOp::kDispatch)
    zc_dispatch_kernel<T, N><<<grid, kRowThreads, 0, s>>>(a);
  else if (op == RowOp::kCombine)
    zc_combine_kernel<T, N><<<grid, kRowThreads, 0, s>>>(a);
  else
    zc_combine_backward_kernel<T, N><<<a.tokens, kRowThreads, 0, s>>>(a);
}

template <class T>
void row_by_alignment(RowOp op, const RowArgs& a, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T);
  const bool wide = host_aligned(a.src, 16) && host_aligned(a.side, 16) && host_aligned(a.dst, 16) &&
                    a.hidden % N == 0 && (op != RowOp::kDispatch || a.stride % N == 0);
  if (wide)
    row_launch<T, N>(op, a, s);
  else
    row_launch<T, 1>(op, a, s);
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
  if (type == ZIPCCL_TYPE_F32)
    row_by_alignment<float>(op, a, s);
  else if (type == ZIPCCL_TYPE_BF16)
    row_by_alignment<__nv_bfloat16>(op, a, s);
  else
    row_by_alignment<__half>(op, a, s);
  return cudaGetLastError() == cudaSuccess ? ZIPCCL_OK : ZIPCCL_ERR_CUDA;
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
