// Layer norm over the rows of T x k activations, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   y = xh gamma + beta
//   dxh = dy gamma,  dx = rstd (dxh - mean(dxh) - xh mean(dxh xh))
//   dgamma (+)= sum over tokens of dy xh,  dbeta (+)= sum over tokens of dy
//
// Activations are BF16 or fp32, weights BF16 or fp32; statistics, sums and the
// weights' gradients are fp32.  Every sum has a fixed order (the gradients of the
// weights: rows within a chunk, then the chunks), so results repeat bit for bit.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kGradRows = 256;  // rows per partial sum of the weights' gradients

__device__ __forceinline__ float get(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float get(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// Sum over the block's threads, the same in every thread.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

template <typename X, typename W>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormForward a) {
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  X* y = static_cast<X*>(a.Y) + row * a.ld_y;
  const W* gamma = static_cast<const W*>(a.gamma);
  const W* beta = static_cast<const W*>(a.beta);
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) s += get(x, i);
  const float mu = block_sum(s) / (float)a.k;
  s = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(x, i) - mu;
    s += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(s) / (float)a.k + a.eps);
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float xh = (get(x, i) - mu) * rstd;
    put(y, i, fmaf(xh, gamma ? get(gamma, i) : 1.f, beta ? get(beta, i) : 0.f));
  }
  if (threadIdx.x == 0) {
    a.mean[row] = mu;
    a.rstd[row] = rstd;
  }
}

template <typename X, typename W>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const NormBackward a) {
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dY) + row * a.ld_dy;
  X* dx = static_cast<X*>(a.dX) + row * a.ld_dx;
  const W* gamma = static_cast<const W*>(a.gamma);
  const float mu = a.mean[row], rstd = a.rstd[row];
  float s0 = 0.f, s1 = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * (gamma ? get(gamma, i) : 1.f);
    s0 += d;
    s1 += d * ((get(x, i) - mu) * rstd);
  }
  s0 = block_sum(s0) / (float)a.k;
  s1 = block_sum(s1) / (float)a.k;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * (gamma ? get(gamma, i) : 1.f);
    put(dx, i, rstd * (d - s0 - ((get(x, i) - mu) * rstd) * s1));
  }
}

// Partial sums over kGradRows rows, one column per thread.
template <typename X>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(const NormBackward a) {
  const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (col >= a.k) return;
  const int64_t r0 = (int64_t)blockIdx.y * kGradRows;
  const int64_t r1 = r0 + kGradRows < a.T ? r0 + kGradRows : a.T;
  const X* X_ = static_cast<const X*>(a.X);
  const X* dY = static_cast<const X*>(a.dY);
  float g = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = get(dY, r * a.ld_dy + col);
    g += d * ((get(X_, r * a.ld_x + col) - a.mean[r]) * a.rstd[r]);
    b += d;
  }
  float* p = a.ws + (int64_t)blockIdx.y * 2 * a.k;
  p[col] = g;
  p[a.k + col] = b;
}

__global__ void __launch_bounds__(kThreads) norm_grad_sum_kernel(const NormBackward a, int chunks) {
  const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (col >= a.k) return;
  float g = 0.f, b = 0.f;
  for (int c = 0; c < chunks; ++c) {
    g += a.ws[(int64_t)c * 2 * a.k + col];
    b += a.ws[(int64_t)c * 2 * a.k + a.k + col];
  }
  if (a.dgamma) a.dgamma[col] = a.overwrite ? g : a.dgamma[col] + g;
  if (a.dbeta) a.dbeta[col] = a.overwrite ? b : a.dbeta[col] + b;
}

template <typename X, typename W>
cudaError_t forward(const NormForward& a, cudaStream_t stream) {
  count_launch();
  norm_forward_kernel<X, W><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename X, typename W>
cudaError_t backward(const NormBackward& a, cudaStream_t stream) {
  if (a.dX) {
    count_launch();
    norm_dx_kernel<X, W><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  }
  if (a.dgamma || a.dbeta) {
    const unsigned cols = (unsigned)ceil_div(a.k, kThreads), chunks = (unsigned)ceil_div(a.T, kGradRows);
    count_launch();
    norm_grad_kernel<X><<<dim3(cols, chunks), kThreads, 0, stream>>>(a);
    count_launch();
    norm_grad_sum_kernel<<<cols, kThreads, 0, stream>>>(a, (int)chunks);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_forward(const NormForward& a, cudaStream_t stream) {
  if (a.x_type == SKETCH_BF16)
    return a.w_type == SKETCH_BF16 ? forward<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                   : forward<__nv_bfloat16, float>(a, stream);
  return a.w_type == SKETCH_BF16 ? forward<float, __nv_bfloat16>(a, stream) : forward<float, float>(a, stream);
}

size_t norm_backward_workspace_bytes(int64_t T, int64_t k) {
  WsCursor cur;
  cur.take<float>((size_t)(ceil_div(T, kGradRows) * 2 * k));
  cur.take<char>(0);
  return cur.offset;
}

cudaError_t launch_norm_backward(const NormBackward& a, cudaStream_t stream) {
  if (a.x_type == SKETCH_BF16)
    return a.w_type == SKETCH_BF16 ? backward<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                   : backward<__nv_bfloat16, float>(a, stream);
  return a.w_type == SKETCH_BF16 ? backward<float, __nv_bfloat16>(a, stream) : backward<float, float>(a, stream);
}

}  // namespace rgs
