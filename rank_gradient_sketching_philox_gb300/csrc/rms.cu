// Root-mean-square norm over the rows of T x k activations, forward with the
// residual's addition and an output in 8 bits, and backward.
//
//   s = x + r, rstd = 1 / sqrt(mean(s^2) + eps), y = s rstd gamma
//   q = e4m3(y / scale), a scale for each row's 128 columns (rows.cuh)
//   xh = s rstd, dxh = dy gamma, dx = rstd (dxh - xh mean(dxh xh)) + ds
//   dgamma (+)= sum over tokens of dy xh
//
// Everything between the inputs and the outputs is fp32: the norm takes the sum x + r
// before S rounds it, q takes y before Y does.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "tc.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPartials = 320;  // partial rows of gamma's gradient

// ---- any alignment, any width --------------------------------------------------------
// A block to a row, a warp to 128 columns, four of them to a lane; rows are read once
// for their sum and again for the output.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = lane_sum<true>(v, 32);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += part[w];
  return v;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) rms_forward_wide_kernel(const RmsForward a) {
  __shared__ float part[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x, groups = ceil_div(a.k, kScaleBlock);
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  const X* r = a.R ? static_cast<const X*>(a.R) + row * a.ld_r : nullptr;
  auto read = [&](int64_t c) { return r ? (float)x[c] + (float)r[c] : (float)x[c]; };
  float sum = 0.f;
  for (int64_t c = threadIdx.x; c < a.k; c += kThreads) sum = fmaf(read(c), read(c), sum);
  const float rstd = 1.f / sqrtf(block_sum(sum, part) / (float)a.k + a.eps);
  for (int64_t g = warp; g < groups; g += kWarps) {
    float y[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = g * kScaleBlock + i * 32 + lane;
      y[i] = 0.f;
      if (c < a.k) {
        const float s = read(c);
        y[i] = s * rstd * weight(a.gamma, a.w_type, c, 1.f);
        if (a.S) store_one(static_cast<X*>(a.S) + row * a.ld_s + c, s);
        if (a.Y) store_one(static_cast<X*>(a.Y) + row * a.ld_y + c, y[i]);
      }
      top = max(top, magnitude(y[i]));
    }
    if (a.Q) {
      float inv;
      const float scale = code_scale(__reduce_max_sync(0xFFFFFFFFu, top), inv);
      if (lane == 0) a.scale[row * groups + g] = scale;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t c = g * kScaleBlock + i * 32 + lane;
        if (c < a.k) a.Q[row * a.ld_q + c] = (uint8_t)codes2(y[i] * inv, 0.f);
      }
    }
  }
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
}

// Partial sums of gamma's gradient over `rows` rows, one column per thread.  Before
// rms_dx_wide_kernel, which may write dX over dY.
template <typename X>
__global__ void __launch_bounds__(kThreads) rms_grad_wide_kernel(const RmsBackward a, int64_t rows) {
  const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (col >= a.k) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows;
  const int64_t r1 = r0 + rows < a.T ? r0 + rows : a.T;
  float g = 0.f;
  for (int64_t r = r0; r < r1; ++r)
    g = fmaf((float)static_cast<const X*>(a.dY)[r * a.ld_dy + col],
             (float)static_cast<const X*>(a.S)[r * a.ld_s + col] * a.rstd[r], g);
  a.ws[(int64_t)blockIdx.y * a.k + col] = g;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) rms_dx_wide_kernel(const RmsBackward a) {
  __shared__ float part[kWarps];
  const int64_t row = blockIdx.x;
  const X* s = static_cast<const X*>(a.S) + row * a.ld_s;
  const X* dy = static_cast<const X*>(a.dY) + row * a.ld_dy;
  const X* ds = a.dS ? static_cast<const X*>(a.dS) + row * a.ld_ds : nullptr;
  X* dx = static_cast<X*>(a.dX) + row * a.ld_dx;
  const float rstd = a.rstd[row];
  float sum = 0.f;
  for (int64_t c = threadIdx.x; c < a.k; c += kThreads)
    sum = fmaf((float)dy[c] * weight(a.gamma, a.w_type, c, 1.f), (float)s[c] * rstd, sum);
  const float mean = block_sum(sum, part) / (float)a.k;
  for (int64_t c = threadIdx.x; c < a.k; c += kThreads) {
    const float d = (float)dy[c] * weight(a.gamma, a.w_type, c, 1.f);
    store_one(dx + c, fmaf(d - (float)s[c] * rstd * mean, rstd, ds ? (float)ds[c] : 0.f));
  }
}

// Adds the partial rows: 32 columns per block, the partials dealt over eight warps.
__global__ void __launch_bounds__(kThreads) rms_grad_sum_kernel(const float* ws, int64_t k, int partials, float* dgamma,
                                                                int overwrite) {
  __shared__ float part[kWarps][32];
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < k) {
#pragma unroll 8
    for (int p = warp; p < partials; p += kWarps) s += ws[(int64_t)p * k + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < k) {
    for (int w = 1; w < kWarps; ++w) s += part[w][lane];
    dgamma[col] = overwrite ? s : dgamma[col] + s;
  }
}

cudaError_t launch_grad_sum(const RmsBackward& a, int partials, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div(a.k, 32), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // its blocks may come up while the kernel before ends
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, rms_grad_sum_kernel, (const float*)a.ws, a.k, partials, a.dgamma, a.overwrite);
}

template <typename X>
cudaError_t forward_any(const RmsForward& a, cudaStream_t stream) {
  count_launch();
  rms_forward_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename X>
cudaError_t backward_any(const RmsBackward& a, cudaStream_t stream) {
  if (a.dgamma) {
    const int64_t rows = ceil_div(a.T, kMaxPartials) > 32 ? ceil_div(a.T, kMaxPartials) : 32;
    const int chunks = (int)ceil_div(a.T, rows);
    count_launch();
    rms_grad_wide_kernel<X><<<dim3((unsigned)ceil_div(a.k, kThreads), (unsigned)chunks), kThreads, 0, stream>>>(a, rows);
    const cudaError_t err = launch_grad_sum(a, chunks, stream);
    if (err != cudaSuccess) return err;
  }
  if (a.dX) {
    count_launch();
    rms_dx_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_forward(const RmsForward& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? forward_any<__nv_bfloat16>(a, stream) : forward_any<float>(a, stream);
}

size_t rms_backward_workspace_bytes(int64_t T, int64_t k) {
  WsCursor cur;
  cur.take<float>((size_t)((T < kMaxPartials ? T : kMaxPartials) * k));
  cur.take<char>(0);
  return cur.offset;
}

cudaError_t launch_rms_backward(const RmsBackward& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? backward_any<__nv_bfloat16>(a, stream) : backward_any<float>(a, stream);
}

}  // namespace rgs
