// Rounding of a matrix to 8 bits with a scale for each block of 128 columns of a row,
// or of 128 rows and 128 columns (rows.cuh), and of its transpose beside it.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A scale per row and 128 columns: a warp to such a piece, four columns to a lane.
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const Quantize a) {
  const int lane = threadIdx.x & 31;
  const int64_t groups = ceil_div(a.k, kScaleBlock), pieces = a.T * groups;
  for (int64_t p = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); p < pieces; p += (int64_t)gridDim.x * kWarps) {
    const int64_t row = p / groups, g = p - row * groups;
    const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
    float v[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = g * kScaleBlock + i * 32 + lane;
      v[i] = c < a.k ? (float)x[c] : 0.f;
      top = max(top, magnitude(v[i]));
    }
    float inv;
    const float scale = code_scale(__reduce_max_sync(0xFFFFFFFFu, top), inv);
    if (lane == 0) a.scale[p] = scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = g * kScaleBlock + i * 32 + lane;
      if (c < a.k) a.Q[row * a.ld_q + c] = (uint8_t)codes2(v[i] * inv, 0.f);
    }
  }
}

// A scale per 128 rows and 128 columns: a block to each, a warp to 16 of its rows.
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_tiles_kernel(const Quantize a) {
  constexpr int kRows = kScaleBlock / kWarps;
  __shared__ uint32_t part[kWarps];
  __shared__ uint8_t tile[kScaleBlock][kScaleBlock + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  const int64_t r0 = blockIdx.x / groups * kScaleBlock, c0 = blockIdx.x % groups * kScaleBlock;
  float v[kRows][4];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t row = r0 + j * kWarps + warp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + i * 32 + lane;
      v[j][i] = row < a.T && c < a.k ? (float)static_cast<const X*>(a.X)[row * a.ld_x + c] : 0.f;
      top = max(top, magnitude(v[j][i]));
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) part[warp] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu, part[lane & (kWarps - 1)]);
  float inv;
  const float scale = code_scale(top, inv);
  if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t row = r0 + j * kWarps + warp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + i * 32 + lane;
      const uint8_t q = (uint8_t)codes2(v[j][i] * inv, 0.f);
      if (a.Q && row < a.T && c < a.k) a.Q[row * a.ld_q + c] = q;
      tile[i * 32 + lane][j * kWarps + warp] = q;
    }
  }
  if (a.Qt == nullptr) return;
  __syncthreads();
  for (int c = warp; c < kScaleBlock; c += kWarps) {
    if (c0 + c >= a.k) break;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i * 32 + lane < a.T) a.Qt[(c0 + c) * a.ld_qt + r0 + i * 32 + lane] = tile[c][i * 32 + lane];
  }
}

template <typename X>
cudaError_t quantize(const Quantize& a, cudaStream_t stream) {
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  count_launch();
  if (a.rows == 1) {
    int64_t blocks = ceil_div(a.T * groups, kWarps);
    if (blocks > (int64_t)num_sms() * 64) blocks = (int64_t)num_sms() * 64;
    quantize_rows_kernel<X><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  } else {
    quantize_tiles_kernel<X><<<(unsigned)(groups * ceil_div(a.T, kScaleBlock)), kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const Quantize& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? quantize<__nv_bfloat16>(a, stream) : quantize<float>(a, stream);
}

}  // namespace rgs
