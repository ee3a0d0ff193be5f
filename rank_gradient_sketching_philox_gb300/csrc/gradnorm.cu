// The global norm of many gradients, the factor that clips it, and the gradients'
// product with a factor on the device.
//
//   norm = sqrt(sum over all tensors of g^2),  scale = 1 where norm <= max_norm, else max_norm / norm
//
// Bound by HBM: the norm reads each gradient once, the scaling reads and writes it.  268M
// BF16 values on one GB300: norm 81 us, 0.98 of the copy rate, scaling 153, 1.03 (a unit to
// a block; 1216 blocks of many units 167), both 238; off 16 bytes the norm takes 151, the
// scaling 600.  114 tensors of 2048 values: 6.4 us on the device, two launches, a call 8 to 10.
//
// The tensors are cut into units of
// kUnit values, dealt to at most kBlocks blocks, whatever the GPU's size, so that the
// sums' order depends on the tensors' sizes alone.  A thread adds its 32
// squares of a unit in fp32 (four chains), the rest in fp64.  Squares that fp32 cannot
// hold (sums that overflow, or small ones of values that are not zero) are taken again
// in fp64, so that the norm is right for every finite gradient.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 32;                  // values of a unit per thread
constexpr int kUnit = kThreads * kEach;
constexpr int kBlocks = 1216;              // partial sums of a launch: eight blocks for each of 152 SMs
constexpr int kScaleBlocks = 1 << 20;      // of a launch that scales: a unit to each up to 8.6 G values
constexpr int kTensors = 256;              // per launch

struct GradBatch {
  sketch_grad_problem p[kTensors];
  int64_t begin[kTensors + 1];  // prefix of the tensors' units
  int n;
};

// Whether 16-byte vectors of the tensor start on 16 bytes.
__device__ __forceinline__ bool on_vector(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every gridDim.x-th unit from this block's first one on, so that the blocks go through
// the tensors together: f(problem, first value).  BACK: from the last unit.
template <bool BACK, typename F>
__device__ __forceinline__ void walk_units(const GradBatch& a, F f) {
  const int64_t units = a.begin[a.n];
  int lo = 0, hi = a.n;
  for (int64_t i = blockIdx.x; i < units; i += gridDim.x) {
    const int64_t u = BACK ? units - 1 - i : i;
    if (BACK) lo = 0;
    else hi = a.n;
    while (hi - lo > 1) {  // the last tensor that begins at or before the unit
      const int mid = (lo + hi) >> 1;
      if (a.begin[mid] <= u) lo = mid;
      else hi = mid;
    }
    f(a.p[lo], (u - a.begin[lo]) * kUnit);
  }
}

// A thread's values of a unit: the vectors threadIdx.x, + 256, ... of it, whole or, where the
// tensor does not start on 16 bytes or ends, element by element, with zeros behind the
// tensor.  Which they are does not depend on the tensor's place, nor does the sums' order.
// (In steps of 256 elements, 268M BF16 values off 16 bytes took 186 us, not 152.)  Not by
// way of the read-only cache: the kernel may come up while the one before still writes the
// gradients.
template <typename G>
__device__ __forceinline__ void load_unit(const G* g, int64_t n, int64_t first, float (&v)[kEach]) {
  constexpr int VE = 16 / (int)sizeof(G);
  const int left = (int)(n - first < kUnit ? n - first : kUnit);
  const G* p = g + first + threadIdx.x * VE;
  if (on_vector(g)) {
    uint4 raw[kEach / VE];
#pragma unroll
    for (int j = 0; j < kEach / VE; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if ((j * kThreads + (int)threadIdx.x + 1) * VE <= left) raw[j] = *reinterpret_cast<const uint4*>(p + j * (kThreads * VE));
    }
#pragma unroll
    for (int j = 0; j < kEach / VE; ++j) {
      Pair q[VE / 2];
      vec_pairs<G>(raw[j], q);
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const float2 f = split(q[i]);
        v[j * VE + 2 * i] = f.x;
        v[j * VE + 2 * i + 1] = f.y;
      }
    }
    if (left % VE == 0 || left / VE % kThreads != (int)threadIdx.x) return;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {  // the tensor's last, cut vector
      if (j / VE != left / VE / kThreads) continue;
      v[j] = j % VE < left % VE ? (float)p[j / VE * (kThreads * VE) + j % VE] : 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int at = j / VE * (kThreads * VE) + j % VE;
      v[j] = at + (int)threadIdx.x * VE < left ? (float)p[at] : 0.f;
    }
  }
}

constexpr float kSmallSum = 8.2718061255302767e-25f;  // 2^-80: squares of 2^-126 and less are lost beside it at 2^-46

__device__ __forceinline__ double unit_sum(const float (&v)[kEach]) {
  Pair s[2] = {0, 0};
  uint32_t any = 0;
#pragma unroll
  for (int j = 0; j < kEach; j += 2) {
    const Pair p = pair(v[j], v[j + 1]);
    s[(j >> 1) & 1] = fma2(p, p, s[(j >> 1) & 1]);
    any |= __float_as_uint(v[j]) | __float_as_uint(v[j + 1]);
  }
  const float sum = sum2(add2(s[0], s[1]));
  if (sum >= kSmallSum && sum < INFINITY) return (double)sum;
  if ((any & 0x7FFFFFFFu) == 0) return 0.0;
  double d = 0.0;
  for (int j = 0; j < kEach; ++j) d = fma((double)v[j], (double)v[j], d);
  return d;
}

__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradBatch a, double* partials) {
  __shared__ double part[kThreads / 32];
  start_early();
  double sum = 0.0;
  walk_units<false>(a, [&](const sketch_grad_problem& p, int64_t first) {
    float v[kEach];
    if (p.type == SKETCH_BF16) load_unit(static_cast<const __nv_bfloat16*>(p.G), p.count, first, v);
    else load_unit(static_cast<const float*>(p.G), p.count, first, v);
    sum += unit_sum(v);
  });
  sum = block_sum(sum, part);
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* partials, int64_t n, float max_norm,
                                                                  float* norm, float* scale) {
  __shared__ double part[kThreads / 32];
  start_early();
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += partials[i];
  sum = sqrt(block_sum(sum, part));
  if (threadIdx.x == 0) {
    *norm = (float)sum;
    if (scale) *scale = sum <= (double)max_norm ? 1.f : (float)((double)max_norm / sum);
  }
}

template <typename G>
__device__ __forceinline__ void scale_unit(const G* g, G* out, int64_t n, int64_t first, float scale) {
  constexpr int VE = 16 / (int)sizeof(G);
  if (first + kUnit <= n && on_vector(g) && on_vector(out)) {
    uint4 raw[kEach / VE];
    const uint4* p = reinterpret_cast<const uint4*>(g + first) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kEach / VE; ++j) raw[j] = p[j * kThreads];
    const Pair s = pair(scale, scale);
#pragma unroll
    for (int j = 0; j < kEach / VE; ++j) {
      Pair q[VE / 2];
      vec_pairs<G>(raw[j], q);
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) q[i] = mul2(q[i], s);
      store_vec<G>(out + first, j * kThreads + threadIdx.x, q);
    }
  } else {
    for (int j = 0; j < kEach; ++j) {
      const int64_t e = first + j * kThreads + threadIdx.x;
      if (e < n) store_one(out + e, (float)g[e] * scale);
    }
  }
}

// From the last unit: what the norm read last is still in L2.
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradBatch a, const float* scale) {
  start_early();
  const float s = *scale;
  walk_units<true>(a, [&](const sketch_grad_problem& p, int64_t first) {
    if (s == 1.f && p.out == p.G) return;
    if (p.type == SKETCH_BF16)
      scale_unit(static_cast<const __nv_bfloat16*>(p.G), static_cast<__nv_bfloat16*>(p.out), p.count, first, s);
    else
      scale_unit(static_cast<const float*>(p.G), static_cast<float*>(p.out), p.count, first, s);
  });
}

// The launches of a batch, up to kTensors tensors each: f(table, blocks).
template <typename F>
cudaError_t for_batches(int n, const sketch_grad_problem* probs, int most, F f) {
  static thread_local GradBatch a;
  for (int i = 0; i < n;) {
    a.n = 0;
    a.begin[0] = 0;
    for (; i < n && a.n < kTensors; ++i) {
      a.p[a.n] = probs[i];
      a.begin[a.n + 1] = a.begin[a.n] + ceil_div(probs[i].count, kUnit);
      ++a.n;
    }
    const int64_t units = a.begin[a.n];
    const cudaError_t err = f(a, (int)(units < 1 ? 1 : units < most ? units : most));
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_workspace_bytes(int64_t n) {
  WsCursor cur;
  cur.take<double>((size_t)(ceil_div(n, kTensors) * kBlocks));
  cur.take<char>(0);
  return cur.offset;
}

cudaError_t launch_grad_norm(int n, const sketch_grad_problem* probs, float max_norm, float* norm, float* scale,
                             double* ws, cudaStream_t stream) {
  int64_t partials = 0;
  const cudaError_t err = for_batches(n, probs, kBlocks, [&](const GradBatch& a, int blocks) {
    double* to = ws + partials;
    partials += blocks;
    return launch_early(grad_norm_kernel, blocks, kThreads, 0, stream, a, to);
  });
  if (err != cudaSuccess) return err;
  return launch_early(grad_norm_join_kernel, 1, kThreads, 0, stream, (const double*)ws, partials, max_norm, norm, scale);
}

cudaError_t launch_grad_scale(int n, const sketch_grad_problem* probs, const float* scale, cudaStream_t stream) {
  return for_batches(n, probs, kScaleBlocks, [&](const GradBatch& a, int blocks) {
    return launch_early(grad_scale_kernel, blocks, kThreads, 0, stream, a, scale);
  });
}

}  // namespace rgs
