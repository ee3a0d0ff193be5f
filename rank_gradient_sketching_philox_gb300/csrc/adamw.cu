// AdamW over many tensors in one launch, with fp32 states or 8-bit states.
//
//   g' = grad_scale g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   w = w (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// BF16 weights are written by stochastic rounding with the library's weight
// stream (a nearest rounding would drop most updates below half a BF16 step).
//
// 8-bit states: blocks of 256 values share an fp32 scale, the largest magnitude
// over 448.  m is held as E4M3 codes of m / scale; of v the root u = sqrt(v) is
// held, so that a block spans 2^18 in u, 2^36 in v.  Both are rounded
// stochastically from streams of their own: a moving average with 1 - b2 = 1e-3
// changes by less than half a step of a 3-bit mantissa, so that a nearest
// rounding would never let it move.  A u that is not zero never rounds to zero,
// since it divides.  On the way to a code every operation is rounded by itself,
// none fused: a code that a last bit decides is the same on any fp32 machine
// (a state that differs by a code is a step apart ever after).  A value that is not finite gets the code NaN and takes no
// part in its block's scale.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace rgs {
namespace {

constexpr uint32_t kTagMoment1 = 3u;
constexpr uint32_t kTagMoment2 = 4u;
constexpr int kBlock = 256;      // values that share a scale; threads per block
constexpr int kAdamBatch = 256;  // tensors per launch

struct AdamBatch {
  sketch_adamw_problem p[kAdamBatch];
  int64_t begin[kAdamBatch + 1];  // prefix of the tensors' blocks of kBlock values
  int n;
  AdamStep h;
  uint64_t seed;
  uint32_t step;
};

// 16 random bits of value e.
__device__ __forceinline__ uint32_t random16(const AdamBatch& a, uint32_t layer, uint32_t tag, int64_t e) {
  const Philox4 r = stream_block(a.seed, layer, a.step, tag, (uint32_t)(e >> 3));
  const int lane = (int)(e & 7);
  const uint32_t w = lane < 4 ? (lane < 2 ? r.w0 : r.w1) : (lane < 6 ? r.w2 : r.w3);
  return (lane & 1) ? w >> 16 : w & 0xFFFFu;
}

// y in [0, 448] to E4M3 with 16 random bits below the kept mantissa.  Below 2^-6
// E4M3's steps are 2^-9, which are those of y + 2^-6.
__device__ __forceinline__ uint32_t sr_e4m3(float y, uint32_t rand16) {
  const bool small = y < 0.015625f;
  const uint32_t bits = __float_as_uint(small ? y + 0.015625f : y) + (rand16 << 4);
  return (bits >> 20) - (small ? 968u : 960u);
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ float block_max(float v) {
  __shared__ float part[kBlock / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kBlock / 32; ++w) v = fmaxf(v, part[w]);
  return v;
}

// Magnitudes below this are dropped from an 8-bit first moment whose whole block
// is as small (the reciprocal of its scale would overflow).
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ void hold8(const AdamBatch& a, const sketch_adamw_problem& p, uint32_t tag, int64_t e, float x,
                                      uint32_t least, uint8_t* codes, float* scales) {
  const bool in = e < p.n;
  const bool finite = in && fabsf(x) <= 3.402823466e38f;
  const float top = block_max(finite ? fabsf(x) : 0.f);
  const float inv = top >= kLeast ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
  if (threadIdx.x == 0) scales[e / kBlock] = inv > 0.f ? __fmul_rn(top, 1.f / 448.f) : 0.f;
  if (!in) return;
  uint32_t c = 0x7Fu;
  if (finite) {
    c = sr_e4m3(fminf(__fmul_rn(fabsf(x), inv), 448.f), random16(a, p.layer, tag, e));
    if (x != 0.f && inv > 0.f && c < least) c = least;
  }
  codes[e] = (uint8_t)(c | (x < 0.f ? 0x80u : 0u));
}

template <bool STATES8>
__global__ void __launch_bounds__(kBlock) adamw_kernel(const __grid_constant__ AdamBatch a) {
  const int64_t block = blockIdx.x;
  int lo = 0, hi = a.n;  // the last tensor that begins at or before this block
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.begin[mid] <= block) lo = mid;
    else hi = mid;
  }
  const sketch_adamw_problem& p = a.p[lo];
  const int64_t e = (block - a.begin[lo]) * kBlock + threadIdx.x;
  const bool in = e < p.n;
  float w = 0.f, g = 0.f, m = 0.f, v = 0.f;
  if (in) {
    w = p.w_type == SKETCH_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p.W)[e])
                                : static_cast<const float*>(p.W)[e];
    g = p.g_type == SKETCH_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p.G)[e])
                                : static_cast<const float*>(p.G)[e];
    if (STATES8) {
      m = __fmul_rn(e4m3_value(static_cast<const uint8_t*>(p.m)[e]), p.m_scale[e / kBlock]);
      v = __fmul_rn(e4m3_value(static_cast<const uint8_t*>(p.v)[e]), p.v_scale[e / kBlock]);
      v = __fmul_rn(v, v);
    } else {
      m = static_cast<const float*>(p.m)[e];
      v = static_cast<const float*>(p.v)[e];
    }
  }
  if (a.h.grad_scale) g *= *a.h.grad_scale;
  m = __fadd_rn(__fmul_rn(a.h.beta1, m), __fmul_rn(a.h.one_beta1, g));
  v = __fadd_rn(__fmul_rn(a.h.beta2, v), __fmul_rn(__fmul_rn(a.h.one_beta2, g), g));
  const float u = __fsqrt_rn(v);
  w = w * a.h.decay - a.h.lr_m * m / (u * a.h.root_v + a.h.eps);
  if (in) {
    if (p.w_type == SKETCH_BF16)
      static_cast<uint16_t*>(p.W)[e] = (uint16_t)sr_bf16_bits(w, random16(a, p.layer, kTagSR, e));
    else
      static_cast<float*>(p.W)[e] = w;
  }
  if (STATES8) {
    __syncthreads();  // the block's scales are read before they are replaced
    hold8(a, p, kTagMoment1, e, m, 0u, static_cast<uint8_t*>(p.m), p.m_scale);
    hold8(a, p, kTagMoment2, e, u, 1u, static_cast<uint8_t*>(p.v), p.v_scale);
  } else if (in) {
    static_cast<float*>(p.m)[e] = m;
    static_cast<float*>(p.v)[e] = v;
  }
}

}  // namespace

cudaError_t launch_adamw(int n, const sketch_adamw_problem* probs, bool states8, const AdamStep& h, uint64_t seed,
                         uint32_t step, cudaStream_t stream) {
  static thread_local AdamBatch a;
  a.h = h;
  a.seed = seed;
  a.step = step;
  int i = 0;
  while (i < n) {
    a.n = 0;
    a.begin[0] = 0;
    for (; i < n && a.n < kAdamBatch; ++i) {
      if (probs[i].n == 0) continue;
      const int64_t blocks = ceil_div(probs[i].n, kBlock);
      if (a.n > 0 && a.begin[a.n] + blocks > (int64_t(1) << 30)) break;
      a.p[a.n] = probs[i];
      a.begin[a.n + 1] = a.begin[a.n] + blocks;
      ++a.n;
    }
    if (a.n == 0) continue;
    count_launch();
    if (states8) adamw_kernel<true><<<(unsigned)a.begin[a.n], kBlock, 0, stream>>>(a);
    else adamw_kernel<false><<<(unsigned)a.begin[a.n], kBlock, 0, stream>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace rgs
