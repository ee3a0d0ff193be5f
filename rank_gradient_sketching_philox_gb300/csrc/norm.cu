// Layer norm over the rows of T x k activations, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   y = xh gamma + beta
//   dxh = dy gamma,  dx = rstd (dxh - mean(dxh) - xh mean(dxh xh))
//   dgamma (+)= sum over tokens of dy xh,  dbeta (+)= sum over tokens of dy
//
// Activations are BF16 or fp32, weights BF16 or fp32; statistics, sums and the
// weights' gradients are fp32.  Both passes are bound by HBM: each row is read
// once and stays in registers while its statistics are formed.
//
// A row belongs to `tpr` threads (a power of two, 8 to 1024), each with NV
// vectors of VE elements (16 bytes; VE = 1 where rows do not start on 16 bytes
// or end inside a vector).  The backward pass keeps a thread's columns fixed over
// the rows that its block walks, so that dgamma and dbeta add up in registers;
// each block leaves one partial row, and norm_grad_sum_kernel adds those.  Rows
// wider than 16384 take the kernels at the end, which read a row again for each
// pass.
//
// Every sum has a fixed order, so results repeat bit for bit.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPartials = 320;  // partial rows of the weights' gradients

// VE elements of a row, as loaded.
template <typename X, int VE>
struct Vec {
  uint4 r;
};
template <typename X>
struct Vec<X, 1> {
  X r;
};
template <typename X, int VE>
__device__ __forceinline__ Vec<X, VE> load_vec(const X* row, int idx) {
  Vec<X, VE> v;
  if constexpr (VE == 1) v.r = row[idx];
  else v.r = __ldcs(reinterpret_cast<const uint4*>(row) + idx);
  return v;
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename X, int VE>
__device__ __forceinline__ void unpack(const Vec<X, VE>& v, float (&f)[VE]) {
  if constexpr (VE == 1) {
    f[0] = to_float(v.r);
  } else {
    const uint32_t r[4] = {v.r.x, v.r.y, v.r.z, v.r.w};
#pragma unroll
    for (int i = 0; i < VE; ++i)
      f[i] = VE == 4 ? __uint_as_float(r[i & 3]) : __uint_as_float((i & 1) ? r[i >> 1] & 0xFFFF0000u : r[i >> 1] << 16);
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename X, int VE>
__device__ __forceinline__ void store_vec(X* row, int idx, const float (&f)[VE]) {
  if constexpr (VE == 1) {
    if constexpr (sizeof(X) == 4) row[idx] = f[0];
    else row[idx] = __float2bfloat16_rn(f[0]);
  } else if constexpr (VE == 4) {
    reinterpret_cast<float4*>(row)[idx] = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    reinterpret_cast<uint4*>(row)[idx] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
}
// VE weights at vector idx; `none` where there are no weights.
template <int VE>
__device__ __forceinline__ void load_weights(const void* w, int type, int idx, float none, float (&f)[VE]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = none;
  } else if (type == SKETCH_FP32) {
    if constexpr (VE == 1) {
      f[0] = __ldg(static_cast<const float*>(w) + idx);
    } else {
      const float4* p = reinterpret_cast<const float4*>(w) + (int64_t)idx * (VE / 4);
#pragma unroll
      for (int i = 0; i < VE / 4; ++i) {
        const float4 v = __ldg(p + i);
        f[4 * i] = v.x;
        f[4 * i + 1] = v.y;
        f[4 * i + 2] = v.z;
        f[4 * i + 3] = v.w;
      }
    }
  } else {
    if constexpr (VE == 1) {
      f[0] = bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(w) + idx));
    } else {
      const uint2* p = reinterpret_cast<const uint2*>(w) + (int64_t)idx * (VE / 4);
#pragma unroll
      for (int i = 0; i < VE / 4; ++i) {
        const uint2 v = __ldg(p + i);
        f[4 * i] = __uint_as_float(v.x << 16);
        f[4 * i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        f[4 * i + 2] = __uint_as_float(v.y << 16);
        f[4 * i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
    }
  }
}

// Sums over the tpr threads of a row, the same in each.  `slots` (one per warp)
// alternate between calls, so that one barrier per call is enough: a thread
// that writes a slot again has passed the barrier of the call between, after
// which nobody reads the old value.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr, float (*slots)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < tpr) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  }
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, first = (threadIdx.x & ~(tpr - 1)) >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slots[warp][i] = v[i];
    }
    if (tpr == (int)blockDim.x) __syncthreads();
    else tc::named_barrier(1 + first / (tpr >> 5), tpr);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < tpr >> 5; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += slots[first + w][i];
    }
  }
}

// ---- forward ---------------------------------------------------------------------
template <typename X, int VE, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_forward_kernel(const NormForward a, int tpr) {
  __shared__ float slots[2][THREADS / 32][1];
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * (THREADS / tpr) + threadIdx.x / tpr;
  const bool in = row < a.T;
  const int nvec = (int)(a.k / VE);
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  Vec<X, VE> raw[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (in && j * tpr + t < nvec) raw[j] = load_vec<X, VE>(x, j * tpr + t);
  const float inv_k = 1.f / (float)a.k;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (in && j * tpr + t < nvec) {
      float f[VE];
      unpack<X, VE>(raw[j], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) s[0] += f[i];
    }
  }
  row_sums<1>(s, tpr, slots[0]);
  const float mu = s[0] * inv_k;
  s[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (in && j * tpr + t < nvec) {
      float f[VE];
      unpack<X, VE>(raw[j], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) s[0] = fmaf(f[i] - mu, f[i] - mu, s[0]);
    }
  }
  row_sums<1>(s, tpr, slots[1]);
  const float rstd = 1.f / sqrtf(s[0] * inv_k + a.eps);
  if (!in) return;
  X* y = static_cast<X*>(a.Y) + row * a.ld_y;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j * tpr + t < nvec) {
      float f[VE], g[VE], b[VE];
      load_weights<VE>(a.gamma, a.w_type, j * tpr + t, 1.f, g);
      load_weights<VE>(a.beta, a.w_type, j * tpr + t, 0.f, b);
      unpack<X, VE>(raw[j], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = fmaf((f[i] - mu) * rstd, g[i], b[i]);
      store_vec<X, VE>(y, j * tpr + t, f);
    }
  }
  if (t == 0) {
    a.mean[row] = mu;
    a.rstd[row] = rstd;
  }
}

// ---- backward --------------------------------------------------------------------
// THREADS per block, one or more rows at a time.  SHARED: rows of more than
// 8192 leave 64 registers a thread, too few for a thread's 16 columns of dgamma
// and dbeta beside its row, so those lie in shared memory.  PREFETCH: the next
// row's loads are issued before this row's sums (BF16 vectors; fp32 rows are
// twice the bytes and have enough in flight without, single elements would take
// a register each).
template <typename X, int VE, int NV, int THREADS, bool SHARED>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) norm_backward_kernel(const NormBackward a, int tpr) {
  constexpr int E = NV * VE;
  constexpr bool PREFETCH = VE == 8;
  extern __shared__ float4 acc_raw[];
  float* acc = reinterpret_cast<float*>(acc_raw);
  __shared__ float slots[2][THREADS / 32][2];
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = THREADS / tpr;
  const int nvec = (int)(a.k / VE), k = (int)a.k;
  const int64_t stride = (int64_t)gridDim.x * groups;
  const int64_t row0 = (int64_t)blockIdx.x * groups + group;
  const int passes = (int)((a.T - (int64_t)blockIdx.x * groups + stride - 1) / stride);  // the same for the whole block
  float dg[SHARED ? 1 : E], db[SHARED ? 1 : E], gamma[SHARED ? 1 : E];
  if constexpr (SHARED) {
    for (int i = threadIdx.x; i < 2 * k; i += THREADS) acc[i] = 0.f;  // each thread's own columns follow after a barrier
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) g[i] = 0.f;
      if (j * tpr + t < nvec) load_weights<VE>(a.gamma, a.w_type, j * tpr + t, 1.f, g);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        gamma[j * VE + i] = g[i];
        dg[j * VE + i] = db[j * VE + i] = 0.f;
      }
    }
  }
  const float inv_k = 1.f / (float)a.k;
  Vec<X, VE> nx[NV], ny[NV];
  float nmu = 0.f, nrs = 0.f;
  auto load = [&](int64_t row) {
    if (row >= a.T) return;
    const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
    const X* y = static_cast<const X*>(a.dY) + row * a.ld_dy;
    nmu = a.mean[row];
    nrs = a.rstd[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j * tpr + t < nvec) {
        nx[j] = load_vec<X, VE>(x, j * tpr + t);
        ny[j] = load_vec<X, VE>(y, j * tpr + t);
      }
    }
  };
  if (PREFETCH) load(row0);
  for (int p = 0; p < passes; ++p) {
    const int64_t row = row0 + p * stride;
    if (!PREFETCH) load(row);
    Vec<X, VE> rx[NV], ry[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rx[j] = nx[j];
      ry[j] = ny[j];
    }
    const float mu = nmu, rs = nrs;
    if (PREFETCH && p + 1 < passes) load(row + stride);
    const bool in = row < a.T;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in && j * tpr + t < nvec) {
        float x[VE], y[VE], g[VE];
        unpack<X, VE>(rx[j], x);
        unpack<X, VE>(ry[j], y);
        if constexpr (SHARED) load_weights<VE>(a.gamma, a.w_type, j * tpr + t, 1.f, g);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float xh = (x[i] - mu) * rs;
          const float d = y[i] * (SHARED ? g[i] : gamma[SHARED ? 0 : j * VE + i]);
          s[0] += d;
          s[1] = fmaf(d, xh, s[1]);
          if constexpr (!SHARED) {
            dg[j * VE + i] = fmaf(y[i], xh, dg[j * VE + i]);
            db[j * VE + i] += y[i];
          }
        }
        if constexpr (SHARED) {
          float* pg = acc + (j * tpr + t) * VE;
#pragma unroll
          for (int i = 0; i < VE; i += (VE == 1 ? 1 : 4)) {
            if constexpr (VE == 1) {
              pg[0] = fmaf(y[0], (x[0] - mu) * rs, pg[0]);
              pg[k] += y[0];
            } else {
              float4 u = *reinterpret_cast<float4*>(pg + i), v = *reinterpret_cast<float4*>(pg + k + i);
              u.x = fmaf(y[i], (x[i] - mu) * rs, u.x);
              u.y = fmaf(y[i + 1], (x[i + 1] - mu) * rs, u.y);
              u.z = fmaf(y[i + 2], (x[i + 2] - mu) * rs, u.z);
              u.w = fmaf(y[i + 3], (x[i + 3] - mu) * rs, u.w);
              v.x += y[i];
              v.y += y[i + 1];
              v.z += y[i + 2];
              v.w += y[i + 3];
              *reinterpret_cast<float4*>(pg + i) = u;
              *reinterpret_cast<float4*>(pg + k + i) = v;
            }
          }
        }
      }
    }
    if (a.dX == nullptr) continue;
    row_sums<2>(s, tpr, slots[p & 1]);
    const float s0 = s[0] * inv_k, s1 = s[1] * inv_k;
    if (!in) continue;
    X* dx = static_cast<X*>(a.dX) + row * a.ld_dx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j * tpr + t < nvec) {
        float x[VE], y[VE], g[VE];
        unpack<X, VE>(rx[j], x);
        unpack<X, VE>(ry[j], y);
        if constexpr (SHARED) load_weights<VE>(a.gamma, a.w_type, j * tpr + t, 1.f, g);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float xh = (x[i] - mu) * rs;
          const float d = y[i] * (SHARED ? g[i] : gamma[SHARED ? 0 : j * VE + i]);
          y[i] = rs * (d - s0 - xh * s1);
        }
        store_vec<X, VE>(dx, j * tpr + t, y);
      }
    }
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return;
  // this block's partial row: the groups' sums added in their order
  float* out = a.ws + (int64_t)blockIdx.x * 2 * k;
  if constexpr (SHARED) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * k; i += THREADS) out[i] = acc[i];
  } else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (groups > 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (j * tpr + t < nvec) acc[group * k + (j * tpr + t) * VE + i] = half ? db[j * VE + i] : dg[j * VE + i];
        __syncthreads();
        for (int c = threadIdx.x; c < k; c += THREADS) {
          float v = 0.f;
          for (int g = 0; g < groups; ++g) v += acc[g * k + c];
          out[half * k + c] = v;
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (j * tpr + t < nvec) out[half * k + (j * tpr + t) * VE + i] = half ? db[j * VE + i] : dg[j * VE + i];
      }
    }
  }
}

// Adds the partial rows: 32 columns per block (of dgamma's k, then dbeta's), the
// partials dealt over eight warps.
__global__ void __launch_bounds__(kThreads) norm_grad_sum_kernel(const float* ws, int64_t k, int partials, float* dgamma,
                                                                 float* dbeta, int overwrite) {
  __shared__ float part[8][32];
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < 2 * k) {
#pragma unroll 8
    for (int p = warp; p < partials; p += 8) s += ws[(int64_t)p * 2 * k + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * k) {
    for (int w = 1; w < 8; ++w) s += part[w][lane];
    float* out = col < k ? dgamma : dbeta;
    if (out) {
      out += col < k ? col : col - k;
      *out = overwrite ? s : *out + s;
    }
  }
}

// ---- rows too wide for registers ----------------------------------------------------
__device__ __forceinline__ float get(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float get(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }
__device__ __forceinline__ float weight(const void* w, int type, int64_t i, float none) {
  if (w == nullptr) return none;
  return type == SKETCH_FP32 ? static_cast<const float*>(w)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(w)[i]);
}

template <typename X>
__global__ void __launch_bounds__(kThreads) norm_forward_wide_kernel(const NormForward a) {
  __shared__ float slots[2][kThreads / 32][1];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  X* y = static_cast<X*>(a.Y) + row * a.ld_y;
  float s[1] = {0.f};
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) s[0] += get(x, i);
  row_sums<1>(s, kThreads, slots[0]);
  const float mu = s[0] / (float)a.k;
  s[0] = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) s[0] = fmaf(get(x, i) - mu, get(x, i) - mu, s[0]);
  row_sums<1>(s, kThreads, slots[1]);
  const float rstd = 1.f / sqrtf(s[0] / (float)a.k + a.eps);
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads)
    put(y, i, fmaf((get(x, i) - mu) * rstd, weight(a.gamma, a.w_type, i, 1.f), weight(a.beta, a.w_type, i, 0.f)));
  if (threadIdx.x == 0) {
    a.mean[row] = mu;
    a.rstd[row] = rstd;
  }
}

// Partial sums of the weights' gradients over `rows` rows, one column per
// thread.  Before norm_dx_wide_kernel, which may write dX over dY.
template <typename X>
__global__ void __launch_bounds__(kThreads) norm_grad_wide_kernel(const NormBackward a, int64_t rows) {
  const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (col >= a.k) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows;
  const int64_t r1 = r0 + rows < a.T ? r0 + rows : a.T;
  float g = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = get(static_cast<const X*>(a.dY), r * a.ld_dy + col);
    g = fmaf(d, (get(static_cast<const X*>(a.X), r * a.ld_x + col) - a.mean[r]) * a.rstd[r], g);
    b += d;
  }
  float* p = a.ws + (int64_t)blockIdx.y * 2 * a.k;
  p[col] = g;
  p[a.k + col] = b;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) norm_dx_wide_kernel(const NormBackward a) {
  __shared__ float slots[kThreads / 32][2];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dY) + row * a.ld_dy;
  X* dx = static_cast<X*>(a.dX) + row * a.ld_dx;
  const float mu = a.mean[row], rs = a.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * weight(a.gamma, a.w_type, i, 1.f);
    s[0] += d;
    s[1] = fmaf(d, (get(x, i) - mu) * rs, s[1]);
  }
  row_sums<2>(s, kThreads, slots);
  const float s0 = s[0] / (float)a.k, s1 = s[1] / (float)a.k;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * weight(a.gamma, a.w_type, i, 1.f);
    put(dx, i, rs * (d - s0 - ((get(x, i) - mu) * rs) * s1));
  }
}

constexpr int64_t kMaxRowWidth = 16384;

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether every row of the matrix starts on 16 bytes and ends with a whole vector.
bool whole_vectors(const void* p, int64_t ld, int64_t k, int ve) { return on16(p) && ld % ve == 0 && k % ve == 0; }

// Threads per row: the fewest that hold a row at `most` vectors each, then more
// while the launch would leave SMs without a block.
int threads_per_row(int64_t nvec, int most, int64_t T, int limit) {
  int tpr = 8;
  while (tpr < limit && (int64_t)tpr * most < nvec) tpr *= 2;
  while (tpr < limit && tpr < 256 && tpr < nvec && T * tpr < 2 * (int64_t)num_sms() * kThreads) tpr *= 2;
  return tpr;
}

template <typename X, int VE, int NV, int THREADS = kThreads>
cudaError_t forward_rows(const NormForward& a, int tpr, cudaStream_t stream) {
  const int64_t blocks = ceil_div(a.T, THREADS / tpr);
  count_launch();
  norm_forward_kernel<X, VE, NV, THREADS><<<(unsigned)blocks, THREADS, 0, stream>>>(a, tpr);
  return cudaGetLastError();
}

template <typename X, int VE>
cudaError_t forward(const NormForward& a, cudaStream_t stream) {
  const int64_t nvec = a.k / VE;
  if constexpr (VE == 1) {  // 16 elements of a row per thread
    const int tpr = threads_per_row(nvec, 16, a.T, 1024);
    const int nv = (int)ceil_div(nvec, tpr);
    if (tpr > kThreads) return forward_rows<X, VE, 16, 1024>(a, 1024, stream);
    return nv <= 4 ? forward_rows<X, VE, 4>(a, tpr, stream) : forward_rows<X, VE, 16>(a, tpr, stream);
  } else {  // 64
    constexpr int kMost = 64 / VE;
    const int tpr = threads_per_row(nvec, kMost, a.T, kThreads);
    const int nv = (int)ceil_div(nvec, tpr);
    if (nv <= 1) return forward_rows<X, VE, 1>(a, tpr, stream);
    if (nv <= 2) return forward_rows<X, VE, 2>(a, tpr, stream);
    if (nv <= 4) return forward_rows<X, VE, 4>(a, tpr, stream);
    if (kMost > 8 && nv <= 8) return forward_rows<X, VE, 8>(a, tpr, stream);
    return forward_rows<X, VE, kMost>(a, tpr, stream);
  }
}

cudaError_t launch_grad_sum(const NormBackward& a, int partials, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div(2 * a.k, 32), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // its blocks may come up while the kernel before ends
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, norm_grad_sum_kernel, (const float*)a.ws, a.k, partials, a.dgamma, a.dbeta,
                            a.overwrite);
}

template <typename X, int VE, int NV, int THREADS, bool SHARED>
cudaError_t backward_rows(const NormBackward& a, int tpr, cudaStream_t stream) {
  const int groups = THREADS / tpr;
  int64_t blocks = ceil_div(a.T, groups);
  const int64_t most = (int64_t)num_sms() * (THREADS == 256 ? 2 : 1);
  if (blocks > most) blocks = most;
  if (blocks > kMaxPartials) blocks = kMaxPartials;
  const size_t smem = SHARED ? (size_t)(2 * a.k) * 4 : groups > 1 ? (size_t)groups * a.k * 4 : 0;
  auto kernel = norm_backward_kernel<X, VE, NV, THREADS, SHARED>;
  if (SHARED) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  count_launch();
  kernel<<<(unsigned)blocks, THREADS, smem, stream>>>(a, tpr);
  cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess && (a.dgamma || a.dbeta)) err = launch_grad_sum(a, (int)blocks, stream);
  return err;
}

template <typename X, int VE>
cudaError_t backward(const NormBackward& a, cudaStream_t stream) {
  const int64_t nvec = a.k / VE;
  if constexpr (VE == 1) {  // eight elements of a row per thread
    const int tpr = threads_per_row(nvec, 8, a.T, 2048);
    if (tpr <= 256) return backward_rows<X, VE, 8, 256, false>(a, tpr, stream);
    if (tpr <= 1024) return backward_rows<X, VE, 8, 1024, false>(a, 1024, stream);
    return backward_rows<X, VE, 16, 1024, true>(a, 1024, stream);
  } else {  // 16
    constexpr int kNV = 16 / VE;
    const int tpr = threads_per_row(nvec, kNV, a.T, 1024);
    if (tpr <= 256) return backward_rows<X, VE, kNV, 256, false>(a, tpr, stream);
    if (tpr == 512) return backward_rows<X, VE, kNV, 512, false>(a, tpr, stream);
    return backward_rows<X, VE, kNV, 1024, true>(a, tpr, stream);
  }
}

template <typename X>
cudaError_t backward_wide(const NormBackward& a, cudaStream_t stream) {
  if (a.dgamma || a.dbeta) {
    const int64_t rows = ceil_div(a.T, kMaxPartials) > 32 ? ceil_div(a.T, kMaxPartials) : 32;
    const int chunks = (int)ceil_div(a.T, rows);
    count_launch();
    norm_grad_wide_kernel<X><<<dim3((unsigned)ceil_div(a.k, kThreads), (unsigned)chunks), kThreads, 0, stream>>>(a, rows);
    const cudaError_t err = launch_grad_sum(a, chunks, stream);
    if (err != cudaSuccess) return err;
  }
  if (a.dX) {
    count_launch();
    norm_dx_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <typename X>
cudaError_t forward_any(const NormForward& a, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(X);
  if (a.k > kMaxRowWidth) {
    count_launch();
    norm_forward_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  if (whole_vectors(a.X, a.ld_x, a.k, VE) && whole_vectors(a.Y, a.ld_y, a.k, VE) && on16(a.gamma) && on16(a.beta))
    return forward<X, VE>(a, stream);
  return forward<X, 1>(a, stream);
}

template <typename X>
cudaError_t backward_any(const NormBackward& a, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(X);
  if (a.k > kMaxRowWidth) return backward_wide<X>(a, stream);
  if (whole_vectors(a.X, a.ld_x, a.k, VE) && whole_vectors(a.dY, a.ld_dy, a.k, VE) && on16(a.gamma) &&
      (a.dX == nullptr || whole_vectors(a.dX, a.ld_dx, a.k, VE)))
    return backward<X, VE>(a, stream);
  return backward<X, 1>(a, stream);
}

}  // namespace

cudaError_t launch_norm_forward(const NormForward& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? forward_any<__nv_bfloat16>(a, stream) : forward_any<float>(a, stream);
}

size_t norm_backward_workspace_bytes(int64_t T, int64_t k) {
  WsCursor cur;
  cur.take<float>((size_t)((T < kMaxPartials ? T : kMaxPartials) * 2 * k));
  cur.take<char>(0);
  return cur.offset;
}

cudaError_t launch_norm_backward(const NormBackward& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? backward_any<__nv_bfloat16>(a, stream) : backward_any<float>(a, stream);
}

}  // namespace rgs
