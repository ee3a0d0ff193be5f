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
//
// Bound by HBM.  One GB300, of the copy rate, 32768 x 4096 BF16: forward with residual,
// BF16 and 8-bit output 188 us, 0.95 (9 bytes a value; with loads that go first from the
// caches 191); with residual and BF16 output 164, 0.97; BF16 output alone 84, 0.94; 8-bit
// output alone 93, 0.64: its instructions take 67 % of the issue slots of warps that have
// 45 % of their places; backward with the stream's gradient 163 us, 0.97 (8 bytes), without
// it 140, 0.85.  8192 x 16384 forward 206 us, 0.87, backward 179, 0.88; fp32 16384 x 4096 185,
// 0.91, and 160, 0.99.  Rows on other places than 16 bytes: 32768 x 4095 forward 289 us, 0.62,
// backward 248, 0.64; the elements' shared memory reads and single stores take the rest.
// Wider rows than 16384 are read twice, value by value: 6554 x 20480 forward 412 us, 0.43,
// backward 742, 0.21.  8 x 2048 forward: 2.7 us on the device, a call 8 to 9; 1021 x 1001
// fp32 backward: 10.2 us on the device, two launches, a call 12 to 14.
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

// Adds the partial rows: 32 columns per block, the partials dealt over 32 warps (over
// eight, 1021 x 1001 fp32 took 12.1 us in all, not 10).
constexpr int kGradThreads = 1024;
__global__ void __launch_bounds__(kGradThreads) rms_grad_sum_kernel(const float* ws, int64_t k, int partials, float* dgamma,
                                                                    int overwrite) {
  __shared__ float part[32][33];
  start_early();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < k) {
#pragma unroll
    for (int i = 0; i < kMaxPartials / 32; ++i) {
      const int p = i * 32 + warp;
      if (p < partials) s += ws[(int64_t)p * k + col];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  s = lane_sum<true>(part[lane][warp], 32);  // warp w joins column w
  const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && mine < k) dgamma[mine] = overwrite ? s : dgamma[mine] + s;
}

cudaError_t launch_grad_sum(const RmsBackward& a, int partials, cudaStream_t stream) {
  return launch_early(rms_grad_sum_kernel, ceil_div(a.k, 32), kGradThreads, 0, stream, (const float*)a.ws, a.k, partials,
                      a.dgamma, a.overwrite);
}

// ---- forward, rows in registers ----------------------------------------------------
// A row belongs to `tpr` threads (a power of two, 32 to 1024), kForwardVectors vectors of
// 16 bytes to each, so that X and R are read once; gamma lies in shared memory as fp32.
// Vector j tpr + t is thread t's j-th, so that 16 neighbouring lanes (BF16; fp32: 32)
// hold the 128 columns of a scale.
constexpr int kForwardVectors = 4;
// Blocks per SM: with the residual two (32768 x 4096 BF16 with codes 191 us, with three
// 200, with four 199), without it four (BF16 output 85.7 us, with three 89.7, two 105).
constexpr int forward_blocks(int threads, bool res) { return threads == 256 ? (res ? 2 : 4) : threads == 512 ? 2 : 1; }

// The row's sum from its threads' ones.  `part` alternates between rows: a thread that
// writes it again has passed the barrier of the row between, after which nobody reads
// the old values.
__device__ __forceinline__ float row_sum(float v, int tpr, float* part) {
  v = lane_sum<true>(v, 32);
  const int warps = tpr >> 5;
  if (warps > 1) {
    const int lane = threadIdx.x & 31, warp0 = (threadIdx.x & ~(tpr - 1)) >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    if (tpr == (int)blockDim.x) __syncthreads();
    else tc::named_barrier(1 + warp0 / warps, tpr);
    float j[1] = {part[warp0 + (lane & (warps - 1))]};
    join_sums(j, warps);
    v = j[0];
  }
  return v;
}

template <typename X, int THREADS, bool RES, bool CODES>
__global__ void __launch_bounds__(THREADS, forward_blocks(THREADS, RES)) rms_forward_kernel(const RmsForward a, int tpr) {
  constexpr int VE = 16 / (int)sizeof(X), NV = kForwardVectors, P = VE / 2;
  extern __shared__ __align__(128) float weights[];
  __shared__ float part[2][THREADS / 32];
  const int t = threadIdx.x & (tpr - 1), lane = threadIdx.x & 31, k = (int)a.k;
  const int nvec = k / VE, groups = (k + kScaleBlock - 1) / kScaleBlock;
  start_early();
  for (int c = threadIdx.x; c < k; c += THREADS) weights[weight_at<VE>(c, k)] = weight(a.gamma, a.w_type, c, 1.f);
  const uint32_t gamma = tc::smem_u32(weights);
  const float inv_k = 1.f / (float)k;
  __syncthreads();
  const int64_t stride = (int64_t)gridDim.x * (THREADS / tpr);
  int p = 0;
  for (int64_t base = (int64_t)blockIdx.x * (THREADS / tpr); base < a.T; base += stride, p ^= 1) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < a.T;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const X*>(a.X) + row * a.ld_x);
    uint4 raw[NV];
    Pair v[RES ? NV : 1][P];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (in && j * tpr + t < nvec) raw[j] = x[j * tpr + t];
    }
    if constexpr (RES) {
      const uint4* r = reinterpret_cast<const uint4*>(static_cast<const X*>(a.R) + row * a.ld_r);
      uint4 add[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        add[j] = make_uint4(0, 0, 0, 0);
        if (in && j * tpr + t < nvec) add[j] = r[j * tpr + t];
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Pair q[P];
        vec_pairs<X>(raw[j], v[j]);
        vec_pairs<X>(add[j], q);
#pragma unroll
        for (int i = 0; i < P; ++i) v[j][i] = add2(v[j][i], q[i]);
      }
    }
    auto values = [&](int j, Pair(&q)[P]) {
      if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < P; ++i) q[i] = v[j][i];
      } else {
        vec_pairs<X>(raw[j], q);
      }
    };
    Pair sum = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pair q[P];
      values(j, q);
#pragma unroll
      for (int i = 0; i < P; ++i) sum = fma2(q[i], q[i], sum);
    }
    if (RES && a.S && in) {
      X* s = static_cast<X*>(a.S) + row * a.ld_s;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j * tpr + t < nvec) store_vec<X>(s, j * tpr + t, v[RES ? j : 0]);
    }
    const float rstd = 1.f / sqrtf(row_sum(sum2(sum), tpr, part[p]) * inv_k + a.eps);
    const Pair r2 = pair(rstd, rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int idx = j * tpr + t;
      const bool has = in && idx < nvec;
      Pair q[P], g[P];
      values(j, q);
      if (has) {
        weight_pairs<VE>(gamma, idx, k, g);
#pragma unroll
        for (int i = 0; i < P; ++i) q[i] = mul2(mul2(q[i], r2), g[i]);
        if (a.Y) store_vec<X>(static_cast<X*>(a.Y) + row * a.ld_y, idx, q);
      }
      if constexpr (CODES) {  // what lies past the row's end counts as zeros
        float y[VE];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 f = split(q[i]);
          y[2 * i] = f.x;
          y[2 * i + 1] = f.y;
        }
        uint32_t top = has ? top_magnitude(y) : 0;
#pragma unroll
        for (int o = 64 / VE; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float inv;
        const float scale = code_scale(top, inv);
        if (has) {
          if ((lane & (128 / VE - 1)) == 0) a.scale[row * groups + idx / (kScaleBlock / VE)] = scale;
          uint32_t c[VE / 4];
#pragma unroll
          for (int i = 0; i < VE / 4; ++i)
            c[i] = codes2(y[4 * i] * inv, y[4 * i + 1] * inv) | codes2(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16;
          uint8_t* out = a.Q + row * a.ld_q + (int64_t)idx * VE;
          if constexpr (VE == 8) *reinterpret_cast<uint2*>(out) = make_uint2(c[0], c[VE / 4 - 1]);
          else *reinterpret_cast<uint32_t*>(out) = c[0];
        }
      }
    }
    if (a.rstd && in && t == 0) a.rstd[row] = rstd;
  }
}

// Rows of any alignment: a warp to 128 columns at a time, four to a lane, G times; `wpr`
// (a power of two) warps to a row.  The rows of X and R come through a ring in shared
// memory, by bulk copies between the 16-byte boundaries around them, and are read there
// once, element by element (read so from global memory, 32768 x 4095 BF16 with residual
// and codes took 711 us).
template <typename X, int G, int THREADS, bool RES>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) rms_forward_ring_kernel(const RmsForward a, const Ring ring, int wpr, int* err) {
  constexpr int NM = RES ? 2 : 1;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ __align__(8) uint64_t full[kMaxSlots];
  __shared__ float part[2][THREADS / 32];
  __shared__ volatile int abort_flag;
  Ring r = ring;
  r.smem = tc::smem_u32(ring_mem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp & (wpr - 1), k = (int)a.k;
  const int groups = (k + kScaleBlock - 1) / kScaleBlock;
  const float inv_k = 1.f / (float)k;
  auto source = [&](const void* p, int64_t ld) {
    return RowSource{static_cast<const char*>(p), ld * (int64_t)sizeof(X), a.T, (uint32_t)(a.k * sizeof(X))};
  };
  RowSource m[NM] = {source(a.X, a.ld_x)};
  if constexpr (RES) m[NM - 1] = source(a.R, a.ld_r);
  const int64_t stride = (int64_t)gridDim.x * r.rows, first = (int64_t)blockIdx.x * r.rows;
  const int passes = first < a.T ? (int)((a.T - first + stride - 1) / stride) : 0;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < r.slots; ++s) tc::mbar_init(&full[s], 1);
    tc::fence_mbar_init();
  }
  start_early();
  __syncthreads();
  int filled = 0;  // warp 0's: sets whose copies have begun
  if (warp == 0)
    for (; filled < passes && filled < r.slots; ++filled)
      fill_slot<true, false, NM>(r, m, filled, first + filled * stride, &full[filled]);
  float gamma[G][4];  // a thread's columns stay the same
#pragma unroll
  for (int j = 0; j < G; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (j * wpr + w) * kScaleBlock + i * 32 + lane;
      gamma[j][i] = c < k ? weight(a.gamma, a.w_type, c, 1.f) : 0.f;
    }
  }
  int64_t row = first + warp / wpr;
  int s = 0;
  uint32_t ph = 0;
  for (int p = 0; p < passes; ++p, row += stride) {
    tc::mbar_wait(&full[s], ph, &abort_flag, err, tc::kErrTimeoutLoad);
    const uint32_t at = r.smem + (uint32_t)s * r.slot + (uint32_t)(warp / wpr) * r.pitch;
    uint32_t from[NM];
#pragma unroll
    for (int i = 0; i < NM; ++i) from[i] = at + (uint32_t)(i * r.rows) * r.pitch + phase(m[i], row);
    const bool in = row < a.T;
    float f[G][4], sum = 0.f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (j * wpr + w) * kScaleBlock + i * 32 + lane;
        f[j][i] = 0.f;
        if (in && c < k) {
          f[j][i] = read_one<X>(from[0] + (uint32_t)(c * sizeof(X)));
          if constexpr (RES) f[j][i] += read_one<X>(from[NM - 1] + (uint32_t)(c * sizeof(X)));
        }
        sum = fmaf(f[j][i], f[j][i], sum);
      }
    }
    sum = lane_sum<true>(sum, 32);
    if (lane == 0) part[p & 1][warp] = sum;  // alternates, as in row_sum
    __syncthreads();
    if (warp == 0 && filled < passes) {  // every thread has its values of this slot
      fill_slot<true, false, NM>(r, m, s, first + filled * stride, &full[s]);
      ++filled;
    }
    float js[1] = {part[p & 1][(warp & ~(wpr - 1)) + (lane & (wpr - 1))]};
    join_sums(js, wpr);
    const float rstd = 1.f / sqrtf(js[0] * inv_k + a.eps);
    if (in) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int g = j * wpr + w;
        if (g >= groups) break;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = g * kScaleBlock + i * 32 + lane;
          y[i] = 0.f;
          if (c < k) {
            y[i] = f[j][i] * rstd * gamma[j][i];
            if (RES && a.S) store_one(static_cast<X*>(a.S) + row * a.ld_s + c, f[j][i]);
            if (a.Y) store_one(static_cast<X*>(a.Y) + row * a.ld_y + c, y[i]);
          }
        }
        if (a.Q) {
          float inv;
          const float scale = code_scale(__reduce_max_sync(0xFFFFFFFFu, top_magnitude(y)), inv);
          if (lane == 0) a.scale[row * groups + g] = scale;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = g * kScaleBlock + i * 32 + lane;
            if (c < k) a.Q[row * a.ld_q + c] = (uint8_t)codes2(y[i] * inv, 0.f);
          }
        }
      }
      if (a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
    }
    if (++s == r.slots) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (threadIdx.x == 0 && abort_flag) drain(full, r.slots, filled);
}

constexpr int64_t kMaxRowWidth = 16384;

template <typename X, int THREADS>
cudaError_t forward_vectors(const RmsForward& a, int tpr, cudaStream_t stream) {
  const size_t smem = (size_t)a.k * 4;
  int64_t blocks = ceil_div(a.T, THREADS / tpr);
  const int64_t most = (int64_t)num_sms() * forward_blocks(THREADS, a.R != nullptr);
  if (blocks > most) blocks = most;
  auto launch = [&](auto kernel) {
    const cudaError_t err = allow_smem(kernel, smem);
    return err == cudaSuccess ? launch_early(kernel, blocks, THREADS, smem, stream, a, tpr) : err;
  };
  if (a.R) return a.Q ? launch(rms_forward_kernel<X, THREADS, true, true>) : launch(rms_forward_kernel<X, THREADS, true, false>);
  return a.Q ? launch(rms_forward_kernel<X, THREADS, false, true>) : launch(rms_forward_kernel<X, THREADS, false, false>);
}

template <typename X, int G, int THREADS, bool RES>
cudaError_t forward_ring(const RmsForward& a, int wpr, cudaStream_t stream) {
  constexpr int kPerSm = THREADS == 256 ? 2 : 1;
  Ring r = {};
  r.rows = THREADS / 32 / wpr;
  r.each = 1;
  r.pitch = (uint32_t)((a.k * sizeof(X) + 15) / 16 * 16 + 16);  // room for the 16-byte boundaries around a row
  r.slot = r.pitch * (uint32_t)(r.rows * (RES ? 2 : 1));
  r.slots = (int)(kMostSmem / kPerSm / r.slot);  // at least one: 128 KB for 16384 fp32 values of X and R
  if (r.slots > kMaxSlots) r.slots = kMaxSlots;
  int64_t blocks = ceil_div(a.T, r.rows);
  if (blocks > kPerSm * (int64_t)num_sms()) blocks = kPerSm * (int64_t)num_sms();
  int* err_word = nullptr;
  cudaError_t err = device_error_word(&err_word);
  if (err != cudaSuccess) return err;
  const size_t smem = (size_t)r.slots * r.slot;
  auto kernel = rms_forward_ring_kernel<X, G, THREADS, RES>;
  err = allow_smem(kernel, smem);
  return err == cudaSuccess ? launch_early(kernel, blocks, THREADS, smem, stream, a, r, wpr, err_word) : err;
}

template <typename X, bool RES>
cudaError_t forward_any_place(const RmsForward& a, cudaStream_t stream) {
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  if (groups > 64) return forward_ring<X, 8, 512, RES>(a, 16, stream);
  if (groups > 32) return forward_ring<X, 4, 512, RES>(a, 16, stream);
  int wpr = 1;
  while (wpr < 8 && 4 * wpr < groups) wpr *= 2;
  while (wpr < 8 && wpr < groups && a.T * wpr < 16 * (int64_t)num_sms()) wpr *= 2;
  return groups <= wpr ? forward_ring<X, 1, 256, RES>(a, wpr, stream) : forward_ring<X, 4, 256, RES>(a, wpr, stream);
}

template <typename X>
cudaError_t forward_any(const RmsForward& a, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(X);
  if (a.k <= kMaxRowWidth) {
    auto whole = [&](const void* p, int64_t ld) { return p == nullptr || whole_vectors(p, ld, a.k, VE, sizeof(X)); };
    if (whole(a.X, a.ld_x) && whole(a.R, a.ld_r) && whole(a.S, a.ld_s) && whole(a.Y, a.ld_y)) {
      int tpr = threads_per_row(a.k / VE, kForwardVectors, a.T, 1024);
      if (tpr < 32) tpr = 32;
      if (tpr <= 256) return forward_vectors<X, 256>(a, tpr, stream);
      if (tpr == 512) return forward_vectors<X, 512>(a, tpr, stream);
      return forward_vectors<X, 1024>(a, tpr, stream);
    }
    return a.R ? forward_any_place<X, true>(a, stream) : forward_any_place<X, false>(a, stream);
  }
  count_launch();
  rms_forward_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ---- backward, rows through a ring in shared memory ----------------------------------
// A thread's columns stay the same over the rows that its block walks, so that dgamma
// adds up in registers; with those and gamma there, the rows of S, dY and (DS) dS come
// through shared memory: bulk copies bring them into a ring of slots, several sets of
// rows ahead, and threads read them there, once for each of the two passes over a row.
// B rows are worked on side by side, so that their sums' shuffles overlap, and one block
// barrier a set both joins the warps' sums and tells that the slot of the set before can
// be filled again.  Each block leaves a partial row of dgamma, which rms_grad_sum_kernel
// adds in a fixed order.
constexpr int backward_blocks(int threads) { return threads == 256 ? 2 : 1; }
constexpr int backward_rows_each(size_t size, int threads) { return threads == 256 && size == 2 ? 2 : 1; }

// A thread's columns: NV vectors of VE elements, as E / 2 pairs.  With VE = 1 (rows of
// any alignment) a pair is the thread's elements 2 q and 2 q + 1, tpr columns apart.
template <typename X, int VE, int NV, int THREADS, bool DS>
__global__ void __launch_bounds__(THREADS, backward_blocks(THREADS))
    rms_backward_kernel(const RmsBackward a, const Ring ring, int tpr, int* err) {
  constexpr int E = NV * VE, B = backward_rows_each(sizeof(X), THREADS), NM = DS ? 3 : 2;
  constexpr int VP = VE == 1 ? 1 : VE / 2, NP = E / 2 / VP;  // pairs per step, steps
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ __align__(8) uint64_t full[kMaxSlots];
  __shared__ float part[2][B][THREADS / 32];
  __shared__ volatile int abort_flag;
  Ring r = ring;
  r.smem = tc::smem_u32(ring_mem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto source = [&](const void* p, int64_t ld) {
    return RowSource{static_cast<const char*>(p), ld * (int64_t)sizeof(X), a.T, (uint32_t)(a.k * sizeof(X))};
  };
  RowSource m[NM] = {source(a.S, a.ld_s), source(a.dY, a.ld_dy)};
  if constexpr (DS) m[NM - 1] = source(a.dS, a.ld_ds);
  const int64_t stride = (int64_t)gridDim.x * r.rows, first = (int64_t)blockIdx.x * r.rows;
  const int passes = first < a.T ? (int)((a.T - first + stride - 1) / stride) : 0;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < r.slots; ++s) tc::mbar_init(&full[s], 1);
    tc::fence_mbar_init();
  }
  start_early();
  __syncthreads();
  int filled = 0;  // warp 0's: sets whose copies have begun
  if (warp == 0)
    for (; filled < passes && filled < r.slots; ++filled)
      fill_slot<VE == 1, false, NM>(r, m, filled, first + filled * stride, &full[filled]);
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = THREADS / tpr, k = (int)a.k;
  const int warps = tpr >> 5, warp0 = (threadIdx.x & ~(tpr - 1)) >> 5;
  const int nvec = k / VE;
  // column of element i of pair q of step j; whether the thread has it
  auto column = [&](int j, int q, int i) { return VE == 1 ? (2 * j + i) * tpr + t : (j * tpr + t) * VE + 2 * q + i; };
  auto has = [&](int j) { return VE == 1 ? 2 * j * tpr + t < k : j * tpr + t < nvec; };
  // VE = 1: the pair's second element may lie past the row; a zero stands for it
  auto read = [&](uint32_t at, int j, Pair(&v)[VP]) {
    if constexpr (VE == 1) {
      const int c = 2 * j * tpr + t;
      const uint32_t p = at + (uint32_t)(c * sizeof(X));
      v[0] = pair(read_one<X>(p), c + tpr < k ? read_one<X>(p + (uint32_t)(tpr * sizeof(X))) : 0.f);
    } else {
      vec_pairs<X>(tc::lds128(at + (uint32_t)j * (16u * tpr)), v);
    }
  };
  Pair dg[E / 2], gamma[E / 2];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      const int c0 = column(j, q, 0), c1 = column(j, q, 1);
      gamma[j * VP + q] = pair(c0 < k ? weight(a.gamma, a.w_type, c0, 1.f) : 0.f, c1 < k ? weight(a.gamma, a.w_type, c1, 1.f) : 0.f);
      dg[j * VP + q] = 0;
    }
  }
  const float inv_k = 1.f / (float)k;
  int64_t row = first + group * r.each;
  float next[B];  // the next set's rstd
  auto load_stats = [&](int64_t at) {
#pragma unroll
    for (int b = 0; b < B; ++b) next[b] = b < r.each && at + b < a.T ? a.rstd[at + b] : 0.f;
  };
  load_stats(row);
  const uint32_t set_at = r.smem + (uint32_t)(group * r.each) * r.pitch, next_m = (uint32_t)r.rows * r.pitch;
  uint32_t slot = set_at;
  int s = 0;
  uint32_t ph = 0;
  for (int p = 0; p < passes; ++p, row += stride) {
    Pair sum[B];
    float rstd[B], v[B];
    uint32_t at[B][NM];
#pragma unroll
    for (int b = 0; b < B; ++b) rstd[b] = next[b];
    if (p + 1 < passes) load_stats(row + stride);
    tc::mbar_wait(&full[s], ph, &abort_flag, err, tc::kErrTimeoutLoad);
    // what lies past the last row is worked on like a row (in shared memory that a row
    // before left) and not kept
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const uint32_t q = b < r.each ? b : 0;
#pragma unroll
      for (int i = 0; i < NM; ++i)
        at[b][i] = slot + q * r.pitch + (uint32_t)i * next_m + (VE == 1 ? phase(m[i], row + q) : 16u * t);
      sum[b] = 0;
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if (has(j)) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          Pair x[VP], y[VP];
          read(at[b][0], j, x);
          read(at[b][1], j, y);
#pragma unroll
          for (int q = 0; q < VP; ++q) sum[b] = fma2(mul2(y[q], gamma[j * VP + q]), x[q], sum[b]);  // times rstd once it is summed up
        }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) v[b] = sum2(sum[b]) * rstd[b];
    lane_sums<true, B>(v, 32);
    float(*q)[THREADS / 32] = part[p & 1];  // alternates, as in row_sum
    if (lane == 0) {
#pragma unroll
      for (int b = 0; b < B; ++b) q[b][warp] = v[b];
    }
    __syncthreads();
    if (warp == 0 && p > 0 && filled < passes && r.slots > 1) {  // every thread is done with the set before
      const int before = s ? s - 1 : r.slots - 1;
      fill_slot<VE == 1, false, NM>(r, m, before, first + filled * stride, &full[before]);
      ++filled;
    }
    if (warps > 1) {
#pragma unroll
      for (int b = 0; b < B; ++b) v[b] = q[b][warp0 + (lane & (warps - 1))];
      join_sums(v, warps);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b >= r.each || row + b >= a.T) continue;
      X* dx = static_cast<X*>(a.dX) + (row + b) * a.ld_dx;
      const float f = -v[b] * inv_k * rstd[b];
      const Pair c = pair(f, f), rs = pair(rstd[b], rstd[b]);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if (has(j)) {
          Pair x[VP], y[VP], d[VP];
          read(at[b][0], j, x);
          read(at[b][1], j, y);
          if constexpr (DS) read(at[b][NM - 1], j, d);
#pragma unroll
          for (int q = 0; q < VP; ++q) {
            const int e = j * VP + q;
            x[q] = mul2(x[q], rs);
            dg[e] = fma2(y[q], x[q], dg[e]);
            x[q] = DS ? fma2(x[q], c, d[q]) : mul2(x[q], c);
            y[q] = fma2(mul2(y[q], gamma[e]), rs, x[q]);
          }
          if (a.dX) {
            if constexpr (VE == 1) {
              const float2 o = split(y[0]);
              const int col = 2 * j * tpr + t;
              store_one(dx + col, o.x);
              if (col + tpr < k) store_one(dx + col + tpr, o.y);
            } else {
              store_vec<X>(dx, j * tpr + t, y);
            }
          }
        }
      }
    }
    if (r.slots == 1 && p + 1 < passes) {  // rows too wide for two slots
      __syncthreads();
      if (warp == 0) fill_slot<VE == 1, false, NM>(r, m, 0, first + filled * stride, &full[0]);
      ++filled;
    }
    slot += r.slot;
    if (++s == r.slots) {
      s = 0;
      ph ^= 1u;
      slot = set_at;
    }
  }
  if (threadIdx.x == 0 && abort_flag) drain(full, r.slots, filled);
  if (a.dgamma == nullptr) return;
  // this block's partial row: the groups' sums added in their order, in the ring's memory
  float* out = a.ws + (int64_t)blockIdx.x * k;
  float* acc = reinterpret_cast<float*>(ring_mem);
  __syncthreads();
  float* to = groups > 1 ? acc + group * k : out;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      const float2 f = split(dg[j * VP + q]);
      const int c0 = column(j, q, 0), c1 = column(j, q, 1);
      if (c0 < k) to[c0] = f.x;
      if (c1 < k) to[c1] = f.y;
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < k; c += THREADS) {
      float v = 0.f;
      for (int g = 0; g < groups; ++g) v += acc[g * k + c];
      out[c] = v;
    }
  }
}

template <typename X, int VE, int NV, int THREADS, bool DS>
cudaError_t backward_rows(const RmsBackward& a, int tpr, cudaStream_t stream) {
  const int groups = THREADS / tpr, matrices = DS ? 3 : 2, per_sm = backward_blocks(THREADS);
  // rows side by side: as many as the kernel takes while every block still has a set
  int each = 1;
  while (each < backward_rows_each(sizeof(X), THREADS) && a.T >= 2 * each * (int64_t)num_sms() * per_sm * groups) each *= 2;
  int64_t blocks = ceil_div(a.T, groups * each);
  if (blocks > (int64_t)num_sms() * per_sm) blocks = (int64_t)num_sms() * per_sm;
  if (blocks > kMaxPartials) blocks = kMaxPartials;
  Ring r = {};
  r.rows = groups * each;
  r.each = each;
  // VE = 1: room for the 16-byte boundaries around a row
  r.pitch = VE > 1 ? (uint32_t)(a.k * sizeof(X)) : (uint32_t)((a.k * sizeof(X) + 15) / 16 * 16 + 16);
  r.slot = r.pitch * (uint32_t)(r.rows * matrices);
  const uint32_t room = (uint32_t)(kMostSmem / per_sm);
  r.slots = (int)(room / r.slot < kMaxSlots ? room / r.slot : kMaxSlots);
  if (r.slots < 1) return cudaErrorInvalidConfiguration;  // the widest set, 16384 fp32 values of three matrices, has 192 KB
  int* err_word = nullptr;
  cudaError_t err = device_error_word(&err_word);
  if (err != cudaSuccess) return err;
  size_t smem = (size_t)r.slots * r.slot;
  if (groups > 1 && smem < (size_t)groups * a.k * 4) smem = (size_t)groups * a.k * 4;
  auto kernel = rms_backward_kernel<X, VE, NV, THREADS, DS>;
  err = allow_smem(kernel, smem);
  if (err != cudaSuccess) return err;
  err = launch_early(kernel, blocks, THREADS, smem, stream, a, r, tpr, err_word);
  if (err == cudaSuccess && a.dgamma) err = launch_grad_sum(a, (int)blocks, stream);
  return err;
}

template <typename X, int VE, bool DS>
cudaError_t backward(const RmsBackward& a, cudaStream_t stream) {
  constexpr int NV = 16 / VE;  // 16 elements of a row per thread, 32 above 8192
  int tpr = threads_per_row(a.k / VE, NV, a.T, 512);
  if (tpr < 32) tpr = 32;
  if (tpr <= 256) return backward_rows<X, VE, NV, 256, DS>(a, tpr, stream);
  if (a.k <= 8192) return backward_rows<X, VE, NV, 512, DS>(a, 512, stream);
  return backward_rows<X, VE, 2 * NV, 512, DS>(a, 512, stream);
}

template <typename X>
cudaError_t backward_any(const RmsBackward& a, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(X);
  if (a.k <= kMaxRowWidth) {
    auto whole = [&](const void* p, int64_t ld) { return p == nullptr || whole_vectors(p, ld, a.k, VE, sizeof(X)); };
    const bool vectors = whole(a.S, a.ld_s) && whole(a.dY, a.ld_dy) && whole(a.dS, a.ld_ds) && whole(a.dX, a.ld_dx);
    if (a.dS) return vectors ? backward<X, VE, true>(a, stream) : backward<X, 1, true>(a, stream);
    return vectors ? backward<X, VE, false>(a, stream) : backward<X, 1, false>(a, stream);
  }
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
