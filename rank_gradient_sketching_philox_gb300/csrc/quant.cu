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

// Codes of a vector's VE values, four to a word.
template <int VE>
__device__ __forceinline__ void vector_codes(const Pair (&v)[VE / 2], float inv, uint32_t (&c)[VE / 4]) {
  const Pair inv2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < VE / 4; ++i) {
    const float2 lo = split(mul2(v[2 * i], inv2)), hi = split(mul2(v[2 * i + 1], inv2));
    c[i] = codes2(lo.x, lo.y) | codes2(hi.x, hi.y) << 16;
  }
}
template <int VE>
__device__ __forceinline__ uint32_t vector_top(const Pair (&v)[VE / 2]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VE / 2; ++i) {
    const float2 f = split(v[i]);
    top = max(top, max(magnitude(f.x), magnitude(f.y)));
  }
  return top;
}
template <int VE>
__device__ __forceinline__ void put_codes(uint8_t* q, const uint32_t (&c)[VE / 4]) {
  if constexpr (VE == 8) *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[VE / 4 - 1]);
  else *reinterpret_cast<uint32_t*>(q) = c[0];
}

// A scale per row and 128 columns, rows of whole 16-byte vectors: 16 lanes (BF16; fp32: 32)
// to such a piece, kPieces of them under way at once.
constexpr int kPieces = 4;
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_row_vectors_kernel(const Quantize a, int64_t pieces) {
  constexpr int VE = 16 / (int)sizeof(X), LANES = kScaleBlock / VE, PER_BLOCK = kThreads / LANES;
  const int t = threadIdx.x % LANES;
  const uint32_t groups = (uint32_t)ceil_div(a.k, kScaleBlock);
  const int64_t first = (int64_t)blockIdx.x * (PER_BLOCK * kPieces) + threadIdx.x / LANES;
  start_early();
  uint4 raw[kPieces];
  int64_t row[kPieces], col[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int64_t p = first + j * PER_BLOCK;
    row[j] = p < (int64_t(1) << 32) ? (uint32_t)p / groups : p / groups;
    col[j] = (p - row[j] * groups) * kScaleBlock + t * VE;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (p < pieces && col[j] < a.k)
      raw[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const X*>(a.X) + row[j] * a.ld_x + col[j]));
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int64_t p = first + j * PER_BLOCK;
    Pair v[VE / 2];
    vec_pairs<X>(raw[j], v);
    uint32_t top = vector_top<VE>(v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (p >= pieces) continue;
    float inv;
    const float scale = code_scale(top, inv);
    if (t == 0) a.scale[p] = scale;
    uint32_t c[VE / 4];
    vector_codes<VE>(v, inv, c);
    if (col[j] < a.k) put_codes<VE>(a.Q + row[j] * a.ld_q + col[j], c);
  }
}

// A scale per 128 rows and 128 columns, rows of whole 16-byte vectors: a block to each.  A
// thread has four rows of VE columns (twice, fp32 four times), whose codes it turns by
// 4 x 4 bytes into words of Qt's rows; those go through shared memory, word w of column
// c at w ^ 4 (c / 8 % 8), where a warp's words meet in a bank twice at most.
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_tile_vectors_kernel(const Quantize a) {
  constexpr int VE = 16 / (int)sizeof(X), LANES = kScaleBlock / VE, QUADS = kThreads / LANES, STEPS = 32 / QUADS;
  __shared__ uint32_t part[kWarps];
  __shared__ __align__(16) uint32_t tile[kScaleBlock][32];
  const int t = threadIdx.x % LANES, quad0 = threadIdx.x / LANES;
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  const int64_t r0 = blockIdx.x / groups * kScaleBlock, c0 = blockIdx.x % groups * kScaleBlock;
  const bool has = c0 + t * VE < a.k;
  start_early();
  uint4 raw[STEPS][4];
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = r0 + (s * QUADS + quad0) * 4 + i;
      raw[s][i] = make_uint4(0, 0, 0, 0);
      if (has && row < a.T)
        raw[s][i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const X*>(a.X) + row * a.ld_x + c0) + t);
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Pair v[VE / 2];
      vec_pairs<X>(raw[s][i], v);
      top = max(top, vector_top<VE>(v));
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu, part[threadIdx.x & (kWarps - 1)]);
  float inv;
  const float scale = code_scale(top, inv);
  if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int quad = s * QUADS + quad0;
    uint32_t c[4][VE / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Pair v[VE / 2];
      vec_pairs<X>(raw[s][i], v);
      vector_codes<VE>(v, inv, c[i]);
      const int64_t row = r0 + quad * 4 + i;
      if (a.Q && has && row < a.T) put_codes<VE>(a.Q + row * a.ld_q + c0 + t * VE, c[i]);
    }
    if (a.Qt) {
#pragma unroll
      for (int h = 0; h < VE / 4; ++h) {
        const uint32_t ab_lo = __byte_perm(c[0][h], c[1][h], 0x5140), ab_hi = __byte_perm(c[0][h], c[1][h], 0x7362);
        const uint32_t cd_lo = __byte_perm(c[2][h], c[3][h], 0x5140), cd_hi = __byte_perm(c[2][h], c[3][h], 0x7362);
        const uint32_t w[4] = {__byte_perm(ab_lo, cd_lo, 0x5410), __byte_perm(ab_lo, cd_lo, 0x7632),
                               __byte_perm(ab_hi, cd_hi, 0x5410), __byte_perm(ab_hi, cd_hi, 0x7632)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = t * VE + 4 * h + i;
          tile[col][quad ^ (4 * ((col >> 3) & 7))] = w[i];
        }
      }
    }
  }
  if (a.Qt == nullptr) return;
  __syncthreads();
#pragma unroll
  for (int e = threadIdx.x; e < kScaleBlock * 8; e += kThreads) {
    const int col = e >> 3, q = e & 7;
    const int64_t row = r0 + 16 * q;  // of X
    if (c0 + col >= a.k || row >= a.T) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(&tile[col][(4 * q) ^ (4 * ((col >> 3) & 7))]);
    uint8_t* out = a.Qt + (c0 + col) * a.ld_qt + row;
    if (row + 16 <= a.T) {
      *reinterpret_cast<uint4*>(out) = w;
    } else {
      const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (row + i < a.T) out[i] = (uint8_t)(r[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <typename X>
cudaError_t quantize(const Quantize& a, cudaStream_t stream) {
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  constexpr int VE = 16 / (int)sizeof(X), PER_BLOCK = kThreads / (kScaleBlock / VE) * kPieces;
  const bool vectors = whole_vectors(a.X, a.ld_x, a.k, VE, sizeof(X));
  if (vectors && a.rows == 1 && ceil_div(a.T * groups, PER_BLOCK) < (int64_t(1) << 31))
    return launch_early(quantize_row_vectors_kernel<X>, ceil_div(a.T * groups, PER_BLOCK), kThreads, 0, stream, a,
                        a.T * groups);
  if (vectors && a.rows == 128)
    return launch_early(quantize_tile_vectors_kernel<X>, groups * ceil_div(a.T, kScaleBlock), kThreads, 0, stream, a);
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
