// Rounding of a matrix to 8 bits with a scale for each block of 128 columns of a row,
// or of 128 rows and 128 columns (rows.cuh), and of its transpose beside it.
//
// Bound by HBM: 3 bytes for a BF16 value, 4 with the transpose.  One GB300, of the copy
// rate: 4096 x 12288 rows 24.1 us, 0.93 (four pieces of a row to a thread 25.6, 64-bit
// divisions for each 28.5); 12288 x 4096 weights with their transpose 32.5 us, 0.91, without
// 24.5; fp32 rows 16384 x 4096 54 us, 0.92, weights 8192 x 4096 with their transpose 32.5,
// 0.91.  Of 6144 x 2048 weights, 9.6 us, 0.77, the blocks are one round, in which all load
// before they store.  Rows that are not whole vectors are gathered from L1, value by value:
// 4096 x 12287 36 us, 12287 x 4095 weights with their transpose 69 (their values cut from
// whole 16-byte pieces took as many instructions: rows 41 to 47 us, weights 64 to 67).
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "tc.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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
  float f[VE];
#pragma unroll
  for (int i = 0; i < VE / 2; ++i) {
    const float2 p = split(v[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
  return top_magnitude(f);
}
// `n` of them (VE at least where rows are whole vectors) to a place in Q.
template <int VE, bool WHOLE>
__device__ __forceinline__ void put_codes(uint8_t* q, const uint32_t (&c)[VE / 4], int64_t n) {
  if (WHOLE || n >= VE) {
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[VE / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(q) = c[0];
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < n) q[i] = (uint8_t)(c[i / 4] >> (8 * (i & 3)));
  }
}
// The first `n` (> 0) values of a vector of X, zeros behind them.  WHOLE: the vector starts
// on 16 bytes and has them all; else they are read singly, which L1 makes one access
// to memory.
template <typename X, bool WHOLE>
__device__ __forceinline__ uint4 get_vector(const X* x, int64_t n) {
  if constexpr (WHOLE) return __ldcs(reinterpret_cast<const uint4*>(x));
  constexpr int VE = 16 / (int)sizeof(X);
  uint32_t r[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    if (i >= n) continue;
    if constexpr (sizeof(X) == 4) r[i & 3] = reinterpret_cast<const uint32_t*>(x)[i];
    else r[(i / 2) & 3] |= (uint32_t)reinterpret_cast<const uint16_t*>(x)[i] << (16 * (i & 1));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Copies of single vectors to shared memory, which their thread alone waits for.
__device__ __forceinline__ void copy_vector(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A scale per row and 128 columns: 16 lanes (BF16; fp32: 32)
// to such a piece, kPieces of them under way at once.
constexpr int kPieces = 2;
template <typename X, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const Quantize a, int64_t pieces, uint32_t groups,
                                                                 uint32_t rows_on, uint32_t groups_on) {
  constexpr int VE = 16 / (int)sizeof(X), LANES = kScaleBlock / VE, PER_BLOCK = kThreads / LANES;
  const int t = threadIdx.x % LANES;
  const int64_t first = (int64_t)blockIdx.x * (PER_BLOCK * kPieces) + threadIdx.x / LANES;
  start_early();
  // a thread's pieces are PER_BLOCK apart: rows_on rows and groups_on groups
  uint32_t row = (uint32_t)(first < (int64_t(1) << 32) ? (uint32_t)first / groups : first / groups);
  uint32_t g = (uint32_t)(first - (int64_t)row * groups);
  uint4 raw[kPieces];
  uint8_t* to[kPieces];
  int left[kPieces];  // values from this thread's first one to the row's end
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int64_t col = (int64_t)g * kScaleBlock + t * VE;
    left[j] = first + j * PER_BLOCK < pieces ? (int)(a.k - col < VE ? a.k - col : VE) : 0;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (left[j] > 0) raw[j] = get_vector<X, WHOLE>(static_cast<const X*>(a.X) + row * a.ld_x + col, left[j]);
    to[j] = a.Q + row * a.ld_q + col;
    row += rows_on;
    g += groups_on;
    if (g >= groups) {
      g -= groups;
      ++row;
    }
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    Pair v[VE / 2];
    vec_pairs<X>(raw[j], v);
    uint32_t top = vector_top<VE>(v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float inv;
    const float scale = code_scale(top, inv);
    if (t == 0 && left[j] > 0) a.scale[first + j * PER_BLOCK] = scale;
    uint32_t c[VE / 4];
    vector_codes<VE>(v, inv, c);
    if (left[j] > 0) put_codes<VE, WHOLE>(to[j], c, left[j]);
  }
}

// A scale per 128 rows and 128 columns: a block to each.  A thread has four rows of VE
// columns (twice, fp32 four times).  Whole vectors wait in shared memory, not in
// registers, where they leave room for five blocks on an SM (fp32 three) instead of three
// (two): 6144 x 2048 BF16 9.6 us for 10.8 (four blocks 10.4, six 10.1), fp32 8192 x 4096 32.2 for
// 40.  A thread turns its codes by 4 x 4 bytes into words of Qt's rows; those go through
// shared memory, too, word w of column c at w ^ 4 (c / 8 % 8), where a warp's words meet
// in a bank twice at most.
template <typename X>
constexpr size_t tile_smem() { return kScaleBlock * kScaleBlock * sizeof(X); }
constexpr int tile_blocks(size_t size, bool whole) { return size == 2 ? (whole ? 5 : 3) : whole ? 3 : 2; }  // per SM

template <typename X, bool WHOLE>
__global__ void __launch_bounds__(kThreads, tile_blocks(sizeof(X), WHOLE)) quantize_tiles_kernel(const Quantize a) {
  constexpr int VE = 16 / (int)sizeof(X), LANES = kScaleBlock / VE, QUADS = kThreads / LANES, STEPS = 32 / QUADS;
  __shared__ uint32_t part[kWarps];
  extern __shared__ __align__(128) uint8_t tile_mem[];  // the vectors; then Qt's words
  const int t = threadIdx.x % LANES, quad0 = threadIdx.x / LANES;
  const int64_t groups = ceil_div(a.k, kScaleBlock);
  const int64_t r0 = blockIdx.x / groups * kScaleBlock, c0 = blockIdx.x % groups * kScaleBlock;
  const int64_t left = a.k - c0 - t * VE;  // columns from this thread's first one on
  const bool has = left > 0;
  const uint32_t mine = tc::smem_u32(tile_mem) + threadIdx.x * 16;  // vector v at + v * kThreads * 16
  start_early();
  uint4 raw[WHOLE ? 1 : STEPS * 4];
  const X* x = static_cast<const X*>(a.X) + (r0 + quad0 * 4) * a.ld_x + c0 + t * VE;
#pragma unroll
  for (int v = 0; v < STEPS * 4; ++v) {
    const int at = v / 4 * QUADS * 4 + v % 4;  // rows from quad0's first one on
    const bool in = has && r0 + quad0 * 4 + at < a.T;
    if constexpr (WHOLE) {
      if (in) copy_vector(mine + v * (kThreads * 16), x + at * a.ld_x);
      else tc::sts128(mine + v * (kThreads * 16), make_uint4(0, 0, 0, 0));
    } else {
      raw[v] = make_uint4(0, 0, 0, 0);
      if (in) raw[v] = get_vector<X, false>(x + at * a.ld_x, left);
    }
  }
  if constexpr (WHOLE) copies_landed();
  auto vector = [&](int v) {
    if constexpr (WHOLE) return tc::lds128(mine + v * (kThreads * 16));
    else return raw[v];
  };
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < STEPS * 4; ++v) {
    Pair p[VE / 2];
    vec_pairs<X>(vector(v), p);
    top = max(top, vector_top<VE>(p));
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu, part[threadIdx.x & (kWarps - 1)]);
  float inv;
  const float scale = code_scale(top, inv);
  if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
  uint32_t c[STEPS * 4][VE / 4];
#pragma unroll
  for (int v = 0; v < STEPS * 4; ++v) {
    Pair p[VE / 2];
    vec_pairs<X>(vector(v), p);
    vector_codes<VE>(p, inv, c[v]);
    const int64_t row = r0 + quad0 * 4 + v / 4 * QUADS * 4 + v % 4;
    if (a.Q && has && row < a.T) put_codes<VE, WHOLE>(a.Q + row * a.ld_q + c0 + t * VE, c[v], left);
  }
  if (a.Qt == nullptr) return;
  if constexpr (WHOLE) __syncthreads();  // every thread has read its vectors
  uint32_t(*tile)[32] = reinterpret_cast<uint32_t(*)[32]>(tile_mem);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int quad = s * QUADS + quad0;
#pragma unroll
    for (int h = 0; h < VE / 4; ++h) {
      const uint32_t c0h = c[4 * s][h], c1h = c[4 * s + 1][h], c2h = c[4 * s + 2][h], c3h = c[4 * s + 3][h];
      const uint32_t ab_lo = __byte_perm(c0h, c1h, 0x5140), ab_hi = __byte_perm(c0h, c1h, 0x7362);
      const uint32_t cd_lo = __byte_perm(c2h, c3h, 0x5140), cd_hi = __byte_perm(c2h, c3h, 0x7362);
      const uint32_t w[4] = {__byte_perm(ab_lo, cd_lo, 0x5410), __byte_perm(ab_lo, cd_lo, 0x7632),
                             __byte_perm(ab_hi, cd_hi, 0x5410), __byte_perm(ab_hi, cd_hi, 0x7632)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = t * VE + 4 * h + i;
        tile[col][quad ^ (4 * ((col >> 3) & 7))] = w[i];
      }
    }
  }
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
  const int64_t blocks = a.rows == 1 ? ceil_div(a.T * groups, PER_BLOCK) : groups * ceil_div(a.T, kScaleBlock);
  const bool whole = whole_vectors(a.X, a.ld_x, a.k, VE, sizeof(X));
  if (a.rows == 1) {
    constexpr int64_t kOn = PER_BLOCK / kPieces;
    return launch_early(whole ? quantize_rows_kernel<X, true> : quantize_rows_kernel<X, false>, blocks, kThreads, 0, stream,
                        a, a.T * groups, (uint32_t)groups, (uint32_t)(kOn / groups), (uint32_t)(kOn % groups));
  }
  auto kernel = whole ? quantize_tiles_kernel<X, true> : quantize_tiles_kernel<X, false>;
  const cudaError_t err = allow_smem(kernel, tile_smem<X>());
  return err == cudaSuccess ? launch_early(kernel, blocks, kThreads, tile_smem<X>(), stream, a) : err;
}

}  // namespace

cudaError_t launch_quantize(const Quantize& a, cudaStream_t stream) {
  return a.x_type == SKETCH_BF16 ? quantize<__nv_bfloat16>(a, stream) : quantize<float>(a, stream);
}

}  // namespace rgs
