// Layer norm over the rows of T x k activations, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   y = xh gamma + beta
//   dxh = dy gamma,  dx = rstd (dxh - mean(dxh) - xh mean(dxh xh))
//   dgamma (+)= sum over tokens of dy xh,  dbeta (+)= sum over tokens of dy
//
// Activations are BF16 or fp32, weights BF16 or fp32; statistics, sums and the
// weights' gradients are fp32.
//
// xh is formed as the formula has it, the difference first: x - mu is exact where
// the two are close, while x rstd - mu rstd would be off by 2^-24 |mu| rstd, which a
// row of little variance far from zero shows (a constant row has xh = 0).
//
// Both passes are bound by HBM, once the instructions for each element are few:
// arithmetic goes two values at a time (packed fp32 pairs).
//
// Forward: a row belongs to `tpr` threads (a power of two, 8 to 1024), each with
// up to 128 bytes of it in registers, so that a row is read once; gamma and beta
// lie in shared memory as fp32, laid out so that a warp's reads of them have no
// bank conflicts.  Blocks walk over the rows.  32768 x 4096 BF16: 90 us, 0.88 of the
// copy rate over the 4 bytes an element that have to move.
//
// Backward: a thread's columns stay the same over the rows that its block walks,
// so that dgamma and dbeta add up in registers; with those and gamma there, rows
// come through shared memory: bulk copies bring them into a ring of slots, several
// sets of rows ahead (HBM wants some 60 KB per SM under way), and threads read them
// there, once for each of the two passes over a row.  B rows are worked on side by
// side, so that their sums' shuffles overlap, and one block barrier a set both
// joins the warps' sums and tells that the slot of the set before can be filled
// again.  32768 x 4096 BF16: 139 us, 0.85 of the copy rate over 6 bytes an element.
//
// Elements come in vectors of 16 bytes (VE of them).  Rows that do not start on 16
// bytes or end inside a vector: both passes take the vectors between a row's first
// and last boundary, and the elements beside those one by one, as long as all
// matrices' rows start on the same place between two boundaries (16384 x 4095 BF16:
// 57 us forward, 0.70 of the copy rate, and 97 us backward, 0.61; single elements all
// along take 148 and 136).  The place comes again after at most 8 rows, and the
// backward pass gives a block rows that far apart, so that its threads' columns stay
// the same.  Its copies start and end at the boundaries around a row (the bytes beyond
// belong to the neighbouring rows; a row at an end of the matrix, which has none, is
// brought in exactly).  Where the matrices' rows start on different places, elements
// are read one by one (backward: VE = 1, from shared memory).
//
// Backward: each block leaves one partial row of dgamma and dbeta, and
// norm_grad_sum_kernel adds those.  Rows wider than 16384 take the kernels at the
// end, which read a row again for each pass.  Every sum has a fixed order, so
// results repeat bit for bit.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace rgs {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPartials = 320;  // partial rows of the weights' gradients
constexpr int kMaxSlots = 8;

// Two BF16 values of a word.
__device__ __forceinline__ Pair pair_bf16(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

// The pairs of a 16-byte vector, and a vector from pairs.
template <typename X>
__device__ __forceinline__ void vec_pairs(const uint4& v, Pair (&p)[8 / sizeof(X)]) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < (int)(8 / sizeof(X)); ++i)
    p[i] = sizeof(X) == 2 ? pair_bf16(r[i & 3])
                          : pair(__uint_as_float(r[(2 * i) & 3]), __uint_as_float(r[(2 * i + 1) & 3]));
}
template <typename X, int N>
__device__ __forceinline__ void store_vec(X* row, int idx, const Pair (&p)[N]) {
  static_assert(N * 2 * sizeof(X) == 16);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = split(p[i]);
    if constexpr (sizeof(X) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      r[2 * i] = __float_as_uint(f.x);
      r[2 * i + 1] = __float_as_uint(f.y);
    }
  }
  reinterpret_cast<uint4*>(row)[idx] = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// One element in shared memory.
template <typename X>
__device__ __forceinline__ float read_one(uint32_t at) {
  if constexpr (sizeof(X) == 4) return tc::lds_f32(at);
  uint16_t h;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
  return bf16_bits_to_float(h);
}
__device__ __forceinline__ float weight(const void* w, int type, int64_t i, float none) {
  if (w == nullptr) return none;
  return type == SKETCH_FP32 ? static_cast<const float*>(w)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(w)[i]);
}
// Sums of N values over the lanes that share a row: a whole warp (WARP) or `tpr`
// lanes of it.  The values' shuffles go side by side.
template <bool WARP, int N>
__device__ __forceinline__ void lane_sums(float (&v)[N], int tpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (WARP || o < tpr) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    }
  }
}
template <bool WARP>
__device__ __forceinline__ float lane_sum(float v, int tpr) {
  float a[1] = {v};
  lane_sums<WARP, 1>(a, tpr);
  return a[0];
}
// Sums of the values of the `warps` warps (2 to 32, a power of two) of a row, held
// by as many neighbouring lanes.
template <int N>
__device__ __forceinline__ void join_sums(float (&v)[N], int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o < warps) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    }
  }
}

// ---- the ring of row sets -----------------------------------------------------------
// One of the matrices that a set's rows come from.
struct RowSource {
  const char* base;
  int64_t ld;         // bytes between rows
  int64_t T;
  uint32_t width;     // bytes of a row
  __device__ const char* end() const { return base + (T - 1) * ld + width; }
};

struct Ring {
  uint32_t smem;      // shared address of the first slot
  uint32_t slot;      // bytes per slot
  uint32_t pitch;     // bytes per row
  int slots;
  int rows;           // rows per set
  int each;           // of them, rows per group of tpr threads
  int classes;        // SHIFT: rows this far apart start on the same place between two 16-byte boundaries
};

// Where row `row` starts inside its place in the slot: its own 16-byte phase.
__device__ __forceinline__ uint32_t phase(const RowSource& m, int64_t row) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(m.base) + (uint64_t)(row * m.ld)) & 15u;
}

// A warp: start the copies of one set of rows into slot `s`, N matrices one after
// another, completing on `bar`.  EDGES: rows that do not start and end on 16 bytes;
// SHIFT: all of them on the same place between two boundaries.
template <bool EDGES, bool SHIFT, int N>
__device__ __forceinline__ void fill_slot(const Ring& r, const RowSource (&m)[N], int s, int64_t first, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  const uint32_t dst0 = r.smem + (uint32_t)s * r.slot;
  const int rows = (int)(m[0].T - first < r.rows ? m[0].T - first : r.rows);
  if constexpr (!EDGES) {
    if (lane == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)(N * rows) * m[0].width);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const char* src = m[i].base + first * m[i].ld;
      const uint32_t dst = dst0 + (uint32_t)(i * r.rows) * r.pitch;
      if (m[i].ld == m[i].width) {  // rows back to back: one copy
        if (lane == 0) tc::bulk_load_1d(dst, src, (uint32_t)rows * m[i].width, bar);
      } else {
        for (int q = lane; q < rows; q += 32)
          tc::bulk_load_1d(dst + (uint32_t)q * r.pitch, src + q * m[i].ld, m[i].width, bar);
      }
    }
  } else if (SHIFT && first > 0 && first + r.rows < m[0].T) {  // no row at an end of the matrix
    const uint32_t ph = phase(m[0], 0), bytes = (ph + m[0].width + 15u) & ~15u;
    if (lane == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)(N * rows) * bytes);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i)
      for (int q = lane; q < rows; q += 32)
        tc::bulk_load_1d(dst0 + (uint32_t)(i * r.rows + q) * r.pitch, m[i].base + (first + q) * m[i].ld - ph, bytes, bar);
  } else {
    // twice over the rows: their bytes (and the single elements), then the copies
    uint32_t sum = 0;
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        for (int q = lane; q < rows; q += 32) {
          const uint32_t ph = phase(m[i], first + q);
          const char* src = m[i].base + (first + q) * m[i].ld - ph;
          uint32_t at = dst0 + (uint32_t)(i * r.rows + q) * r.pitch;
          uint32_t bytes = (ph + m[i].width + 15u) & ~15u;
          if (src < m[i].base || src + bytes > m[i].end()) {  // whole 16 bytes inside the row, the rest singly
            const uint32_t lo = (ph + 15u) & ~15u, hi = (ph + m[i].width) & ~15u;
            if (turn == 0) {
              const uint32_t end = ph + m[i].width;
              for (uint32_t b = ph; b < end && b < lo; b += 2) tc::sts16(at + b, *reinterpret_cast<const uint16_t*>(src + b));
              for (uint32_t b = hi > lo ? hi : lo; b < end; b += 2)
                tc::sts16(at + b, *reinterpret_cast<const uint16_t*>(src + b));
              tc::fence_proxy_async_smem();  // a later set's copy writes over them
            }
            src += lo;
            at += lo;
            bytes = hi > lo ? hi - lo : 0u;
          }
          if (turn == 0) sum += bytes;
          else if (bytes) tc::bulk_load_1d(at, src, bytes, bar);
        }
      }
      if (turn == 0) {
        sum = __reduce_add_sync(0xFFFFFFFFu, sum);
        __syncwarp();  // the single elements are written before the slot's barrier can complete
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, sum);
        __syncwarp();
      }
    }
  }
}

// If a copy never landed: wait, with a limit, for those still under way.
__device__ __forceinline__ void drain(uint64_t* full, int slots, int filled) {
  volatile int none = 0;
  for (int i = filled > slots ? filled - slots : 0; i < filled; ++i)
    tc::mbar_wait(&full[i % slots], (i / slots) & 1, &none, nullptr, 0, 100000000ull);
}

// ---- forward ---------------------------------------------------------------------
// Bytes of a row per thread, and blocks per SM: two, with three the threads have 80
// registers and spill (32768 x 4096 BF16: 96 against 91 us); threads that read
// single elements hold less and do better with three (16384 x 4095 BF16: 148 against
// 187 us).
constexpr int forward_bytes(int threads) { return threads == 256 ? 128 : 64; }
constexpr int forward_blocks(int threads) { return threads == 256 ? 2 : 1; }
constexpr int kSingles = 32;  // elements per thread
constexpr int single_blocks(int threads) { return threads == 256 ? 3 : 1; }

// Where column c of a weight lies in shared memory: for eight-element vectors
// the first and the second four columns of each go to halves of their own, so that
// a thread's two 16-byte reads are 16 bytes from its neighbour's.
template <int VE>
__device__ __forceinline__ int weight_at(int c, int k) {
  return VE == 8 ? (c >> 3) * 4 + (c & 3) + ((c & 4) ? k / 2 : 0) : c;
}
// The pairs of the weights of vector idx.
template <int VE>
__device__ __forceinline__ void weight_pairs(uint32_t base, int idx, int k, Pair (&p)[VE / 2]) {
#pragma unroll
  for (int h = 0; h < VE / 4; ++h) {
    const uint4 v = tc::lds128(base + 16u * idx + (h ? 2u * k : 0u));
    p[2 * h] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    p[2 * h + 1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
}

__device__ __forceinline__ float2 lds_f32x2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// Statistics of the row whose elements this thread's share sums to `sum` and,
// around a mean, to dev(mean): first the warp's mean over its `n` elements and
// squared deviations from it, then the row's from its warps', n (mean_w - mean)^2
// more each (no difference of squares, so that a row far from zero loses nothing).
// Means are quotients, not products with a rounded 1 / n: where the sum is exact, as
// for a row of equal integers, so is the mean if it can be.  `part` alternates
// between rows: a thread that writes it again has passed the barrier of the row
// between, after which nobody reads the old values.
template <bool WARP, typename Dev, typename Count>
__device__ __forceinline__ void row_moments(float sum, Dev dev, int tpr, float n_warp, float k, Count counts,
                                            float2* part, float& mu, float& m2) {
  mu = lane_sum<WARP>(sum, tpr) / (n_warp > 0.f ? n_warp : 1.f);
  m2 = lane_sum<WARP>(dev(mu), tpr);
  const int warps = tpr >> 5;
  if (WARP && warps > 1) {
    const int lane = threadIdx.x & 31, warp0 = (threadIdx.x & ~(tpr - 1)) >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = make_float2(mu, m2);
    if (tpr == (int)blockDim.x) __syncthreads();
    else tc::named_barrier(1 + warp0 / warps, tpr);
    const int w = warp0 + (lane & (warps - 1));  // every `warps` lanes join the row's warps
    const float2 v = part[w];
    const float n = counts(w);
    float j[1] = {n * v.x};
    join_sums(j, warps);
    mu = j[0] / k;
    j[0] = fmaf(n * (v.x - mu), v.x - mu, v.y);
    join_sums(j, warps);
    m2 = j[0];
  }
}

// Rows of whole 16-byte vectors.  FULL: every thread has NV of them.  WARP: a row has a
// warp at least.
template <typename X, int THREADS, bool FULL, bool WARP>
__global__ void __launch_bounds__(THREADS, forward_blocks(THREADS)) norm_forward_kernel(const NormForward a, int tpr) {
  constexpr int VE = 16 / (int)sizeof(X), NV = forward_bytes(THREADS) / 16;
  extern __shared__ __align__(128) float weights[];
  __shared__ float2 part[2][THREADS / 32];
  __shared__ float counts[THREADS / 32];
  const int t = threadIdx.x & (tpr - 1), groups = THREADS / tpr, k = (int)a.k;
  const int nvec = k / VE;
  for (int c = threadIdx.x; c < k; c += THREADS) {
    weights[weight_at<VE>(c, k)] = weight(a.gamma, a.w_type, c, 1.f);
    weights[k + weight_at<VE>(c, k)] = weight(a.beta, a.w_type, c, 0.f);
  }
  const uint32_t gamma = tc::smem_u32(weights), beta = gamma + 4u * k;
  // elements of the row that this warp holds (the whole row's, where it is one of several in the warp)
  int mine = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) mine += j * tpr + t < nvec ? VE : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  const float inv_k = 1.f / (float)k;
  if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = (float)mine;
  __syncthreads();
  const int64_t stride = (int64_t)gridDim.x * groups;
  int p = 0;
  for (int64_t base = (int64_t)blockIdx.x * groups; base < a.T; base += stride, p ^= 1) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < a.T;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const X*>(a.X) + row * a.ld_x);
    uint4 raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (in && (FULL || j * tpr + t < nvec)) raw[j] = __ldcs(x + j * tpr + t);
    }
    Pair s = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pair v[VE / 2];
      vec_pairs<X>(raw[j], v);
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) s = add2(s, v[i]);
    }
    float mu, m2;
    row_moments<WARP>(
        sum2(s),
        [&](float m) {
          const Pair neg = pair(-m, -m);
          Pair q = 0;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (FULL || j * tpr + t < nvec) {
              Pair v[VE / 2];
              vec_pairs<X>(raw[j], v);
#pragma unroll
              for (int i = 0; i < VE / 2; ++i) {
                v[i] = add2(v[i], neg);
                q = fma2(v[i], v[i], q);
              }
            }
          }
          return sum2(q);
        },
        tpr, (float)mine, (float)k, [&](int w) { return counts[w]; }, part[p], mu, m2);
    const float rstd = 1.f / sqrtf(m2 * inv_k + a.eps);
    if (!in) continue;
    const Pair r2 = pair(rstd, rstd), neg = pair(-mu, -mu);
    X* y = static_cast<X*>(a.Y) + row * a.ld_y;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (FULL || j * tpr + t < nvec) {
        Pair v[VE / 2], g[VE / 2], b[VE / 2];
        vec_pairs<X>(raw[j], v);
        weight_pairs<VE>(gamma, j * tpr + t, k, g);
        weight_pairs<VE>(beta, j * tpr + t, k, b);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) v[i] = fma2(mul2(add2(v[i], neg), r2), g[i], b[i]);
        store_vec<X>(y, j * tpr + t, v);
      }
    }
    if (t == 0) {
      a.mean[row] = mu;
      a.rstd[row] = rstd;
    }
  }
}

// Rows of X and Y that start on the same, any, place between two 16-byte
// boundaries: the vectors between a row's first and last boundary, and the elements
// before and behind those, one to a thread.  gamma and beta lie side by side, column
// c at [c % VE][c / VE]: whichever column the vectors start at, a warp reads 32
// neighbours.
template <typename X, int THREADS, bool WARP>
__global__ void __launch_bounds__(THREADS, forward_blocks(THREADS)) norm_forward_shifted_kernel(const NormForward a, int tpr) {
  constexpr int VE = 16 / (int)sizeof(X), NV = forward_bytes(THREADS) / 16;
  extern __shared__ __align__(128) float weights[];
  __shared__ float2 part[2][THREADS / 32];
  const int t = threadIdx.x & (tpr - 1), groups = THREADS / tpr, k = (int)a.k;
  const int pitch = k / VE + 1;
  float2* gb = reinterpret_cast<float2*>(weights);
  for (int c = threadIdx.x; c < k; c += THREADS)
    gb[(c & (VE - 1)) * pitch + c / VE] = make_float2(weight(a.gamma, a.w_type, c, 1.f), weight(a.beta, a.w_type, c, 0.f));
  __syncthreads();
  const uint32_t gb0 = tc::smem_u32(weights) + 8u * t;
  const float inv_k = 1.f / (float)k;
  const int64_t stride = (int64_t)gridDim.x * groups;
  const int log_tpr = 31 - __clz(tpr);
  int p = 0;
  for (int64_t base = (int64_t)blockIdx.x * groups; base < a.T; base += stride, p ^= 1) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < a.T;
    const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
    const int ahead = (int)(-(reinterpret_cast<uintptr_t>(x) / sizeof(X)) & (VE - 1));  // elements before the first vector
    const int lead = ahead < k ? ahead : k, nvec = (k - lead) / VE, behind = k - lead - nvec * VE;
    // this thread's single element: one of the first `lead`, or of the last
    const int one = t < lead ? t : t - VE;
    const bool has_one = t < lead || (t >= VE && t < VE + behind);
    const int col = t < lead ? one : lead + nvec * VE + one;
    const bool take = in && has_one;
    X single = X(0.f);
    if (take) single = __ldcs(x + col);
    uint4 raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (in && j * tpr + t < nvec) raw[j] = __ldcs(reinterpret_cast<const uint4*>(x + lead) + j * tpr + t);
    }
    Pair s = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pair v[VE / 2];
      vec_pairs<X>(raw[j], v);
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) s = add2(s, v[i]);
    }
    const float e = (float)single;
    // elements of the row's warp `w` of the block
    auto count = [&](int w) {
      const int t0 = (w * 32) & (tpr - 1), whole = nvec >> log_tpr;
      const int rest = min(max(nvec - (whole << log_tpr) - t0, 0), 32);
      return (float)((whole * 32 + rest) * VE + (t0 == 0 ? lead + behind : 0));
    };
    const float n = WARP ? count(threadIdx.x >> 5) : (float)k;
    float mu, m2;
    row_moments<WARP>(
        sum2(s) + e,
        [&](float m) {
          const Pair neg = pair(-m, -m);
          Pair q = 0;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (j * tpr + t < nvec) {
              Pair v[VE / 2];
              vec_pairs<X>(raw[j], v);
#pragma unroll
              for (int i = 0; i < VE / 2; ++i) {
                v[i] = add2(v[i], neg);
                q = fma2(v[i], v[i], q);
              }
            }
          }
          return has_one ? fmaf(e - m, e - m, sum2(q)) : sum2(q);
        },
        tpr, n, (float)k, count, part[p], mu, m2);
    const float rstd = 1.f / sqrtf(m2 * inv_k + a.eps);
    if (!in) continue;
    const Pair r2 = pair(rstd, rstd), neg = pair(-mu, -mu);
    X* y = static_cast<X*>(a.Y) + row * a.ld_y;
    uint32_t at[VE];  // of the weights of the thread's first vector
#pragma unroll
    for (int i = 0; i < VE; ++i) at[i] = gb0 + 8u * (uint32_t)(((lead + i) & (VE - 1)) * pitch + ((lead + i) / VE));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j * tpr + t < nvec) {
        Pair v[VE / 2];
        vec_pairs<X>(raw[j], v);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
          const float2 f = split(mul2(add2(v[i], neg), r2));
          const float2 w0 = lds_f32x2(at[2 * i] + 8u * (uint32_t)(j * tpr)), w1 = lds_f32x2(at[2 * i + 1] + 8u * (uint32_t)(j * tpr));
          v[i] = pair(fmaf(f.x, w0.x, w0.y), fmaf(f.y, w1.x, w1.y));
        }
        store_vec<X>(y + lead, j * tpr + t, v);
      }
    }
    if (take) {
      const float2 w = gb[(col & (VE - 1)) * pitch + col / VE];
      store_one(y + col, fmaf((e - mu) * rstd, w.x, w.y));
    }
    if (t == 0) {
      a.mean[row] = mu;
      a.rstd[row] = rstd;
    }
  }
}

// Rows of X and of Y that start on different places: elements one by one, NV of them
// per thread.
template <typename X, int NV, int THREADS, bool WARP>
__global__ void __launch_bounds__(THREADS, single_blocks(THREADS)) norm_forward_single_kernel(const NormForward a, int tpr) {
  extern __shared__ __align__(128) float weights[];
  __shared__ float2 part[2][THREADS / 32];
  __shared__ float counts[THREADS / 32];
  const int t = threadIdx.x & (tpr - 1), groups = THREADS / tpr, k = (int)a.k;
  for (int c = threadIdx.x; c < k; c += THREADS) {
    weights[c] = weight(a.gamma, a.w_type, c, 1.f);
    weights[k + c] = weight(a.beta, a.w_type, c, 0.f);
  }
  int mine = (k - t + tpr - 1) / tpr;  // this thread's elements: columns t, t + tpr, ...
  if (mine < 0) mine = 0;
  int warp_n = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) warp_n += __shfl_xor_sync(0xFFFFFFFFu, warp_n, o);
  const float inv_k = 1.f / (float)k;
  if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = (float)warp_n;
  __syncthreads();
  const int64_t stride = (int64_t)gridDim.x * groups;
  int p = 0;
  for (int64_t base = (int64_t)blockIdx.x * groups; base < a.T; base += stride, p ^= 1) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < a.T;
    const X* x = static_cast<const X*>(a.X) + row * a.ld_x + t;
    float f[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) f[j] = (in && j < mine) ? (float)__ldcs(x + j * tpr) : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) sum += f[j];
    float mu, m2;
    row_moments<WARP>(
        sum,
        [&](float m) {
          float q = 0.f;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (j < mine) q = fmaf(f[j] - m, f[j] - m, q);
          return q;
        },
        tpr, (float)warp_n, (float)k, [&](int w) { return counts[w]; }, part[p], mu, m2);
    const float rstd = 1.f / sqrtf(m2 * inv_k + a.eps);
    if (!in) continue;
    X* y = static_cast<X*>(a.Y) + row * a.ld_y + t;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j < mine) store_one(y + j * tpr, fmaf((f[j] - mu) * rstd, weights[j * tpr + t], weights[k + j * tpr + t]));
    if (t == 0) {
      a.mean[row] = mu;
      a.rstd[row] = rstd;
    }
  }
}

// ---- backward --------------------------------------------------------------------
constexpr int blocks_per_sm(int threads) { return threads == 256 ? 2 : 1; }
constexpr int backward_rows_each(size_t size, int threads) { return threads == 256 && size == 2 ? 2 : 1; }

// A thread's columns: NV vectors of VE elements, as E / 2 pairs.  With VE = 1 a pair
// is the thread's elements 2 q and 2 q + 1, tpr columns apart.  SHIFT: the vectors
// between a row's first and last 16-byte boundary, and one of the elements beside
// those; a block keeps to rows that start on the same place, `classes` apart.
template <typename X, int VE, int NV, int THREADS, bool FULL, bool WARP, bool SHIFT = false>
__global__ void __launch_bounds__(THREADS, blocks_per_sm(THREADS))
    norm_backward_kernel(const NormBackward a, const Ring ring, int tpr, int* err) {
  constexpr int E = NV * VE, B = backward_rows_each(sizeof(X), THREADS);
  constexpr int VP = VE == 1 ? 1 : VE / 2, NP = E / 2 / VP;  // pairs per step, steps
  constexpr bool HOLD = E <= 16;  // gamma stays in registers
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ __align__(8) uint64_t full[kMaxSlots];
  __shared__ float2 part[2][B][THREADS / 32];
  __shared__ volatile int abort_flag;
  Ring r = ring;
  r.smem = tc::smem_u32(ring_mem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // SHIFT: the block's class of rows as matrices of their own
  const int classes = SHIFT ? r.classes : 1, cls = SHIFT ? (int)blockIdx.x % classes : 0;
  const int64_t block = SHIFT ? blockIdx.x / classes : blockIdx.x, blocks = SHIFT ? gridDim.x / classes : gridDim.x;
  const int64_t rows_in = SHIFT ? (a.T - cls + classes - 1) / classes : a.T;
  auto source = [&](const void* p, int64_t ld) {
    ld *= (int64_t)sizeof(X);
    return RowSource{static_cast<const char*>(p) + cls * ld, ld * classes, rows_in, (uint32_t)(a.k * sizeof(X))};
  };
  const RowSource m[2] = {source(a.X, a.ld_x), source(a.dY, a.ld_dy)};
  const float *mean = a.mean + cls, *row_rstd = a.rstd + cls;
  const int64_t stride = blocks * r.rows;
  const int64_t first = block * r.rows;
  const int passes = first < rows_in ? (int)((rows_in - first + stride - 1) / stride) : 0;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < r.slots; ++s) tc::mbar_init(&full[s], 1);
    tc::fence_mbar_init();
  }
  cudaTriggerProgrammaticLaunchCompletion();  // norm_grad_sum_kernel may come up as blocks leave
  __syncthreads();
  int filled = 0;  // warp 0's: sets whose copies have begun
  if (warp == 0)
    for (; filled < passes && filled < r.slots; ++filled) fill_slot<VE == 1 || SHIFT, SHIFT, 2>(r, m, filled, first + filled * stride, &full[filled]);
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = THREADS / tpr, k = (int)a.k;
  const int warps = tpr >> 5, warp0 = (threadIdx.x & ~(tpr - 1)) >> 5;
  // SHIFT: elements before the first vector; the place of a row's first element, of its first vector
  const uint32_t place = SHIFT ? phase(m[0], 0) : 0u, vec_place = (place + 15u) & ~15u;
  const int lead = SHIFT ? min((int)((vec_place - place) / sizeof(X)), k) : 0;
  const int nvec = (k - lead) / VE, end = SHIFT ? lead + nvec * VE : k;
  // this thread's element beside the vectors: one of the first `lead`, or of those
  // behind; the row's last threads have them, the first warp having the copies
  const int u = t - (tpr - 2 * VE);
  const bool has_one = SHIFT && u >= 0 && (u < lead || (u >= VE && u < VE + k - end));
  const int one = u < lead ? u : end + u - VE;
  // column of element i of pair q of step j; whether the thread has it
  auto column = [&](int j, int q, int i) { return VE == 1 ? (2 * j + i) * tpr + t : lead + (j * tpr + t) * VE + 2 * q + i; };
  auto has = [&](int j) { return FULL || (VE == 1 ? 2 * j * tpr + t < k : j * tpr + t < nvec); };
  // VE = 1: the pair's second element may lie past the row; a zero stands for it
  auto read = [&](uint32_t at, int j, Pair (&v)[VP]) {
    if constexpr (VE == 1) {
      const int c = 2 * j * tpr + t;
      const uint32_t p = r.smem + at + (uint32_t)(c * sizeof(X));
      v[0] = pair(read_one<X>(p), c + tpr < k ? read_one<X>(p + (uint32_t)(tpr * sizeof(X))) : 0.f);
    } else {
      // `at` is the thread's first vector; plain loads, which the compiler may move
      // ahead, where registers allow it
      const uint32_t p = at + (uint32_t)j * (16u * tpr);
      if constexpr (FULL && HOLD) vec_pairs<X>(*reinterpret_cast<const uint4*>(ring_mem + p), v);
      else vec_pairs<X>(tc::lds128(r.smem + p), v);
    }
  };
  Pair dg[E / 2], db[E / 2], gamma[HOLD ? E / 2 : 1];
  float dg_one = 0.f, db_one = 0.f;
  // wide rows: gamma behind the ring, as the forward pass lays it out
  float* gmem = reinterpret_cast<float*>(ring_mem + (size_t)r.slots * r.slot);
  {
    auto gamma_pairs = [&](int j, Pair (&g)[VP]) {
      if constexpr (VE == 1) {
        const int c = 2 * j * tpr + t;
        g[0] = pair(gmem[c], c + tpr < k ? gmem[c + tpr] : 0.f);
      } else {
        weight_pairs<VE>(tc::smem_u32(gmem), j * tpr + t, end - lead, g);
      }
    };
    if constexpr (!HOLD) {
      for (int c = lead + threadIdx.x; c < end; c += THREADS)
        gmem[weight_at<VE>(c - lead, end - lead)] = weight(a.gamma, a.w_type, c, 1.f);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
#pragma unroll
      for (int q = 0; q < VP; ++q) {
        const int c0 = column(j, q, 0), c1 = column(j, q, 1);
        if constexpr (HOLD)
          gamma[j * VP + q] = pair(FULL || c0 < end ? weight(a.gamma, a.w_type, c0, 1.f) : 0.f,
                                   FULL || c1 < end ? weight(a.gamma, a.w_type, c1, 1.f) : 0.f);
        dg[j * VP + q] = db[j * VP + q] = 0;
      }
    }
    const float gamma_one = has_one ? weight(a.gamma, a.w_type, one, 1.f) : 0.f;
    const float inv_k = 1.f / (float)k;
    // rows, row strides (below 2^31) and their products in 32 x 32 -> 64 bits
    const uint32_t T = (uint32_t)rows_in, step = (uint32_t)stride;
    using Stride = std::conditional_t<SHIFT, uint64_t, uint32_t>;
    const Stride ld_dx = (Stride)((a.ld_dx * sizeof(X) >> 1) * classes);
    auto row_dx = [&](uint32_t i) {
      char* p = static_cast<char*>(a.dX) + 2 * ((uint64_t)i * ld_dx);
      return reinterpret_cast<X*>(SHIFT ? p + cls * a.ld_dx * (int64_t)sizeof(X) : p);
    };
    uint32_t row = (uint32_t)first + group * r.each;
    float nmu[B], nrs[B];  // the next set's
    auto load_stats = [&](uint32_t at) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        nmu[b] = nrs[b] = 0.f;
        if (b < r.each && at + b < T) {
          nmu[b] = mean[(at + b) * classes];
          nrs[b] = row_rstd[(at + b) * classes];
        }
      }
    };
    load_stats(row);
    const uint32_t vec0 = 16u * t + vec_place;
    const uint32_t one_at = r.smem + place + (uint32_t)(one * (int)sizeof(X)) - vec0;  // from the thread's first vector
    const uint32_t set_at = (uint32_t)(group * r.each) * r.pitch, y_at = (uint32_t)r.rows * r.pitch;
    uint32_t slot = set_at;  // in the ring
    int s = 0;
    uint32_t ph = 0;
    for (int p = 0; p < passes; ++p, row += step) {
      Pair rs[B], neg[B], s0[B], s1[B];
      float rstd[B], mu[B];
      uint32_t ax[B], ay[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        rstd[b] = nrs[b];
        mu[b] = nmu[b];
        rs[b] = pair(nrs[b], nrs[b]);
        neg[b] = pair(-nmu[b], -nmu[b]);
      }
      if (p + 1 < passes) load_stats(row + step);
      tc::mbar_wait(&full[s], ph, &abort_flag, err, tc::kErrTimeoutLoad);
      // what lies past the last row is worked on like a row (in shared memory that
      // a row before left) and not kept
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t q = b < r.each ? b : 0;
        ax[b] = slot + q * r.pitch;
        ay[b] = ax[b] + y_at;
        if constexpr (VE == 1) {
          ax[b] += phase(m[0], row + q);
          ay[b] += phase(m[1], row + q);
        } else {
          ax[b] += vec0;
          ay[b] += vec0;
        }
        s0[b] = s1[b] = 0;
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if (has(j)) {
          Pair g[VP];
          if constexpr (!HOLD) gamma_pairs(j, g);
#pragma unroll
          for (int b = 0; b < B; ++b) {
            Pair x[VP], y[VP];
            read(ax[b], j, x);
            read(ay[b], j, y);
#pragma unroll
            for (int q = 0; q < VP; ++q) {
              const Pair d = mul2(y[q], HOLD ? gamma[HOLD ? j * VP + q : 0] : g[q]);
              s0[b] = add2(s0[b], d);
              s1[b] = fma2(d, add2(x[q], neg[b]), s1[b]);  // times rstd once it is summed up
            }
          }
        }
      }
      float v[2 * B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        v[2 * b] = sum2(s0[b]);
        v[2 * b + 1] = sum2(s1[b]);
        if (SHIFT && has_one) {
          const float d = read_one<X>(ay[b] + one_at) * gamma_one;
          v[2 * b] += d;
          v[2 * b + 1] = fmaf(d, read_one<X>(ax[b] + one_at) - mu[b], v[2 * b + 1]);
        }
        v[2 * b + 1] *= rstd[b];
      }
      lane_sums<WARP, 2 * B>(v, tpr);
      float2(*q)[THREADS / 32] = part[p & 1];  // alternates, as in row_moments
      if (WARP && lane == 0) {
#pragma unroll
        for (int b = 0; b < B; ++b) q[b][warp] = make_float2(v[2 * b], v[2 * b + 1]);
      }
      __syncthreads();
      if (warp == 0 && p > 0 && filled < passes && r.slots > 1) {  // every thread is done with the set before
        const int before = s ? s - 1 : r.slots - 1;
        fill_slot<VE == 1 || SHIFT, SHIFT, 2>(r, m, before, first + filled * stride, &full[before]);
        ++filled;
      }
      if (WARP && warps > 1) {
        const int b = lane >> (31 - __clz(warps)), w = lane & (warps - 1);  // lane (row, warp) joins
        const float2 u = q[b < B ? b : 0][warp0 + w];
        float j[2] = {u.x, u.y};
        join_sums(j, warps);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          v[2 * i] = __shfl_sync(0xFFFFFFFFu, j[0], i * warps);
          v[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, j[1], i * warps);
        }
      }
      // the gradients; WHOLE: all of the block's rows of this set exist
      auto second = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (!WHOLE && (b >= r.each || row + b >= T)) continue;
          X* dx = row_dx(row + b);
          const float f0 = -v[2 * b] * inv_k * rstd[b], f1 = -v[2 * b + 1] * inv_k * rstd[b];
          const Pair c0 = pair(f0, f0), c1 = pair(f1, f1);
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            if (has(j)) {
              Pair x[VP], y[VP], g[VP];
              read(ax[b], j, x);
              read(ay[b], j, y);
              if constexpr (!HOLD) gamma_pairs(j, g);
#pragma unroll
              for (int q = 0; q < VP; ++q) {
                const int e = j * VP + q;
                x[q] = mul2(add2(x[q], neg[b]), rs[b]);
                dg[e] = fma2(y[q], x[q], dg[e]);
                db[e] = add2(db[e], y[q]);
                y[q] = fma2(mul2(y[q], HOLD ? gamma[HOLD ? e : 0] : g[q]), rs[b], fma2(x[q], c1, c0));
              }
              if constexpr (VE == 1) {
                if (a.dX) {
                  const float2 f = split(y[0]);
                  const int c = 2 * j * tpr + t;
                  store_one(dx + c, f.x);
                  if (c + tpr < k) store_one(dx + c + tpr, f.y);
                }
              } else {
                if (a.dX) store_vec<X>(dx + lead, j * tpr + t, y);
              }
            }
          }
          if (SHIFT && has_one) {
            const float x = (read_one<X>(ax[b] + one_at) - mu[b]) * rstd[b], y = read_one<X>(ay[b] + one_at);
            dg_one = fmaf(y, x, dg_one);
            db_one += y;
            if (a.dX) store_one(dx + one, fmaf(y * gamma_one, rstd[b], fmaf(x, f1, f0)));
          }
        }
      };
      if (FULL && HOLD && r.each == B && row - group * r.each + r.rows <= T) second(std::bool_constant<FULL && HOLD>{});
      else second(std::false_type{});
      if (r.slots == 1 && p + 1 < passes) {  // fp32 rows too wide for two slots
        __syncthreads();
        if (warp == 0) fill_slot<VE == 1 || SHIFT, SHIFT, 2>(r, m, 0, first + filled * stride, &full[0]);
        ++filled;
      }
      slot += r.slot;
      if (++s == r.slots) {
        s = 0;
        ph ^= 1u;
        slot = set_at;
      }
    }
  }
  if (threadIdx.x == 0 && abort_flag) drain(full, r.slots, filled);
  if (a.dgamma == nullptr && a.dbeta == nullptr) return;
  // this block's partial row: the groups' sums added in their order, in the ring's memory
  float* out = a.ws + (int64_t)blockIdx.x * 2 * k;
  float* acc = reinterpret_cast<float*>(ring_mem);
  __syncthreads();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    {
      float* to = groups > 1 ? acc + group * k : out + half * k;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
#pragma unroll
        for (int q = 0; q < VP; ++q) {
          const float2 f = split(half ? db[j * VP + q] : dg[j * VP + q]);
          const int c0 = column(j, q, 0), c1 = column(j, q, 1);
          if (FULL || c0 < end) to[c0] = f.x;
          if (FULL || c1 < end) to[c1] = f.y;
        }
      }
      if (has_one) to[one] = half ? db_one : dg_one;
    }
    if (groups > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < k; c += THREADS) {
        float v = 0.f;
        for (int g = 0; g < groups; ++g) v += acc[g * k + c];
        out[half * k + c] = v;
      }
      __syncthreads();
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

__device__ __forceinline__ float block_sum(float v, float* part) {
  v = lane_sum<true>(v, 32);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) norm_forward_wide_kernel(const NormForward a) {
  __shared__ float part[2][kThreads / 32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  X* y = static_cast<X*>(a.Y) + row * a.ld_y;
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) s += get(x, i);
  const float mu = block_sum(s, part[0]) / (float)a.k;
  s = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) s = fmaf(get(x, i) - mu, get(x, i) - mu, s);
  const float rstd = 1.f / sqrtf(block_sum(s, part[1]) / (float)a.k + a.eps);
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
  __shared__ float part[2][kThreads / 32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.X) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dY) + row * a.ld_dy;
  X* dx = static_cast<X*>(a.dX) + row * a.ld_dx;
  const float mu = a.mean[row], rs = a.rstd[row];
  float s0 = 0.f, s1 = 0.f;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * weight(a.gamma, a.w_type, i, 1.f);
    s0 += d;
    s1 = fmaf(d, (get(x, i) - mu) * rs, s1);
  }
  s0 = block_sum(s0, part[0]) / (float)a.k;
  s1 = block_sum(s1, part[1]) / (float)a.k;
  for (int64_t i = threadIdx.x; i < a.k; i += kThreads) {
    const float d = get(dy, i) * weight(a.gamma, a.w_type, i, 1.f);
    put(dx, i, rs * (d - s0 - ((get(x, i) - mu) * rs) * s1));
  }
}

constexpr int64_t kMaxRowWidth = 16384;
constexpr size_t kMostSmem = 216u << 10;  // dynamic shared memory of a launch

// Whether every row of the matrix starts on a vector of ve elements and ends with a whole one.
bool whole_vectors(const void* p, int64_t ld, int64_t k, int ve, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % (ve * size) == 0 && ld % ve == 0 && k % ve == 0;
}

// Whether each row of Y starts as far from a 16-byte boundary as the one of X.
bool same_places(const void* x, int64_t ld_x, const void* y, int64_t ld_y, size_t size) {
  return (reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(y)) % 16 == 0 && (ld_x - ld_y) * (int64_t)size % 16 == 0;
}

// Threads per row: the fewest (of at most `limit`) that hold a row at `most`
// vectors each, then more while the launch would leave SMs without a block.
int threads_per_row(int64_t nvec, int most, int64_t T, int limit) {
  int tpr = 8;
  while (tpr < limit && (int64_t)tpr * most < nvec) tpr *= 2;
  while (tpr < 256 && tpr < nvec && T * tpr < 2 * (int64_t)num_sms() * kThreads) tpr *= 2;
  return tpr;
}

// Let a kernel have `smem` bytes of dynamic shared memory, kMostSmem at most.  Static
// and dynamic parts of up to 48 KB together need no asking; the kernels' static parts
// stay below 1 KB.  The limit is the kernel's, not the launch's: it is the same for
// every size, so that another host thread's launch never finds it lowered.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t smem) {
  if (smem <= (47u << 10)) return cudaSuccess;
  if (smem > kMostSmem) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
}

template <int THREADS, typename Kernel>
cudaError_t launch_forward(Kernel kernel, const NormForward& a, int tpr, int per_sm, cudaStream_t stream) {
  const size_t smem = ((size_t)a.k + 8) * 8;  // the shifted kernel's pitch rounds up
  const cudaError_t err = allow_smem(kernel, smem);
  if (err != cudaSuccess) return err;
  int64_t blocks = ceil_div(a.T, THREADS / tpr);
  const int64_t most = (int64_t)num_sms() * per_sm;
  if (blocks > most) blocks = most;
  count_launch();
  kernel<<<(unsigned)blocks, THREADS, smem, stream>>>(a, tpr);
  return cudaGetLastError();
}

// Blocks of 256 threads, two to an SM, up to rows of 4096, else one of 1024
// (whose threads have half the registers).
template <typename X, int THREADS>
cudaError_t forward_vectors(const NormForward& a, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(X), kMost = forward_bytes(THREADS) / 16, kPerSm = forward_blocks(THREADS);
  const int tpr = threads_per_row(a.k / VE, kMost, a.T, THREADS);
  if constexpr (THREADS == 256) {
    if (tpr < 32)
      return launch_forward<THREADS>(norm_forward_kernel<X, THREADS, false, false>, a, tpr, kPerSm, stream);
  }
  if (a.k == (int64_t)VE * kMost * tpr)
    return launch_forward<THREADS>(norm_forward_kernel<X, THREADS, true, true>, a, tpr, kPerSm, stream);
  return launch_forward<THREADS>(norm_forward_kernel<X, THREADS, false, true>, a, tpr, kPerSm, stream);
}
template <typename X, int THREADS>
cudaError_t forward_shifted(const NormForward& a, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(X);
  int tpr = threads_per_row(a.k / VE, forward_bytes(THREADS) / 16, a.T, THREADS);
  if (tpr < 2 * VE) tpr = 2 * VE;  // a thread for each of the elements beside the vectors
  if constexpr (THREADS == 256) {
    if (tpr < 32)
      return launch_forward<THREADS>(norm_forward_shifted_kernel<X, THREADS, false>, a, tpr, forward_blocks(THREADS), stream);
  }
  return launch_forward<THREADS>(norm_forward_shifted_kernel<X, THREADS, true>, a, tpr, forward_blocks(THREADS), stream);
}
template <typename X>
cudaError_t forward_singles(const NormForward& a, cudaStream_t stream) {
  const int tpr = threads_per_row(a.k, kSingles, a.T, 512);
  if (tpr < 32) return launch_forward<256>(norm_forward_single_kernel<X, kSingles, 256, false>, a, tpr, single_blocks(256), stream);
  if (tpr <= 256) return launch_forward<256>(norm_forward_single_kernel<X, kSingles, 256, true>, a, tpr, single_blocks(256), stream);
  return launch_forward<512>(norm_forward_single_kernel<X, kSingles, 512, true>, a, tpr, single_blocks(512), stream);
}

// The ring for sets of rows of `matrices` matrices, with `beside` bytes of shared
// memory behind it; 0 slots where not even one fits.
Ring make_ring(int64_t k, size_t size, bool edges, int groups, int each, int matrices, int threads, size_t beside) {
  Ring r = {};
  r.rows = groups * each;
  r.each = each;
  // edges: room for 16-byte boundaries around a row
  r.pitch = !edges ? (uint32_t)(k * size) : (uint32_t)((k * size + 15) / 16 * 16 + 16);
  r.slot = r.pitch * (uint32_t)(r.rows * matrices);
  const uint32_t room = (uint32_t)(kMostSmem / blocks_per_sm(threads) - beside);
  r.slots = (int)(room / r.slot < kMaxSlots ? room / r.slot : kMaxSlots);
  return r;
}

// Rows side by side: as many as `most` while every block still has a set.
int rows_each(int most, int64_t T, int groups, int threads) {
  const int64_t sets = (int64_t)num_sms() * blocks_per_sm(threads) * groups;
  int each = 1;
  while (each < most && T >= 2 * each * sets) each *= 2;
  return each;
}

// A launch of `kernel` over row sets; `room`: shared memory that it needs at least.
template <typename Args, typename Kernel>
cudaError_t launch_rows(Kernel kernel, const Args& a, const Ring& r, int tpr, int threads, int64_t blocks, size_t room,
                        cudaStream_t stream) {
  int* err_word = nullptr;
  cudaError_t err = device_error_word(&err_word);
  if (err != cudaSuccess) return err;
  size_t smem = (size_t)r.slots * r.slot;
  if (smem < room) smem = room;
  err = allow_smem(kernel, smem);
  if (err != cudaSuccess) return err;
  count_launch();
  kernel<<<(unsigned)blocks, threads, smem, stream>>>(a, r, tpr, err_word);
  return cudaGetLastError();
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

template <typename X, int VE, int NV, int THREADS, bool SHIFT>
cudaError_t backward_rows(const NormBackward& a, int tpr, int classes, bool& done, cudaStream_t stream) {
  const int groups = THREADS / tpr;
  const int each = rows_each(backward_rows_each(sizeof(X), THREADS), a.T, groups, THREADS);
  int64_t blocks = ceil_div(a.T, groups * each);
  const int64_t most = (int64_t)num_sms() * blocks_per_sm(THREADS);
  if (blocks > most) blocks = most;
  if (blocks > kMaxPartials) blocks = kMaxPartials;
  if (SHIFT) blocks = blocks < classes ? classes : blocks / classes * classes;
  const size_t beside = VE * NV > 16 ? (size_t)a.k * 4 : 0;  // gamma
  Ring r = make_ring(a.k, sizeof(X), VE == 1 || SHIFT, groups, each, 2, THREADS, beside);
  r.classes = classes;
  if (r.slots < 1) return cudaSuccess;
  done = true;
  const size_t room = groups > 1 ? (size_t)groups * a.k * 4 : (size_t)r.slots * r.slot + beside;
  cudaError_t err = cudaSuccess;
  bool full = false;
  if constexpr (VE > 1 && !SHIFT) {
    full = a.k == (int64_t)VE * NV * tpr && tpr >= 32;
    if (full)
      err = launch_rows(norm_backward_kernel<X, VE, NV, THREADS, true, true>, a, r, tpr, THREADS, blocks, room, stream);
  }
  if constexpr (THREADS == 256) {
    if (tpr < 32) {
      full = true;
      err = launch_rows(norm_backward_kernel<X, VE, NV, THREADS, false, false, SHIFT>, a, r, tpr, THREADS, blocks, room, stream);
    }
  }
  if (!full)
    err = launch_rows(norm_backward_kernel<X, VE, NV, THREADS, false, true, SHIFT>, a, r, tpr, THREADS, blocks, room, stream);
  if (err == cudaSuccess && (a.dgamma || a.dbeta)) err = launch_grad_sum(a, (int)blocks, stream);
  return err;
}

template <typename X, int VE, bool SHIFT>
cudaError_t backward(const NormBackward& a, int classes, bool& done, cudaStream_t stream) {
  constexpr int kNV = 16 / VE;  // 16 elements of a row per thread, 32 above 8192
  int tpr = threads_per_row(a.k / VE, kNV, a.T, 512);
  if (SHIFT && tpr < 2 * VE) tpr = 2 * VE;  // a thread for each of the elements beside the vectors
  if (tpr <= 256) return backward_rows<X, VE, kNV, 256, SHIFT>(a, tpr, classes, done, stream);
  if (a.k <= 8192) return backward_rows<X, VE, kNV, 512, SHIFT>(a, 512, classes, done, stream);
  return backward_rows<X, VE, 2 * kNV, 512, SHIFT>(a, 512, classes, done, stream);
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
  constexpr int VE = 16 / (int)sizeof(X);
  if (a.k <= kMaxRowWidth) {
    if (whole_vectors(a.X, a.ld_x, a.k, VE, sizeof(X)) && whole_vectors(a.Y, a.ld_y, a.k, VE, sizeof(X)))
      return a.k <= 4096 ? forward_vectors<X, 256>(a, stream) : forward_vectors<X, 1024>(a, stream);
    if (same_places(a.X, a.ld_x, a.Y, a.ld_y, sizeof(X)))
      return a.k <= 4096 ? forward_shifted<X, 256>(a, stream) : forward_shifted<X, 1024>(a, stream);
    return forward_singles<X>(a, stream);
  }
  count_launch();
  norm_forward_wide_kernel<X><<<(unsigned)a.T, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename X>
cudaError_t backward_any(const NormBackward& a, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(X);
  bool done = false;
  cudaError_t err = cudaSuccess;
  if (a.k <= kMaxRowWidth) {
    auto vectors = [&](const void* p, int64_t ld) { return p == nullptr || whole_vectors(p, ld, a.k, VE, sizeof(X)); };
    auto same = [&](const void* p, int64_t ld) { return p == nullptr || same_places(a.X, a.ld_x, p, ld, sizeof(X)); };
    int classes = 1;  // rows after which the place between two boundaries comes again
    while (a.ld_x * (int64_t)sizeof(X) * classes % 16 != 0) classes *= 2;
    if (vectors(a.X, a.ld_x) && vectors(a.dY, a.ld_dy) && vectors(a.dX, a.ld_dx))
      err = backward<X, VE, false>(a, 1, done, stream);
    else if (a.T >= classes && same(a.dY, a.ld_dy) && same(a.dX, a.ld_dx))
      err = backward<X, VE, true>(a, classes, done, stream);
    else
      err = backward<X, 1, false>(a, 1, done, stream);
  }
  return (done || err != cudaSuccess) ? err : backward_wide<X>(a, stream);
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
