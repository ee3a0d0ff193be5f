// What kernels over the rows of an activation matrix share: vectors of 16 bytes as
// packed pairs, sums over the threads of a row, and a ring of row sets in shared
// memory that bulk copies fill.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace rgs {

constexpr int kMaxSlots = 8;                // of a ring
constexpr size_t kMostSmem = 216u << 10;    // dynamic shared memory of a launch

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

// ---- 8-bit values ------------------------------------------------------------------
// E4M3 codes with an fp32 scale for each block of 128 columns: value = code * scale,
// scale = (the block's largest magnitude) / 448, at least the smallest normal number,
// so that its reciprocal is finite.  A block with an infinity or a NaN has a NaN scale
// and NaN codes.
constexpr int kScaleBlock = 128;
constexpr float kScaleLeast = 1.17549435e-38f;  // 2^-126

// Bits of a magnitude: as integers they are ordered like the numbers, NaN above all.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
// Bits of the largest magnitude of N values (an even number of them); NaN where one is.
template <int N>
__device__ __forceinline__ uint32_t top_magnitude(const float (&x)[N]) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < N; i += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(x[i])), "f"(fabsf(x[i + 1 < N ? i + 1 : i])));
  return __float_as_uint(top);
}

// A block's scale from the bits of its largest magnitude, and what its values are
// multiplied by.  Both roundings are choices: the scale is the magnitude times the rounded
// 1 / 448, within 2^-23 of the quotient, and the reciprocal an approximate one, good to
// 2^-23, so that a value comes within 2^-22 of its quotient by the scale before its code's own
// rounding, 2^-4.  One value in some 200,000 lies that near to the middle between two codes.  The
// scale is a normal number, so that the reciprocal is one too.
__device__ __forceinline__ float code_scale(uint32_t top, float& inv) {
  float scale = fmaxf(__uint_as_float(top) * (1.f / 448.f), kScaleLeast);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  if (top >= 0x7F800000u) scale = inv = __uint_as_float(0x7FC00000u);
  return scale;
}
// Two values' codes (the first in the low byte), rounded to nearest, ties to even; a
// product that the reciprocal's rounding took past 448 stays 448.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// ---- launches --------------------------------------------------------------------
// Whether every row of the matrix starts on a vector of ve elements and ends with a whole one.
inline bool whole_vectors(const void* p, int64_t ld, int64_t k, int ve, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % (ve * size) == 0 && ld % ve == 0 && k % ve == 0;
}

// Threads per row: the fewest (of at most `limit`) that hold a row at `most`
// vectors each, then more while the launch would leave SMs without a block.
inline int threads_per_row(int64_t nvec, int most, int64_t T, int limit) {
  int tpr = 8;
  while (tpr < limit && (int64_t)tpr * most < nvec) tpr *= 2;
  while (tpr < 256 && tpr < nvec && T * tpr < 2 * (int64_t)num_sms() * 256) tpr *= 2;
  return tpr;
}

// Let a kernel have `smem` bytes of dynamic shared memory, kMostSmem at most.  Static
// and dynamic parts of up to 48 KB together need no asking; the static parts of the kernels
// that come here with up to 47 KB stay below 1 KB.  The limit is the kernel's, not the launch's: it is the same for
// every size, so that another host thread's launch never finds it lowered.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t smem) {
  if (smem <= (47u << 10)) return cudaSuccess;
  if (smem > kMostSmem) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
}

// A launch whose blocks may come up while the kernel before it in the stream ends.  The
// kernel waits for that one's results itself, before it touches global memory.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), int64_t blocks, int threads, size_t smem, cudaStream_t stream,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// The other half, at a kernel's start: the kernel after this one may come up as blocks
// leave; the one before has ended.  A kernel that takes TMEM takes it between the two: it
// holds none while it waits for the kernel before, which may still want some, and nothing
// after it comes up before it has its own.
__device__ __forceinline__ void start_early() {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
}

}  // namespace rgs
