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
// (a state that differs by a code is a step apart ever after).  A value that is not
// finite gets the code NaN and takes no part in its block's scale.
//
// A thread works on eight values at a time, one Philox block for each stream; a
// warp's 256 values are one block of an 8-bit state.  fp32 states are bound by HBM
// (268M BF16 weights: 866 us, 1.01 of the copy rate over 22 bytes a value); 8-bit
// states by instruction issue: 68 instructions a value at 0.71 of the issue slots, 15
// of them the three Philox streams, against the 55 that the 10 bytes' time would allow
// at a full issue rate (638 us, 0.62 of the copy rate).  Arithmetic goes in packed pairs.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace rgs {
namespace {

constexpr uint32_t kTagMoment1 = 3u;
constexpr uint32_t kTagMoment2 = 4u;
constexpr int kAdamThreads = 256;
constexpr int kUnit = 8;                         // values per thread: one Philox block of 16-bit lanes
constexpr int kStep = kAdamThreads * kUnit;      // values per block and pass
constexpr int kAdamBatch = 256;                  // tensors per launch

struct AdamBatch {
  sketch_adamw_problem p[kAdamBatch];
  int begin[kAdamBatch + 1];  // prefix of the tensors' chunks
  int n;
  int chunk;                  // values per block, a multiple of kStep
  AdamStep h;
  uint32_t step;
  uint32_t rk0[10], rk1[10];  // Philox round keys of the seed
};

// What a thread loads for its eight values; converted once the values of the
// pass before are done.
template <bool STATES8, bool WF32, bool GF32>
struct Loaded {
  uint4 w[WF32 ? 2 : 1], g[GF32 ? 2 : 1];
  uint4 m[STATES8 ? 1 : 2], v[STATES8 ? 1 : 2];  // 8-bit states: eight codes in x and y
  float ms, vs;
};

// FULL: all of the chunk's values lie inside the tensor.
template <bool F32, bool FULL>
__device__ __forceinline__ void load_values(const void* base, int64_t e, int64_t n, uint4* out) {
  if (FULL || e + kUnit <= n) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + e * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) out[i] = __ldcs(p + i);
    return;
  }
  uint32_t r[F32 ? 8 : 4] = {};
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {  // the tensor's ragged end
    if (e + i < n) {
      if (F32) r[i] = static_cast<const uint32_t*>(base)[e + i];
      else r[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(base)[e + i] << (16 * (i & 1));
    }
  }
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) out[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}
template <bool F32, bool FULL>
__device__ __forceinline__ void store_values(void* base, int64_t e, int64_t n, const uint4* v) {
  if (FULL || e + kUnit <= n) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + e * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) __stcs(p + i, v[i]);
    return;
  }
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    if (e + i < n) {
      if (F32) static_cast<uint32_t*>(base)[e + i] = r[i];
      else static_cast<uint16_t*>(base)[e + i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
    }
  }
}
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const void* base, int64_t e, int64_t n) {
  const uint8_t* c = static_cast<const uint8_t*>(base) + e;
  if (FULL || e + kUnit <= n) return __ldcs(reinterpret_cast<const uint2*>(c));
  uint64_t r = 0;
  for (int i = 0; e + i < n; ++i) r |= (uint64_t)c[i] << (8 * i);
  return make_uint2((uint32_t)r, (uint32_t)(r >> 32));
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void* base, int64_t e, int64_t n, uint2 v) {
  uint8_t* c = static_cast<uint8_t*>(base) + e;
  if (FULL || e + kUnit <= n) {
    __stcs(reinterpret_cast<uint2*>(c), v);
    return;
  }
  const uint64_t r = ((uint64_t)v.y << 32) | v.x;
  for (int i = 0; e + i < n; ++i) c[i] = (uint8_t)(r >> (8 * i));
}

constexpr int kPairs = kUnit / 2;
template <bool F32>
__device__ __forceinline__ void unpack(const uint4* v, Pair (&f)[kPairs]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    f[i] = F32 ? pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]))
               : pair(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack_codes(uint32_t x, uint32_t y, Pair (&f)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((i < 2 ? x : y) >> (16 * (i & 1))), __NV_E4M3);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[i] = pair(v.x, v.y);
  }
}
__device__ __forceinline__ void values(const Pair (&p)[kPairs], float (&f)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 v = split(p[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// t plus the 16 random bits of value i, as the stream lays them out.
__device__ __forceinline__ uint32_t plus_random(uint32_t t, const uint32_t (&r)[4], int i) {
  return (i & 1) ? mad_hi(r[i >> 1], 65536u, t) : t + (r[i >> 1] & 0xFFFFu);
}

// Maximum of top and the magnitudes of a and b; NaN when one of them is.
__device__ __forceinline__ float max3_abs(float top, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float max8_abs(const float (&x)[kUnit]) {
  float top = fabsf(x[0]);
  top = max3_abs(top, x[1], x[2]);
  top = max3_abs(top, x[3], x[4]);
  top = max3_abs(top, x[5], x[6]);
  return max3_abs(top, x[7], x[7]);
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Magnitudes below this are dropped from an 8-bit first moment whose whole block
// is as small (the reciprocal of its scale would overflow).
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100
constexpr uint32_t kInfBits = 0x7F800000u;

// A block's largest finite magnitude from each lane's largest magnitude (or NaN)
// `top`; `odd`: some value of the block is not finite.
__device__ __forceinline__ float block_top(const float (&x)[kUnit], float top, bool& odd) {
  uint32_t t = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
  odd = t >= kInfBits;  // the same in every lane
  if (odd) {
    t = 0;
    for (int i = 0; i < kUnit; ++i) {
      const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      t = max(t, b < kInfBits ? b : 0u);
    }
    t = __reduce_max_sync(0xFFFFFFFFu, t);
  }
  return __uint_as_float(t);
}

// A block's reciprocal scale (0: the block is held as zeros); lane 0 stores the scale.
__device__ __forceinline__ float block_scale(float top, float* scale) {
  const float inv = top >= kLeast ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
  if ((threadIdx.x & 31) == 0) *scale = inv > 0.f ? __fmul_rn(top, 1.f / 448.f) : 0.f;
  return inv;
}

// E4M3 codes in bits 16 to 22 of c.  y = x / scale lies in [-448, 448]; times
// 2^-120 its exponent field is E4M3's (bias 7 for 127) and its subnormals are
// E4M3's, so that the code of |y| is bits 20 to 26, with 16 random bits added below
// them and the rest cut off; the sign stays clear of it.
__device__ __forceinline__ void codes8(const Pair (&x)[kPairs], float inv, const uint32_t (&r)[4], uint32_t (&c)[kUnit]) {
  const Pair inv2 = pair(inv, inv), shift = pair(7.523163845262640e-37f, 7.523163845262640e-37f);  // 2^-120
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 y = split(mul2(mul2(x[i], inv2), shift));
    c[2 * i] = plus_random(__float_as_uint(y.x) >> 4, r, 2 * i);
    c[2 * i + 1] = plus_random(__float_as_uint(y.y) >> 4, r, 2 * i + 1);
  }
}
// Bytes B of four words.
template <int B>
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, B | (B + 4) << 4), __byte_perm(c, d, B << 8 | (B + 4) << 12), 0x7610);
}
__device__ __forceinline__ uint32_t any_zero_byte(uint32_t x) { return (x - 0x01010101u) & ~x & 0x80808080u; }

__device__ __forceinline__ uint2 hold_m(const Pair (&m2)[kPairs], const uint32_t (&r)[4], float* scale) {
  float m[kUnit];
  values(m2, m);
  bool odd;
  const float inv = block_scale(block_top(m, max8_abs(m), odd), scale);
  uint32_t c[kUnit], out[2];
  codes8(m2, inv, r, c);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    out[h] = gather_bytes<2>(c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]) |
             (gather_bytes<3>(__float_as_uint(m[4 * h]), __float_as_uint(m[4 * h + 1]), __float_as_uint(m[4 * h + 2]),
                              __float_as_uint(m[4 * h + 3])) &
              0x80808080u);
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if ((__float_as_uint(m[i]) & 0x7FFFFFFFu) >= kInfBits) out[i >> 2] |= 0x7Fu << (8 * (i & 3));
  }
  return make_uint2(out[0], out[1]);
}

// The roots u of v, good to 2^-22, as codes.  A code is that of the correctly
// rounded root all the same: where the approximate one leaves the random bits'
// sum at an edge (one lane in 4000), the roots are taken again, and the scale
// comes from the correctly rounded root of the largest v, which is the largest
// of the roots.
__device__ __forceinline__ uint2 hold_u(const Pair (&v2)[kPairs], Pair (&u)[kPairs], const uint32_t (&r)[4], float* scale) {
  float v[kUnit];
  values(v2, v);
  bool odd;
  const float inv = block_scale(__fsqrt_rn(block_top(v, max8_abs(v), odd)), scale);
  uint32_t c[kUnit], out[2], edge = 0xFFFFFFFFu;
  codes8(u, inv, r, c);
#pragma unroll
  for (int i = 0; i < kUnit; i += 2)  // two sums' low halves, plus one: 0 or 1 at an edge
    edge = __viaddmin_u16x2(__byte_perm(c[i], c[i + 1], 0x5410), 0x00010001u, edge);
  if ((edge & 0xFFFFu) < 2u || (edge >> 16) < 2u) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) u[i] = pair(__fsqrt_rn(v[2 * i]), __fsqrt_rn(v[2 * i + 1]));
    codes8(u, inv, r, c);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) out[h] = gather_bytes<2>(c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]);
  if (odd || any_zero_byte(out[0]) || any_zero_byte(out[1])) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const uint32_t at = 8 * (i & 3);
      if (v[i] > 0.f && inv > 0.f && ((out[i >> 2] >> at) & 0xFFu) == 0) out[i >> 2] |= 1u << at;  // never zero
      if ((__float_as_uint(v[i]) & 0x7FFFFFFFu) >= kInfBits) out[i >> 2] |= 0x7Fu << at;
    }
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a + b with scalar additions: a packed addition of a packed product is compiled
// to a fused multiply-add (a fifth of the scales came out a last bit apart).
__device__ __forceinline__ Pair add_unfused(Pair a, Pair b) {
  const float2 x = split(a), y = split(b);
  return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One chunk of one tensor: passes of kStep values, a pass's loads issued before
// the values of the pass before are worked on.
template <bool STATES8, bool WF32, bool GF32, bool FULL>
__device__ __forceinline__ void adamw_chunk(const AdamBatch& a, const sketch_adamw_problem& p, int64_t begin) {
  const int64_t n = p.n;
  const int64_t left = n - begin < a.chunk ? n - begin : a.chunk;
  const int passes = (int)(((FULL ? a.chunk : left) + kStep - 1) / kStep);
  int64_t e = begin + (int64_t)threadIdx.x * kUnit;
  using L = Loaded<STATES8, WF32, GF32>;
  auto load = [&](L& l, int64_t at) {
    load_values<WF32, FULL>(p.W, at, n, l.w);
    load_values<GF32, FULL>(p.G, at, n, l.g);
    if constexpr (STATES8) {
      const uint2 m = load_codes<FULL>(p.m, at, n), v = load_codes<FULL>(p.v, at, n);
      l.m[0] = make_uint4(m.x, m.y, 0, 0);
      l.v[0] = make_uint4(v.x, v.y, 0, 0);
      const bool block = FULL || (at & ~int64_t(255)) < n;
      l.ms = block ? p.m_scale[at >> 8] : 0.f;
      l.vs = block ? p.v_scale[at >> 8] : 0.f;
    } else {
      load_values<true, FULL>(p.m, at, n, l.m);
      load_values<true, FULL>(p.v, at, n, l.v);
    }
  };
  L next;
  load(next, e);
  for (int i = 0; i < passes; ++i, e += kStep) {
    const L l = next;
    if (i + 1 < passes) load(next, e + kStep);
    if (!FULL && (e & ~int64_t(255)) >= n) break;  // the warp's values lie past the end
    Pair w[kPairs], g[kPairs], m[kPairs], v[kPairs], u[kPairs];
    unpack<WF32>(l.w, w);
    unpack<GF32>(l.g, g);
    if constexpr (STATES8) {
      unpack_codes(l.m[0].x, l.m[0].y, m);
      unpack_codes(l.v[0].x, l.v[0].y, v);
      const Pair ms = pair(l.ms, l.ms), vs = pair(l.vs, l.vs);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        m[j] = mul2(m[j], ms);
        v[j] = mul2(v[j], vs);
        v[j] = mul2(v[j], v[j]);
      }
    } else {
      unpack<true>(l.m, m);
      unpack<true>(l.v, v);
    }
    if (a.h.grad_scale) {
      const float gs = *a.h.grad_scale;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) g[j] = mul2(g[j], pair(gs, gs));
    }
    const Pair beta1 = pair(a.h.beta1, a.h.beta1), one_beta1 = pair(a.h.one_beta1, a.h.one_beta1);
    const Pair beta2 = pair(a.h.beta2, a.h.beta2), one_beta2 = pair(a.h.one_beta2, a.h.one_beta2);
    const Pair decay = pair(a.h.decay, a.h.decay), lr = pair(-a.h.lr_m, -a.h.lr_m);
    const Pair root = pair(a.h.root_v, a.h.root_v), eps = pair(a.h.eps, a.h.eps);
    float least = FLT_MAX;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      m[j] = add_unfused(mul2(beta1, m[j]), mul2(one_beta1, g[j]));
      v[j] = add_unfused(mul2(beta2, v[j]), mul2(mul2(one_beta2, g[j]), g[j]));
      const float2 f = split(v[j]);
      u[j] = pair(sqrt_approx(f.x), sqrt_approx(f.y));
      least = min3(least, f.x, f.y);
    }
    if (least < FLT_MIN) {  // the approximate root takes subnormals for zeros
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float2 f = split(v[j]);
        u[j] = pair(__fsqrt_rn(f.x), __fsqrt_rn(f.y));
      }
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const float2 d = split(fma2(u[j], root, eps));  // at least eps, a normal number
      w[j] = fma2(mul2(lr, m[j]), pair(rcp_approx(d.x), rcp_approx(d.y)), mul2(w[j], decay));
    }
    float wf[kUnit];
    values(w, wf);
    const uint32_t block = (uint32_t)(e >> 3);
    if constexpr (WF32) {
      uint4 o[2];
      float* f = reinterpret_cast<float*>(o);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) f[j] = wf[j];
      store_values<true, FULL>(p.W, e, n, o);
    } else {
      const Philox4 rw = philox4x32_10_rk(block, a.step, p.layer, kTagSR, a.rk0, a.rk1);
      const uint32_t r[4] = {rw.w0, rw.w1, rw.w2, rw.w3};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __byte_perm(plus_random(__float_as_uint(wf[2 * j]), r, 2 * j),
                           plus_random(__float_as_uint(wf[2 * j + 1]), r, 2 * j + 1), 0x7632);
      if (__float_as_uint(max8_abs(wf)) > kInfBits) {  // a NaN among the eight
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = sr_bf16_bits(wf[2 * j], r[j] & 0xFFFFu) | (sr_bf16_bits(wf[2 * j + 1], r[j] >> 16) << 16);
      }
      const uint4 ov = make_uint4(o[0], o[1], o[2], o[3]);
      store_values<false, FULL>(p.W, e, n, &ov);
    }
    if constexpr (STATES8) {
      const Philox4 pm = philox4x32_10_rk(block, a.step, p.layer, kTagMoment1, a.rk0, a.rk1);
      const uint32_t rm[4] = {pm.w0, pm.w1, pm.w2, pm.w3};
      store_codes<FULL>(p.m, e, n, hold_m(m, rm, p.m_scale + (e >> 8)));
      const Philox4 pu = philox4x32_10_rk(block, a.step, p.layer, kTagMoment2, a.rk0, a.rk1);
      const uint32_t ru[4] = {pu.w0, pu.w1, pu.w2, pu.w3};
      store_codes<FULL>(p.v, e, n, hold_u(v, u, ru, p.v_scale + (e >> 8)));
    } else {
      uint4 o[2];
      float f[kUnit];
      values(m, f);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) reinterpret_cast<float*>(o)[j] = f[j];
      store_values<true, FULL>(p.m, e, n, o);
      values(v, f);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) reinterpret_cast<float*>(o)[j] = f[j];
      store_values<true, FULL>(p.v, e, n, o);
    }
  }
}

template <bool STATES8, bool WF32, bool GF32>
__device__ __forceinline__ void adamw_block(const AdamBatch& a, const sketch_adamw_problem& p, int64_t begin) {
  if (begin + a.chunk <= p.n) adamw_chunk<STATES8, WF32, GF32, true>(a, p, begin);
  else adamw_chunk<STATES8, WF32, GF32, false>(a, p, begin);
}

template <bool STATES8>
__global__ void __launch_bounds__(kAdamThreads, STATES8 ? 4 : 2) adamw_kernel(const __grid_constant__ AdamBatch a) {
  const int block = blockIdx.x;
  int lo = 0, hi = a.n;  // the last tensor that begins at or before this block
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.begin[mid] <= block) lo = mid;
    else hi = mid;
  }
  const sketch_adamw_problem& p = a.p[lo];
  const int64_t begin = (int64_t)(block - a.begin[lo]) * a.chunk;
  if (p.w_type == SKETCH_BF16) {
    if (p.g_type == SKETCH_BF16) adamw_block<STATES8, false, false>(a, p, begin);
    else adamw_block<STATES8, false, true>(a, p, begin);
  } else {
    if (p.g_type == SKETCH_BF16) adamw_block<STATES8, true, false>(a, p, begin);
    else adamw_block<STATES8, true, true>(a, p, begin);
  }
}

}  // namespace

cudaError_t launch_adamw(int n, const sketch_adamw_problem* probs, bool states8, const AdamStep& h, uint64_t seed,
                         uint32_t step, cudaStream_t stream) {
  static thread_local AdamBatch a;
  a.h = h;
  philox_round_keys(seed, a.rk0, a.rk1);
  a.step = step;
  // a block's passes overlap, so it makes up to eight, as long as every SM gets
  // some sixteen blocks (268M values: 638 us with eight passes, 650 with four)
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += probs[i].n;
  int64_t passes = total / ((int64_t)num_sms() * 16 * kStep);
  passes = passes < 1 ? 1 : passes > 8 ? 8 : passes;
  a.chunk = (int)passes * kStep;
  int i = 0;
  while (i < n) {
    a.n = 0;
    a.begin[0] = 0;
    for (; i < n && a.n < kAdamBatch; ++i) {
      if (probs[i].n == 0) continue;
      const int64_t blocks = ceil_div(probs[i].n, a.chunk);  // at most 2^24
      if (a.begin[a.n] + blocks > (int64_t(1) << 30)) break;
      a.p[a.n] = probs[i];
      a.begin[a.n + 1] = (int)(a.begin[a.n] + blocks);
      ++a.n;
    }
    if (a.n == 0) continue;
    count_launch();
    if (states8) adamw_kernel<true><<<(unsigned)a.begin[a.n], kAdamThreads, 0, stream>>>(a);
    else adamw_kernel<false><<<(unsigned)a.begin[a.n], kAdamThreads, 0, stream>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace rgs
