// Matrix product of two 8-bit matrices with block scales.
//
//   Y[t, n] (+)= sum over groups g of 128 columns  a_scale[t, g] b_scale[n / 128, g] P_g[t, n],
//   P_g[t, n] = sum over the group's columns of A[t, j] B[n, j]
//
// A: T x k and B: N x k E4M3 codes.  The tensor cores (tcgen05, kind::f8f6f4) form a
// group's P_g in TMEM from 128-byte rows that TMA brings in, one K = 32 slice after
// another; each group's result is read back, multiplied by its scales and added up in
// fp32 registers, groups in their order.
//
// What bounds it, one GB300.  Many tokens: the sums.  8192 x 12288 x 4096 (T x N x k)
// takes 285 us, 2.9 PFLOP/s, and in a long run of passes, at the power limit, 321 to 328; a
// library product with one scale for each matrix takes 221 and 244.  An fp32 Y, whose 400 MB
// are 59 us of writing, takes 330 to 340 there, one that is added to 355 to 370.  Rows of
// scales off 16 bytes cost nothing: 8192 x 12288 takes 8.4 us for each group at k = 11008 (86
// groups) and at 11264 (88).  Without the sums the kernel takes 222 us: a group's MMAs take
// 512 cycles, and in that time eight warps have to see their end, read 256 columns of 128
// rows from TMEM, add them, times their scales, and hand the accumulators back.  Without the
// multiply-adds it takes 240, without the loads from TMEM 266, without either 238: what
// is left is the accumulators' way between the CTAs, some 800 cycles of the 1024 that TMEM
// holds, and the multiply-adds.  What brought it there, each step from the time before it:
// an arrival on the other CTA's barrier without a release to the cluster (870 to 395 us),
// the scales through shared memory (363), whole warps that walk the issuing loops (352), four
// accumulators and two MMA warps with the loads from TMEM beside the sums (302), scales
// multiplied ahead and four boxes a warp (294), fewer and wider loads of the scales and
// the registers that they leave (285).  Tried and dropped, against the kernel of their day:
// MMAs of each CTA alone, B's rows sent to both (1 % longer; these MMAs by themselves take
// as long as the whole kernel), an arrival of one thread for a CTA (8 %), scales by
// asynchronous copies (3 %), pieces of 24 columns (as long), of 32 (as long, but 4096 x 4096 x
// 12288 9 % longer); slower, too, were pieces of 64 columns, 16 warps of 64 columns, the next
// group's scales or barrier looked at ahead, and waits that spin.
//
// Few tokens: B's bytes and the start: 16 x 4096 x 4096 7.4 us on the device, of which 2.5
// are its 17 MB, 16 x 12288 x 4096 12.0 (50 MB, 7.4); a call takes 8 to 10.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "tc.cuh"
#include "tmem.h"

namespace rgs {
namespace {

constexpr int kChunk = 128;            // a group of columns: one 128-byte swizzle row
constexpr uint32_t kRowsBytes = 128 * kChunk;  // 128 rows of a group

struct Product8 {
  CUtensorMap tmA, tmB, tmY;
  const float* a_scale;
  int64_t ld_as;
  const float* b_scale;
  int64_t bs_row, bs_col;
  void* Y;
  int64_t ld_y;
  int y_type, overwrite;
  int T, N, chunks;
  int stages, m_tiles, n_tiles;
  int first, items;  // tiles of a launch of many tokens' kernel
  int* err;
};

// Four values of a row of Y from column `col` on, as far as N goes.
__device__ __forceinline__ void put4(const Product8& a, int64_t row, int col, float4 v) {
  if (a.y_type == SKETCH_BF16) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.Y) + row * a.ld_y + col;
    if (col + 4 <= a.N) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(y) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      return;
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 4 && col + i < a.N; ++i) y[i] = __float2bfloat16_rn(f[i]);
    return;
  }
  float* y = static_cast<float*>(a.Y) + row * a.ld_y + col;
  if (col + 4 <= a.N) {
    if (!a.overwrite) {
      const float4 o = *reinterpret_cast<const float4*>(y);
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *reinterpret_cast<float4*>(y) = v;
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
  for (int i = 0; i < 4 && col + i < a.N; ++i) y[i] = a.overwrite ? f[i] : y[i] + f[i];
}

// ---- few tokens --------------------------------------------------------------------
// B's rows are the MMA's M (128 of them), TN tokens its N.  A cluster of S CTAs splits
// the groups of a tile and joins its parts through distributed shared memory, each CTA
// a share of the tokens, in the CTAs' order.
constexpr int kFewStages = 5;   // at most
// Tokens of a thread of the sums' warps: 32 at most, then two warps share 32 rows of B.
constexpr int few_cols(int TN) { return TN <= 32 ? TN : TN / 2; }
constexpr int few_warps(int TN) { return 4 * (TN / few_cols(TN)); }
constexpr int few_threads(int TN) { return 64 + 32 * few_warps(TN); }  // copies, MMAs, sums
constexpr uint32_t few_stage_bytes(int TN) { return kRowsBytes + TN * kChunk; }

template <int TN>
__global__ void __launch_bounds__(few_threads(TN), few_resident(TN)) matmul8_few_kernel(const __grid_constant__ Product8 a) {
  constexpr int kBuffers = few_buffers(TN), kCols = few_cols(TN), kSums = few_warps(TN);
  constexpr uint32_t kStageBytes = few_stage_bytes(TN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kFewStages], empty_bar[kFewStages];
  __shared__ __align__(8) uint64_t tfull_bar[kBuffers], tempty_bar[kBuffers];
  __shared__ __align__(16) float factor[kSums][2][kCols];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int issued, consumed;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = tc::cluster_ctarank();
  const int tile = (int)(blockIdx.x / S);
  const int n0 = tile % a.n_tiles * 128, t0 = tile / a.n_tiles * TN;
  const int c0 = (int)((int64_t)a.chunks * rank / S), n_mine = (int)((int64_t)a.chunks * (rank + 1) / S) - c0;

  auto fetch = [&](int i, int s) {
    uint8_t* st = smem + (size_t)s * kStageBytes;
    tc::mbar_arrive_expect_tx(&full_bar[s], kStageBytes);
    tc::tma_load_2d(st, &a.tmB, &full_bar[s], (c0 + i) * kChunk, n0);
    tc::tma_load_2d(st + kRowsBytes, &a.tmA, &full_bar[s], (c0 + i) * kChunk, t0);
  };
  const int early = n_mine < a.stages ? n_mine : a.stages;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&a.tmA);
    tc::prefetch_tmap(&a.tmB);
    abort_flag = 0;
    issued = early;
    consumed = 0;
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(&full_bar[s], 1);
      tc::mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < kBuffers; ++b) {
      tc::mbar_init(&tfull_bar[b], 1);
      tc::mbar_init(&tempty_bar[b], kSums);
    }
    tc::fence_mbar_init();
    tc::fence_proxy_async_smem();
    cudaGridDependencySynchronize();
    for (int i = 0; i < early; ++i) fetch(i, i);  // while the others set up
  }
  cudaGridDependencySynchronize();
  if (warp == 1) tc::tmem_alloc(&tmem_slot, few_columns(TN));
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  cudaTriggerProgrammaticLaunchCompletion();
  const uint32_t tmem = tmem_slot;
  Pair acc[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;

  if (warp == 0) {
    // ---- copies ----
    if (lane == 0) {
      int s = early % a.stages;
      uint32_t ph = 0;
      for (int i = early; i < n_mine; ++i) {
        if (!tc::mbar_wait(&empty_bar[s], ph, &abort_flag, a.err, tc::kErrTimeoutStage)) break;
        fetch(i, s);
        issued = i + 1;
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMAs: a group to an accumulator ----
    constexpr uint32_t idesc = tc::idesc_e4m3(128, TN);
    int s = 0, b = 0;
    uint32_t ph = 0, bph = 0;
    for (int i = 0; i < n_mine; ++i) {
      bool live = tc::mbar_wait(&full_bar[s], ph, &abort_flag, a.err, tc::kErrTimeoutLoad);
      if (i >= kBuffers) live = tc::mbar_wait(&tempty_bar[b], bph ^ 1u, &abort_flag, a.err, tc::kErrTimeoutStage) && live;
      if (!__all_sync(0xFFFFFFFFu, live)) break;
      tc::tc_fence_after();
      const uint32_t sa = tc::smem_u32(smem + (size_t)s * kStageBytes);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kChunk / 32; ++kk)
          tc::mma_e4m3(tmem + (uint32_t)(b * TN), tc::sdesc_sw128(sa + kk * 32, 16, 1024),
                       tc::sdesc_sw128(sa + kRowsBytes + kk * 32, 16, 1024), idesc, kk > 0);
        tc::mma_commit(&tfull_bar[b]);
        tc::mma_commit(&empty_bar[s]);
        consumed = i + 1;
      }
      __syncwarp();
      if (++s == a.stages) {
        s = 0;
        ph ^= 1u;
      }
      if (++b == kBuffers) {
        b = 0;
        bph ^= 1u;
      }
    }
  } else {
    // ---- sums: a row of B to a thread ----
    const int quarter = warp & 3;  // TMEM lanes 32 (warp % 4) .. +31
    const int col = (warp - 2) / 4 * kCols;
    float(*f)[kCols] = factor[warp - 2];
    const uint32_t f0 = tc::smem_u32(f);
    constexpr int kMine = (kCols + 31) / 32;
    const float* as[kMine];
    float next[kMine];
    float next_b = 0.f;
    const float* bs = a.b_scale + (int64_t)(n0 / kScaleBlock) * a.bs_row;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int t = t0 + col + i * 32 + lane;
      as[i] = (kCols >= 32 || lane < kCols) && t < a.T ? a.a_scale + t * a.ld_as : nullptr;
    }
    auto load = [&](int c) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) next[i] = as[i] ? as[i][c] : 0.f;
      next_b = bs[c * a.bs_col];
    };
    if (n_mine > 0) load(c0);
    int b = 0;
    uint32_t bph = 0;
    for (int i = 0; i < n_mine; ++i) {
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        if (kCols >= 32 || lane < kCols) f[i & 1][j * 32 + lane] = next[j] * next_b;
      __syncwarp();
      if (i + 1 < n_mine) load(c0 + i + 1);
      const bool live = tc::mbar_wait(&tfull_bar[b], bph, &abort_flag, a.err, tc::kErrTimeoutMma);
      if (!__all_sync(0xFFFFFFFFu, live)) break;
      tc::tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * TN + col);
      constexpr int kLoad = kCols < 32 ? kCols : 32;
#pragma unroll
      for (int cg = 0; cg < kCols / kLoad; ++cg) {
        uint32_t v[kLoad];
        tc::tmem_ld_32x32b<kLoad>(at + cg * kLoad, v);
        tc::tmem_wait_ld_regs(v);
        if (cg == kCols / kLoad - 1) {  // the accumulator is read
          tc::tc_fence_before();
          if (tc::elect_one()) tc::mbar_arrive(&tempty_bar[b]);
        }
#pragma unroll
        for (int q = 0; q < kLoad / 4; ++q) {
          const uint4 w = tc::lds128(f0 + (uint32_t)(((i & 1) * kCols + cg * kLoad + 4 * q) * 4));
          Pair* p = acc + (cg * kLoad + 4 * q) / 2;
          p[0] = fma2(pair(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])),
                      pair(__uint_as_float(w.x), __uint_as_float(w.y)), p[0]);
          p[1] = fma2(pair(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])),
                      pair(__uint_as_float(w.z), __uint_as_float(w.w)), p[1]);
        }
      }
      if (++b == kBuffers) {
        b = 0;
        bph ^= 1u;
      }
    }
  }
  __syncwarp();
  // ---- the parts' sum; the MMAs that read the stages are done once the sums' warps get here ----
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);  // [token][row of B]
  if (warp >= 2) {
    const int q = (warp & 3) * 32 + lane, col = (warp - 2) / 4 * kCols;
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const float2 v = split(acc[i]);
      red[(col + 2 * i) * 128 + q] = v.x;
      red[(col + 2 * i + 1) * 128 + q] = v.y;
    }
  }
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  const uint32_t red0 = tc::smem_u32(red);
  const int tokens = a.T - t0 < TN ? a.T - t0 : TN;
  for (int e = threadIdx.x; e < tokens * 32; e += few_threads(TN)) {
    const int t = e >> 5, n = (e & 31) * 4;
    if (t % (int)S != (int)rank || n0 + n >= a.N) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t off = red0 + (uint32_t)(t * 128 + n) * 4;
    for (uint32_t r = 0; r < S; ++r) {
      const float4 v = tc::ld_dsmem_f4(tc::mapa_shared(off, r));
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    if (!abort_flag) put4(a, t0 + t, n0 + n, sum);
  }
  // ---- on a timeout, give copies still in flight a bounded chance to land ----
  if (threadIdx.x == 0 && abort_flag) {
    volatile int dummy = 0;
    for (int i = consumed; i < issued; ++i)
      tc::mbar_wait(&full_bar[i % a.stages], (i / a.stages) & 1, &dummy, nullptr, 0, 100000000ull);
  }
  __syncthreads();
  if (S > 1) tc::cluster_sync();  // no CTA leaves while its part may still be read
  if (warp == 1) tc::tmem_dealloc(tmem, few_columns(TN));
}

// Clusters' size for `tiles` tiles, and the groups one after another, over the rounds that
// the CTAs take.  As many CTAs as the GPU holds at once (in two rounds 64 x 12288 x 4096
// takes 25 us, with clusters of 3 beside each other 14.8), not five to seven to a cluster
// (clusters of 6 do not all fit beside each other: 32 x 6144 x 2048 takes 15.9 us with
// them, 6.9 with 4), and more where that saves three groups at least (16 x 2048 x 2048:
// 4.3 us with 4, 4.9 with 8; 16 x 1024 x 4096: 5.7 and 4.6).
unsigned few_split(int64_t tiles, int chunks, int resident, int64_t* steps) {
  const int64_t slots = (int64_t)num_sms() * resident;
  unsigned S = 1;
  *steps = ceil_div(tiles, slots) * chunks;
  for (int s : {2, 3, 4, 8}) {
    if (s > chunks || tiles * s > slots) break;
    const int64_t n = ceil_div(chunks, s);
    if (n + 3 <= *steps) {
      *steps = n;
      S = (unsigned)s;
    }
  }
  return S;
}

template <int TN>
cudaError_t launch_few(Product8& p, const MatmulBlocks& a, cudaStream_t stream) {
  constexpr uint32_t kStageBytes = few_stage_bytes(TN);
  cudaError_t err = make_tmap_u8_2d(&p.tmA, a.A, (uint64_t)a.k, (uint64_t)a.T, (uint64_t)a.ld_a, kChunk, TN);
  if (err == cudaSuccess)
    err = make_tmap_u8_2d(&p.tmB, a.B, (uint64_t)a.k, (uint64_t)a.N, (uint64_t)a.ld_b, kChunk, 128);
  if (err != cudaSuccess) return err;
  p.n_tiles = (int)ceil_div(a.N, 128);
  const int64_t tiles = (int64_t)p.n_tiles * ceil_div(a.T, TN);
  int64_t steps;
  const unsigned S = few_split(tiles, p.chunks, few_resident(TN), &steps);
  p.stages = (int)ceil_div(p.chunks, S);
  static std::atomic<size_t> known;
  size_t fixed = 0;
  err = static_smem(matmul8_few_kernel<TN>, known, &fixed);
  if (err != cudaSuccess) return err;
  const size_t smem = few_smem(TN, fixed);
  const int most = (int)((smem - 1024) / kStageBytes);  // 1 KB: the stages' alignment
  if (most < 3 || TN * 512 > smem - 1024 || !tmem_safe(few_columns(TN), smem + fixed + kBlockSmem, true))
    return cudaErrorInvalidConfiguration;  // stages, a part of the sum, TMEM
  if (p.stages > most) p.stages = most;
  if (p.stages > kFewStages) p.stages = kFewStages;
  err = allow_smem(matmul8_few_kernel<TN>, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S), 1, 1);
  cfg.blockDim = dim3(few_threads(TN), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // comes up while the kernel before ends
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, matmul8_few_kernel<TN>, p);
}

// ---- many tokens -------------------------------------------------------------------
// Pairs of CTAs (cta_group::2) on 256 x 256 tiles, persistent.  A group's MMAs fill two
// of four accumulators in TMEM (256 x 128 each, 512 columns in all) while eight warps of
// each CTA add the others, times their scales, to the tile's sums in registers: 128
// columns of a row to a thread.  Where there are few tiles, a cluster of several pairs
// takes one, each pair a part of its groups; the parts meet in shared memory and are
// added in the pairs' order.
constexpr int kTile = 256;
constexpr int kTileStages = 5;  // 8192 x 12288 x 4096 284 us, with four and twice the boxes 286
constexpr uint32_t kTileStageBytes = 2 * kRowsBytes;  // 128 rows of A, 128 of B
constexpr int kSumWarps = 8;
constexpr int kTileThreads = 128 + 32 * kSumWarps;    // copies, MMAs, scales, an idle warp; sums
constexpr int kSumCols = 128;                         // of a thread
constexpr int kLoads = kSumCols / 16;                 // from TMEM, of 16 columns
// Registers: the launch has 168 for each thread, 384 * 168 = 128 * 88 + 256 * 208.  8192 x
// 12288 x 4096 takes 4 to 5 % longer with 72 and 216, 104 and 200, or 120 and 192.
constexpr int kFewRegisters = 88, kSumRegisters = 208;
constexpr uint32_t kBoxBytes = 32 * 64;               // a warp's 32 rows of 64 bytes, on their way to Y
constexpr int kBoxes = 2;                             // of a warp
constexpr int kScaleGroups = 8;                       // groups whose scales are handed over together
constexpr size_t kTileSmem = kTileStages * kTileStageBytes + kSumWarps * kBoxes * kBoxBytes + 1024;
static_assert(tmem_alone(kTileSmem));
constexpr int kGroupM = 16;                           // tile rows walked together
constexpr int kMostPairs = 4;                         // of a cluster

// acc += f * (16 columns in v), while the next 16 columns come from TMEM into w.  One
// piece, so that nothing touches w between the load and its wait.
__device__ __forceinline__ void add_and_load(Pair (&acc)[8], const uint32_t (&v)[16], Pair f, uint32_t (&w)[16], uint32_t taddr) {
  asm volatile(
      "{\n\t.reg .b64 p;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%41];\n\t"
      "mov.b64 p, {%24, %25};\n\tfma.rn.f32x2 %16, p, %40, %16;\n\t"
      "mov.b64 p, {%26, %27};\n\tfma.rn.f32x2 %17, p, %40, %17;\n\t"
      "mov.b64 p, {%28, %29};\n\tfma.rn.f32x2 %18, p, %40, %18;\n\t"
      "mov.b64 p, {%30, %31};\n\tfma.rn.f32x2 %19, p, %40, %19;\n\t"
      "mov.b64 p, {%32, %33};\n\tfma.rn.f32x2 %20, p, %40, %20;\n\t"
      "mov.b64 p, {%34, %35};\n\tfma.rn.f32x2 %21, p, %40, %21;\n\t"
      "mov.b64 p, {%36, %37};\n\tfma.rn.f32x2 %22, p, %40, %22;\n\t"
      "mov.b64 p, {%38, %39};\n\tfma.rn.f32x2 %23, p, %40, %23;\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]), "=&r"(w[4]), "=&r"(w[5]), "=&r"(w[6]), "=&r"(w[7]), 
        "=&r"(w[8]), "=&r"(w[9]), "=&r"(w[10]), "=&r"(w[11]), "=&r"(w[12]), "=&r"(w[13]), "=&r"(w[14]), "=&r"(w[15]),
        "+l"(acc[0]), "+l"(acc[1]), "+l"(acc[2]), "+l"(acc[3]), "+l"(acc[4]), "+l"(acc[5]), "+l"(acc[6]), "+l"(acc[7])
      : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), 
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "l"(f), "r"(taddr)
      : "memory");
}

// The last values of a row of Y from its 64 bytes in shared memory.
__device__ __noinline__ void put_end(const Product8& a, int64_t row, int col, uint32_t mine, uint32_t swizzle) {
  const bool fp32 = a.y_type == SKETCH_FP32;
  for (int e = 0; col + e < a.N; ++e) {
    const uint32_t byte = (uint32_t)e * (fp32 ? 4u : 2u), at = mine + (((byte >> 4) ^ swizzle) << 4) + (byte & 15u);
    if (fp32) {
      float* y = static_cast<float*>(a.Y) + row * a.ld_y + col + e;
      *y = a.overwrite ? tc::lds_f32(at) : *y + tc::lds_f32(at);
    } else {
      store_one(static_cast<__nv_bfloat16*>(a.Y) + row * a.ld_y + col + e, read_one<__nv_bfloat16>(at));
    }
  }
}

// SPLIT: clusters of several pairs (one kernel for both took 4 % longer for 8192 x 12288 x
// 4096).
template <bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1) matmul8_tile_kernel(const __grid_constant__ Product8 a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kTileStages];   // the even CTA's: both CTAs' rows have landed
  __shared__ __align__(8) uint64_t empty_bar[kTileStages];  // each CTA's: the stage may be refilled
  __shared__ __align__(8) uint64_t tfull_bar[4];            // each CTA's: half a group's products are complete
  __shared__ __align__(8) uint64_t tempty_bar[4];           // the even CTA's: both CTAs have read them
  __shared__ __align__(8) uint64_t scale_bar[2];  // each CTA's: the scales of some groups are there
  __shared__ __align__(8) uint64_t read_bar[2];   // each CTA's: its sums' warps have read them
  __shared__ float scales[2][kScaleGroups][2][128];  // of a row, times those of the tile's two column blocks
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int issued, consumed[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ctas = 2;
  if constexpr (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  // the CTA in its pair, the pair's even CTA, the pair's part of a tile's groups
  const uint32_t in_cluster = tc::cluster_ctarank(), rank = in_cluster & 1u, even = SPLIT ? in_cluster & ~1u : 0u;
  const uint16_t both = (uint16_t)(3u << even);
  const int pairs = SPLIT ? (int)ctas >> 1 : 1, part = (int)even >> 1;
  const int c0 = (int)((int64_t)a.chunks * part / pairs), chunks = (int)((int64_t)a.chunks * (part + 1) / pairs) - c0;
  const int first_item = (int)(blockIdx.x / ctas), step = (int)(gridDim.x / ctas), items = a.items;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    issued = 0;
    consumed[0] = consumed[1] = 0;
    for (int s = 0; s < kTileStages; ++s) {
      tc::mbar_init(&full_bar[s], 1);
      tc::mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 4; ++b) {
      tc::mbar_init(&tfull_bar[b], 1);
      tc::mbar_init(&tempty_bar[b], kSumWarps);  // half of them, of both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&scale_bar[b], 1);
      tc::mbar_init(&read_bar[b], kSumWarps);
    }
    tc::fence_mbar_init();
  }
  cudaGridDependencySynchronize();
  if (warp == 0) tc::tmem_alloc_pair(&tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  cudaTriggerProgrammaticLaunchCompletion();
  tc::cluster_sync();  // both CTAs' barriers exist before either signals one
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // first row and column of a tile
  auto place = [&](int item, int& m0, int& n0) {
    item += a.first;
    const int per_group = kGroupM * a.n_tiles, g = item / per_group, rem = item - g * per_group;
    const int left = a.m_tiles - g * kGroupM, gm = left < kGroupM ? left : kGroupM;
    const int n = rem / gm;
    n0 = n * kTile;
    m0 = (g * kGroupM + rem - n * gm) * kTile;
  };

  if (warp < 4) {
  tc::fewer_registers<kFewRegisters>();
  if (warp == 0) {
    // ---- copies: this CTA's half of each operand's rows ----
    // The whole warp walks, one thread issues: what it needs stays in uniform registers,
    // and a stage takes it less than its MMAs' 512 cycles beside the sums' warps.
    const uint32_t full0 = tc::mapa_shared(tc::smem_u32(full_bar), even);  // the even CTA's
    const uint32_t mine0 = tc::smem_u32(full_bar), empty0 = tc::smem_u32(empty_bar), stage0 = tc::smem_u32(smem);
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool stop = false;
    for (int item = first_item; item < items && !stop; item += step) {
      int m0, n0;
      place(item, m0, n0);
      const int ar = m0 + 128 * (int)rank, br = n0 + 64 * (int)rank;  // of each 128 columns, half from each CTA
      for (int c = c0; c < c0 + chunks; ++c, ++it) {
        if (it >= kTileStages) {
          stop = !tc::mbar_wait(empty0 + 8u * s, ph ^ 1u, &abort_flag, a.err, tc::kErrTimeoutStage);
          stop = __any_sync(0xFFFFFFFFu, stop);
          if (stop) break;
        }
        const uint32_t st = stage0 + (uint32_t)s * kTileStageBytes, bar = full0 + 8u * s;
        if (tc::elect_one()) {
          if (rank == 0) tc::mbar_arrive_expect_tx(mine0 + 8u * s, 2 * kTileStageBytes);
          tc::tma_load_2d_pair(st, &a.tmA, bar, c * kChunk, ar);
          tc::tma_load_2d_pair(st + kRowsBytes, &a.tmB, bar, c * kChunk, br);
          tc::tma_load_2d_pair(st + kRowsBytes + kRowsBytes / 2, &a.tmB, bar, c * kChunk, br + 128);
        }
        __syncwarp();
        if (++s == kTileStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) issued = it;
    // the even CTA's commits have arrived on this one's barriers before it leaves
    for (int i = it > kTileStages ? it - kTileStages : 0; i < it && !stop; ++i) {
      stop = !tc::mbar_wait(empty0 + 8u * (i % kTileStages), (i / kTileStages) & 1, &abort_flag, a.err, tc::kErrTimeoutStage);
      stop = __any_sync(0xFFFFFFFFu, stop);
    }
  } else if ((warp & 1) && rank == 0) {
    // ---- MMAs, for both CTAs: warp 1 the even groups, warp 3 the odd ones ----
    // A group's waits, MMAs and commits take a warp some 800 cycles, one after another,
    // the MMAs 512; the accumulators are not the same, so the order does not matter.
    constexpr uint32_t idesc = tc::idesc_e4m3(kTile, kTile / 2);
    const uint64_t ad0 = tc::sdesc_sw128(tc::smem_u32(smem), 16, 1024);
    const uint64_t bd0 = tc::sdesc_sw128(tc::smem_u32(smem) + kRowsBytes, 16, 1024);
    const uint32_t a_hi = (uint32_t)(ad0 >> 32), b_hi = (uint32_t)(bd0 >> 32);
    const uint32_t b0 = (uint32_t)(warp & 2);  // the first of this warp's two accumulators
    const uint32_t full0 = tc::smem_u32(full_bar), tempty0 = tc::smem_u32(tempty_bar) + 8u * b0;
    int total = 0;
    for (int item = first_item; item < items; item += step) total += chunks;
    int s = warp >> 1, it = warp >> 1;
    uint32_t ph = 0, tph = 1;
    bool live = true;
    for (; it < total; it += 2) {
      live = tc::mbar_wait(full0 + 8u * s, ph, &abort_flag, a.err, tc::kErrTimeoutLoad) && live;
      const uint32_t al = (uint32_t)ad0 + (uint32_t)s * (kTileStageBytes >> 4);
      const uint32_t bl = (uint32_t)bd0 + (uint32_t)s * (kTileStageBytes >> 4);
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        if (it >= 2) live = tc::mbar_wait(tempty0 + 8u * h, tph, &abort_flag, a.err, tc::kErrTimeoutStage) && live;
        __syncwarp();
        tc::tc_fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kChunk / 32; ++kk)
            tc::mma_e4m3_pair(tmem + (b0 + h) * (kTile / 2), al + kk * 2, a_hi, bl + h * (kRowsBytes / 2 >> 4) + kk * 2,
                              b_hi, idesc, kk > 0);
          tc::mma_commit_pair(&tfull_bar[b0 + h], both);
          if (h == 1) tc::mma_commit_pair(&empty_bar[s], both);
        }
        __syncwarp();
      }
      // a wait that gives up makes all later ones give up too; looked at now and then (each
      // time, 8192 x 12288 x 4096 took 2 % longer)
      if ((it & 14) == 14 && !__all_sync(0xFFFFFFFFu, live)) break;
      tph ^= 1u;
      s += 2;
      if (s >= kTileStages) {
        s -= kTileStages;
        ph ^= 1u;
      }
    }
    if (lane == 0 && live) consumed[warp >> 1] = it;
  } else if (warp == 2) {
    // ---- scales: of the CTA's 128 rows, times those of the tile's two column blocks ----
    // Four groups' of a row in one load, where they lie on 16 bytes.  With each read singly,
    // the columns' by every lane, this warp took longer than eight groups' MMAs, or the
    // registers that the sums' warps want (8192 x 12288 x 4096 8 % longer with 88).  Rows off 16
    // bytes, four loads for one, keep up (8.4 us a group at 86 groups and at 88).
    const bool fours = ((reinterpret_cast<uintptr_t>(a.a_scale) | (uintptr_t)(a.ld_as * 4) | (uintptr_t)(c0 * 4)) & 15u) == 0;
    int batch = 0;
    bool live = true;
    for (int item = first_item; item < items && live; item += step) {
      int m0, n0;
      place(item, m0, n0);
      const int row = m0 + 128 * (int)rank + lane, left = a.T - row;
      const float* as = a.a_scale + (int64_t)(left > 0 ? row : 0) * a.ld_as + c0;
      // lane c + 8 j: group c's, column block j's
      const int block = n0 / kScaleBlock + ((lane >> 3) & 1);
      const float* bs = a.b_scale + (int64_t)(block * kScaleBlock < a.N ? block : 0) * a.bs_row + (int64_t)c0 * a.bs_col;
      for (int first = 0; first < chunks && live; first += kScaleGroups, ++batch) {
        const int slot = batch & 1;
        const float mine = block * kScaleBlock < a.N && first + (lane & 7) < chunks ? bs[(int64_t)(first + (lane & 7)) * a.bs_col] : 0.f;
#pragma unroll
        for (int half = 0; half < kScaleGroups; half += 4) {
          float sa[4][4];  // row, group
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* from = as + (int64_t)(32 * i) * a.ld_as + first + half;
            if (fours && first + half + 4 <= chunks) {
              const float4 v = 32 * i < left ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
              sa[i][0] = v.x, sa[i][1] = v.y, sa[i][2] = v.z, sa[i][3] = v.w;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) sa[i][j] = 32 * i < left && first + half + j < chunks ? from[j] : 0.f;
            }
          }
          if (half == 0 && batch >= 2)
            live = tc::mbar_wait(&read_bar[slot], ((batch >> 1) - 1) & 1, &abort_flag, a.err, tc::kErrTimeoutStage);
          live = __all_sync(0xFFFFFFFFu, live);
          if (!live) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float b0 = __shfl_sync(0xFFFFFFFFu, mine, half + j), b1 = __shfl_sync(0xFFFFFFFFu, mine, half + j + 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              scales[slot][half + j][0][32 * i + lane] = sa[i][j] * b0;
              scales[slot][half + j][1][32 * i + lane] = sa[i][j] * b1;
            }
          }
        }
        if (!live) break;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&scale_bar[slot]);
      }
    }
  }
  } else {
    // ---- sums: 128 columns of a row to a thread ----
    tc::more_registers<kSumRegisters>();
    const int quarter = warp & 3;  // TMEM lanes 32 (warp % 4) .. +31
    const uint32_t half = (uint32_t)(warp - 4) >> 2;
    const int col = (int)half * kSumCols;
    const uint32_t at0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)col;
    const uint32_t tempty0 = tc::mapa_shared(tc::smem_u32(tempty_bar), even) + 8u * half;
    const uint32_t tfull0 = tc::smem_u32(tfull_bar) + 8u * half;
    const uint32_t box = tc::smem_u32(smem) + kTileStages * kTileStageBytes + (uint32_t)(warp - 4) * (kBoxes * kBoxBytes);
    const uint32_t scale0 = tc::smem_u32(scales) + half * 512u + (uint32_t)(quarter * 32 + lane) * 4u;
    uint32_t b = 0, ph = 0;  // accumulators of the next group, and their barriers' parity
    uint32_t slot = 0, slot_ph = 0;
    bool live = true;
    for (int item = first_item; item < items && live; item += step) {
      int m0, n0;
      place(item, m0, n0);
      const int row0 = m0 + 128 * (int)rank + quarter * 32, col0 = n0 + col;
      Pair acc[kLoads][8];
#pragma unroll
      for (int i = 0; i < kSumCols / 2; ++i) acc[i / 8][i % 8] = 0;
      // A wait that gives up makes all later ones give up too; that is looked at once in
      // eight groups.
      auto group = [&](uint32_t scale) {
        const float f = tc::lds_f32(scale);
        const Pair f2 = pair(f, f);
        live = tc::mbar_wait(tfull0 + 16u * b, ph, &abort_flag, a.err, tc::kErrTimeoutMma) && live;
        __syncwarp();  // the loads are the whole warp's
        tc::tc_fence_after();
        const uint32_t at = at0 + b * kTile;
        uint32_t v[2][16];
        tc::tmem_ld_32x32b_x16(at, v[0]);
        tc::tmem_wait_ld_regs(v[0]);
#pragma unroll
        for (int h = 0; h + 1 < kLoads; ++h) add_and_load(acc[h], v[h & 1], f2, v[(h + 1) & 1], at + 16 * (h + 1));
        tc::tc_fence_before();  // the accumulator is read
        if (tc::elect_one()) tc::mbar_arrive_pair(tempty0 + 16u * b);
        const uint32_t* w = v[(kLoads - 1) & 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          Pair& s = acc[kLoads - 1][i];
          s = fma2(pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), f2, s);
        }
        b ^= 1u;
        ph ^= b ^ 1u;
      };
      for (int c = 0; c < chunks; c += kScaleGroups) {
        live = tc::mbar_wait(&scale_bar[slot], slot_ph, &abort_flag, a.err, tc::kErrTimeoutStage) && live;
        const uint32_t scale = scale0 + slot * (kScaleGroups * 1024u);
        const int n = chunks - c;
#pragma unroll
        for (uint32_t j = 0; j < kScaleGroups; ++j)
          if ((int)j < n) group(scale + j * 1024u);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&read_bar[slot]);
        slot ^= 1u;
        slot_ph ^= slot ^ 1u;
        live = __all_sync(0xFFFFFFFFu, live);
        if (!live) break;
      }
      if constexpr (SPLIT) {
        // the part to where the stages were, 16 bytes of a row's 1024 at 16 (i ^ row % 8);
        // every warp has seen the last MMAs' end (or given up)
        tc::named_barrier(1, 32 * kSumWarps);
        if (!live) break;
        const uint32_t to = tc::smem_u32(smem) + (uint32_t)(quarter * 32 + lane) * 1024u + half * 512u;
#pragma unroll
        for (uint32_t i = 0; i < kSumCols / 4; ++i) {
          const float2 lo = split(acc[i / 4][2 * (i % 4)]), hi = split(acc[i / 4][2 * (i % 4) + 1]);
          tc::sts128(to + ((i ^ ((uint32_t)lane & 7u)) << 4), make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y),
                                                                        __float_as_uint(hi.x), __float_as_uint(hi.y)));
        }
        break;
      }
      if (!live) break;
      // to Y, 64 bytes of 32 rows at a time, in TMA's 64-byte swizzle; a row's last values
      // singly where they do not fill 16 bytes, which TMA would write whole
      const bool fp32 = a.y_type == SKETCH_FP32;
      const uint32_t swizzle = (uint32_t)(lane >> 1) & 3u;
      auto send = [&](int c, int at, const uint4(&w)[4]) {  // in box `at` of the warp's
        const uint32_t to = box + (uint32_t)(at % kBoxes) * kBoxBytes, mine = to + (uint32_t)lane * 64u;
        if (at % kBoxes == 0) {  // the boxes' last copies have left
          if (lane == 0) tc::bulk_wait_read<0>();
          __syncwarp();
        }
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) tc::sts128(mine + ((j ^ swizzle) << 4), w[j]);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (a.N - c < (fp32 ? 16 : 32) && (a.N & (fp32 ? 3 : 7)) != 0) {
          if (row0 + lane < a.T) put_end(a, row0 + lane, c, mine, swizzle);
        } else if (lane == 0 && row0 < a.T && c < a.N) {
          if (fp32 && !a.overwrite) tc::tma_add_2d(&a.tmY, to, c, row0);
          else tc::tma_store_2d_at(&a.tmY, to, c, row0);
          tc::bulk_commit();
        }
      };
      uint4 w[4];
      if (!fp32) {
#pragma unroll
        for (int h = 0; h < kSumCols / 32; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = split(acc[2 * h + j / 2][4 * (j % 2) + i]);
              const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
              r[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            w[j] = make_uint4(r[0], r[1], r[2], r[3]);
          }
          send(col0 + 32 * h, h, w);
        }
      } else {
#pragma unroll
        for (int h = 0; h < kSumCols / 16; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 lo = split(acc[h][2 * j]), hi = split(acc[h][2 * j + 1]);
            w[j] = make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y));
          }
          send(col0 + 16 * h, h, w);
        }
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }
  __syncwarp();
  // ---- on a timeout, give copies still in flight a bounded chance to land ----
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_flag) {
    volatile int dummy = 0;
    if (rank == 0) {
      for (int i = consumed[0] < consumed[1] ? consumed[0] : consumed[1]; i < issued; ++i)
        tc::mbar_wait(&full_bar[i % kTileStages], (i / kTileStages) & 1, &dummy, nullptr, 0, 100000000ull);
    } else {
      const uint64_t t0 = tc::globaltimer();
      while (tc::globaltimer() - t0 < 100000000ull) {
      }
    }
  }
  __syncthreads();
  tc::cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 0) tc::tmem_dealloc_pair(tmem, 512);
  if constexpr (!SPLIT) return;
  // ---- the parts' sum: a share of the CTA's 128 rows for each pair ----
  int m0, n0;
  place(first_item, m0, n0);
  const int row_end = 128 * (part + 1) / pairs;
  const uint32_t from = tc::smem_u32(smem);
  for (int e = 128 * part / pairs * 64 + (int)threadIdx.x; e < row_end * 64; e += kTileThreads) {
    const int r = e >> 6, i = e & 63, row = m0 + 128 * (int)rank + r, col = n0 + 4 * i;
    if (row >= a.T || col >= a.N) continue;
    const uint32_t at = from + (uint32_t)r * 1024u + (uint32_t)((i ^ (r & 7)) << 4);
    float4 v[kMostPairs];
#pragma unroll
    for (int q = 0; q < kMostPairs; ++q) {
      v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < pairs) v[q] = tc::ld_dsmem_f4(tc::mapa_shared(at, 2u * (uint32_t)q + rank));
    }
#pragma unroll
    for (int q = 1; q < kMostPairs; ++q)
      v[0] = make_float4(v[0].x + v[q].x, v[0].y + v[q].y, v[0].z + v[q].z, v[0].w + v[q].w);
    if (!abort_flag) put4(a, row, col, v[0]);
  }
  tc::cluster_sync();  // no CTA leaves while its part may still be read
}

cudaLaunchConfig_t tile_config(int clusters, int pairs, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(clusters * pairs), 1, 1);
  cfg.blockDim = dim3(kTileThreads, 1, 1);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * (unsigned)pairs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of 1 to kMostPairs pairs that the device holds at once (its SMs need not all
// find a place in one).
cudaError_t tile_clusters(int (&out)[kMostPairs + 1]) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices][kMostPairs + 1];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (known[dev][1] == 0) {
    for (auto kernel : {matmul8_tile_kernel<false>, matmul8_tile_kernel<true>}) {
      // what the warpgroups take must be there, or they would wait for it forever
      cudaFuncAttributes f;
      err = cudaFuncGetAttributes(&f, kernel);
      if (err != cudaSuccess) return err;
      if (f.numRegs * kTileThreads < 128 * kFewRegisters + 32 * kSumWarps * kSumRegisters) return cudaErrorInvalidConfiguration;
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTileSmem);
      if (err != cudaSuccess) return err;
    }
    for (int p = kMostPairs; p >= 1; --p) {  // the first entry last: it says that all are there
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = tile_config(num_sms(), p, nullptr, attr);
      cfg.numAttrs = 1;
      int n = 0;
      err = cudaOccupancyMaxActiveClusters(&n, p > 1 ? matmul8_tile_kernel<true> : matmul8_tile_kernel<false>, &cfg);
      if (err != cudaSuccess) return err;
      if (n < 1 && p == 1) return cudaErrorInvalidConfiguration;
      known[dev][p] = n;
    }
  }
  for (int p = 1; p <= kMostPairs; ++p) out[p] = known[dev][p];
  return cudaSuccess;
}

// Tiles [first, first + items), `pairs` pairs to each, `clusters` at once.
cudaError_t launch_tiles(Product8& p, int first, int items, int clusters, int pairs, cudaStream_t stream) {
  p.first = first;
  p.items = items;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = tile_config(clusters, pairs, stream, attr);
  count_launch();
  return cudaLaunchKernelEx(&cfg, pairs > 1 ? matmul8_tile_kernel<true> : matmul8_tile_kernel<false>, p);
}

}  // namespace

cudaError_t launch_matmul_blocks(const MatmulBlocks& a, cudaStream_t stream) {
  Product8 p = {};
  cudaError_t err = device_error_word(&p.err);
  if (err != cudaSuccess) return err;
  p.a_scale = a.a_scale;
  p.ld_as = a.ld_as;
  p.b_scale = a.b_scale;
  p.bs_row = a.bs_row;
  p.bs_col = a.bs_col;
  p.Y = a.Y;
  p.ld_y = a.ld_y;
  p.y_type = a.y_type;
  p.overwrite = a.overwrite;
  p.T = (int)a.T;
  p.N = (int)a.N;
  p.chunks = (int)ceil_div(a.k, kChunk);
  if (a.T <= 16) return launch_few<16>(p, a, stream);
  if (a.T <= 32) return launch_few<32>(p, a, stream);
  // Which takes less, in us as measured: few tokens' kernel 5 and 0.85 for each group one
  // after another; the pairs of CTAs 5 and 0.37 for each group, 1.5 for each further round
  // of tiles, and 4 more for the join where several pairs share a tile (two groups or
  // more each).  Of BF16 outputs; what an fp32 one takes longer (256 tokens, 4096 x 4096,
  // 15.5 for 14.2, added to 16.8) is left out of the rule.
  // 4096 x 4096 with 64 tokens 9.6 against 12.9, with 192 15.9 against 13.4;
  // 12288 x 4096 with 64 16.1 against 17.3, with 96 25 against 17.7; 4096 x 12288 with
  // 256 tokens 21.7 with three pairs to a tile, 42 with one.
  int fit[kMostPairs + 1];
  err = tile_clusters(fit);
  if (err != cudaSuccess) return err;
  p.m_tiles = (int)ceil_div(a.T, kTile);
  p.n_tiles = (int)ceil_div(a.N, kTile);
  const int items = p.m_tiles * p.n_tiles, rounds = (int)ceil_div(items, fit[1]);
  double best = 0.37 * ((double)rounds * p.chunks) + 1.5 * (rounds - 1);
  int pairs = 1;
  for (int q = 2; q <= kMostPairs && 2 * q <= p.chunks; ++q) {
    const double us = 0.37 * (double)ceil_div(p.chunks, q) + 4.0;
    if (items <= fit[q] && us < best) {
      best = us;
      pairs = q;
    }
  }
  int64_t steps;
  few_split(ceil_div(a.T, 64) * ceil_div(a.N, 128), p.chunks, few_resident(64), &steps);
  if (0.85 * (double)steps <= best) return launch_few<64>(p, a, stream);
  err = make_tmap_u8_2d(&p.tmA, a.A, (uint64_t)a.k, (uint64_t)a.T, (uint64_t)a.ld_a, kChunk, 128);
  if (err == cudaSuccess)
    err = make_tmap_u8_2d(&p.tmB, a.B, (uint64_t)a.k, (uint64_t)a.N, (uint64_t)a.ld_b, kChunk, 64);
  const uint32_t size = a.y_type == SKETCH_BF16 ? 2 : 4;
  if (err == cudaSuccess)
    err = make_tmap_out_2d(&p.tmY, a.y_type, a.Y, (uint64_t)a.N, (uint64_t)a.T, (uint64_t)a.ld_y * size, 64 / size, 32);
  if (err != cudaSuccess) return err;
  if (pairs > 1) return launch_tiles(p, 0, items, items, pairs, stream);
  // The last round's tiles, where they are few: two or more pairs to each in a launch of
  // their own, which costs some 18 us (4096 x 5120 x 16384 268 us without, 253 with;
  // 4096 x 4096 x 12288 163 and 160; 4096 x 4096 x 6144 85 and 91).
  const int whole = items / fit[1] * fit[1], last = items - whole;
  if (whole > 0 && last > 0) {
    int q = kMostPairs;
    while (q > 1 && last > fit[q]) --q;
    if (q > 1 && 0.4 * (double)(p.chunks - ceil_div(p.chunks, q)) > 18.0) {
      err = launch_tiles(p, 0, whole, fit[1], 1, stream);
      return err == cudaSuccess ? launch_tiles(p, whole, last, last, q, stream) : err;
    }
  }
  return launch_tiles(p, 0, items, items < fit[1] ? items : fit[1], 1, stream);
}

}  // namespace rgs
