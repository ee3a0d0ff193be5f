// Softmax cross entropy of a linear head over a large vocabulary, without
// storing its logits.
//
//   l = scale X W^T,  lse = log sum_v exp l_v,  loss = lse - l[target]
//   D = g scale (exp(l - lse) - onehot(target))
//   dX = D W,   dW = D^T X   (or the sketch C (+)= D^T XP of dW)
//
// X: T x k and W: V x k BF16; a token whose target is negative is ignored
// (loss 0, no gradient).  Every product runs in one persistent kernel,
// head_gemm_kernel: pairs of CTAs (cta_group::2) on 256 x 256 tiles, K streamed
// in 64-wide chunks by TMA into a ring of stages, tcgen05 BF16 MMAs into two
// TMEM accumulators in turn, so that one tile's epilogue overlaps the next
// tile's MMAs.  Its epilogues:
//   stats   each row's maximum and sum of exponentials over 128 columns, the
//           target's left out; head_combine_kernel joins them per row
//   dlogit  D from the logits and the row's lse, rounded to BF16 (as every D of
//           this library is: the tensor cores take 16-bit operands; 2^-9 of each
//           entry, independent over the terms that dX and dW add up).  D is in
//           units of the largest |g scale|, which its products' results are
//           multiplied by in fp32: with the usual mean over tokens all weights are
//           that one, and the targets' entries, close to -1 for a small exp(l - lse),
//           keep their values, where -g scale would be rounded the same way for
//           every token (up to 0.2% of all gradients).  A target's exp(l - lse) - 1
//           comes from the fp32 dot product that the forward pass put into lse, so
//           that 1 - p of a confident token is off by lse's own rounding (2^-24 of it),
//           where the tensor cores' truncating sum leaves 1.5e-6 of l.  What a target's
//           entry lost in rounding all the same is added to dX at the end, in fp32; up to 128 tokens
//           the rest of every entry takes part in dW's sum as a row of its own
//   dx      rows of dX, added up over the vocabulary's pieces in fp32
//   dw      rows of dW; BF16 ones in 64-byte pieces (single 16-byte ones: 314 us for
//           300 at 1000 x 2048 x 32771)
// The backward pass walks the vocabulary in pieces, so that only T x piece
// logit gradients exist at a time.  One launch forms a piece's rows of dW, its
// part of dX and the next piece's D.  Ignored tokens are dropped beforehand: the
// kept rows of X are gathered to the front (head_gather_kernel), the products
// run over those alone, and what an ignored row of X holds, infinities or NaN
// too, reaches no result.
//
// Tiles of different lengths share a launch, so pairs take them from a counter,
// the longest kind first.  Where dX has too few tiles for the pairs, the
// vocabulary of a tile is split over several, whose fp32 parts head_dx_sum_kernel
// adds.
//
// What bounds it, tokens x k x vocabulary, times in a long run of passes: many tokens
// the tensor cores' rate, which the power limit sets (8192 x 4096 x 131072 forward 5.2
// ms, 1.70 PFLOP/s, where a plain matrix product of that length runs at 1.72; 4096 x
// 4096 x 65536 backward with a tenth of the tokens ignored 3.7 to 3.8 ms, 1.56 to 1.61
// PFLOP/s over the kept ones, and 3.4 ms on a cool GPU); few tokens the stream of W (16
// x 2048 x 32768 forward: 38 us, 0.52 of the copy rate: 128 tiles are two rounds for 76
// pairs, and 11 us go to starts, ends and the join); a backward pass over few tokens
// the epilogues of dW, whose tiles have few chunks of MMAs (19 x 3624 x 47943: 383 us,
// 0.27 of the copy rate; logits and D take 83 of it, dX and dW 271, of which 2820
// tiles of dW at some 4 us a pair, 2.5 of them reading TMEM and packing, 1.8 storing,
// are 148); 1000 x 2048 x 32771 backward (300 us, 0.63 of the kept tokens' MMAs' time)
// the same, with 16 chunks to a tile; small k the epilogues' reads of TMEM, beside which
// MMAs run slower (8192 x 512 x 32768 forward: 295 us, 195 without them).
//
// Softmax statistics and every sum are fp32.  A tile's result is written by one
// thread after a fixed-order accumulation, so results do not depend on timing.
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace rgs {
namespace {

constexpr int kChunk = 64;                  // K elements per stage: one 128-byte swizzle row
constexpr int kTile = 256;                  // rows and columns of a pair's tile
constexpr int kHalf = 128;                  // rows of A and of B that each CTA of the pair loads
constexpr uint32_t kOperandBytes = kHalf * kChunk * 2;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;                // four lane quarters x two column halves
constexpr int kHeadThreads = 64 + 32 * kEpiWarps + 32;  // copies, MMAs, epilogue, tiles
constexpr int kMaxProducts = 3;
constexpr int kTileSlots = 4;                // tiles handed out ahead of the slowest reader
constexpr int kTileReaders = 2 * (1 + kEpiWarps) + 1;  // both CTAs' copies and epilogues, the MMAs
// Tile rows walked together, so that their operands stay in L2: with 16 the forward
// pass takes 5.25 ms (8192 x 4096 x 131072), with 8 5.36, with 4 and 32 more; the
// backward pass the same with 8 and 16.
constexpr int kGroupM = 16;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Epilogue { kEpiStats = 0, kEpiDlogit = 1, kEpiDx = 2, kEpiDw = 3 };

// One product A B^T (M x N, K): operands K-major (rows x K) or MN-major (K x rows).
struct Product {
  CUtensorMap tmA, tmB;
  int a_mn, b_mn;
  int a_row, a_k;       // coordinates of A's first row and K element
  int b_row, b_k;
  int M, N, K;          // M or K is replaced by the number of kept rows where kept_m / kept_k says so
  int kept_m, kept_k;
  int splits;           // parts of K, each a tile of its own (1 or more)
  int a_box;            // rows of K-major A that the even CTA loads; where M <= 128 fewer than 128, and the odd CTA none
  int epi;
};

struct HeadLaunch {
  Product p[kMaxProducts];
  int n;
  const int* kept;      // device: number of kept rows, null where all are
  int* counter;         // device, 0: tiles taken beyond the pairs' first ones; null: every n-th tile
  int* err;
  int64_t T;
  // stats
  const int64_t* targets;
  float scale_log2;     // scale * log2(e)
  float2* partials;     // [128-column block][T]: (maximum, sum) in log2 units, without the target's
  // dlogit
  const float* lse_log2;  // per kept row: lse * log2(e)
  const float* weight;    // per kept row: g * scale
  const float* factor;    // D is in units of it
  const int* target;      // per kept row
  const float* hit;       // per kept row: its target's exp(l - lse) - 1
  uint16_t* D;
  int64_t ld_d;
  int two_terms;          // D's rows kHalf and on hold what its first kHalf rows lost in rounding
  float* rest;            // per kept row: what its target's entry of D lost
  int d_first;            // the vocabulary entry of D's first column
  // dx
  const int* row_of;      // the row of X that each kept row came from
  float* acc;             // kept rows x k, fp32; of the piece's first part where K is split
  int64_t acc_part;       // values of a part
  int dx_first, dx_last;  // no value to add to / the sum is complete and goes to dX
  uint16_t* dX;
  int64_t ld_dx;
  const uint16_t* W;
  int64_t ld_w;
  // dw
  void* dW;               // of the piece's first row
  int64_t ld_dw;
  int dw_mode;            // 0: BF16; 1: fp32; 2: added to fp32
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Columns 2 i and 2 i + 1 of a row's 32 in registers.
__device__ __forceinline__ Pair columns(const uint32_t (&v)[32], int i) {
  return pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What a finite value lost when it was rounded to the one with these bits.
__device__ __forceinline__ float rest_of(float x, uint32_t rounded) {
  const float r = x - __uint_as_float(rounded);
  return fabsf(x) <= FLT_MAX && fabsf(__uint_as_float(rounded)) <= FLT_MAX ? r : 0.f;
}
// f += c * (eight BF16 values)
__device__ __forceinline__ void add_scaled(float (&f)[8], float c, const uint16_t* w) {
  const uint4 q = *reinterpret_cast<const uint4*>(w);
  const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = fmaf(c, __uint_as_float(r[i] << 16), f[2 * i]);
    f[2 * i + 1] = fmaf(c, __uint_as_float(r[i] & 0xFFFF0000u), f[2 * i + 1]);
  }
}

// Four 16-byte pieces of a row in each lane, dealt anew among every four lanes: piece
// i then belongs to the row of the four's lane i, and is the one whose number is the
// lane's own.  A warp's store then covers 64 bytes of eight rows, not 16 of 32.
__device__ __forceinline__ void deal_rows(uint32_t (&d)[16], int lane) {
#pragma unroll
  for (int o = 1; o <= 2; o *= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & o) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t &lo = d[4 * i + w], &hi = d[4 * (i + o) + w];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, o);
        if (up) lo = got;
        else hi = got;
      }
    }
  }
}

struct Tile {
  int p, m, n;              // product (-1: no more tiles), first row, first column
  int part;                 // of a split K
  int a_row, a_k, b_row, b_k;  // the even CTA's first coordinates
  int chunks;
  int a_mn, b_mn;
  int a_box;
};

struct TileOrder {
  int begin[kMaxProducts + 1];
  int m_tiles[kMaxProducts], n_tiles[kMaxProducts];
  int kchunks[kMaxProducts], splits[kMaxProducts];
  __device__ Tile at(const HeadLaunch& a, int item) const {
    Tile t;
    t.p = 0;
    while (t.p + 1 < a.n && begin[t.p + 1] <= item) ++t.p;
    const int tiles = m_tiles[t.p] * n_tiles[t.p];
    t.part = (item - begin[t.p]) / tiles;
    const int c0 = (int)((int64_t)kchunks[t.p] * t.part / splits[t.p]);
    t.chunks = (int)((int64_t)kchunks[t.p] * (t.part + 1) / splits[t.p]) - c0;
    const int local = item - begin[t.p] - t.part * tiles;
    const int per_group = kGroupM * n_tiles[t.p];
    const int g = local / per_group, rem = local - g * per_group;
    const int left = m_tiles[t.p] - g * kGroupM;
    const int gm = left < kGroupM ? left : kGroupM;
    t.n = rem / gm;
    t.m = (g * kGroupM + (rem - t.n * gm)) * kTile;
    t.n *= kTile;
    const Product& pr = a.p[t.p];
    t.a_row = pr.a_row + t.m;
    t.b_row = pr.b_row + t.n;
    t.a_k = pr.a_k + c0 * kChunk;
    t.b_k = pr.b_k + c0 * kChunk;
    t.a_mn = pr.a_mn;
    t.b_mn = pr.b_mn;
    t.a_box = pr.a_box;
    return t;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kHeadThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadLaunch a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kStages];   // the even CTA's: both CTAs' tiles have landed
  __shared__ __align__(8) uint64_t empty_bar[kStages];  // each CTA's: the stage may be refilled
  __shared__ __align__(8) uint64_t tfull_bar[2];        // each CTA's: an accumulator is complete
  __shared__ __align__(8) uint64_t tempty_bar[2];       // the even CTA's: both CTAs have read an accumulator
  __shared__ __align__(8) uint64_t tile_bar[kTileSlots];  // each CTA's: tiles[slot] is there
  __shared__ __align__(8) uint64_t read_bar[kTileSlots];  // the even CTA's: every role of both CTAs has read it
  __shared__ __align__(16) Tile tiles[kTileSlots];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int issued, consumed;
  __shared__ TileOrder order;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const int my_pair = (int)blockIdx.x >> 1, n_pairs = (int)gridDim.x >> 1;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    issued = 0;
    consumed = 0;
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full_bar[s], 1);
      tc::mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&tfull_bar[b], 1);
      tc::mbar_init(&tempty_bar[b], 2 * kEpiWarps);
    }
    for (int i = 0; i < kTileSlots; ++i) {
      tc::mbar_init(&tile_bar[i], 1);
      tc::mbar_init(&read_bar[i], kTileReaders);
    }
    tc::fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc_pair(&tmem_slot, 512);
  // the kernel after this one may come up as this one's blocks leave, and this
  // one has come up while the one before it ends: now its results are needed
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  if (threadIdx.x == 0) {
    // with no kept row at all one tile of zero rows still runs, so that dW is written
    int kept = a.kept ? *a.kept : 0;
    if (kept < 1) kept = 1;
    order.begin[0] = 0;
    for (int p = 0; p < a.n; ++p) {
      const Product& pr = a.p[p];
      order.m_tiles[p] = ((pr.kept_m ? kept : pr.M) + kTile - 1) / kTile;
      order.n_tiles[p] = (pr.N + kTile - 1) / kTile;
      const int K = !pr.kept_k ? pr.K : a.two_terms && kept ? kHalf + kept : kept;
      order.kchunks[p] = (K + kChunk - 1) / kChunk;
      order.splits[p] = pr.splits;
      order.begin[p + 1] = order.begin[p] + order.m_tiles[p] * order.n_tiles[p] * pr.splits;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers exist before either signals one
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int n_items = order.begin[a.n];
  // The pair's j-th tile.  The even CTA's tile warp works tiles out ahead and
  // hands them to the other roles of both CTAs through slots (worked out by each
  // role itself, between one tile's chunks and the next one's, it held the copies
  // and the MMAs up by some 4000 cycles a tile).  A thread that has read a slot
  // says so, one per warp.
  auto next_tile = [&](int j) -> Tile {
    const int slot = j & (kTileSlots - 1);
    Tile t;
    t.p = -1;
    t.chunks = 0;
    if (tc::mbar_wait<true>(&tile_bar[slot], (uint32_t)(j / kTileSlots) & 1u, &abort_flag, a.err, tc::kErrTimeoutStage))
      t = tiles[slot];
    return t;
  };
  auto tile_read = [&](int j) {
    tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&read_bar[j & (kTileSlots - 1)]), 0));
  };

  if (warp == 0 && lane == 0) {
    // ---- producer: this CTA's half of each operand ----
    // This thread paces the kernel: its time for a chunk has to stay below that of
    // the chunk's MMAs, 512 cycles, and every instruction in its loop shows (with a
    // product's fields looked up for each chunk it took 700 cycles, with the next
    // tile read in the loop 780).
    const uint32_t full0 = tc::mapa_shared(tc::smem_u32(full_bar), 0);  // the even CTA's
    const uint32_t empty0 = tc::smem_u32(empty_bar), stage0 = tc::smem_u32(smem);
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool stop = false;
    for (int j = 0; !stop; ++j) {
      const Tile t = next_tile(j);
      if (t.p < 0) break;
      tile_read(j);
      const CUtensorMap *tmA = &a.p[t.p].tmA, *tmB = &a.p[t.p].tmB;
      const int ar = t.a_row + kHalf * (int)rank, br = t.b_row + kHalf * (int)rank;
      // few rows: the rest of A's tile keeps what it holds, which reaches only
      // rows of the product that are not kept
      const uint32_t bytes = kOperandBytes * 2 + (t.a_box == kHalf ? 2 * kOperandBytes : (uint32_t)t.a_box * kChunk * 2);
      auto run = [&](auto a_is_mn, auto b_is_mn, auto loads_a) {
        constexpr bool A_MN = decltype(a_is_mn)::value, B_MN = decltype(b_is_mn)::value;
        int ak = t.a_k, bk = t.b_k;
        for (int c = t.chunks; c > 0; --c, ++it, ak += kChunk, bk += kChunk) {
          if (it >= kStages && !tc::mbar_wait(empty0 + 8u * s, ph ^ 1u, &abort_flag, a.err, tc::kErrTimeoutStage)) {
            stop = true;
            break;
          }
          const uint32_t st = stage0 + (uint32_t)s * kStageBytes, bar = full0 + 8u * s;
          if (rank == 0) tc::mbar_arrive_expect_tx(tc::smem_u32(full_bar) + 8u * s, bytes);
          if constexpr (decltype(loads_a)::value) {
            if constexpr (A_MN) {  // two boxes of [64 k][64 rows]
              tc::tma_load_2d_pair(st, tmA, bar, ar, ak);
              tc::tma_load_2d_pair(st + kOperandBytes / 2, tmA, bar, ar + 64, ak);
            } else {  // one box of [128 rows][64 k]
              tc::tma_load_2d_pair(st, tmA, bar, ak, ar);
            }
          }
          if constexpr (B_MN) {
            tc::tma_load_2d_pair(st + kOperandBytes, tmB, bar, br, bk);
            tc::tma_load_2d_pair(st + kOperandBytes + kOperandBytes / 2, tmB, bar, br + 64, bk);
          } else {
            tc::tma_load_2d_pair(st + kOperandBytes, tmB, bar, bk, br);
          }
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      };
      const bool loads_a = rank == 0 || t.a_box == kHalf;
      if (t.a_mn) run(std::true_type{}, std::true_type{}, std::true_type{});
      else if (t.b_mn && loads_a) run(std::false_type{}, std::true_type{}, std::true_type{});
      else if (t.b_mn) run(std::false_type{}, std::true_type{}, std::false_type{});
      else if (loads_a) run(std::false_type{}, std::false_type{}, std::true_type{});
      else run(std::false_type{}, std::false_type{}, std::false_type{});
    }
    issued = it;
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issuer, for both CTAs ----
    int s = 0, it = 0, j = 0;
    uint32_t ph = 0;
    bool stop = false;
    const uint32_t full0 = tc::smem_u32(full_bar);
    for (; !stop; ++j) {
      const Tile t = next_tile(j);
      if (t.p < 0) break;
      tile_read(j);
      const int b = j & 1;
      if (j >= 2 && !tc::mbar_wait<true>(&tempty_bar[b], ((j >> 1) - 1) & 1, &abort_flag, a.err, tc::kErrTimeoutStage))
        break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(b * kTile);
      // the chunks' MMAs, with everything but the stage fixed at compile time: this
      // thread shares its scheduler with two warps of the epilogue
      auto run = [&](auto a_is_mn, auto b_is_mn) {
        constexpr bool A_MN = decltype(a_is_mn)::value, B_MN = decltype(b_is_mn)::value;
        // a 16-wide K step: 32 bytes along a K-major swizzle row, 16 rows of 128 bytes of an MN-major tile
        constexpr uint32_t kStepA = (A_MN ? 2048u : 32u) >> 4, kStepB = (B_MN ? 2048u : 32u) >> 4;
        constexpr uint32_t idesc = tc::idesc_bf16(kTile, kTile, A_MN, B_MN);
        const uint64_t ad0 = tc::sdesc_sw128(tc::smem_u32(smem), A_MN ? 8192u : 16u, 1024);
        const uint64_t bd0 = tc::sdesc_sw128(tc::smem_u32(smem) + kOperandBytes, B_MN ? 8192u : 16u, 1024);
        const uint32_t a_hi = (uint32_t)(ad0 >> 32), b_hi = (uint32_t)(bd0 >> 32);
        uint32_t more = 0;  // the tile's first MMA overwrites the accumulator
        for (int c = t.chunks; c > 0; --c) {
          if (!tc::mbar_wait(full0 + 8u * s, ph, &abort_flag, a.err, tc::kErrTimeoutLoad)) {
            stop = true;
            break;
          }
          tc::tc_fence_after();
          // a stage further: its size in the descriptors' address fields (16-byte units)
          const uint32_t al = (uint32_t)ad0 + (uint32_t)s * (kStageBytes >> 4);
          const uint32_t bl = (uint32_t)bd0 + (uint32_t)s * (kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk) {
            tc::mma_bf16_pair(acc, al + kk * kStepA, a_hi, bl + kk * kStepB, b_hi, idesc, kk == 0 ? more : 1u);
          }
          more = 1;
          tc::mma_commit_pair(&empty_bar[s]);
          ++it;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      };
      if (t.a_mn) run(std::true_type{}, std::true_type{});  // dW
      else if (t.b_mn) run(std::false_type{}, std::true_type{});
      else run(std::false_type{}, std::false_type{});
      if (!stop) tc::mma_commit_pair(&tfull_bar[b]);
    }
    consumed = it;
  } else if (warp == 2 + kEpiWarps) {
    // ---- tiles: every n-th, or as a counter deals them out ----
    if (lane == 0 && rank == 0) {
      int item = my_pair;
      for (int j = 0;; ++j) {
        const int slot = j & (kTileSlots - 1);
        if (j >= kTileSlots && !tc::mbar_wait<true>(&read_bar[slot], (uint32_t)(j / kTileSlots - 1) & 1u, &abort_flag,
                                                    a.err, tc::kErrTimeoutStage))
          break;
        Tile t = {};
        t.p = -1;
        if (item < n_items) t = order.at(a, item);
        tiles[slot] = t;
        const uint32_t there = tc::mapa_shared(tc::smem_u32(&tiles[slot]), 1);
        const int4* q = reinterpret_cast<const int4*>(&tiles[slot]);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Tile) / 16); ++i) {
          const int4 v = q[i];
          asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(there + 16 * i), "r"(v.x), "r"(v.y),
                       "r"(v.z), "r"(v.w)
                       : "memory");
        }
        tc::mbar_arrive(&tile_bar[slot]);
        tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&tile_bar[slot]), 1));
        if (item >= n_items) break;
        item = a.counter ? n_pairs + atomicAdd(a.counter, 1) : item + n_pairs;
      }
    }
  } else if (warp >= 2) {
    // ---- epilogue: one row per thread, half of the tile's columns ----
    const int quarter = warp & 3;  // TMEM lanes 32 (warp % 4) .. +31
    const int half = (warp - 2) >> 2;
    const int q = quarter * 32 + lane;
    const int kept = a.kept ? *a.kept : 0;
    const float unit = a.factor ? *a.factor : 1.f;
    int j = 0;
    for (;; ++j) {
      const Tile t = next_tile(j);
      if (!__all_sync(0xFFFFFFFFu, t.p >= 0)) break;
      __syncwarp();
      if (lane == 0) tile_read(j);
      const Product& pr = a.p[t.p];
      const int b = j & 1;
      const int row = t.m + kHalf * (int)rank + q;
      const int col0 = t.n + half * kHalf;
      const int N = pr.N;
      // what the epilogue wants of its row, read while the MMAs run
      const bool in = pr.epi == kEpiStats || pr.epi == kEpiDw ? row < pr.M : row < kept;
      float w = 0.f, l2 = 0.f, hit = 0.f;
      int tcol = -1;  // column of the row's target among the tile's
      if (pr.epi == kEpiStats) {
        const int64_t target = in ? a.targets[row] : -1;
        if (target >= col0 && target < col0 + kHalf && target < N) tcol = (int)(target - col0);
      } else if (pr.epi == kEpiDlogit && in) {
        w = a.weight[row] / unit;
        l2 = a.lse_log2[row];
        hit = a.hit[row];
        tcol = a.target[row] - (a.d_first + col0);
      }
      const bool live = tc::mbar_wait(&tfull_bar[b], (j >> 1) & 1, &abort_flag, a.err, tc::kErrTimeoutMma);
      if (!__all_sync(0xFFFFFFFFu, live)) break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * kTile + half * kHalf);
      uint32_t v[32];
      if (pr.epi == kEpiStats) {
        const Pair scale2 = pair(a.scale_log2, a.scale_log2);
        float mx = -INFINITY;
        Pair sum = 0;
        for (int cg = 0; cg < kHalf / 32; ++cg) {
          __syncwarp();  // the load is the whole warp's
          tc::tmem_ld_32x32b_x32(acc + cg * 32, v);
          tc::tmem_wait_ld_regs(v);
          const int c0 = col0 + cg * 32;
          if (c0 + 32 > N) {  // past the vocabulary: no logits
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c0 + i >= N) v[i] = __float_as_uint(-INFINITY);
          }
          if (tcol >= 0 && (tcol >> 5) == cg) {  // the target's own term is added by head_combine_kernel
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((tcol & 31) == i) v[i] = __float_as_uint(-INFINITY);
          }
          float g = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[31]));
#pragma unroll
          for (int i = 2; i < 30; i += 2) g = max3(g, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          const float top = fmaxf(mx, fmaxf(g, __uint_as_float(v[30])) * a.scale_log2);  // scale > 0
          const float ref = top == -INFINITY ? 0.f : top;
          const Pair neg = pair(-ref, -ref);
          const float keep = ex2(mx - ref);
          sum = mul2(sum, pair(keep, keep));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = split(fma2(columns(v, i), scale2, neg));
            sum = add2(sum, pair(ex2(e.x), ex2(e.y)));
          }
          mx = top;
        }
        if (in && col0 < N) a.partials[(int64_t)(col0 / kHalf) * a.T + row] = make_float2(mx, sum2(sum));
      } else if (pr.epi == kEpiDlogit) {
        // rows past the kept ones are written as zeros up to the tile's end,
        // since they take part in dW's sum over rows
        uint16_t* out = a.D + (int64_t)row * a.ld_d + col0;
        auto dlogit = [&](auto two_terms) {
          constexpr bool TWO = decltype(two_terms)::value;
          for (int cg = 0; cg < kHalf / 32; ++cg) {
            __syncwarp();  // the load is the whole warp's
            tc::tmem_ld_32x32b_x32(acc + cg * 32, v);
            tc::tmem_wait_ld_regs(v);
            uint32_t d[16], e[TWO ? 16 : 1];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float p0 = ex2(fmaf(__uint_as_float(v[2 * i]), a.scale_log2, -l2));
              float p1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]), a.scale_log2, -l2));
              if (tcol == cg * 32 + 2 * i) p0 = hit;
              if (tcol == cg * 32 + 2 * i + 1) p1 = hit;
              d[i] = in ? pack_bf16(p0 * w, p1 * w) : 0u;
              if constexpr (TWO)
                e[i] = in ? pack_bf16(rest_of(p0 * w, d[i] << 16), rest_of(p1 * w, d[i] & 0xFFFF0000u)) : 0u;
            }
            if ((unsigned)(tcol - cg * 32) < 32u) a.rest[row] = rest_of(hit * w, pack_bf16(0.f, hit * w) & 0xFFFF0000u);
            if (TWO && row >= kHalf) continue;  // written with the row before
            // D's row stride is a multiple of the tile's width
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              reinterpret_cast<uint4*>(out + cg * 32)[i] = make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
              if constexpr (TWO)
                reinterpret_cast<uint4*>(out + kHalf * a.ld_d + cg * 32)[i] =
                    make_uint4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
            }
          }
        };
        if (a.two_terms) dlogit(std::true_type{});
        else dlogit(std::false_type{});
      } else if (pr.epi == kEpiDx) {
        float* sum = a.acc + t.part * a.acc_part + (int64_t)row * N + col0;
        uint16_t* out = (in && a.dx_last) ? a.dX + (int64_t)a.row_of[row] * a.ld_dx + col0 : nullptr;
        const float rest = (in && a.dx_last) ? a.rest[row] : 0.f;
        const uint16_t* wt = (in && a.dx_last) ? a.W + (int64_t)a.target[row] * a.ld_w + col0 : nullptr;
        for (int cg = 0; cg < kHalf / 32; ++cg) {
          __syncwarp();  // the load is the whole warp's
          tc::tmem_ld_32x32b_x32(acc + cg * 32, v);
          tc::tmem_wait_ld_regs(v);
          if (!in) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // k is a multiple of 8
            const int c = cg * 32 + 8 * i;
            if (col0 + c >= N) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * i + e]);
            if (!a.dx_first) {
              const float4 x = *reinterpret_cast<const float4*>(sum + c), y = *reinterpret_cast<const float4*>(sum + c + 4);
              f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
              f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
            }
            if (a.dx_last) {
              add_scaled(f, rest, wt + c);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] *= unit;
              *reinterpret_cast<uint4*>(out + c) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                              pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            } else {
              *reinterpret_cast<float4*>(sum + c) = make_float4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<float4*>(sum + c + 4) = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
      } else {
        auto dw = [&](auto bf16) {
          for (int cg = 0; cg < kHalf / 32; ++cg) {
            __syncwarp();  // the load is the whole warp's
            tc::tmem_ld_32x32b_x32(acc + cg * 32, v);
            tc::tmem_wait_ld_regs(v);
            const int col = col0 + cg * 32;
            // unfused: adding a gradient to itself doubles it
            auto value = [&](int i) { return __fmul_rn(__uint_as_float(v[i]), unit); };
            if constexpr (decltype(bf16)::value) {
              uint32_t d[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) d[i] = pack_bf16(value(2 * i), value(2 * i + 1));
              deal_rows(d, lane);
              const int first = row - (lane & 3), c = col + 8 * (lane & 3);
              uint16_t* out = static_cast<uint16_t*>(a.dW) + (int64_t)first * a.ld_dw + c;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (first + i < pr.M && c < N)
                  *reinterpret_cast<uint4*>(out + i * a.ld_dw) = make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
            } else {
              if (!in) continue;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (col + 4 * i >= N) break;
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.dW) + (int64_t)row * a.ld_dw + col) + i;
                float4 x = make_float4(value(4 * i), value(4 * i + 1), value(4 * i + 2), value(4 * i + 3));
                if (a.dw_mode == 2) {
                  const float4 y = *o;
                  x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                }
                *o = x;
              }
            }
          }
        };
        if (a.dw_mode == 0) dw(std::true_type{});
        else dw(std::false_type{});
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&tempty_bar[b]), 0));
    }
  }
  __syncwarp();
  // ---- on a timeout, give copies still in flight a bounded chance to land ----
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_flag) {
    volatile int dummy = 0;
    if (rank == 0) {
      for (int i = consumed; i < issued; ++i)
        tc::mbar_wait(&full_bar[i % kStages], (i / kStages) & 1, &dummy, nullptr, 0, 100000000ull);
    } else {
      const uint64_t t0 = tc::globaltimer();
      while (tc::globaltimer() - t0 < 100000000ull) {
      }
    }
  }
  __syncthreads();
  tc::cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 0) tc::tmem_dealloc_pair(tmem, 512);
}

__device__ __forceinline__ void join(float& mx, float& sum, float mx1, float sum1) {
  const float top = fmaxf(mx, mx1);
  const float ref = top == -INFINITY ? 0.f : top;
  sum = sum * ex2(mx - ref) + sum1 * ex2(mx1 - ref);
  mx = top;
}

// Dot product of two BF16 rows by a warp, in fp32: the same bits wherever it is taken.
// COPY: x is also copied to y.
template <bool COPY>
__device__ __forceinline__ float warp_dot(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w, int64_t k,
                                          uint16_t* __restrict__ y) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int64_t i = threadIdx.x & 31; i < k / 8; i += 32) {
    const uint4 a = reinterpret_cast<const uint4*>(x)[i], b = reinterpret_cast<const uint4*>(w)[i];
    if (COPY) reinterpret_cast<uint4*>(y)[i] = a;
    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s0 = fmaf(__uint_as_float(p[e] << 16), __uint_as_float(q[e] << 16), s0);
      s1 = fmaf(__uint_as_float(p[e] & 0xFFFF0000u), __uint_as_float(q[e] & 0xFFFF0000u), s1);
    }
  }
  float dot = s0 + s1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  return dot;
}

// Join a row's partial statistics with its target's logit.  That logit is a dot
// product of its own in fp32 (the tensor cores' accumulation truncates, which
// the loss would show at a relative 1.5e-6 for k = 4096; so 6e-7) and stands
// both in the sum and in loss = lse - logit.  Where it is the largest, the loss is
// log(1 + s), s the other exponentials' sum over its own: taken from s itself, so
// that a confident token's small loss keeps its digits (1 + s loses all of an s
// below 2^-24).  Block: eight rows; a warp for each dot product, and 32 threads for
// each row's partials.
constexpr int kCombineRows = 8;
__global__ void __launch_bounds__(256) head_combine_kernel(const float2* partials, const uint16_t* X, int64_t ld_x,
                                                           const uint16_t* W, int64_t ld_w, int64_t k,
                                                           const int64_t* targets, float scale, float scale_log2,
                                                           int64_t T, int64_t V, int blocks, float* loss, float* lse,
                                                           int32_t* status) {
  cudaGridDependencySynchronize();
  __shared__ float2 part[32][kCombineRows];
  __shared__ float hit[kCombineRows];
  __shared__ int bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * kCombineRows;
  const int64_t row = row0 + (threadIdx.x & 7);
  float mx = -INFINITY, sum = 0.f;
  if (row < T) {
#pragma unroll 4
    for (int i = threadIdx.x >> 3; i < blocks; i += 32) {
      const float2 v = partials[(int64_t)i * T + row];
      join(mx, sum, v.x, v.y);
    }
  }
  part[threadIdx.x >> 3][threadIdx.x & 7] = make_float2(mx, sum);
  const int64_t drow = row0 + warp;
  const int64_t target = drow < T ? targets[drow] : -1;
  float dot = 0.f;
  if (target >= 0 && target < V) dot = warp_dot<false>(X + drow * ld_x, W + target * ld_w, k, nullptr);
  if (lane == 0) hit[warp] = dot;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  if (threadIdx.x < kCombineRows && row < T) {
    for (int i = 1; i < 32; ++i) join(mx, sum, part[i][threadIdx.x].x, part[i][threadIdx.x].y);
    const int64_t t = targets[row];
    const bool is_logit = t >= 0 && t < V;
    const float h = hit[threadIdx.x] * scale_log2;
    if (is_logit && h >= mx) {
      const float l = log1pf(sum * ex2(mx - h)) + (h - h);  // NaN for an infinite logit, as inf - inf is
      lse[row] = fmaf(hit[threadIdx.x], scale, l);
      loss[row] = l;
    } else {
      if (is_logit) join(mx, sum, h, 1.f);
      const float l2 = (mx == -INFINITY ? 0.f : mx) + log2f(sum);
      lse[row] = l2 * kLn2;
      loss[row] = t < 0 ? 0.f : t >= V ? NAN : (((mx - h) + log2f(sum)) * kLn2);
    }
  }
  if (status != nullptr && blockIdx.x == 0) {
    int found = 0;
    for (int64_t i = threadIdx.x; i < T; i += blockDim.x) found |= targets[i] >= V;
    if (found) bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *status = bad ? SKETCH_DEV_BAD_TARGET : 0;
  }
}

// Gather the kept tokens' rows to the front, in order.  Block: `per_block` rows,
// eight at a time, one per warp.  Each block counts the kept tokens before its own,
// so that no pass over the targets comes first; blocks are longer for many tokens,
// so that this counting stays small (T = 131072: 1 GB read from L2 in all, beside
// 1 GB of X).  A kept token's target gets its exp(l - lse) - 1 here, from the same
// dot product as in the forward pass.  Compact rows past the kept ones, up to `fill` (a multiple of the
// tile's rows), are zeroed.
struct Gather {
  const uint16_t* X;
  int64_t T, k, ld_x;
  const uint16_t* XP;  // nullable
  int64_t ld_xp, r;
  const uint16_t* W;
  int64_t V, ld_w;
  const int64_t* targets;
  const float* lse;
  const float* g;
  float scale;
  uint16_t* Xc;   // rows x k
  uint16_t* XPc;  // rows x ld_xpc
  int64_t ld_xpc;
  float* lse_log2;
  float* weight;
  float* factor;  // the largest finite |weight|, 1 where that is 0
  int* target;
  float* hit;
  int* row_of;
  int* kept;
  int* counters;  // n_counters of them, set to 0
  int n_counters;
  uint16_t* dX;  // nullable
  int64_t ld_dx;
  int64_t rows;  // compact rows the buffers hold
  int two_terms;  // each kept row once more, kHalf rows on
  int per_block;
  int all_rows;  // zero every compact row past the kept ones, not only the last tile's
  int32_t* status;
};

__global__ void __launch_bounds__(256) head_gather_kernel(const __grid_constant__ Gather a) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  __shared__ int before_s, total_s, bad_s, top_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.x * a.per_block;
  if (threadIdx.x == 0) before_s = total_s = bad_s = top_s = 0;
  __syncthreads();
  int before = 0, total = 0, bad = 0;
  float top = 0.f;
  for (int64_t i = threadIdx.x; i < a.T; i += blockDim.x) {
    const int64_t t = a.targets[i];
    const int keep = t >= 0 && t < a.V;
    total += keep;
    before += keep && i < base;
    bad |= t >= a.V;
    if (blockIdx.x == 0 && keep) {
      const float w = fabsf(a.g[i] * a.scale);
      if (w <= FLT_MAX) top = fmaxf(top, w);
    }
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane == 0) {  // integer sums: the same in any order
    atomicAdd(&before_s, before);
    atomicAdd(&total_s, total);
    if (bad) bad_s = 1;
  }
  if (top > 0.f) atomicMax(&top_s, __float_as_int(top));  // block 0's alone; positive floats compare as integers do
  __syncthreads();
  total = total_s;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.n_counters; i += blockDim.x) a.counters[i] = 0;
    if (threadIdx.x == 0) {
      *a.kept = total;
      *a.factor = top_s > 0 ? __int_as_float(top_s) : 1.f;
      if (a.status) *a.status = bad_s ? SKETCH_DEV_BAD_TARGET : 0;
    }
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int64_t fill = total < 1 ? 1 : total;
  fill = a.all_rows ? a.rows : (fill + kTile - 1) / kTile * kTile;
  int64_t next = before_s;  // compact row of the first kept one among the eight rows
  const int64_t end = base + a.per_block < a.rows ? base + a.per_block : a.rows;
  for (int64_t first = base; first < end; first += 8) {
    const int64_t row = first + warp;
    int64_t dst = next, t = -1;
    for (int w = 0; w < 8; ++w) {
      const int64_t u = first + w < a.T ? a.targets[first + w] : -1;
      const int keep = u >= 0 && u < a.V;
      next += keep;
      if (w < warp) dst += keep;
      if (w == warp) t = u;
    }
    if (row < a.T) {
      if (t >= 0 && t < a.V) {
        const float dot = warp_dot<true>(a.X + row * a.ld_x, a.W + t * a.ld_w, a.k, a.Xc + dst * a.k);
        if (a.XP)
          for (int64_t i = lane; i < a.r; i += 32) a.XPc[dst * a.ld_xpc + i] = a.XP[row * a.ld_xp + i];
        if (a.two_terms) {
          const uint4* x = reinterpret_cast<const uint4*>(a.X + row * a.ld_x);
          uint4* z = reinterpret_cast<uint4*>(a.Xc + (dst + kHalf) * a.k);
          for (int64_t i = lane; i < a.k / 8; i += 32) z[i] = x[i];
          if (a.XP)
            for (int64_t i = lane; i < a.r; i += 32) a.XPc[(dst + kHalf) * a.ld_xpc + i] = a.XP[row * a.ld_xp + i];
        }
        if (lane == 0) {
          a.hit[dst] = expm1f(fmaf(dot, a.scale, -a.lse[row]));
          a.lse_log2[dst] = a.lse[row] * kLog2e;
          a.weight[dst] = a.g[row] * a.scale;
          a.target[dst] = (int)t;
          a.row_of[dst] = (int)row;
        }
      } else if (a.dX) {
        uint4* y = reinterpret_cast<uint4*>(a.dX + row * a.ld_dx);
        for (int64_t i = lane; i < a.k / 8; i += 32) y[i] = zero;
      }
    }
    if (row >= total && row < fill && !(a.two_terms && row >= kHalf && row < kHalf + total)) {
      uint4* y = reinterpret_cast<uint4*>(a.Xc + row * a.k);
      for (int64_t i = lane; i < a.k / 8; i += 32) y[i] = zero;
      if (a.XP)
        for (int64_t i = lane; i < a.r; i += 32) a.XPc[row * a.ld_xpc + i] = 0;
    }
  }
}

// dX's kept rows from their `parts` fp32 parts, eight columns per thread.
__global__ void __launch_bounds__(256) head_dx_sum_kernel(const float* acc, int64_t part, int parts, int64_t k,
                                                          const int* kept, const float* factor, const int* row_of,
                                                          const int* target, const float* rest, const uint16_t* W,
                                                          int64_t ld_w, uint16_t* dX, int64_t ld_dx) {
  cudaGridDependencySynchronize();
  const float unit = *factor;
  const int64_t per_row = k / 8, n = *kept * per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / per_row, c = (i - row * per_row) * 8;
    const float4* p = reinterpret_cast<const float4*>(acc + row * k + c);
    float4 x = p[0], y = p[1];
#pragma unroll 4
    for (int q = 1; q < parts; ++q) {
      const float4* r = reinterpret_cast<const float4*>(acc + q * part + row * k + c);
      const float4 u = r[0], v = r[1];
      x.x += u.x; x.y += u.y; x.z += u.z; x.w += u.w;
      y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
    }
    float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    add_scaled(f, rest[row], W + (int64_t)target[row] * ld_w + c);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= unit;
    *reinterpret_cast<uint4*>(dX + (int64_t)row_of[row] * ld_dx + c) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
}

// C (+)= factor S, for a piece of the vocabulary.
__global__ void __launch_bounds__(256) head_sketch_add_kernel(const float* S, int64_t n, const float* factor, int overwrite,
                                                              float* C) {
  const float unit = *factor;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    C[i] = overwrite ? unit * S[i] : __fadd_rn(C[i], __fmul_rn(unit, S[i]));  // unfused, as dW's sum
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Vocabulary entries per piece: as many whole tiles as 256 MB of BF16 logit
// gradients hold.
int64_t piece_width(int64_t T, int64_t V) {
  const int64_t rows = round_up(T, kTile);
  int64_t w = (int64_t(256) << 20) / (2 * rows) / kTile * kTile;
  if (w < 4 * kTile) w = 4 * kTile;
  const int64_t all = round_up(V, kTile);
  return w < all ? w : all;
}

// Parts that a dX tile's sum over a piece's vocabulary is split into: as many as
// give every pair a tile, of 16 chunks (1024 entries) at least.  (T = 1000, k =
// 2048, V = 32771: 32 tiles of 513 chunks, beside 1032 tiles of dW of 16.)
int dx_parts(int64_t T, int64_t V, int64_t k) {
  const int64_t tiles = ceil_div(T, kTile) * ceil_div(k, kTile), pairs = num_sms() / 2;
  const int64_t chunks = ceil_div(piece_width(T, V) < V ? piece_width(T, V) : V, kChunk);
  int parts = 1;
  while (tiles * parts * 2 <= pairs && chunks / (parts * 2) >= 16) parts *= 2;
  return parts;
}

constexpr size_t kHeadSmem = (size_t)kStages * kStageBytes + 1024;

// CTA pairs that the device holds at once (its SMs need not all pair up).
cudaError_t head_pairs(int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> pairs[kMaxDevices];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (pairs[dev] == 0) {
    err = cudaFuncSetAttribute(head_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kHeadSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)num_sms(), 1, 1);
    cfg.blockDim = dim3(kHeadThreads, 1, 1);
    cfg.dynamicSmemBytes = kHeadSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    err = cudaOccupancyMaxActiveClusters(&n, head_gemm_kernel, &cfg);
    if (err != cudaSuccess) return err;
    if (n < 1) return cudaErrorInvalidConfiguration;
    pairs[dev] = n;
  }
  *out = pairs[dev];
  return cudaSuccess;
}

// A launch whose blocks may come up while the kernel before it in the stream ends
// (each kernel here waits for that one's results itself).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

cudaError_t launch_products(const HeadLaunch& a, cudaStream_t stream) {
  int64_t items = 0;
  for (int p = 0; p < a.n; ++p) items += ceil_div(a.p[p].M, kTile) * ceil_div(a.p[p].N, kTile) * a.p[p].splits;
  int pairs = 0;
  cudaError_t err = head_pairs(&pairs);
  if (err != cudaSuccess) return err;
  if (items < pairs) pairs = (int)items;
  return launch_after(head_gemm_kernel, 2 * (unsigned)pairs, kHeadThreads, kHeadSmem, stream, a);
}

// Operand rows x K, K contiguous (box 64 x 128), or K x rows, rows contiguous (box 64 x 64).
cudaError_t k_major(CUtensorMap* map, const uint16_t* p, int64_t rows, int64_t K, int64_t ld, int box = kHalf) {
  return encode_tmap_bf16_2d(map, p, (uint64_t)K, (uint64_t)rows, (uint64_t)ld * 2, kChunk, (uint32_t)box);
}
// Rows of a K-major A of M rows that a tile's even CTA loads.
int a_box(int64_t M) { return M <= kHalf ? (int)((M + 7) / 8 * 8) : kHalf; }
cudaError_t mn_major(CUtensorMap* map, const uint16_t* p, int64_t rows, int64_t K, int64_t ld) {
  return encode_tmap_bf16_2d(map, p, (uint64_t)rows, (uint64_t)K, (uint64_t)ld * 2, 64, kChunk);
}

struct BackwardWorkspace {
  uint16_t* Xc;
  uint16_t* XPc;
  int64_t ld_xpc;
  uint16_t* D[2];
  float* acc;
  float* S;           // a piece of the sketch, in units of the factor
  float* lse_log2;
  float* weight;
  float* factor;
  float* rest;
  int* target;
  float* hit;
  int* row_of;
  int* kept;
  int* counters;
  int parts;  // of dX's sum over a piece
  size_t bytes;
};
BackwardWorkspace carve_backward(void* base, int64_t T, int64_t V, int64_t k, int64_t r) {
  WsCursor cur;
  cur.base = static_cast<char*>(base);
  const int64_t rows = round_up(T, kTile), piece = piece_width(T, V);
  const int64_t pieces = ceil_div(V, piece);
  BackwardWorkspace w;
  w.parts = dx_parts(T, V, k);
  w.Xc = cur.take<uint16_t>((size_t)(rows * k));
  w.ld_xpc = round_up(r, 8);
  w.XPc = cur.take<uint16_t>((size_t)(rows * w.ld_xpc));
  for (int i = 0; i < 2; ++i) w.D[i] = cur.take<uint16_t>((size_t)((i == 0 || pieces > 1) ? rows * piece : 0));
  // split sums keep a part per piece and split, others are added up over the pieces
  w.acc = cur.take<float>((size_t)(w.parts > 1 ? pieces * w.parts * rows * k : pieces > 1 ? rows * k : 0));
  w.S = cur.take<float>((size_t)((piece < V ? piece : V) * r));
  w.lse_log2 = cur.take<float>((size_t)rows);
  w.weight = cur.take<float>((size_t)rows);
  w.factor = cur.take<float>(1);
  w.rest = cur.take<float>((size_t)rows);
  w.target = cur.take<int>((size_t)rows);
  w.hit = cur.take<float>((size_t)rows);
  w.row_of = cur.take<int>((size_t)rows);
  w.kept = cur.take<int>(1);
  w.counters = cur.take<int>((size_t)(pieces + 1));
  cur.take<char>(0);
  w.bytes = cur.offset;
  return w;
}

}  // namespace

size_t head_forward_workspace_bytes(int64_t T, int64_t V) {
  WsCursor cur;
  cur.take<float2>((size_t)(ceil_div(V, kHalf) * T));
  cur.take<char>(0);
  return cur.offset;
}

cudaError_t launch_head_forward(const HeadForward& f, void* ws, cudaStream_t stream) {
  WsCursor cur;
  cur.base = static_cast<char*>(ws);
  const int blocks = (int)ceil_div(f.V, kHalf);
  HeadLaunch a = {};
  a.partials = cur.take<float2>((size_t)(blocks * f.T));
  cudaError_t err = device_error_word(&a.err);
  if (err != cudaSuccess) return err;
  a.n = 1;
  a.T = f.T;
  a.targets = f.targets;
  a.scale_log2 = f.scale * kLog2e;
  Product& p = a.p[0];
  p.M = (int)f.T;
  p.N = (int)f.V;
  p.K = (int)f.k;
  p.epi = kEpiStats;
  p.splits = 1;
  p.a_box = a_box(f.T);
  err = k_major(&p.tmA, f.X, f.T, f.k, f.ld_x, p.a_box);
  if (err == cudaSuccess) err = k_major(&p.tmB, f.W, f.V, f.k, f.ld_w);
  if (err == cudaSuccess) err = launch_products(a, stream);
  if (err != cudaSuccess) return err;
  return launch_after(head_combine_kernel, (unsigned)ceil_div(f.T, kCombineRows), 256, 0, stream, a.partials, f.X,
                      f.ld_x, f.W, f.ld_w, f.k, f.targets, f.scale, a.scale_log2, f.T, f.V, blocks, f.loss, f.lse,
                      f.dev_status);
}

size_t head_backward_workspace_bytes(int64_t T, int64_t V, int64_t k, int64_t r) {
  return carve_backward(nullptr, T, V, k, r).bytes;
}

cudaError_t launch_head_backward(const HeadBackward& f, void* ws, cudaStream_t stream) {
  const bool sketch = f.C != nullptr;
  const BackwardWorkspace w = carve_backward(ws, f.T, f.V, f.k, sketch ? f.r : 0);
  const int64_t rows = round_up(f.T, kTile), piece = piece_width(f.T, f.V);
  const int pieces = (int)ceil_div(f.V, piece);

  // Few tokens' rounding errors do not average out in dW, and D's tile has room
  // beside them for what its entries lose (120 x 2048 x 32768: 219 us, 211 without)
  const int two_terms = f.T <= kHalf && (f.dW || sketch);
  Gather g = {};
  g.X = f.X; g.T = f.T; g.k = f.k; g.ld_x = f.ld_x;
  g.XP = sketch ? f.XP : nullptr; g.ld_xp = f.ld_xp; g.r = f.r;
  g.W = f.W; g.V = f.V; g.ld_w = f.ld_w; g.targets = f.targets; g.lse = f.lse; g.g = f.g; g.scale = f.scale;
  g.Xc = w.Xc; g.XPc = w.XPc; g.ld_xpc = w.ld_xpc;
  g.lse_log2 = w.lse_log2; g.weight = w.weight; g.factor = w.factor; g.target = w.target; g.hit = w.hit;
  g.row_of = w.row_of; g.kept = w.kept;
  g.dX = f.dX; g.ld_dx = f.ld_dx;
  g.counters = w.counters; g.n_counters = pieces + 1;
  g.two_terms = two_terms; g.rows = rows; g.all_rows = sketch; g.status = f.dev_status;
  g.per_block = 8 * (int)(ceil_div(rows, 8192) < 64 ? ceil_div(rows, 8192) : 64);
  cudaError_t err = launch_after(head_gather_kernel, (unsigned)ceil_div(rows, g.per_block), 256, 0, stream, g);
  if (err != cudaSuccess) return err;

  HeadLaunch a = {};
  err = device_error_word(&a.err);
  if (err != cudaSuccess) return err;
  a.kept = w.kept;
  a.T = f.T;
  a.scale_log2 = f.scale * kLog2e;
  a.lse_log2 = w.lse_log2;
  a.weight = w.weight;
  a.factor = w.factor;
  a.two_terms = two_terms;
  a.rest = w.rest;
  a.W = f.W;
  a.ld_w = f.ld_w;
  a.target = w.target;
  a.hit = w.hit;
  a.row_of = w.row_of;
  a.ld_d = piece;
  a.dX = f.dX;
  a.ld_dx = f.ld_dx;
  a.ld_dw = f.ld_dw;
  a.dw_mode = f.dw_type == SKETCH_BF16 ? 0 : f.overwrite ? 1 : 2;
  int dx_sum_parts = 0;
  // step i: dX and dW of piece i - 1, and D of piece i
  for (int i = 0; i <= pieces; ++i) {
    a.n = 0;
    a.counter = w.counters + i;
    if (i > 0) {
      const int64_t v0 = (i - 1) * piece, width = f.V - v0 < piece ? f.V - v0 : piece;
      const uint16_t* D = w.D[(i - 1) & 1];
      if (f.dX) {
        Product& p = a.p[a.n++];
        p = Product{};
        p.a_box = a_box(f.T);
        err = k_major(&p.tmA, D, rows, width, piece, p.a_box);
        if (err == cudaSuccess) err = mn_major(&p.tmB, f.W, f.k, f.V, f.ld_w);
        if (err != cudaSuccess) return err;
        p.b_mn = 1;
        p.b_k = (int)v0;
        p.M = (int)f.T;
        p.kept_m = 1;
        p.N = (int)f.k;
        p.K = (int)width;
        p.epi = kEpiDx;
        p.splits = w.parts < ceil_div(width, kChunk) ? w.parts : (int)ceil_div(width, kChunk);  // a chunk each at least
        dx_sum_parts += p.splits;
        a.acc = w.acc + (w.parts > 1 ? (i - 1) * w.parts * rows * f.k : 0);
        a.acc_part = rows * f.k;
        a.dx_first = i == 1 || w.parts > 1;
        a.dx_last = i == pieces && w.parts == 1;
      }
      if (f.dW) {
        Product& p = a.p[a.n++];
        p = Product{};
        p.a_box = kHalf;
        err = mn_major(&p.tmA, D, width, rows, piece);
        if (err == cudaSuccess) err = mn_major(&p.tmB, w.Xc, f.k, rows, f.k);
        if (err != cudaSuccess) return err;
        p.a_mn = p.b_mn = 1;
        p.M = (int)width;
        p.N = (int)f.k;
        p.K = (int)f.T;
        p.kept_k = 1;
        p.epi = kEpiDw;
        p.splits = 1;
        const size_t size = f.dw_type == SKETCH_BF16 ? 2 : 4;
        a.dW = static_cast<char*>(f.dW) + (size_t)(v0 * f.ld_dw) * size;
      }
      if (sketch) {
        AccumulateProblem ap = {D, rows, width, piece, w.XPc, w.ld_xpc, w.S};
        err = launch_accumulate(1, &ap, (int)f.r, 1, stream);
        if (err != cudaSuccess) return err;
        const int64_t n = width * f.r, blocks = ceil_div(n, 256), most = 8 * (int64_t)num_sms();
        count_launch();
        head_sketch_add_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(w.S, n, w.factor, f.overwrite,
                                                                                            f.C + v0 * f.r);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
      }
    }
    if (i < pieces) {
      const int64_t v0 = i * piece, width = f.V - v0 < piece ? f.V - v0 : piece;
      Product& p = a.p[a.n++];
      p = Product{};
      p.a_box = a_box(sketch ? rows : f.T);
      err = k_major(&p.tmA, w.Xc, rows, f.k, f.k, p.a_box);
      if (err == cudaSuccess) err = k_major(&p.tmB, f.W, f.V, f.k, f.ld_w);
      if (err != cudaSuccess) return err;
      p.b_row = (int)v0;
      p.M = (int)(sketch ? rows : f.T);
      p.kept_m = !sketch;  // the sketch's sum runs over every compact row
      p.N = (int)width;
      p.K = (int)f.k;
      p.epi = kEpiDlogit;
      p.splits = 1;
      a.D = w.D[i & 1];
      a.d_first = (int)v0;
    }
    if (a.n > 0) {
      err = launch_products(a, stream);
      if (err != cudaSuccess) return err;
    }
  }
  if (f.dX && w.parts > 1) {
    const int64_t blocks = ceil_div(f.T * (f.k / 8), 256), most = 8 * (int64_t)num_sms();
    return launch_after(head_dx_sum_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, stream, w.acc,
                        rows * f.k, dx_sum_parts, f.k, w.kept, w.factor, w.row_of, w.target, w.rest, f.W, f.ld_w,
                        f.dX, f.ld_dx);
  }
  return cudaSuccess;
}

}  // namespace rgs
