// Tensor memory beside shared memory: how much of an SM's each kernel takes.
//
// tcgen05.alloc waits, without a limit, until the SM has the columns.  A block that waits
// so while its cluster's other blocks hold columns on other SMs can wait for a cluster
// that waits for those.  So no block of a cluster ever finds fewer columns than it wants
// because other clusters' blocks hold them, whatever streams the launches are on.  What
// bounds the blocks of an SM is its shared memory, and every kernel that takes TMEM asks
// for so much of it (tmem_safe) that one of these holds for its blocks:
//   alone  no other block that takes TMEM fits beside it;
//   share  it has at least the part of the SM's shared memory that its columns are of the
//          SM's TMEM (in clusters, a quarter of the SM at least);
//   half   it is in no cluster and has more than half of the shared memory.
// Of the blocks on an SM let two or more be in clusters.  None is `alone`, and none is
// `half`, which two quarters leave no place for.  So all have their shares, and their columns
// add up to no more than there are.  With a single cluster's block on the SM the others
// are in no cluster: they wait for nobody but each other and it, and never while they
// hold columns, so that those that hold some end.
#pragma once

#include "internal.h"

namespace rgs {

constexpr size_t kSmSmem = 228u << 10;     // shared memory of an SM
constexpr size_t kBlockSmem = 1u << 10;    // of it, the system's for each block
constexpr uint32_t kSmTmem = 512;          // TMEM columns of an SM
constexpr size_t kTmemLeast = 38u << 10;   // no kernel that takes TMEM has blocks with less: triangular products, rank 16

// Shared memory of an SM for its part of this many columns.
constexpr size_t tmem_share(uint32_t columns) { return kSmSmem / kSmTmem * columns; }

// `bytes`: dynamic, static and the system's.
constexpr bool tmem_safe(uint32_t columns, size_t bytes, bool clusters) {
  if (columns > kSmTmem || bytes < kTmemLeast || bytes > kSmSmem) return false;
  if (bytes + kTmemLeast > kSmSmem) return true;
  if (bytes >= tmem_share(columns)) return !clusters || 4 * bytes >= kSmSmem;
  return !clusters && 2 * bytes > kSmSmem;
}

// Dynamic shared memory beside `fixed` static bytes: `want`, and the share of the columns at least.
constexpr size_t tmem_smem(uint32_t columns, size_t fixed, size_t want) {
  const size_t least = tmem_share(columns) - kBlockSmem - fixed;
  return want < least ? least : want;
}

// Columns are taken as a power of two, 32 at least.
constexpr uint32_t tmem_cols_for(int n) {
  uint32_t c = 32;
  while ((int)c < n) c <<= 1;
  return c;
}

// ---- products with a projection or a sketch (skinny.cu) ------------------------------
constexpr int kSkinnyMaxStages = 8;

struct SkinnySizes {
  uint32_t stage_bytes;
  int stages;
  int red_stride;      // floats per row of the reduction tile
  uint32_t tmem_cols;
  size_t smem;         // dynamic
};
// Clusters that split K: `operands` tiles of B, b_bytes each, beside one of A in a stage.
inline SkinnySizes skinny_sizes(int n_pad, uint32_t a_bytes, uint32_t b_bytes, int operands, size_t fixed) {
  SkinnySizes z;
  z.stage_bytes = a_bytes + operands * b_bytes;
  // two CTAs per SM when the stages fit in half of shared memory; stages wider
  // than 48 KB (a B of 192+ rank columns, as grouped projections have) get
  // the whole SM, since two of them per CTA would leave too few K chunks in
  // flight to cover the loads
  const uint32_t budget = z.stage_bytes > 48u * 1024u ? 208u * 1024u : 96u * 1024u;
  z.stages = (int)(budget / z.stage_bytes);
  if (z.stages < 2) z.stages = 2;
  if (z.stages > kSkinnyMaxStages) z.stages = kSkinnyMaxStages;
  z.red_stride = (n_pad + 31) / 32 * 32 + 4;
  z.tmem_cols = tmem_cols_for(n_pad);
  size_t smem = (size_t)z.stages * z.stage_bytes;
  const size_t red_bytes = (size_t)128 * z.red_stride * sizeof(float);
  if (red_bytes > smem) smem = red_bytes;
  // at most two CTAs per SM
  if (smem < 80 * 1024) smem = 80 * 1024;
  smem += 1024;  // alignment slack
  z.smem = tmem_smem(z.tmem_cols, fixed, smem);
  return z;
}

// Persistent CTAs, one per SM.
struct PersistentSizes {
  uint32_t stage_bytes;
  int stages;          // below two: the launch is refused
  uint32_t tmem_cols;
  size_t smem;         // dynamic
};
inline PersistentSizes persistent_sizes(uint32_t stage_bytes, int columns) {
  PersistentSizes z;
  z.stage_bytes = stage_bytes;
  z.stages = (int)((200u * 1024u) / stage_bytes);
  if (z.stages > kSkinnyMaxStages) z.stages = kSkinnyMaxStages;
  z.tmem_cols = tmem_cols_for(columns);
  z.smem = (size_t)z.stages * stage_bytes + 1024;
  return z;
}
// Sketches: strips of `tiles` tiles of 128 rows, two TMEM buffers.
inline PersistentSizes accumulate_sizes(int n_pad, uint32_t b_bytes, int tiles, int operands) {
  return persistent_sizes(tiles * 16384u + operands * b_bytes, 2 * tiles * n_pad);
}
// Projected inputs.
struct ProjectSizes {
  int chunks;     // 64-wide K chunks per stage
  bool stack;     // both parts of the split in one MMA
  int k_parts;    // partial accumulators per tile
  int acc_bufs;   // tiles in flight
  PersistentSizes p;
};
inline ProjectSizes project_sizes(int n_pad, uint32_t a_bytes, uint32_t b_bytes) {
  ProjectSizes z;
  // two 64-wide K chunks per stage (longer runs of each token row of X, half
  // the per-stage work of the issuing threads) where three such stages fit
  const uint32_t one = a_bytes + 2 * b_bytes;
  z.chunks = (3 * 2 * one <= 200u * 1024u) ? 2 : 1;
  // both parts of the split in one MMA (N = 2 n_pad): half the MMA
  // instructions.  Up to rank 64 this keeps two tiles of accumulators in
  // TMEM; above, the wider accumulators would leave room for one tile only,
  // which measured slower than twice the MMAs (rank 128: 0.66 against 0.67 of HBM)
  z.stack = n_pad <= 64;
  const int acc_n = z.stack ? 2 * n_pad : n_pad;
  // partial accumulators: up to 4 per tile, two tiles in flight where TMEM
  // holds them, else one tile of two
  z.acc_bufs = 2;
  z.k_parts = 4;
  while (z.k_parts > 1 && z.acc_bufs * z.k_parts * acc_n > 512) z.k_parts >>= 1;
  if (z.k_parts == 1) {
    z.acc_bufs = 1;
    z.k_parts = 2;
  }
  z.p = persistent_sizes(z.chunks * one, z.acc_bufs * z.k_parts * acc_n);
  return z;
}

// ---- Gram matrices (gram.cu) ------------------------------------------------------------
constexpr int kGtcStep = 64;  // rows per step: one 128-byte swizzled row of FP16 per column of A
constexpr int kGtcMaxRaw = 4;
__host__ __device__ inline int gtc_mpad(int r) { return r <= 128 ? 128 : 256; }
__host__ __device__ inline int gtc_npad(int r) { return (r + 15) / 16 * 16; }
// TMEM columns: the accumulators (nacc x M halves x npad), and at least the
// span the epilogue's 32-column reads cover
__host__ __device__ inline uint32_t gtc_tmem_cols(int r) {
  const int npad = gtc_npad(r), nmh = gtc_mpad(r) / 128, nacc = gram_tc_accs(r);
  const int reads = (nacc * nmh - 1) * npad + (npad + 31) / 32 * 32;
  const int cols = nacc * nmh * npad > reads ? nacc * nmh * npad : reads;
  uint32_t c = 32;
  while ((int)c < cols) c <<= 1;
  return c;
}
struct GramSizes {
  int raw_stages;  // of the ring of fp32 row copies (0: none)
  size_t smem;     // dynamic
};
inline GramSizes gram_sizes(int r, size_t fixed) {
  // two buffers of two tiles, or more, so that the blocks resident on an SM never ask
  // for more than its 512 TMEM columns
  const size_t tiles = (size_t)4 * gtc_mpad(r) * 128 + 1024;
  const uint32_t columns = gtc_tmem_cols(r);
  const size_t max_blocks = kSmTmem / columns;
  GramSizes z;
  z.smem = max_blocks > 1 ? tmem_smem(columns, fixed, tiles) : kSmSmem / 2 - kBlockSmem + 16;
  if (z.smem < tiles) z.smem = tiles;
  // the ring in what the blocks an SM's TMEM admits leave (each block also holds 1 KB
  // reserved by the system and the kernel's static shared memory)
  const size_t per_block = kSmSmem / max_blocks - kBlockSmem - fixed;
  const size_t raw_bytes = (size_t)kGtcStep * r * 4;
  z.raw_stages = per_block > tiles ? (int)((per_block - tiles) / raw_bytes) : 0;
  if (z.raw_stages > kGtcMaxRaw) z.raw_stages = kGtcMaxRaw;
  if (z.raw_stages < 2 || r > 128) z.raw_stages = 0;
  return z;
}
// With the ring.
inline size_t gram_ring_smem(const GramSizes& z, int r, int raw_stages) {
  const size_t with = (size_t)4 * gtc_mpad(r) * 128 + 1024 + (size_t)raw_stages * kGtcStep * r * 4;
  return raw_stages > 0 && with > z.smem ? with : z.smem;
}

// ---- triangular products (projection.cu) --------------------------------------------------
__host__ __device__ inline int ttc_npad(int r) { return (r + 15) / 16 * 16; }
__host__ __device__ inline int ttc_kc(int r) { return (ttc_npad(r) + 63) / 64; }
// chunks of X^T held at once: all of them up to rank 128, else one at a time
__host__ __device__ inline int ttc_bchunks(int r) { return ttc_kc(r) <= 2 ? ttc_kc(r) : 1; }
__host__ __device__ inline size_t ttc_smem_bytes(int r) {
  return (size_t)ttc_kc(r) * 2 * 16384 + (size_t)ttc_bchunks(r) * 2 * ttc_npad(r) * 128 + 1024;
}
__host__ __device__ inline uint32_t ttc_tmem_cols(int r) {
  uint32_t c = 32;
  while ((int)c < ttc_npad(r)) c <<= 1;
  return c;
}

// ---- updates (update.cu) --------------------------------------------------------------------
constexpr int kMaxStagesUpd = 8;
constexpr int kTmemBufs = 4;                      // accumulator tiles in flight
struct UpdateSizes {
  int p_stages, w_stages;  // w_stages below one: the launch is refused
  size_t smem;             // dynamic
};
// What the opt-in limit leaves next to the static arrays: `c_bytes` of C, P stages of
// p_stage bytes, and the rest for the ring of W tiles.
inline UpdateSizes update_sizes(int kchunks, size_t c_bytes, size_t p_stage, size_t w_bytes, size_t fixed_smem) {
  const size_t max_smem = 227 * 1024 - fixed_smem;
  const size_t fixed = c_bytes + 1024;
  UpdateSizes z;
  // P stages (each one 64-wide chunk of r): up to rank 128 two, when they
  // still leave three W stages (W comes from HBM and needs the deeper ring),
  // else one; above, as many as leave two W stages (rank 256: a tile's four
  // chunks, 4% faster than two).  The rest of shared memory goes to the W ring.
  z.p_stages = (fixed + 2 * p_stage + 3 * w_bytes <= max_smem) ? 2 : 1;
  if (kchunks > 2) {
    z.p_stages = 2 * kchunks;
    while (z.p_stages > 1 && fixed + z.p_stages * p_stage + 2 * w_bytes > max_smem) --z.p_stages;
  }
  z.w_stages = (int)((max_smem - fixed - z.p_stages * p_stage) / w_bytes);
  if (z.w_stages > kMaxStagesUpd) z.w_stages = kMaxStagesUpd;
  z.smem = fixed + z.p_stages * p_stage + (size_t)(z.w_stages < 1 ? 0 : z.w_stages) * w_bytes;
  return z;
}

// ---- 8-bit products of few tokens (matmul8.cu) -----------------------------------------------
constexpr int few_buffers(int TN) { return TN == 64 ? 4 : 8; }
constexpr uint32_t few_columns(int TN) { return TN * few_buffers(TN); }  // of TMEM: 128 or 256 of 512
// CTAs per SM: as many as TMEM has columns for (16 tokens, 12288 x 4096: 12.1 us with four,
// 14 to 15 with two).
constexpr int few_resident(int TN) { return (int)(kSmTmem / few_columns(TN)); }
// Dynamic shared memory of a launch, whatever it needs: its columns' share.
constexpr size_t few_smem(int TN, size_t fixed) { return tmem_smem(few_columns(TN), fixed, 0); }

// ---- pairs of CTAs that take all of TMEM (matmul8.cu, head.cu) -------------------------------
constexpr bool tmem_alone(size_t dynamic) { return tmem_safe(kSmTmem, dynamic + kBlockSmem, true); }

}  // namespace rgs
