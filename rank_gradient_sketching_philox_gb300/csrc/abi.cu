// C ABI of the sketching library: argument checks, workspace carving and
// dispatch to the kernels.  Every check happens on the host before anything is
// launched; see include/sketch.h for the contract of each entry point.
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <vector>

#include "common.cuh"
#include "internal.h"
#include "sketch.h"

namespace {

thread_local char g_last_error[512] = "";

sketch_status fail(sketch_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

sketch_status ok() {
  g_last_error[0] = '\0';
  return SKETCH_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define CHECK_PTR(p)                                                                   \
  do {                                                                                 \
    if ((p) == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "%s is NULL", #p);         \
    if (!aligned16(p)) return fail(SKETCH_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

#define CHECK_OPT_ALIGN(p, a)                                                          \
  do {                                                                                 \
    if ((p) != nullptr && (reinterpret_cast<uintptr_t>(p) % (a)) != 0)                \
      return fail(SKETCH_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, (int)(a));  \
  } while (0)

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

sketch_status check_dim(const char* name, int64_t v) {
  if (v < 1 || v > kMaxDim) return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld out of [1, 2^31)", name, (long long)v);
  return SKETCH_OK;
}

sketch_status check_rank(int64_t r) {
  if (r < 1 || r > rgs::kMaxRank)
    return fail(SKETCH_ERR_INVALID_ARG, "r=%lld out of [1, %d]", (long long)r, rgs::kMaxRank);
  return SKETCH_OK;
}

sketch_status check_ld(const char* name, int64_t ld, int64_t width) {
  if (ld < width) return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld < row width %lld", name, (long long)ld, (long long)width);
  if (ld % 8 != 0) return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld is not a multiple of 8", name, (long long)ld);
  if (ld > kMaxDim) return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld too large", name, (long long)ld);
  return SKETCH_OK;
}

sketch_status check_k(int64_t k) {
  sketch_status st = check_dim("k", k);
  if (st) return st;
  if (k % 8 != 0) return fail(SKETCH_ERR_INVALID_ARG, "k=%lld is not a multiple of 8", (long long)k);
  return SKETCH_OK;
}

sketch_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return SKETCH_OK;
  if (ws == nullptr) return fail(SKETCH_ERR_WORKSPACE, "workspace of %zu bytes required, got NULL", need);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(SKETCH_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need) return fail(SKETCH_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, need);
  return SKETCH_OK;
}

sketch_status launch_result(cudaError_t err, const char* what) {
  if (err != cudaSuccess) return fail(SKETCH_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
  return ok();
}

#define TRY(expr)                  \
  do {                             \
    sketch_status st_ = (expr);    \
    if (st_ != SKETCH_OK) return st_; \
  } while (0)

size_t qr_ws_bytes(int64_t k, int64_t r) {
  rgs::WsCursor cur;
  rgs::carve_qr_workspace(cur, k, (int)r, nullptr);
  cur.take<int32_t>(1);  // scratch status word
  cur.take<char>(0);
  return cur.offset;
}

size_t update_ws_bytes(bool normsgd, int64_t d, int64_t k, int64_t r) {
  rgs::WsCursor cur;
  return rgs::carve_update_workspace(cur, d, k, (int)r, normsgd, nullptr);
}

// Cross entropy: tokens, vocabulary and width whose tile coordinates and numbers of tiles stay below 2^31.
bool head_sizes_ok(int64_t T, int64_t V, int64_t k) {
  if (T < 1 || T > rgs::kMaxHeadDim || V < 1 || V > rgs::kMaxHeadDim || k < 8 || k % 8 != 0 || k > rgs::kMaxHeadDim)
    return false;
  const int64_t t = rgs::ceil_div(T, 256), v = rgs::ceil_div(V, 256), w = rgs::ceil_div(k, 256);
  return t * v <= rgs::kMaxHeadTiles && t * w <= rgs::kMaxHeadTiles && v * w <= rgs::kMaxHeadTiles;
}

size_t op_ws_bytes(sketch_op op, int64_t T, int64_t d, int64_t k, int64_t r) {
  switch (op) {  // the training operators, whose sizes are checked as the calls check them
    case SKETCH_OP_LAYER_NORM_BACKWARD:
      return (T >= 1 && T <= kMaxDim && k >= 1 && k <= kMaxDim) ? rgs::norm_backward_workspace_bytes(T, k) : 0;
    case SKETCH_OP_CROSS_ENTROPY_FORWARD:
      return head_sizes_ok(T, d, 8) ? rgs::head_forward_workspace_bytes(T, d) : 0;
    case SKETCH_OP_CROSS_ENTROPY_BACKWARD:
      return (head_sizes_ok(T, d, k) && r >= 0 && r <= rgs::kMaxRank)
                 ? rgs::head_backward_workspace_bytes(T, d, k, r)
                 : 0;
    case SKETCH_OP_RMS_NORM_BACKWARD:
      return (T >= 1 && T <= kMaxDim && k >= 1 && k <= kMaxDim) ? rgs::rms_backward_workspace_bytes(T, k) : 0;
    case SKETCH_OP_GRAD_NORM: return (T >= 1 && T <= (1 << 20)) ? rgs::grad_norm_workspace_bytes(T) : 0;
    default: break;
  }
  if (r < 1 || r > rgs::kMaxRank) return 0;
  switch (op) {
    case SKETCH_OP_SAMPLE_PROJECTION: return (k >= 1) ? qr_ws_bytes(k, r) : 0;
    case SKETCH_OP_PROJECT_INPUTS: return (T >= 1 && k >= 1) ? rgs::project_workspace_bytes(T, k, r) : 0;
    case SKETCH_OP_ACCUMULATE: return (T >= 1 && d >= 1) ? rgs::accumulate_workspace_bytes(T, d, r) : 0;
    case SKETCH_OP_UPDATE_NORMSGD: return (d >= 1 && k >= 1) ? update_ws_bytes(true, d, k, r) : 0;
    case SKETCH_OP_UPDATE_SGD: return (d >= 1 && k >= 1) ? update_ws_bytes(false, d, k, r) : 0;
    default: break;
  }
  return 0;
}

sketch_status check_n(int n) {
  if (n < 1 || n > (1 << 20)) return fail(SKETCH_ERR_INVALID_ARG, "n=%d out of [1, 2^20]", n);
  return SKETCH_OK;
}

// ---- per-problem checks ------------------------------------------------------
sketch_status check_projection(const sketch_projection_problem& p) {
  TRY(check_k(p.k));
  CHECK_PTR(p.P);
  return SKETCH_OK;
}

sketch_status check_project(const sketch_project_problem& p, int64_t r) {
  TRY(check_dim("T", p.T));
  TRY(check_k(p.k));
  TRY(check_ld("ld_x", p.ld_x, p.k));
  TRY(check_ld("ld_xp", p.ld_xp, r));
  CHECK_PTR(p.X);
  if (p.P == nullptr && p.P_split == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "P and P_split are both NULL");
  CHECK_PTR(p.XP);
  return SKETCH_OK;
}

sketch_status check_accumulate(const sketch_accumulate_problem& p, int64_t r) {
  TRY(check_dim("T", p.T));
  TRY(check_dim("d", p.d));
  TRY(check_ld("ld_d", p.ld_d, p.d));
  TRY(check_ld("ld_xp", p.ld_xp, r));
  CHECK_PTR(p.D);
  CHECK_PTR(p.XP);
  CHECK_PTR(p.C);
  return SKETCH_OK;
}

sketch_status check_update(const sketch_update_problem& p) {
  TRY(check_dim("d", p.d));
  TRY(check_k(p.k));
  TRY(check_ld("ld_w", p.ld_w, p.k));
  CHECK_PTR(p.W);
  CHECK_PTR(p.C);
  CHECK_PTR(p.P);
  CHECK_OPT_ALIGN(p.wnorm2_in, 8);
  CHECK_OPT_ALIGN(p.wnorm2_out, 8);
  CHECK_OPT_ALIGN(p.dev_status, 4);
  if (p.d * p.k >= (int64_t(1) << 40)) return fail(SKETCH_ERR_INVALID_ARG, "d*k too large");
  if ((p.d * p.k) / 8 > (int64_t)UINT32_MAX)
    return fail(SKETCH_ERR_INVALID_ARG, "d*k exceeds the 2^35 weights one rounding stream covers");
  return SKETCH_OK;
}

// ---- batched implementations --------------------------------------------------
sketch_status do_sample(sketch_proj_kind kind, uint64_t seed, uint32_t step, int n,
                        const sketch_projection_problem* probs, int64_t r, int32_t* dev_status, void* ws,
                        size_t ws_bytes, cudaStream_t s) {
  if (kind != SKETCH_PROJ_RADEMACHER && kind != SKETCH_PROJ_GAUSSIAN_QR)
    return fail(SKETCH_ERR_INVALID_ARG, "unknown projection kind %d", (int)kind);
  TRY(check_n(n));
  if (probs == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  TRY(check_rank(r));
  CHECK_OPT_ALIGN(dev_status, 4);
  size_t need = 0;
  for (int i = 0; i < n; ++i) {
    TRY(check_projection(probs[i]));
    if (probs[i].k * r > (int64_t(1) << 34)) return fail(SKETCH_ERR_INVALID_ARG, "k*r too large");
    if (kind == SKETCH_PROJ_GAUSSIAN_QR) {
      if (r > probs[i].k)
        return fail(SKETCH_ERR_INVALID_ARG, "Gaussian-QR projection needs r <= k (k=%lld, r=%lld)",
                    (long long)probs[i].k, (long long)r);
      need += qr_ws_bytes(probs[i].k, r);
    }
  }
  if (kind == SKETCH_PROJ_GAUSSIAN_QR) TRY(check_ws(ws, ws_bytes, need));
  // Up to two batches are filled at once: CholeskyQR2 frames (and Rademacher
  // draws) in `batch`, fp64 Householder frames (r <= k < 4r) in `wide`; each is
  // launched when full and at the end.
  static thread_local rgs::ProjBatch batch, wide;
  for (rgs::ProjBatch* b : {&batch, &wide}) {
    b->n = 0;
    b->r = (int)r;
    b->seed = seed;
    rgs::philox_round_keys(seed, b->rk0, b->rk1);
    b->step = step;
  }
  rgs::WsCursor cur;
  cur.base = static_cast<char*>(ws);
  int32_t* status = dev_status;
  cudaError_t err = cudaSuccess;
  int64_t max_k = 0;
  auto flush = [&](rgs::ProjBatch& b) {
    if (b.n == 0 || err != cudaSuccess) return;
    if (kind == SKETCH_PROJ_RADEMACHER) {
      err = rgs::launch_rademacher(b, max_k, s);
    } else {
      b.status = status;
      err = (&b == &wide) ? rgs::launch_wide_qr(b, s) : rgs::launch_gaussian_qr(b, max_k, s);
    }
    if (&b == &batch) max_k = 0;
    b.n = 0;
  };
  for (int i = 0; i < n && err == cudaSuccess; ++i) {
    const sketch_projection_problem& pr = probs[i];
    const bool is_wide = kind == SKETCH_PROJ_GAUSSIAN_QR && rgs::qr_is_wide(pr.k, r);
    rgs::ProjBatch& b = is_wide ? wide : batch;
    rgs::ProjProblem& pb = b.p[b.n++];
    pb.P = pr.P;
    pb.k = pr.k;
    pb.layer = pr.layer;
    if (kind == SKETCH_PROJ_RADEMACHER) {
      pb.scale = (float)(1.0 / std::sqrt((double)r));
    } else {
      rgs::carve_qr_workspace(cur, pr.k, (int)r, &pb);
      int32_t* scratch = cur.take<int32_t>(1);
      cur.take<char>(0);
      if (status == nullptr) status = scratch;
      pb.scale = (float)std::sqrt((double)pr.k / (double)r);
      if (i == 0) err = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    }
    if (!is_wide) max_k = pr.k > max_k ? pr.k : max_k;
    if (b.n == rgs::kMaxBatch) flush(b);
  }
  flush(batch);
  flush(wide);
  if (err == cudaSuccess && kind == SKETCH_PROJ_RADEMACHER && dev_status)
    err = cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s);
  return launch_result(err, "sample_projection");
}

// XP width: r columns, or the BF16 pair of the fp32-accurate form (2 * round16(r)).
int64_t xp_width(int64_t r, bool xp_split) { return xp_split ? 2 * ((r + 15) / 16 * 16) : r; }

sketch_status do_project(int n, const sketch_project_problem* probs, int64_t r, void* ws, size_t ws_bytes,
                         cudaStream_t s, bool xp_split = false) {
  TRY(check_n(n));
  if (probs == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  TRY(check_rank(r));
  size_t need = 0;
  std::vector<rgs::ProjectProblem> v((size_t)n);
  for (int i = 0; i < n; ++i) {
    TRY(check_project(probs[i], r));
    TRY(check_ld("ld_xp", probs[i].ld_xp, xp_width(r, xp_split)));
    need += rgs::project_workspace_bytes(probs[i].T, probs[i].k, r);
    v[i] = rgs::ProjectProblem{probs[i].X, probs[i].T, probs[i].k, probs[i].ld_x, probs[i].P, probs[i].XP,
                               probs[i].ld_xp, probs[i].P_split};
  }
  TRY(check_ws(ws, ws_bytes, need));
  return launch_result(rgs::launch_project_inputs(n, v.data(), (int)r, ws, s, xp_split), "project_inputs");
}

sketch_status do_accumulate(int n, const sketch_accumulate_problem* probs, int64_t r, int overwrite, void* ws,
                            size_t ws_bytes, cudaStream_t s, bool xp_split = false) {
  TRY(check_n(n));
  if (probs == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  TRY(check_rank(r));
  if (overwrite != 0 && overwrite != 1) return fail(SKETCH_ERR_INVALID_ARG, "overwrite must be 0 or 1");
  size_t need = 0;
  std::vector<rgs::AccumulateProblem> v((size_t)n);
  for (int i = 0; i < n; ++i) {
    TRY(check_accumulate(probs[i], r));
    TRY(check_ld("ld_xp", probs[i].ld_xp, xp_width(r, xp_split)));
    need += rgs::accumulate_workspace_bytes(probs[i].T, probs[i].d, r);
    v[i] = rgs::AccumulateProblem{probs[i].D, probs[i].T, probs[i].d, probs[i].ld_d, probs[i].XP, probs[i].ld_xp,
                                  probs[i].C};
  }
  TRY(check_ws(ws, ws_bytes, need));
  return launch_result(rgs::launch_accumulate(n, v.data(), (int)r, overwrite, s, xp_split), "accumulate");
}

sketch_status do_update(bool normsgd, int n, const sketch_update_problem* probs, int64_t r, float step_size,
                        uint64_t seed, uint32_t step, void* ws, size_t ws_bytes, cudaStream_t s) {
  TRY(check_n(n));
  if (probs == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  TRY(check_rank(r));
  if (!std::isfinite(step_size)) return fail(SKETCH_ERR_INVALID_ARG, "%s is not finite", normsgd ? "tau" : "alpha_eta");
  size_t need = 0;
  for (int i = 0; i < n; ++i) {
    TRY(check_update(probs[i]));
    need += update_ws_bytes(normsgd, probs[i].d, probs[i].k, r);
  }
  TRY(check_ws(ws, ws_bytes, need));
  std::vector<rgs::UpdateProblem> v((size_t)n);
  std::vector<rgs::UpdateWorkspace> w((size_t)n);
  rgs::WsCursor cur;
  cur.base = static_cast<char*>(ws);
  for (int i = 0; i < n; ++i) {
    const sketch_update_problem& p = probs[i];
    v[i] = rgs::UpdateProblem{p.W, p.d, p.k, p.ld_w, p.C, p.P, p.layer,
                              normsgd ? p.wnorm2_in : nullptr, normsgd ? p.wnorm2_out : nullptr, p.dev_status};
    rgs::carve_update_workspace(cur, p.d, p.k, (int)r, normsgd, &w[i]);
  }
  cudaError_t err = normsgd ? rgs::launch_update_normsgd(n, v.data(), w.data(), (int)r, step_size, seed, step, s)
                            : rgs::launch_update_sgd(n, v.data(), w.data(), (int)r, step_size, seed, step, s);
  return launch_result(err, normsgd ? "apply_update_normsgd" : "apply_update_sgd");
}

// ---- training operators ---------------------------------------------------------
bool is_dtype(int t) { return t == SKETCH_BF16 || t == SKETCH_FP32; }

#define CHECK_DTYPE(t)                                                                      \
  do {                                                                                      \
    if (!is_dtype((int)(t))) return fail(SKETCH_ERR_INVALID_ARG, "unknown %s %d", #t, (int)(t)); \
  } while (0)

#define CHECK_ELEM_PTR(p, type)                                                             \
  do {                                                                                      \
    if ((p) == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "%s is NULL", #p);              \
    CHECK_OPT_ALIGN(p, (type) == SKETCH_BF16 ? 2 : 4);                                      \
  } while (0)

// A row stride of the layer norm: at least the row, no alignment of its own.
sketch_status check_row_stride(const char* name, int64_t ld, int64_t width) {
  if (ld < width || ld > kMaxDim)
    return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld out of [%lld, 2^31)", name, (long long)ld, (long long)width);
  return SKETCH_OK;
}

sketch_status check_head(const uint16_t* X, int64_t T, int64_t k, int64_t ld_x, const uint16_t* W, int64_t V,
                         int64_t ld_w, const int64_t* targets, float scale, const int32_t* dev_status) {
  TRY(check_dim("T", T));
  TRY(check_dim("V", V));
  TRY(check_k(k));
  if (!head_sizes_ok(T, V, k))
    return fail(SKETCH_ERR_UNSUPPORTED, "T=%lld, V=%lld, k=%lld: one exceeds 2^24, or two have more than 2^28 tiles of 256 x 256",
                (long long)T, (long long)V, (long long)k);
  TRY(check_ld("ld_x", ld_x, k));
  TRY(check_ld("ld_w", ld_w, k));
  CHECK_PTR(X);
  CHECK_PTR(W);
  if (targets == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "targets is NULL");
  CHECK_OPT_ALIGN(targets, 8);
  CHECK_OPT_ALIGN(dev_status, 4);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(SKETCH_ERR_INVALID_ARG, "scale is not finite and > 0");
  return SKETCH_OK;
}

sketch_status check_adamw(const sketch_adamw_problem& p, bool states8) {
  if (p.n < 0 || p.n > (int64_t(1) << 35)) return fail(SKETCH_ERR_INVALID_ARG, "n=%lld out of [0, 2^35]", (long long)p.n);
  CHECK_DTYPE(p.w_type);
  CHECK_DTYPE(p.g_type);
  if ((p.m_scale != nullptr) != states8 || (p.v_scale != nullptr) != states8)
    return fail(SKETCH_ERR_INVALID_ARG, "m_scale and v_scale are given for all tensors of a call or for none");
  if (p.n == 0) return SKETCH_OK;
  CHECK_PTR(p.W);
  CHECK_PTR(p.G);
  CHECK_PTR(p.m);
  CHECK_PTR(p.v);
  CHECK_OPT_ALIGN(p.m_scale, 4);
  CHECK_OPT_ALIGN(p.v_scale, 4);
  return SKETCH_OK;
}

// Rows of 8-bit codes: 16-byte aligned, as TMA reads them.
sketch_status check_ld_codes(const char* name, int64_t ld, int64_t width) {
  if (ld < width || ld > kMaxDim)
    return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld out of [%lld, 2^31)", name, (long long)ld, (long long)width);
  if (ld % 16 != 0) return fail(SKETCH_ERR_INVALID_ARG, "%s=%lld is not a multiple of 16", name, (long long)ld);
  return SKETCH_OK;
}

sketch_status check_grads(int n, const sketch_grad_problem* problems, bool out) {
  TRY(check_n(n));
  if (problems == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  for (int i = 0; i < n; ++i) {
    const sketch_grad_problem& p = problems[i];
    if (p.count < 0 || p.count > (int64_t(1) << 40))
      return fail(SKETCH_ERR_INVALID_ARG, "count=%lld out of [0, 2^40]", (long long)p.count);
    CHECK_DTYPE(p.type);
    if (p.count == 0) continue;
    CHECK_ELEM_PTR(p.G, p.type);
    if (out) CHECK_ELEM_PTR(p.out, p.type);
  }
  return SKETCH_OK;
}

}  // namespace

namespace rgs {
void set_last_error(const char* message) {
  snprintf(g_last_error, sizeof(g_last_error), "%s", message);
}
}  // namespace rgs

extern "C" {

const char* sketch_status_string(sketch_status status) {
  switch (status) {
    case SKETCH_OK: return "ok";
    case SKETCH_ERR_INVALID_ARG: return "invalid argument";
    case SKETCH_ERR_UNSUPPORTED: return "unsupported";
    case SKETCH_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case SKETCH_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

const char* sketch_last_error(void) { return g_last_error; }

size_t sketch_workspace_bytes(sketch_op op, int64_t T, int64_t d, int64_t k, int64_t r) {
  return op_ws_bytes(op, T, d, k, r);
}

size_t sketch_workspace_bytes_batched(sketch_op op, int n, const int64_t* T, const int64_t* d, const int64_t* k,
                                      int64_t r) {
  size_t total = 0;
  for (int i = 0; i < n; ++i)
    total += op_ws_bytes(op, T ? T[i] : 0, d ? d[i] : 0, k ? k[i] : 0, r);
  return total;
}

sketch_status sketch_sample_projection(sketch_proj_kind kind, uint64_t seed, uint32_t layer, uint32_t step,
                                       int64_t k, int64_t r, float* P, int32_t* dev_status, void* ws,
                                       size_t ws_bytes, void* stream) {
  const sketch_projection_problem p{P, k, layer};
  return do_sample(kind, seed, step, 1, &p, r, dev_status, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_sample_projection_batched(sketch_proj_kind kind, uint64_t seed, uint32_t step, int n,
                                               const sketch_projection_problem* problems, int64_t r,
                                               int32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  return do_sample(kind, seed, step, n, problems, r, dev_status, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_project_inputs(const uint16_t* X, int64_t T, int64_t k, int64_t ld_x, const float* P,
                                    int64_t r, uint16_t* XP, int64_t ld_xp, void* ws, size_t ws_bytes,
                                    void* stream) {
  const sketch_project_problem p{X, T, k, ld_x, P, XP, ld_xp};
  return do_project(1, &p, r, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_project_inputs_batched(int n, const sketch_project_problem* problems, int64_t r, void* ws,
                                            size_t ws_bytes, void* stream) {
  return do_project(n, problems, r, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_project_inputs_fp32xp_batched(int n, const sketch_project_problem* problems, int64_t r,
                                                   void* ws, size_t ws_bytes, void* stream) {
  return do_project(n, problems, r, ws, ws_bytes, static_cast<cudaStream_t>(stream), true);
}

sketch_status sketch_accumulate_fp32xp_batched(int n, const sketch_accumulate_problem* problems, int64_t r,
                                               int overwrite, void* ws, size_t ws_bytes, void* stream) {
  return do_accumulate(n, problems, r, overwrite, ws, ws_bytes, static_cast<cudaStream_t>(stream), true);
}

size_t sketch_projection_split_elems(int64_t k, int64_t r) {
  if (k < 1 || k > kMaxDim || k % 8 != 0 || r < 1 || r > rgs::kMaxRank) return 0;
  return (size_t)2 * (size_t)((r + 15) / 16 * 16) * (size_t)k;
}

sketch_status sketch_split_projection_batched(int n, const sketch_split_problem* problems, int64_t r,
                                              void* stream) {
  TRY(check_n(n));
  if (problems == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  TRY(check_rank(r));
  std::vector<const float*> P((size_t)n);
  std::vector<int64_t> k((size_t)n);
  std::vector<uint16_t*> out((size_t)n);
  for (int i = 0; i < n; ++i) {
    TRY(check_k(problems[i].k));
    CHECK_PTR(problems[i].P);
    CHECK_PTR(problems[i].P_split);
    P[i] = problems[i].P;
    k[i] = problems[i].k;
    out[i] = problems[i].P_split;
  }
  return launch_result(rgs::launch_split_projection(n, P.data(), k.data(), out.data(), (int)r,
                                                    static_cast<cudaStream_t>(stream)),
                       "split_projection");
}

sketch_status sketch_split_projection_grouped(int n, const sketch_split_group* groups, int64_t r, void* stream) {
  TRY(check_n(n));
  if (groups == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "groups is NULL");
  TRY(check_rank(r));
  std::vector<rgs::SplitGroup> g((size_t)n);
  for (int i = 0; i < n; ++i) {
    const sketch_split_group& gr = groups[i];
    if (gr.m < 1 || gr.m > rgs::kMaxGroup)
      return fail(SKETCH_ERR_INVALID_ARG, "group %d: m=%d out of [1, %d]", i, gr.m, rgs::kMaxGroup);
    if ((int64_t)gr.m * r > rgs::kMaxRank)
      return fail(SKETCH_ERR_INVALID_ARG, "group %d: m*r=%lld exceeds %d", i, (long long)gr.m * r, rgs::kMaxRank);
    if (gr.m > 1 && r % 8 != 0)
      return fail(SKETCH_ERR_INVALID_ARG, "group %d: r=%lld must be a multiple of 8 when m > 1", i, (long long)r);
    if (gr.P == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "group %d: P is NULL", i);
    TRY(check_k(gr.k));
    CHECK_PTR(gr.P_split);
    g[i].m = gr.m;
    g[i].k = gr.k;
    g[i].out = gr.P_split;
    for (int q = 0; q < gr.m; ++q) {
      CHECK_PTR(gr.P[q]);
      g[i].P[q] = gr.P[q];
    }
  }
  return launch_result(rgs::launch_split_projection_grouped(n, g.data(), (int)r, static_cast<cudaStream_t>(stream)),
                       "split_projection_grouped");
}

sketch_status sketch_accumulate(const uint16_t* D, int64_t T, int64_t d, int64_t ld_d, const uint16_t* XP,
                                int64_t ld_xp, int64_t r, float* C, int overwrite, void* ws, size_t ws_bytes,
                                void* stream) {
  const sketch_accumulate_problem p{D, T, d, ld_d, XP, ld_xp, C};
  return do_accumulate(1, &p, r, overwrite, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_accumulate_batched(int n, const sketch_accumulate_problem* problems, int64_t r, int overwrite,
                                        void* ws, size_t ws_bytes, void* stream) {
  return do_accumulate(n, problems, r, overwrite, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_apply_update_normsgd(uint16_t* W, int64_t d, int64_t k, int64_t ld_w, const float* C,
                                          const float* P, int64_t r, float tau, uint64_t seed, uint32_t layer,
                                          uint32_t step, const double* wnorm2_in, double* wnorm2_out,
                                          int32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  const sketch_update_problem p{W, d, k, ld_w, C, P, layer, wnorm2_in, wnorm2_out, dev_status};
  return do_update(true, 1, &p, r, tau, seed, step, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_apply_update_normsgd_batched(int n, const sketch_update_problem* problems, int64_t r,
                                                  float tau, uint64_t seed, uint32_t step, void* ws,
                                                  size_t ws_bytes, void* stream) {
  return do_update(true, n, problems, r, tau, seed, step, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_apply_update_sgd(uint16_t* W, int64_t d, int64_t k, int64_t ld_w, const float* C,
                                      const float* P, int64_t r, float alpha_eta, uint64_t seed, uint32_t layer,
                                      uint32_t step, int32_t* dev_status, void* ws, size_t ws_bytes,
                                      void* stream) {
  const sketch_update_problem p{W, d, k, ld_w, C, P, layer, nullptr, nullptr, dev_status};
  return do_update(false, 1, &p, r, alpha_eta, seed, step, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

sketch_status sketch_apply_update_sgd_batched(int n, const sketch_update_problem* problems, int64_t r,
                                              float alpha_eta, uint64_t seed, uint32_t step, void* ws,
                                              size_t ws_bytes, void* stream) {
  return do_update(false, n, problems, r, alpha_eta, seed, step, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

uint64_t sketch_kernel_launches(void) { return rgs::launches_issued(); }

sketch_status sketch_layer_norm_forward(const void* X, sketch_dtype x_type, int64_t T, int64_t k, int64_t ld_x,
                                        const void* gamma, const void* beta, sketch_dtype w_type, float eps, void* Y,
                                        int64_t ld_y, float* mean, float* rstd, void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("k", k));
  CHECK_DTYPE(x_type);
  CHECK_DTYPE(w_type);
  TRY(check_row_stride("ld_x", ld_x, k));
  TRY(check_row_stride("ld_y", ld_y, k));
  if (!std::isfinite(eps) || eps < 0.f) return fail(SKETCH_ERR_INVALID_ARG, "eps is not finite and >= 0");
  CHECK_ELEM_PTR(X, x_type);
  CHECK_ELEM_PTR(Y, x_type);
  CHECK_OPT_ALIGN(gamma, w_type == SKETCH_BF16 ? 2 : 4);
  CHECK_OPT_ALIGN(beta, w_type == SKETCH_BF16 ? 2 : 4);
  CHECK_ELEM_PTR(mean, SKETCH_FP32);
  CHECK_ELEM_PTR(rstd, SKETCH_FP32);
  const rgs::NormForward a = {X, (int)x_type, T, k, ld_x, gamma, beta, (int)w_type, eps, Y, ld_y, mean, rstd};
  return launch_result(rgs::launch_norm_forward(a, static_cast<cudaStream_t>(stream)), "layer_norm_forward");
}

sketch_status sketch_layer_norm_backward(const void* dY, int64_t ld_dy, const void* X, sketch_dtype x_type, int64_t T,
                                         int64_t k, int64_t ld_x, const void* gamma, sketch_dtype w_type,
                                         const float* mean, const float* rstd, void* dX, int64_t ld_dx, float* dgamma,
                                         float* dbeta, int overwrite, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("k", k));
  CHECK_DTYPE(x_type);
  CHECK_DTYPE(w_type);
  TRY(check_row_stride("ld_dy", ld_dy, k));
  TRY(check_row_stride("ld_x", ld_x, k));
  if (dX) TRY(check_row_stride("ld_dx", ld_dx, k));
  if (overwrite != 0 && overwrite != 1) return fail(SKETCH_ERR_INVALID_ARG, "overwrite must be 0 or 1");
  CHECK_ELEM_PTR(dY, x_type);
  CHECK_ELEM_PTR(X, x_type);
  CHECK_OPT_ALIGN(gamma, w_type == SKETCH_BF16 ? 2 : 4);
  CHECK_ELEM_PTR(mean, SKETCH_FP32);
  CHECK_ELEM_PTR(rstd, SKETCH_FP32);
  if (!dX && !dgamma && !dbeta) return fail(SKETCH_ERR_INVALID_ARG, "dX, dgamma and dbeta are all NULL");
  CHECK_OPT_ALIGN(dX, x_type == SKETCH_BF16 ? 2 : 4);
  CHECK_OPT_ALIGN(dgamma, 4);
  CHECK_OPT_ALIGN(dbeta, 4);
  TRY(check_ws(ws, ws_bytes, rgs::norm_backward_workspace_bytes(T, k)));
  const rgs::NormBackward a = {dY,   X,    (int)x_type, T,  k,     ld_dy,  ld_x,  gamma,     (int)w_type,
                               mean, rstd, dX,          ld_dx, dgamma, dbeta, overwrite, static_cast<float*>(ws)};
  return launch_result(rgs::launch_norm_backward(a, static_cast<cudaStream_t>(stream)), "layer_norm_backward");
}

sketch_status sketch_cross_entropy_forward(const uint16_t* X, int64_t T, int64_t k, int64_t ld_x, const uint16_t* W,
                                           int64_t V, int64_t ld_w, const int64_t* targets, float scale, float* loss,
                                           float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                                           void* stream) {
  TRY(check_head(X, T, k, ld_x, W, V, ld_w, targets, scale, dev_status));
  CHECK_ELEM_PTR(loss, SKETCH_FP32);
  CHECK_ELEM_PTR(lse, SKETCH_FP32);
  TRY(check_ws(ws, ws_bytes, rgs::head_forward_workspace_bytes(T, V)));
  const rgs::HeadForward a = {X, T, k, ld_x, W, V, ld_w, targets, scale, loss, lse, dev_status};
  return launch_result(rgs::launch_head_forward(a, ws, static_cast<cudaStream_t>(stream)), "cross_entropy_forward");
}

sketch_status sketch_cross_entropy_backward(const uint16_t* X, int64_t T, int64_t k, int64_t ld_x, const uint16_t* W,
                                            int64_t V, int64_t ld_w, const int64_t* targets, float scale,
                                            const float* lse, const float* g, uint16_t* dX, int64_t ld_dx, void* dW,
                                            sketch_dtype dw_type, int64_t ld_dw, const uint16_t* XP, int64_t ld_xp,
                                            int64_t r, float* C, int overwrite, int32_t* dev_status, void* ws,
                                            size_t ws_bytes, void* stream) {
  TRY(check_head(X, T, k, ld_x, W, V, ld_w, targets, scale, dev_status));
  CHECK_ELEM_PTR(lse, SKETCH_FP32);
  CHECK_ELEM_PTR(g, SKETCH_FP32);
  if (overwrite != 0 && overwrite != 1) return fail(SKETCH_ERR_INVALID_ARG, "overwrite must be 0 or 1");
  if (!dX && !dW && !C) return fail(SKETCH_ERR_INVALID_ARG, "dX, dW and C are all NULL");
  if (dX) {
    TRY(check_ld("ld_dx", ld_dx, k));
    CHECK_PTR(dX);
  }
  if (dW) {
    CHECK_DTYPE(dw_type);
    TRY(check_ld("ld_dw", ld_dw, k));
    CHECK_PTR(dW);
  }
  if ((C != nullptr) != (XP != nullptr)) return fail(SKETCH_ERR_INVALID_ARG, "C and XP are given together");
  if (C) {
    TRY(check_rank(r));
    TRY(check_ld("ld_xp", ld_xp, r));
    CHECK_PTR(C);
    CHECK_PTR(XP);
  }
  TRY(check_ws(ws, ws_bytes, rgs::head_backward_workspace_bytes(T, V, k, C ? r : 0)));
  const rgs::HeadBackward a = {X,  T,  k,     ld_x, W,            V,     ld_w, targets, scale, lse, g,         dX,
                               ld_dx, dW, (int)dw_type, ld_dw, XP,   ld_xp,   r,     C,   overwrite, dev_status};
  return launch_result(rgs::launch_head_backward(a, ws, static_cast<cudaStream_t>(stream)), "cross_entropy_backward");
}

sketch_status sketch_adamw_batched(int n, const sketch_adamw_problem* problems, double lr, double beta1,
                                   double beta2, double eps, double weight_decay, const float* grad_scale,
                                   uint64_t seed, uint32_t step, void* stream) {
  TRY(check_n(n));
  if (problems == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "problems is NULL");
  if (!std::isfinite(lr) || !std::isfinite(weight_decay))
    return fail(SKETCH_ERR_INVALID_ARG, "lr or weight_decay is not finite");
  // in fp32 a beta just below 1 would round to 1
  if (!(beta1 >= 0.0 && (float)beta1 < 1.f) || !(beta2 >= 0.0 && (float)beta2 < 1.f))
    return fail(SKETCH_ERR_INVALID_ARG, "beta1 or beta2 out of [0, 1)");
  if (!std::isfinite(eps) || !((float)eps >= FLT_MIN))
    return fail(SKETCH_ERR_INVALID_ARG, "eps is not finite and at least the smallest normal fp32");
  CHECK_OPT_ALIGN(grad_scale, 4);
  const bool states8 = problems[0].m_scale != nullptr;
  for (int i = 0; i < n; ++i) TRY(check_adamw(problems[i], states8));
  const double t = (double)step + 1.0;
  rgs::AdamStep h = {};
  h.decay = (float)(1.0 - lr * weight_decay);
  h.lr_m = (float)(lr / (1.0 - std::pow(beta1, t)));
  h.root_v = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  h.beta1 = (float)beta1;
  h.beta2 = (float)beta2;
  h.one_beta1 = (float)(1.0 - beta1);
  h.one_beta2 = (float)(1.0 - beta2);
  h.eps = (float)eps;
  h.grad_scale = grad_scale;
  return launch_result(rgs::launch_adamw(n, problems, states8, h, seed, step, static_cast<cudaStream_t>(stream)),
                       "adamw");
}

sketch_status sketch_rms_norm_forward(const void* X, sketch_dtype x_type, int64_t T, int64_t k, int64_t ld_x,
                                      const void* R, int64_t ld_r, void* S, int64_t ld_s, const void* gamma,
                                      sketch_dtype w_type, float eps, void* Y, int64_t ld_y, uint8_t* Q, int64_t ld_q,
                                      float* scale, float* rstd, void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("k", k));
  CHECK_DTYPE(x_type);
  CHECK_DTYPE(w_type);
  TRY(check_row_stride("ld_x", ld_x, k));
  CHECK_ELEM_PTR(X, x_type);
  if (!std::isfinite(eps) || eps < 0.f) return fail(SKETCH_ERR_INVALID_ARG, "eps is not finite and >= 0");
  if (R) {
    TRY(check_row_stride("ld_r", ld_r, k));
    CHECK_ELEM_PTR(R, x_type);
  }
  if (S) {
    if (!R) return fail(SKETCH_ERR_INVALID_ARG, "S is given without R");
    TRY(check_row_stride("ld_s", ld_s, k));
    CHECK_ELEM_PTR(S, x_type);
  }
  if (!Y && !Q) return fail(SKETCH_ERR_INVALID_ARG, "Y and Q are both NULL");
  if (Y) {
    TRY(check_row_stride("ld_y", ld_y, k));
    CHECK_ELEM_PTR(Y, x_type);
    if (Y == S) return fail(SKETCH_ERR_INVALID_ARG, "Y and S are one buffer");
  }
  if ((Q != nullptr) != (scale != nullptr)) return fail(SKETCH_ERR_INVALID_ARG, "Q and scale are given together");
  if (Q) {
    TRY(check_ld_codes("ld_q", ld_q, k));
    CHECK_PTR(Q);
    CHECK_ELEM_PTR(scale, SKETCH_FP32);
  }
  CHECK_OPT_ALIGN(gamma, w_type == SKETCH_BF16 ? 2 : 4);
  CHECK_OPT_ALIGN(rstd, 4);
  const rgs::RmsForward a = {X,   (int)x_type, T, k,    ld_x, R,    ld_r,  S,   ld_s, gamma, (int)w_type,
                             eps, Y,           ld_y, Q, ld_q, scale, rstd};
  return launch_result(rgs::launch_rms_forward(a, static_cast<cudaStream_t>(stream)), "rms_norm_forward");
}

sketch_status sketch_rms_norm_backward(const void* dY, int64_t ld_dy, const void* S, sketch_dtype x_type, int64_t T,
                                       int64_t k, int64_t ld_s, const void* gamma, sketch_dtype w_type,
                                       const float* rstd, const void* dS, int64_t ld_ds, void* dX, int64_t ld_dx,
                                       float* dgamma, int overwrite, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("k", k));
  CHECK_DTYPE(x_type);
  CHECK_DTYPE(w_type);
  TRY(check_row_stride("ld_dy", ld_dy, k));
  TRY(check_row_stride("ld_s", ld_s, k));
  CHECK_ELEM_PTR(dY, x_type);
  CHECK_ELEM_PTR(S, x_type);
  CHECK_OPT_ALIGN(gamma, w_type == SKETCH_BF16 ? 2 : 4);
  CHECK_ELEM_PTR(rstd, SKETCH_FP32);
  if (overwrite != 0 && overwrite != 1) return fail(SKETCH_ERR_INVALID_ARG, "overwrite must be 0 or 1");
  if (!dX && !dgamma) return fail(SKETCH_ERR_INVALID_ARG, "dX and dgamma are both NULL");
  if (dX) {
    TRY(check_row_stride("ld_dx", ld_dx, k));
    CHECK_ELEM_PTR(dX, x_type);
  }
  if (dS) {
    if (!dX) return fail(SKETCH_ERR_INVALID_ARG, "dS is given without dX");
    TRY(check_row_stride("ld_ds", ld_ds, k));
    CHECK_ELEM_PTR(dS, x_type);
  }
  CHECK_OPT_ALIGN(dgamma, 4);
  if (dgamma) TRY(check_ws(ws, ws_bytes, rgs::rms_backward_workspace_bytes(T, k)));
  const rgs::RmsBackward a = {dY,   S,  (int)x_type, T,  k,     ld_dy,  ld_s,      gamma, (int)w_type,
                              rstd, dS, ld_ds,       dX, ld_dx, dgamma, overwrite, static_cast<float*>(ws)};
  return launch_result(rgs::launch_rms_backward(a, static_cast<cudaStream_t>(stream)), "rms_norm_backward");
}

sketch_status sketch_quantize_blocks(const void* X, sketch_dtype x_type, int64_t T, int64_t k, int64_t ld_x, int rows,
                                     uint8_t* Q, int64_t ld_q, float* scale, uint8_t* Qt, int64_t ld_qt,
                                     void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("k", k));
  CHECK_DTYPE(x_type);
  TRY(check_row_stride("ld_x", ld_x, k));
  CHECK_ELEM_PTR(X, x_type);
  if (rows != 1 && rows != 128) return fail(SKETCH_ERR_INVALID_ARG, "rows=%d is neither 1 nor 128", rows);
  if (rows == 1 && Qt) return fail(SKETCH_ERR_INVALID_ARG, "Qt needs rows=128");
  if (!Q && !Qt) return fail(SKETCH_ERR_INVALID_ARG, "Q and Qt are both NULL");
  if (Q) {
    TRY(check_ld_codes("ld_q", ld_q, k));
    CHECK_PTR(Q);
  }
  if (Qt) {
    TRY(check_ld_codes("ld_qt", ld_qt, T));
    CHECK_PTR(Qt);
  }
  CHECK_ELEM_PTR(scale, SKETCH_FP32);
  if (rgs::ceil_div(T, rows == 1 ? 16 : 128) * rgs::ceil_div(k, 128) > kMaxDim)  // a launch's blocks of threads
    return fail(SKETCH_ERR_UNSUPPORTED, "T=%lld and k=%lld span 2^31 blocks or more", (long long)T, (long long)k);
  const rgs::Quantize a = {X, (int)x_type, T, k, ld_x, rows, Q, ld_q, scale, Qt, ld_qt};
  return launch_result(rgs::launch_quantize(a, static_cast<cudaStream_t>(stream)), "quantize_blocks");
}

sketch_status sketch_matmul_blocks(const uint8_t* A, int64_t T, int64_t k, int64_t ld_a, const float* a_scale,
                                   int64_t ld_as, const uint8_t* B, int64_t N, int64_t ld_b, const float* b_scale,
                                   int64_t bs_row, int64_t bs_col, void* Y, sketch_dtype y_type, int64_t ld_y,
                                   int overwrite, void* stream) {
  TRY(check_dim("T", T));
  TRY(check_dim("N", N));
  TRY(check_dim("k", k));
  if (T > rgs::kMaxHeadDim || N > rgs::kMaxHeadDim || k > rgs::kMaxHeadDim ||
      rgs::ceil_div(T, 256) * rgs::ceil_div(N, 256) > rgs::kMaxHeadTiles)
    return fail(SKETCH_ERR_UNSUPPORTED, "T=%lld, N=%lld, k=%lld: at most 2^24 each and 2^28 tiles of 256 x 256",
                (long long)T, (long long)N, (long long)k);
  const int64_t groups = rgs::ceil_div(k, 128);
  CHECK_DTYPE(y_type);
  TRY(check_ld_codes("ld_a", ld_a, k));
  TRY(check_ld_codes("ld_b", ld_b, k));
  TRY(check_row_stride("ld_as", ld_as, groups));
  if (bs_row < 0 || bs_row > kMaxDim || bs_col < 0 || bs_col > kMaxDim)
    return fail(SKETCH_ERR_INVALID_ARG, "bs_row=%lld or bs_col=%lld out of [0, 2^31)", (long long)bs_row,
                (long long)bs_col);
  TRY(check_ld("ld_y", ld_y, N));
  CHECK_PTR(A);
  CHECK_ELEM_PTR(a_scale, SKETCH_FP32);
  CHECK_PTR(B);
  CHECK_ELEM_PTR(b_scale, SKETCH_FP32);
  CHECK_PTR(Y);
  if (overwrite != 0 && overwrite != 1) return fail(SKETCH_ERR_INVALID_ARG, "overwrite must be 0 or 1");
  if (!overwrite && y_type == SKETCH_BF16) return fail(SKETCH_ERR_INVALID_ARG, "overwrite=0 needs an fp32 Y");
  const rgs::MatmulBlocks a = {A,       T,      k,      ld_a, a_scale,     ld_as, B,        N,
                               ld_b,    b_scale, bs_row, bs_col, Y, (int)y_type, ld_y, overwrite};
  return launch_result(rgs::launch_matmul_blocks(a, static_cast<cudaStream_t>(stream)), "matmul_blocks");
}

sketch_status sketch_grad_norm_batched(int n, const sketch_grad_problem* problems, float max_norm, float* norm,
                                       float* scale, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_grads(n, problems, false));
  if (scale && !(std::isfinite(max_norm) && max_norm > 0.f))
    return fail(SKETCH_ERR_INVALID_ARG, "max_norm is not finite and > 0");
  CHECK_ELEM_PTR(norm, SKETCH_FP32);
  CHECK_OPT_ALIGN(scale, 4);
  TRY(check_ws(ws, ws_bytes, rgs::grad_norm_workspace_bytes(n)));
  return launch_result(rgs::launch_grad_norm(n, problems, max_norm, norm, scale, static_cast<double*>(ws),
                                             static_cast<cudaStream_t>(stream)),
                       "grad_norm");
}

sketch_status sketch_grad_scale_batched(int n, const sketch_grad_problem* problems, const float* scale, void* stream) {
  TRY(check_grads(n, problems, true));
  CHECK_ELEM_PTR(scale, SKETCH_FP32);
  return launch_result(rgs::launch_grad_scale(n, problems, scale, static_cast<cudaStream_t>(stream)), "grad_scale");
}

sketch_status sketch_read_device_errors(int32_t* flags, void* stream) {
  if (flags == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "flags is NULL");
  int* word = nullptr;
  cudaError_t err = rgs::device_error_word(&word);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t host = 0;
  if (err == cudaSuccess) err = cudaMemcpyAsync(&host, word, sizeof(int32_t), cudaMemcpyDeviceToHost, s);
  if (err == cudaSuccess) err = cudaMemsetAsync(word, 0, sizeof(int32_t), s);
  if (err == cudaSuccess) err = cudaStreamSynchronize(s);
  *flags = host;
  return launch_result(err, "read_device_errors");
}

sketch_status sketch_read_exact_count(uint64_t* count, void* stream) {
  if (count == nullptr) return fail(SKETCH_ERR_INVALID_ARG, "count is NULL");
  unsigned long long* word = nullptr;
  cudaError_t err = rgs::device_exact_counter(&word);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned long long host = 0;
  if (err == cudaSuccess) err = cudaMemcpyAsync(&host, word, sizeof(host), cudaMemcpyDeviceToHost, s);
  if (err == cudaSuccess) err = cudaMemsetAsync(word, 0, sizeof(host), s);
  if (err == cudaSuccess) err = cudaStreamSynchronize(s);
  *count = (uint64_t)host;
  return launch_result(err, "read_exact_count");
}

}  // extern "C"
