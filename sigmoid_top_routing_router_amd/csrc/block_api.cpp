// C ABI of the operators around the layer (the residual norm and the balance
// loss, forward and backward) and of the layer's backward pass.  Argument
// checks, workspace carving and the launches on the caller's stream; nothing
// else.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/moe_mi355x.h"
#include "api_internal.h"
#include "kernels.h"

namespace {

moe_status_t fail(moe_status_t s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return moe::set_error(s, buf);
}

moe_status_t done(hipError_t e, const char* where) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
  return moe::set_error(MOE_OK, "");
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr size_t kAlign = 256;
size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

moe_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, kAlign))
    return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
  if (have < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < required %zu", have, need);
  return MOE_OK;
}

// ---- norm
constexpr int64_t kNormMaxN = int64_t(1) << 27;

moe_status_t check_norm(int64_t n, int32_t d, float eps, uint32_t flags) {
  if (n < 0 || n > kNormMaxN || d < 1 || d > moe::kNormMaxD)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n=%lld d=%d: need 0 <= n <= 2^27 and 1 <= d <= %d",
                (long long)n, d, moe::kNormMaxD);
  if (!std::isfinite(eps) || eps < 0.0f)
    return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (flags & ~(MOE_NORM_STREAM_F32 | MOE_NORM_WEIGHT_F32))
    return fail(MOE_ERR_INVALID_ARGUMENT, "unknown flag bits 0x%x", flags);
  return MOE_OK;
}

moe_status_t check_aligned(const void* const* p, int count, size_t a, const char* what) {
  for (int i = 0; i < count; ++i)
    if (p[i] && !aligned(p[i], a))
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s must be %zu-byte aligned", what, a);
  return MOE_OK;
}

// A buffer of a call (p NULL: absent).  inplace: the input and the output that
// may be one buffer.
struct Span {
  const void* p;
  size_t bytes;
  bool inplace = false;
};

// No output (the workspace is one) shares memory with an input or another
// output: a launch would overwrite what a later one still reads.
moe_status_t check_alias(const Span* in, int n_in, const Span* out, int n_out) {
  auto share = [](const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
  };
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (share(in[i], out[o]) && !(in[i].inplace && out[o].inplace && in[i].p == out[o].p))
        return fail(MOE_ERR_INVALID_ARGUMENT, "an output aliases an input");
    for (int j = 0; j < o; ++j)
      if (share(out[j], out[o]))
        return fail(MOE_ERR_INVALID_ARGUMENT, "two outputs alias each other");
  }
  return MOE_OK;
}

template <int I, int O>
moe_status_t check_alias(const Span (&in)[I], const Span (&out)[O]) {
  return check_alias(in, I, out, O);
}

// ---- balance loss
constexpr int32_t kMaxSegments = 1 << 20;

bool balance_sizes_ok(int64_t N, int32_t E, int32_t n_seg) {
  return N >= 1 && N <= (int64_t(1) << 24) && E >= 2 && E <= MOE_MAX_E && n_seg >= 1 &&
         n_seg <= kMaxSegments;
}

moe_status_t check_balance(int64_t N, int32_t E, int32_t n_seg, const int32_t* begin,
                           const int32_t* end, int32_t score, float coef) {
  if (!balance_sizes_ok(N, E, n_seg))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "N=%lld E=%d n_seg=%d: need 1 <= N <= 2^24, 2 <= E <= %d, 1 <= n_seg <= 2^20",
                (long long)N, E, n_seg, MOE_MAX_E);
  if ((begin == nullptr) != (end == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "seg_begin and seg_end: both or neither");
  if (!begin && n_seg != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_seg=%d needs seg_begin and seg_end", n_seg);
  if (score < MOE_SCORE_SIGMOID || score > MOE_SCORE_SOFTMAX)
    return fail(MOE_ERR_INVALID_ARGUMENT, "score=%d outside [0, 2]", score);
  if (!std::isfinite(coef)) return fail(MOE_ERR_INVALID_ARGUMENT, "coef must be finite");
  return MOE_OK;
}

moe::BalanceWork carve_balance(void* ws, int64_t N, int32_t E, int32_t n_seg, size_t* bytes) {
  const size_t rows = (size_t)moe::balance_slots(N, n_seg) * (size_t)E;
  const size_t terms = (size_t)n_seg * (size_t)((E + 63) / 64) * 2;
  char* p = (char*)ws;
  moe::BalanceWork w;
  w.sums = (float*)p;
  p += up(rows * sizeof(float));
  w.loads = (uint32_t*)p;
  p += up(rows * sizeof(uint32_t));
  w.terms = (double*)p;
  p += up(terms * sizeof(double));
  w.ticket = (uint32_t*)p;
  p += kAlign;
  *bytes = (size_t)(p - (char*)ws);
  return w;
}

// ---- layer backward
struct GradLayout {
  int32_t *ids, *counts, *offsets, *sorted_src, *src_pos, *tiles, *n_tiles, *row_tiles, *n_row_tiles;
  uint32_t* tok;
  uint32_t* block_counts;
  float *S, *Q, *Qs, *dscore, *dXp, *base;
  uint16_t *hid, *hids, *dzb;
  int64_t ld, lds;  // row pitch of hid and of hids (the shared expert's)
  int64_t max_tiles, max_row_tiles;
  int ldb;
  size_t bytes;
};
// Rows of dG | dU | s H in whole 128-byte lines.
int64_t hidden_pitch(int h) { return (3 * (int64_t)h + 63) / 64 * 64; }
GradLayout carve_grad(void* ws, const moe_problem_t& p) {
  char* const base = (char*)ws;
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    void* q = base ? base + off : nullptr;
    off += up(bytes);
    return q;
  };
  GradLayout l{};
  const size_t N = (size_t)p.N, pairs = N * p.K, hs = p.n_shared ? (size_t)p.h_shared : 0;
  l.ldb = (p.E + 63) / 64 * 64;
  l.ids = (int32_t*)take(pairs * 4);
  l.S = (float*)take(pairs * 4);
  l.block_counts = (uint32_t*)take((size_t)moe::perm_count_rows((int64_t)pairs) * p.E * 4);
  l.counts = (int32_t*)take((size_t)p.E * 4);
  l.offsets = (int32_t*)take(((size_t)p.E + 1) * 4);
  l.sorted_src = (int32_t*)take(pairs * 4);
  l.src_pos = (int32_t*)take(pairs * 4);
  l.max_tiles = moe::perm_max_tiles((int64_t)pairs, p.E, moe::gemm_bm());
  l.tiles = (int32_t*)take((size_t)l.max_tiles * 16);
  l.n_tiles = (int32_t*)take(16);
  l.max_row_tiles = moe::perm_max_tiles((int64_t)pairs, p.E, moe::grad_tile_rows());
  l.row_tiles = (int32_t*)take((size_t)l.max_row_tiles * 16);
  l.n_row_tiles = (int32_t*)take(16);
  l.tok = (uint32_t*)take(pairs * 4);
  // Q is read for the last time before the pairs' part of grad_x is written
  l.Q = l.dXp = (float*)take(pairs * (size_t)(p.h > p.d ? p.h : p.d) * 4);
  l.ld = hidden_pitch(p.h);
  l.lds = hidden_pitch((int)hs);
  l.hid = (uint16_t*)take(pairs * l.ld * 2);
  l.dscore = (float*)take(pairs * (size_t)moe::gateup_col_tiles(p.h) * 4);
  l.Qs = (float*)take(N * hs * 4);
  l.hids = (uint16_t*)take(hs ? N * l.lds * 2 : 0);
  l.dzb = (uint16_t*)take(N * (size_t)l.ldb * 2);
  l.base = (float*)take(N * p.d * 4);
  l.bytes = off;
  return l;
}

moe_status_t check_grad_problem(const moe_problem_t* p) {
  const moe_status_t s = moe::check_layer(p);
  if (s != MOE_OK) return s;
  if (p->flags & MOE_PACKED_GATEUP)
    return fail(MOE_ERR_INVALID_ARGUMENT, "the backward pass takes row-major weights only");
  const uint64_t most = moe::kGradMaxOperandBytes;
  if ((uint64_t)p->N * p->d * 2 > most || (uint64_t)p->N * p->K * p->h * 2 > most ||
      (p->n_shared && (uint64_t)p->N * p->h_shared * 2 > most))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "N=%lld too large: x and the hidden rows must each be "
                "at most 4 GiB - 128 KiB", (long long)p->N);
  return MOE_OK;
}

#define MOE_TRY(expr, where)                                  \
  do {                                                        \
    const hipError_t _e = (expr);                             \
    if (_e != hipSuccess) return done(_e, "moe_backward: " where); \
  } while (0)

moe_status_t backward_launches(const moe_problem_t& p, const moe_weights_t& w, const uint16_t* x,
                               const uint16_t* dy, const float* Z, const int32_t* ids,
                               const float* grad_logits, const moe_grads_t& g, const GradLayout& l,
                               hipStream_t st) {
  const int64_t N = p.N, pairs = N * p.K;
  const int d = p.d, h = p.h, hs = p.h_shared, E = p.E, K = p.K;
  const bool shared = p.n_shared == 1, router = w.w_router != nullptr;
  // the pairs' weights and their grouping by expert
  MOE_TRY(moe::launch_pairs(ids, Z, pairs, E, K, l.ids, l.S, st), "pairs");
  moe::PermWork pw;
  pw.block_counts = l.block_counts;
  pw.counts = l.counts;
  pw.offsets = l.offsets;
  pw.sorted_src = l.sorted_src;
  pw.src_pos = l.src_pos;
  pw.tiles = l.tiles;
  pw.n_tiles = l.n_tiles;
  MOE_TRY(moe::launch_permute(l.ids, N, E, K, moe::gemm_bm(), moe::gemm_xrows(), pw, st),
          "grouping");
  MOE_TRY(moe::launch_grouped_rows(l.sorted_src, l.S, pairs, K, (uint32_t)d * 2u, l.offsets, E, l.tok,
                                   l.row_tiles, l.n_row_tiles, st),
          "grouped rows");

  auto pair_rows = [&] {
    moe::RowsProblem r{};
    r.tiles = l.row_tiles;
    r.n_tiles = l.n_row_tiles;
    r.max_tiles = l.max_row_tiles;
    return r;
  };
  auto token_rows = [&] {
    moe::RowsProblem r{};
    r.rows_dense = N;
    return r;
  };
  // Q = dy W_d
  {
    moe::RowsProblem r = pair_rows(), t = token_rows();
    r.seg[0] = {dy, d, w.w_down, (int64_t)d * h, d};
    r.n_seg = 1;
    r.gather = l.tok;
    r.a_rows = N;
    r.ncols = h;
    r.out = l.Q;
    r.ldo = h;
    if (shared) {
      t.seg[0] = {dy, d, w.ws_down, 0, d};
      t.n_seg = 1;
      t.ncols = hs;
      t.out = l.Qs;
      t.ldo = hs;
    }
    MOE_TRY(moe::launch_rows(shared ? &t : nullptr, r, st), "hidden gradient");
  }
  // G, U again; dG, dU, s H and the score gradients
  {
    const moe::GateUpGrad r{w.w_gate, w.w_up, h, l.Q, l.hid, l.ld};
    const moe::GateUpGrad t{w.ws_gate, w.ws_up, hs, l.Qs, l.hids, l.lds};
    MOE_TRY(moe::launch_gateup_grad(x, N, l.sorted_src, K, l.tiles, l.n_tiles, l.max_tiles, d, l.S,
                                    l.dscore, r, shared ? &t : nullptr, st),
            "gate/up gradient");
  }
  MOE_TRY(moe::launch_logits_grad(Z, ids, l.src_pos, l.dscore, moe::gateup_col_tiles(h), N, E, K,
                                  grad_logits, g.logits, router ? l.dzb : nullptr, l.ldb, st),
          "logits gradient");
  // grad_x: the pairs' parts, and the tokens' (shared expert and router)
  moe::RowsProblem r = pair_rows(), t = token_rows();
  const int64_t es = (int64_t)h * d;
  r.seg[0] = {l.hid, l.ld, w.w_gate, es, h};
  r.seg[1] = {l.hid + h, l.ld, w.w_up, es, h};
  r.n_seg = 2;
  r.ncols = d;
  r.out = l.dXp;
  r.ldo = d;
  if (shared) {
    t.seg[t.n_seg++] = {l.hids, l.lds, w.ws_gate, 0, hs};
    t.seg[t.n_seg++] = {l.hids + hs, l.lds, w.ws_up, 0, hs};
  }
  if (router) t.seg[t.n_seg++] = {l.dzb, l.ldb, w.w_router, 0, E};
  t.ncols = d;
  t.out = l.base;
  t.ldo = d;
  // the weights' gradients
  moe::WeightsLaunch wl{};
  auto problem = [&](const uint16_t* A, int64_t lda, int a_cols, const uint16_t* B, int64_t ldb,
                     int b_cols, uint16_t* out) {
    moe::WeightsProblem q{};
    q.A = A;
    q.lda = lda;
    q.a_cols = a_cols;
    q.B = B;
    q.ldb = ldb;
    q.b_cols = b_cols;
    q.rows_dense = N;
    q.out = out;
    q.offsets = l.offsets;
    q.tok = l.tok;
    q.tok_rows = N;
    q.out_stride = (int64_t)h * d;
    return q;
  };
  if (shared) {
    wl.dense[wl.n_dense++] = problem(l.hids, l.lds, hs, x, d, d, g.ws_gate);
    wl.dense[wl.n_dense++] = problem(l.hids + hs, l.lds, hs, x, d, d, g.ws_up);
    wl.dense[wl.n_dense++] = problem(dy, d, d, l.hids + 2 * hs, l.lds, hs, g.ws_down);
  }
  if (router) wl.dense[wl.n_dense++] = problem(l.dzb, l.ldb, E, x, d, d, g.w_router);
  wl.expert[0] = problem(l.hid, l.ld, h, x, d, d, g.w_gate);
  wl.expert[1] = problem(l.hid + h, l.ld, h, x, d, d, g.w_up);
  wl.expert[2] = problem(dy, d, d, l.hid + 2 * h, l.ld, h, g.w_down);
  wl.E = E;
  MOE_TRY(moe::launch_gradients(t.n_seg ? &t : nullptr, r, wl, st), "x and weight gradients");
  MOE_TRY(moe::launch_sum_pairs(t.n_seg ? l.base : nullptr, l.dXp, l.src_pos, N, K, d, g.x, st),
          "x gradient sum");
  return moe::set_error(MOE_OK, "");
}

}  // namespace

extern "C" {

size_t moe_backward_workspace_bytes(const moe_problem_t* p) {
  if (check_grad_problem(p) != MOE_OK) return 0;
  return carve_grad(nullptr, *p).bytes;
}

moe_status_t moe_backward(const moe_problem_t* p, const moe_weights_t* w, const uint16_t* x,
                          const uint16_t* grad_y, const float* logits, const int32_t* topk_ids,
                          const float* grad_logits, const moe_grads_t* g, void* workspace,
                          size_t workspace_bytes, void* stream) {
  moe_status_t s = check_grad_problem(p);
  if (s != MOE_OK) return s;
  if (!w || !x || !grad_y || !logits || !topk_ids || !g)
    return fail(MOE_ERR_INVALID_ARGUMENT,
                "weights, x, grad_y, logits, topk_ids and gradients are required");
  if (!w->w_gate || !w->w_up || !w->w_down || !g->w_gate || !g->w_up || !g->w_down || !g->x ||
      !g->logits)
    return fail(MOE_ERR_INVALID_ARGUMENT,
                "routed expert weights and the gradients of x, logits and them are required");
  if ((w->w_router != nullptr) != (g->w_router != nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "w_router and its gradient: both or neither");
  if (p->n_shared == 1 && (!w->ws_gate || !w->ws_up || !w->ws_down || !g->ws_gate || !g->ws_up ||
                           !g->ws_down))
    return fail(MOE_ERR_INVALID_ARGUMENT, "shared expert weights and gradients are required");
  const void* in[] = {x, grad_y, w->w_router, w->w_gate, w->w_up, w->w_down, w->ws_gate, w->ws_up,
                      w->ws_down};
  const void* out[] = {g->x, g->w_router, g->w_gate, g->w_up, g->w_down, g->ws_gate, g->ws_up,
                       g->ws_down};
  const void* f4[] = {logits, topk_ids, grad_logits, g->logits};
  if ((s = check_aligned(in, 9, 16, "bf16 inputs")) != MOE_OK) return s;
  if ((s = check_aligned(out, 8, 16, "bf16 gradients")) != MOE_OK) return s;
  if ((s = check_aligned(f4, 4, 4, "logits and ids")) != MOE_OK) return s;
  const GradLayout need = carve_grad(nullptr, *p);
  if ((s = check_workspace(workspace, workspace_bytes, need.bytes)) != MOE_OK) return s;
  const size_t xb = (size_t)p->N * p->d * 2, zb = (size_t)p->N * p->E * 4;
  const size_t rb = (size_t)p->E * p->d * 2, eb = rb * p->h;
  const size_t sb = p->n_shared == 1 ? (size_t)p->h_shared * p->d * 2 : 0;
  const Span ins[] = {{x, xb}, {grad_y, xb}, {logits, zb}, {topk_ids, (size_t)p->N * p->K * 4},
                      {grad_logits, zb, true}, {w->w_router, rb}, {w->w_gate, eb}, {w->w_up, eb},
                      {w->w_down, eb}, {w->ws_gate, sb}, {w->ws_up, sb}, {w->ws_down, sb}};
  const Span outs[] = {{g->x, xb}, {g->logits, zb, true}, {g->w_router, rb}, {g->w_gate, eb},
                       {g->w_up, eb}, {g->w_down, eb}, {g->ws_gate, sb}, {g->ws_up, sb},
                       {g->ws_down, sb}, {workspace, need.bytes}};
  if ((s = check_alias(ins, outs)) != MOE_OK) return s;
  return backward_launches(*p, *w, x, grad_y, logits, topk_ids, grad_logits, *g,
                           carve_grad(workspace, *p), (hipStream_t)stream);
}

moe_status_t moe_rms_norm(const uint16_t* x, const void* residual, const void* post_weight,
                          const void* weight, int64_t n, int32_t d, float eps, uint32_t flags,
                          uint16_t* y, void* residual_out, uint8_t* codes, float* scales,
                          void* stream) {
  moe_status_t s = check_norm(n, d, eps, flags);
  if (s != MOE_OK) return s;
  if (codes && d % 128)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "d=%d: codes need a multiple of 128", d);
  if (n == 0) return moe::set_error(MOE_OK, "");
  if ((codes == nullptr) != (scales == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "codes and scales: both or neither");
  if (!y && !residual_out && !codes)
    return fail(MOE_ERR_INVALID_ARGUMENT, "y, residual_out or codes is required");
  if (!x || !weight) return fail(MOE_ERR_INVALID_ARGUMENT, "x and weight are required");
  const bool sf = (flags & MOE_NORM_STREAM_F32) != 0, wf = (flags & MOE_NORM_WEIGHT_F32) != 0;
  const void* bf[] = {x, y};
  const void* st[] = {residual, residual_out};
  const void* wt[] = {weight, post_weight};
  const void* sc[] = {scales};
  if ((s = check_aligned(bf, 2, 2, "x and y")) != MOE_OK) return s;
  if ((s = check_aligned(st, 2, sf ? 4 : 2, "residual and residual_out")) != MOE_OK) return s;
  if ((s = check_aligned(wt, 2, wf ? 4 : 2, "weights")) != MOE_OK) return s;
  if ((s = check_aligned(sc, 1, 4, "scales")) != MOE_OK) return s;
  if (codes) {
    const void* all[] = {x, y, residual, residual_out, weight, post_weight, codes};
    if ((s = check_aligned(all, 7, 16, "buffers of a call with codes")) != MOE_OK) return s;
  }
  const size_t m = (size_t)n * d, sm = m * (sf ? 4 : 2), wm = (size_t)d * (wf ? 4 : 2);
  const Span in[] = {{x, m * 2}, {residual, sm, true}, {weight, wm}, {post_weight, wm}};
  const Span out[] = {{y, m * 2}, {residual_out, sm, true}, {codes, m}, {scales, m / 128 * 4}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_rms_norm(x, residual, post_weight, weight, n, d, eps, sf, wf, y,
                                   residual_out, codes, scales, (hipStream_t)stream),
              "moe_rms_norm");
}

size_t moe_rms_norm_backward_workspace_bytes(int64_t n, int32_t d) {
  if (n < 0 || n > kNormMaxN || d < 1 || d > moe::kNormMaxD) return 0;
  return up((size_t)moe::rms_norm_grad_blocks(n, d) * 2u * (size_t)d * sizeof(float));
}

moe_status_t moe_rms_norm_backward(const uint16_t* grad_y, const void* r, const uint16_t* x,
                                   const void* grad_residual, const void* weight,
                                   const void* post_weight, int64_t n, int32_t d, float eps,
                                   uint32_t flags, uint16_t* grad_x, void* grad_residual_out,
                                   float* grad_weight, float* grad_post_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  moe_status_t s = check_norm(n, d, eps, flags);
  if (s != MOE_OK) return s;
  if (!weight) return fail(MOE_ERR_INVALID_ARGUMENT, "weight is required");
  if (n > 0 && (!grad_y || !r)) return fail(MOE_ERR_INVALID_ARGUMENT, "grad_y and r are required");
  if (n > 0 && (x != nullptr) != (post_weight != nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "x belongs to post_weight: both or neither");
  if (grad_post_weight && !post_weight)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_post_weight needs post_weight");
  // the gradients of no rows are empty (and may be NULL); those of the weights are zeros
  if (n == 0 && !grad_weight && !grad_post_weight) return moe::set_error(MOE_OK, "");
  if (!grad_x && !grad_residual_out && !grad_weight && !grad_post_weight)
    return fail(MOE_ERR_INVALID_ARGUMENT, "an output is required");
  const bool sf = (flags & MOE_NORM_STREAM_F32) != 0, wf = (flags & MOE_NORM_WEIGHT_F32) != 0;
  const void* bf[] = {grad_y, x, grad_x};
  const void* st[] = {r, grad_residual, grad_residual_out};
  const void* wt[] = {weight, post_weight};
  const void* f4[] = {grad_weight, grad_post_weight};
  if ((s = check_aligned(bf, 3, 2, "grad_y, x and grad_x")) != MOE_OK) return s;
  if ((s = check_aligned(st, 3, sf ? 4 : 2, "r and the residual's gradients")) != MOE_OK) return s;
  if ((s = check_aligned(wt, 2, wf ? 4 : 2, "weights")) != MOE_OK) return s;
  if ((s = check_aligned(f4, 2, 4, "weight gradients")) != MOE_OK) return s;
  const size_t need = moe_rms_norm_backward_workspace_bytes(n, d);
  if ((s = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return s;
  const size_t m = (size_t)n * d, sm = m * (sf ? 4 : 2), wm = (size_t)d * (wf ? 4 : 2);
  const Span in[] = {{grad_y, m * 2}, {r, sm}, {x, m * 2}, {grad_residual, sm}, {weight, wm},
                     {post_weight, wm}};
  const Span out[] = {{grad_x, m * 2}, {grad_residual_out, sm}, {grad_weight, (size_t)d * 4},
                      {grad_post_weight, (size_t)d * 4}, {workspace, need}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_rms_norm_grad(grad_y, r, x, grad_residual, weight, post_weight, n, d,
                                        eps, sf, wf, grad_x, grad_residual_out, grad_weight,
                                        grad_post_weight, (float*)workspace, (hipStream_t)stream),
              "moe_rms_norm_backward");
}

size_t moe_balance_workspace_bytes(int64_t N, int32_t E, int32_t n_seg) {
  if (!balance_sizes_ok(N, E, n_seg)) return 0;
  size_t bytes;
  (void)carve_balance(nullptr, N, E, n_seg, &bytes);
  return bytes;
}

moe_status_t moe_balance_loss(const float* logits, const int32_t* topk_ids,
                              const int32_t* counts_in, const int32_t* seg_begin,
                              const int32_t* seg_end, int64_t N, int32_t E, int32_t K,
                              int32_t n_seg, int32_t score, float coef, float* loss,
                              int32_t* counts_out, float* mean_scores, void* workspace,
                              size_t workspace_bytes, void* stream) {
  moe_status_t s = check_balance(N, E, n_seg, seg_begin, seg_end, score, coef);
  if (s != MOE_OK) return s;
  if (K < 1 || K > MOE_MAX_K || K >= E)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "K=%d must satisfy 1 <= K <= %d and K < E", K, MOE_MAX_K);
  if (!logits || !loss) return fail(MOE_ERR_INVALID_ARGUMENT, "logits and loss are required");
  if (!topk_ids && !counts_in)
    return fail(MOE_ERR_INVALID_ARGUMENT, "topk_ids or counts_in is required");
  const void* p4[] = {logits, topk_ids, counts_in, seg_begin, seg_end, loss, counts_out, mean_scores};
  if ((s = check_aligned(p4, 8, 4, "buffers")) != MOE_OK) return s;
  const size_t need = moe_balance_workspace_bytes(N, E, n_seg);
  if ((s = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return s;
  const size_t gb = (size_t)n_seg * 4, cb = gb * E;
  const Span in[] = {{logits, (size_t)N * E * 4}, {topk_ids, (size_t)N * K * 4}, {counts_in, cb},
                     {seg_begin, gb}, {seg_end, gb}};
  const Span out[] = {{loss, 4}, {counts_out, cb}, {mean_scores, cb}, {workspace, need}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  size_t bytes;
  const moe::BalanceWork w = carve_balance(workspace, N, E, n_seg, &bytes);
  return done(moe::launch_balance_loss(logits, topk_ids, counts_in, seg_begin, seg_end, N, E, K,
                                       n_seg, score, coef, w, loss, counts_out, mean_scores,
                                       (hipStream_t)stream),
              "moe_balance_loss");
}

moe_status_t moe_balance_loss_backward(const float* logits, const int32_t* counts,
                                       const int32_t* seg_begin, const int32_t* seg_end,
                                       int64_t N, int32_t E, int32_t n_seg, int32_t score,
                                       float coef, const float* grad_loss,
                                       const float* grad_logits, float* grad_logits_out,
                                       void* stream) {
  moe_status_t s = check_balance(N, E, n_seg, seg_begin, seg_end, score, coef);
  if (s != MOE_OK) return s;
  if (!logits || !counts || !grad_logits_out)
    return fail(MOE_ERR_INVALID_ARGUMENT, "logits, counts and grad_logits_out are required");
  const void* p4[] = {logits, counts, seg_begin, seg_end, grad_loss, grad_logits, grad_logits_out};
  if ((s = check_aligned(p4, 7, 4, "buffers")) != MOE_OK) return s;
  const size_t zb = (size_t)N * E * 4, gb = (size_t)n_seg * 4;
  const Span in[] = {{logits, zb}, {counts, gb * E}, {seg_begin, gb}, {seg_end, gb},
                     {grad_loss, 4}, {grad_logits, zb, true}};
  const Span out[] = {{grad_logits_out, zb, true}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_balance_grad(logits, counts, seg_begin, seg_end, N, E, n_seg, score, coef,
                                       grad_loss, grad_logits, grad_logits_out,
                                       (hipStream_t)stream),
              "moe_balance_loss_backward");
}

}  // extern "C"
