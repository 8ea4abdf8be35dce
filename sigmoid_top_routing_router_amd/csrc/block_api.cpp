// C ABI of the operators around the layer: the residual norm and the balance
// loss, forward and backward.  Argument checks, workspace carving and the
// launches on the caller's stream; nothing else.
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

}  // namespace

extern "C" {

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
  const void* in[] = {x, weight, post_weight, residual};
  const void* out[] = {y, codes, scales, residual_out};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (in[i] && in[i] == out[j] && !(in[i] == residual && out[j] == residual_out))
        return fail(MOE_ERR_INVALID_ARGUMENT, "an output aliases an input");
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
  const void* in[] = {grad_y, r, x, grad_residual, weight, post_weight};
  const void* out[] = {grad_x, grad_residual_out, grad_weight, grad_post_weight};
  for (const void* i : in)
    for (const void* o : out)
      if (i && i == o) return fail(MOE_ERR_INVALID_ARGUMENT, "an output aliases an input");
  s = check_workspace(workspace, workspace_bytes, moe_rms_norm_backward_workspace_bytes(n, d));
  if (s != MOE_OK) return s;
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
  if (counts_in && counts_in == counts_out)
    return fail(MOE_ERR_INVALID_ARGUMENT, "counts_out aliases counts_in");
  s = check_workspace(workspace, workspace_bytes, moe_balance_workspace_bytes(N, E, n_seg));
  if (s != MOE_OK) return s;
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
  if (grad_logits_out == logits)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_logits_out must not be logits");
  return done(moe::launch_balance_grad(logits, counts, seg_begin, seg_end, N, E, n_seg, score, coef,
                                       grad_loss, grad_logits, grad_logits_out,
                                       (hipStream_t)stream),
              "moe_balance_loss_backward");
}

}  // extern "C"
