// C ABI of the operators that take the layer apart: grouping, rows to the
// experts and back with their gradients, and the 8-bit integer products.
// Argument checks and the launches on the caller's stream; nothing else.
#include <hip/hip_runtime.h>

#include "../../include/moe_mi355x.h"
#include "api_checks.h"
#include "kernels.h"

using namespace moe::api;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxRows = kMaxTokens * MOE_MAX_K;
constexpr int kMaxD = 8192, kMaxDepth = moe::kInt8MaxDepth;

bool group_sizes_ok(int64_t N, int32_t E, int32_t K) {
  return N >= 0 && N <= kMaxTokens && E >= 1 && E <= MOE_MAX_E && K >= 1 && K <= MOE_MAX_K;
}

// Sizes, flags and alignment of the row calls.  kept: rows in 8 bits take part;
// rows: the buffers whose rows move; f32s: those of 32-bit words.
template <int R, int F>
moe_status_t check_rows(int64_t N, int32_t d, int32_t K, uint32_t flags, bool kept,
                        const void* const (&rows)[R], const void* const (&f32s)[F]) {
  if (N < 0 || N > kMaxTokens || d < 1 || d > kMaxD || K < 1 || K > MOE_MAX_K)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "N=%lld d=%d K=%d: need 0 <= N <= 2^24, 1 <= d <= %d and 1 <= K <= %d",
                (long long)N, d, K, kMaxD, MOE_MAX_K);
  if (flags & ~MOE_ROWS_F32) return fail(MOE_ERR_INVALID_ARGUMENT, "unknown flag bits 0x%x", flags);
  if (kept && (flags & MOE_ROWS_F32))
    return fail(MOE_ERR_INVALID_ARGUMENT, "rows kept in 8 bits belong to bf16 rows");
  if (kept && d % 128)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "d=%d: rows kept in 8 bits need a multiple of 128", d);
  moe_status_t s = check_aligned(rows, R, kept ? 16 : (flags & MOE_ROWS_F32) ? 4 : 2,
                                 kept ? "rows of a call with codes" : "rows");
  if (s != MOE_OK) return s;
  return check_aligned(f32s, F, 4, "src_pos, weights and scales");
}

size_t row_bytes(uint32_t flags) { return (flags & MOE_ROWS_F32) ? 4 : 2; }

}  // namespace

extern "C" {

size_t moe_group_workspace_bytes(int64_t N, int32_t E, int32_t K) {
  if (!group_sizes_ok(N, E, K)) return 0;
  return up(moe::group_work_words(N * K, E) * 4 + 4);
}

moe_status_t moe_group(const int32_t* topk_ids, int64_t N, int32_t E, int32_t K, int32_t* counts,
                       int32_t* offsets, int32_t* sorted_src, int32_t* src_pos, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!group_sizes_ok(N, E, K))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "N=%lld E=%d K=%d: need 0 <= N <= 2^24, 1 <= E <= %d and 1 <= K <= %d",
                (long long)N, E, K, MOE_MAX_E, MOE_MAX_K);
  if (!counts || !offsets)
    return fail(MOE_ERR_INVALID_ARGUMENT, "counts and offsets are required");
  if (N > 0 && (!topk_ids || !sorted_src || !src_pos))
    return fail(MOE_ERR_INVALID_ARGUMENT, "topk_ids, sorted_src and src_pos are required");
  const void* p4[] = {topk_ids, counts, offsets, sorted_src, src_pos};
  moe_status_t s = check_aligned(p4, 5, 4, "buffers");
  if (s != MOE_OK) return s;
  const size_t need = moe_group_workspace_bytes(N, E, K);
  if ((s = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return s;
  const size_t pb = (size_t)N * K * 4;
  const Span in[] = {{topk_ids, pb}};
  const Span out[] = {{counts, (size_t)E * 4}, {offsets, (size_t)E * 4 + 4}, {sorted_src, pb},
                      {src_pos, pb}, {workspace, need}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_group(topk_ids, N * K, E, counts, offsets, sorted_src, src_pos,
                                (uint32_t*)workspace, (hipStream_t)stream),
              "moe_group");
}

moe_status_t moe_permute(const void* x, const float* x_scales, const int32_t* src_pos, int64_t N,
                         int32_t d, int32_t K, uint32_t flags, void* rows, void* stream) {
  const bool kept = x_scales != nullptr;
  const void* r[] = {x, rows};
  const void* f[] = {src_pos, x_scales};
  moe_status_t s = check_rows(N, d, K, flags, kept, r, f);
  if (s != MOE_OK) return s;
  if (N == 0) return moe::set_error(MOE_OK, "");
  if (!x || !src_pos || !rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "x, src_pos and rows are required");
  const size_t m = (size_t)N * d, es = row_bytes(flags);
  const Span in[] = {{x, kept ? m : m * es}, {x_scales, m / 128 * 4}, {src_pos, (size_t)N * K * 4}};
  const Span out[] = {{rows, m * K * es}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_permute_rows(x, x_scales, src_pos, N, d, K, es == 4, rows,
                                       (hipStream_t)stream),
              "moe_permute");
}

moe_status_t moe_permute_backward(const void* grad_rows, const int32_t* src_pos, int64_t N,
                                  int32_t d, int32_t K, uint32_t flags, void* grad_x,
                                  void* stream) {
  const void* r[] = {grad_rows, grad_x};
  const void* f[] = {src_pos};
  moe_status_t s = check_rows(N, d, K, flags, false, r, f);
  if (s != MOE_OK) return s;
  if (N == 0) return moe::set_error(MOE_OK, "");
  if (!grad_rows || !src_pos || !grad_x)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_rows, src_pos and grad_x are required");
  const size_t m = (size_t)N * d * row_bytes(flags);
  const Span in[] = {{grad_rows, m * K}, {src_pos, (size_t)N * K * 4}};
  const Span out[] = {{grad_x, m}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_unpermute_rows(grad_rows, src_pos, nullptr, nullptr, N, d, K,
                                         (flags & MOE_ROWS_F32) != 0, grad_x, nullptr, nullptr,
                                         (hipStream_t)stream),
              "moe_permute_backward");
}

moe_status_t moe_unpermute(const void* rows, const int32_t* src_pos, const float* weights,
                           const void* base, int64_t N, int32_t d, int32_t K, uint32_t flags,
                           void* y, uint8_t* codes, float* scales, void* stream) {
  const bool kept = codes != nullptr;
  const void* r[] = {rows, base, y, codes};
  const void* f[] = {src_pos, weights, scales};
  moe_status_t s = check_rows(N, d, K, flags, kept, r, f);
  if (s != MOE_OK) return s;
  if (N == 0) return moe::set_error(MOE_OK, "");
  if ((codes == nullptr) != (scales == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "codes and scales: both or neither");
  if (!rows || !src_pos || !y)
    return fail(MOE_ERR_INVALID_ARGUMENT, "rows, src_pos and y are required");
  const size_t m = (size_t)N * d, es = row_bytes(flags), pb = (size_t)N * K * 4;
  const Span in[] = {{rows, m * K * es}, {src_pos, pb}, {weights, pb}, {base, m * es}};
  const Span out[] = {{y, m * es}, {codes, m * K}, {scales, m * K / 128 * 4}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_unpermute_rows(rows, src_pos, weights, base, N, d, K, es == 4, y, codes,
                                         scales, (hipStream_t)stream),
              "moe_unpermute");
}

moe_status_t moe_unpermute_backward(const void* grad_y, const void* rows, const float* row_scales,
                                    const int32_t* src_pos, const float* weights, int64_t N,
                                    int32_t d, int32_t K, uint32_t flags, void* grad_rows,
                                    float* grad_weights, void* stream) {
  const bool kept = row_scales != nullptr;
  const void* r[] = {grad_y, rows, grad_rows};
  const void* f[] = {src_pos, weights, row_scales, grad_weights};
  moe_status_t s = check_rows(N, d, K, flags, kept, r, f);
  if (s != MOE_OK) return s;
  if (N == 0) return moe::set_error(MOE_OK, "");
  if (!grad_rows && !grad_weights)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_rows or grad_weights is required");
  if (!grad_y || !src_pos)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_y and src_pos are required");
  if (grad_weights && !rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "grad_weights needs rows");
  const size_t m = (size_t)N * d, es = row_bytes(flags), pb = (size_t)N * K * 4;
  const Span in[] = {{grad_y, m * es}, {rows, m * K * (kept ? 1 : es)},
                     {row_scales, m * K / 128 * 4}, {src_pos, pb}, {weights, pb}};
  const Span out[] = {{grad_rows, m * K * es}, {grad_weights, pb}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_unpermute_grad(grad_y, rows, row_scales, src_pos, weights, N, d, K,
                                         es == 4, grad_rows, grad_weights, (hipStream_t)stream),
              "moe_unpermute_backward");
}

moe_status_t moe_int8_quantize_rows(const uint16_t* x, int64_t n, int32_t cols, int8_t* codes,
                                    float* scales, void* stream) {
  if (n < 0 || n > kMaxRows || cols < 16 || cols > kMaxDepth || cols % 16)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "n=%lld cols=%d: need 0 <= n <= 2^27 and 16 <= cols <= %d, cols %% 16 == 0",
                (long long)n, cols, kMaxDepth);
  if (n == 0) return moe::set_error(MOE_OK, "");
  if (!x || !codes || !scales)
    return fail(MOE_ERR_INVALID_ARGUMENT, "x, codes and scales are required");
  const void* r[] = {x, codes};
  const void* f[] = {scales};
  moe_status_t s = check_aligned(r, 2, 16, "x and codes");
  if (s != MOE_OK) return s;
  if ((s = check_aligned(f, 1, 4, "scales")) != MOE_OK) return s;
  const size_t m = (size_t)n * cols;
  const Span in[] = {{x, m * 2}};
  const Span out[] = {{codes, m}, {scales, (size_t)n * 4}};
  if ((s = check_alias(in, out)) != MOE_OK) return s;
  return done(moe::launch_quant_int8(x, n, cols, codes, scales, (hipStream_t)stream),
              "moe_int8_quantize_rows");
}

moe_status_t moe_int8_matmul(const moe_int8_matmul_t* p, uint16_t* out, void* stream) {
  if (!p) return fail(MOE_ERR_INVALID_ARGUMENT, "problem is NULL");
  if (p->rows < 0 || p->rows > kMaxRows || p->a_rows < 0 || p->a_rows > kMaxRows || p->k < 16 ||
      p->k > kMaxDepth || p->k % 16 || p->cols < 8 || p->cols > kMaxDepth || p->cols % 8 ||
      p->E < 1 || p->E > MOE_MAX_E || p->K < 1 || p->K > MOE_MAX_K)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "rows=%lld a_rows=%lld k=%d cols=%d E=%d K=%d: need 0 <= rows, a_rows <= 2^27, "
                "16 <= k <= %d, k %% 16 == 0, 8 <= cols <= %d, cols %% 8 == 0, 1 <= E <= %d, "
                "1 <= K <= %d",
                (long long)p->rows, (long long)p->a_rows, p->k, p->cols, p->E, p->K, kMaxDepth,
                kMaxDepth, MOE_MAX_E, MOE_MAX_K);
  if (!p->offsets && (p->E != 1 || p->sorted_src))
    return fail(MOE_ERR_INVALID_ARGUMENT, "without offsets there is one weight and no sorted_src");
  if ((p->w_up == nullptr) != (p->w_up_scales == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "w_up and w_up_scales: both or neither");
  if (!p->sorted_src && p->a_rows != p->rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "without sorted_src a_rows must be rows");
  if (p->sorted_src && (uint64_t)p->a_rows * p->k > moe::kInt8MaxGathered)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "a_rows=%lld k=%d: a gathered a must be at most 4 GiB - "
                "512 KiB", (long long)p->a_rows, p->k);
  if (p->rows == 0) return moe::set_error(MOE_OK, "");
  if (p->a_rows == 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rows of an empty a");
  if (!p->a || !p->a_scales || !p->w || !p->w_scales || !out)
    return fail(MOE_ERR_INVALID_ARGUMENT, "a, w, their scales and out are required");
  const void* wide[] = {p->a, p->w, p->w_up, out};
  const void* f4[] = {p->a_scales, p->w_scales, p->w_up_scales, p->offsets, p->sorted_src};
  moe_status_t s = check_aligned(wide, 4, 16, "a, w, w_up and out");
  if (s != MOE_OK) return s;
  if ((s = check_aligned(f4, 5, 4, "scales, offsets and sorted_src")) != MOE_OK) return s;
  const size_t wr = (size_t)p->E * p->cols, wb = wr * p->k;
  const Span in[] = {{p->a, (size_t)p->a_rows * p->k}, {p->a_scales, (size_t)p->a_rows * 4},
                     {p->w, wb}, {p->w_scales, wr * 4}, {p->w_up, wb}, {p->w_up_scales, wr * 4},
                     {p->offsets, (size_t)p->E * 4 + 4}, {p->sorted_src, (size_t)p->rows * 4}};
  const Span outs[] = {{out, (size_t)p->rows * p->cols * 2}};
  if ((s = check_alias(in, outs)) != MOE_OK) return s;
  moe::Int8Args a{};
  a.a = p->a;
  a.a_scales = p->a_scales;
  a.w = p->w;
  a.w_scales = p->w_scales;
  a.w_up = p->w_up;
  a.w_up_scales = p->w_up_scales;
  a.offsets = p->offsets;
  a.sorted_src = p->sorted_src;
  a.out = out;
  a.a_rows = p->a_rows;
  a.rows = p->rows;
  a.k = p->k;
  a.cols = p->cols;
  a.E = p->E;
  a.K = p->K;
  return done(moe::launch_int8_matmul(a, (hipStream_t)stream), "moe_int8_matmul");
}

}  // extern "C"
