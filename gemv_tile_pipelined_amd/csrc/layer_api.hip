// layer_api.hip -- the C ABI of the operators around the products (4-bit
// weights, norm, routing, rows): argument checks and launches, as in api.hip.
#include "api_common.hpp"
#include "kernels.hpp"

namespace {

using gt::misaligned;
using gt::to_status;

constexpr int64_t kMax32 = (int64_t{1} << 31) - 512;
// A grid's threads along x are counted in 32 bits, its workgroups along y in 16.
constexpr int64_t kMaxFp4N = int64_t{1} << 25;
constexpr int64_t kMaxFp4M = int64_t{1} << 19;
constexpr int64_t kMaxFp4K = 4194272;
constexpr int64_t kMaxFp4Elements = (int64_t{1} << 36) - 4096;
constexpr int64_t kMaxNormC = 32768;
constexpr int64_t kMaxTopkT = (int64_t{1} << 26) - 64;
constexpr int64_t kMaxExperts = 1024, kMaxChoices = 32, kMaxExpertGroups = 64;
constexpr int64_t kMaxTokens = (int64_t{1} << 24) - 1;
constexpr int64_t kMaxRowK = int64_t{1} << 20;

int run_quantize_fp4(int dtype, const void *x, void *q, void *scale, int64_t N, int64_t K, void *stream) {
  if (N < 0 || K < 0) return GEMVTILE_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return GEMVTILE_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return GEMVTILE_ERR_INVALID_ARG;
  if (K % 32 != 0 || N > kMaxFp4Elements / K) return GEMVTILE_ERR_UNSUPPORTED;
  if (misaligned(x, 16) || misaligned(q, 16)) return GEMVTILE_ERR_UNSUPPORTED;
  return to_status(gt::launch_quantize_fp4(dtype, x, q, scale, N * K, static_cast<hipStream_t>(stream)));
}

int run_gemv_fp4(int dtype, const void *x, const void *W, const void *sW, void *y, int64_t M, int64_t N, int64_t K,
                 void *stream) {
  if (M < 0 || N < 0 || K < 0) return GEMVTILE_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMVTILE_OK;
  if (y == nullptr || (K > 0 && (x == nullptr || W == nullptr || sW == nullptr))) return GEMVTILE_ERR_INVALID_ARG;
  if (M > kMaxFp4M || N > kMaxFp4N || K > kMaxFp4K || K % 32 != 0) return GEMVTILE_ERR_UNSUPPORTED;
  if (misaligned(y, 2) || (K > 0 && (misaligned(x, 16) || misaligned(W, 16)))) return GEMVTILE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (K == 0) return to_status(gt::launch_fill_zero_f16(y, M * N, s));
  int cus = 0;
  const int st = gt::current_cu_count(&cus);
  if (st != GEMVTILE_OK) return st;
  return to_status(
      gt::launch_gemv_fp4(dtype, x, W, sW, y, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), cus, s));
}

// fp8: q and scale wanted, y optional; otherwise y wanted.
int run_rmsnorm(int dtype, bool fp8, const void *x, const void *residual, const void *weight, void *h, void *y, void *q,
                float *scale, float *rstd, int64_t T, int64_t C, double eps, void *stream) {
  if (T < 0 || C < 0 || !(eps >= 0.0)) return GEMVTILE_ERR_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr)) {
    if (T > 0 && C > 0) return GEMVTILE_ERR_INVALID_ARG;
  }
  if (T == 0 || C == 0) return GEMVTILE_OK;
  if (x == nullptr || weight == nullptr || (fp8 ? q == nullptr || scale == nullptr : y == nullptr))
    return GEMVTILE_ERR_INVALID_ARG;
  if (T > kMax32 || C > kMaxNormC || C % (fp8 ? 16 : 8) != 0) return GEMVTILE_ERR_UNSUPPORTED;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(weight, 16) || misaligned(h, 16) || misaligned(y, 16) ||
      misaligned(q, 16) || misaligned(scale, 4) || misaligned(rstd, 4))
    return GEMVTILE_ERR_UNSUPPORTED;
  const gt::NormArgs a = {x, residual, weight, h, y, q, scale, rstd, static_cast<int>(T), static_cast<int>(C), eps};
  return to_status(gt::launch_rmsnorm(dtype, a, static_cast<hipStream_t>(stream)));
}

int run_rmsnorm_grad(int dtype, const void *dy, const void *dh, const void *h, const void *weight, const float *rstd, void *dx,
                     float *dweight, int64_t T, int64_t C, void *workspace, int64_t workspace_bytes, void *stream) {
  if (T < 0 || C < 0 || workspace_bytes < 0) return GEMVTILE_ERR_INVALID_ARG;
  if (C == 0) return GEMVTILE_OK;
  if (dweight == nullptr) return GEMVTILE_ERR_INVALID_ARG;
  if (T > 0 && (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr))
    return GEMVTILE_ERR_INVALID_ARG;
  if (T > kMax32 || C > kMaxNormC || C % 8 != 0) return GEMVTILE_ERR_UNSUPPORTED;
  const int64_t need = gemvtile_rmsnorm_grad_workspace(T, C);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GEMVTILE_ERR_INVALID_ARG;
  if (misaligned(dweight, 4) || (T > 0 && (misaligned(dy, 16) || misaligned(dh, 16) || misaligned(h, 16) ||
                                           misaligned(weight, 16) || misaligned(rstd, 4) || misaligned(dx, 16) ||
                                           misaligned(workspace, 16))))
    return GEMVTILE_ERR_UNSUPPORTED;
  const gt::NormGradArgs a = {dy,      dh,      h, weight, rstd, dx, dweight, static_cast<float *>(workspace), static_cast<int>(T),
                              static_cast<int>(C)};
  return to_status(gt::launch_rmsnorm_grad(dtype, a, static_cast<hipStream_t>(stream)));
}

bool score_exists(int score) { return score == GEMVTILE_SCORE_SOFTMAX || score == GEMVTILE_SCORE_SIGMOID; }

int run_topk(int dtype, const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E, int64_t k,
             int64_t groups, int64_t top_groups, int group_best, int score, int norm, float scale, void *stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      k > top_groups * (E / groups) || (group_best != 1 && group_best != 2) || !score_exists(score) || (norm != 0 && norm != 1))
    return GEMVTILE_ERR_INVALID_ARG;
  if (T == 0) return GEMVTILE_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return GEMVTILE_ERR_INVALID_ARG;
  if (T > kMaxTopkT || E > kMaxExperts || k > kMaxChoices || groups > kMaxExpertGroups) return GEMVTILE_ERR_UNSUPPORTED;
  if (misaligned(logits, 16) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4))
    return GEMVTILE_ERR_UNSUPPORTED;
  const gt::RouteArgs r = {T, static_cast<int>(E), static_cast<int>(k), static_cast<int>(groups), static_cast<int>(top_groups),
                           group_best, score, norm, scale};
  return to_status(gt::launch_route_topk(dtype, logits, bias, ids, weights, r, static_cast<hipStream_t>(stream)));
}

int run_topk_grad(int dtype, const void *logits, const int32_t *ids, const float *dweights, void *dlogits, int64_t T, int64_t E,
                  int64_t k, int score, int norm, float scale, void *stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || !score_exists(score) || (norm != 0 && norm != 1)) return GEMVTILE_ERR_INVALID_ARG;
  if (T == 0) return GEMVTILE_OK;
  if (logits == nullptr || ids == nullptr || dweights == nullptr || dlogits == nullptr) return GEMVTILE_ERR_INVALID_ARG;
  if (T > kMaxTopkT || E > kMaxExperts || k > kMaxChoices) return GEMVTILE_ERR_UNSUPPORTED;
  if (misaligned(logits, 16) || misaligned(dlogits, 16) || misaligned(ids, 4) || misaligned(dweights, 4))
    return GEMVTILE_ERR_UNSUPPORTED;
  const gt::RouteArgs r = {T, static_cast<int>(E), static_cast<int>(k), 1, 1, 1, score, norm, scale};
  return to_status(gt::launch_route_topk_grad(dtype, logits, ids, dweights, dlogits, r, static_cast<hipStream_t>(stream)));
}

// The sizes that the row movers share; `step` divides K.
int check_rows(int64_t T, int64_t k, int64_t R, int64_t K, int step) {
  if (T < 0 || k < 1 || R < 0 || K < 0) return GEMVTILE_ERR_INVALID_ARG;
  if (T > kMaxTokens || k > kMaxChoices || R > kMax32 || K > kMaxRowK || K % step != 0) return GEMVTILE_ERR_UNSUPPORTED;
  return GEMVTILE_OK;
}

int run_gather(bool fp8, const void *X, const float *scale, const int32_t *pos, void *Xs, float *scales, int64_t T, int64_t k,
               int64_t R, int64_t K, void *stream) {
  const int st = check_rows(T, k, R, K, fp8 ? 16 : 8);
  if (st != GEMVTILE_OK || T == 0 || K == 0 || R == 0) return st;
  if (X == nullptr || pos == nullptr || Xs == nullptr || (fp8 && (scale == nullptr || scales == nullptr)))
    return GEMVTILE_ERR_INVALID_ARG;
  if (misaligned(X, 16) || misaligned(Xs, 16) || misaligned(pos, 4) || misaligned(scale, 4) || misaligned(scales, 4))
    return GEMVTILE_ERR_UNSUPPORTED;
  return to_status(gt::launch_route_gather(X, scale, pos, Xs, scales, T, R, static_cast<int>(fp8 ? K / 16 : K / 8),
                                           fp8 ? static_cast<int>((K + 127) / 128) : 0, static_cast<int>(k),
                                           static_cast<hipStream_t>(stream)));
}

int run_combine(int dtype, const void *D, const int32_t *pos, const float *weights, void *Y, int64_t T, int64_t k, int64_t R,
                int64_t K, void *stream) {
  const int st = check_rows(T, k, R, K, 8);
  if (st != GEMVTILE_OK || T == 0 || K == 0) return st;
  if (pos == nullptr || Y == nullptr || (R > 0 && D == nullptr)) return GEMVTILE_ERR_INVALID_ARG;
  if (misaligned(D, 16) || misaligned(Y, 16) || misaligned(pos, 4) || misaligned(weights, 4)) return GEMVTILE_ERR_UNSUPPORTED;
  return to_status(gt::launch_route_combine(dtype, D, pos, weights, Y, T, R, static_cast<int>(K / 8), static_cast<int>(k),
                                            static_cast<hipStream_t>(stream)));
}

int run_combine_grad(int dtype, const void *dY, const void *D, const int32_t *pos, const float *weights, void *dD,
                     float *dweights, int64_t T, int64_t k, int64_t R, int64_t K, void *stream) {
  const int st = check_rows(T, k, R, K, 8);
  if (st != GEMVTILE_OK || T == 0) return st;
  if (pos == nullptr || weights == nullptr || dweights == nullptr || (K > 0 && dY == nullptr) ||
      (K > 0 && R > 0 && (D == nullptr || dD == nullptr)))
    return GEMVTILE_ERR_INVALID_ARG;
  if (misaligned(dY, 16) || misaligned(D, 16) || misaligned(dD, 16) || misaligned(pos, 4) || misaligned(weights, 4) ||
      misaligned(dweights, 4))
    return GEMVTILE_ERR_UNSUPPORTED;
  return to_status(gt::launch_route_combine_grad(dtype, dY, D, pos, weights, dD, dweights, T, R, static_cast<int>(K / 8),
                                                 static_cast<int>(k), static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t gemvtile_rmsnorm_grad_workspace(int64_t T, int64_t C) {
  if (T <= 0 || C <= 0 || T > kMax32 || C > kMaxNormC) return 0;
  return int64_t{4} * gt::rmsnorm_grad_parts(T) * C;
}

int64_t gemvtile_route_sort_workspace(int64_t T, int64_t k, int64_t E) {
  if (T <= 0 || k <= 0 || E <= 0 || E > kMaxExperts || T > kMax32 / k) return 0;
  const int blocks = gt::route_sort_blocks(T * k);
  return blocks > 1 ? int64_t{4} * blocks * E : 0;
}

int route_sort(const int32_t *ids, int32_t *offsets, int32_t *pos, int64_t T, int64_t k, int64_t E, void *workspace,
               int64_t workspace_bytes, void *stream) {
  if (T < 0 || k < 1 || E < 1 || workspace_bytes < 0) return GEMVTILE_ERR_INVALID_ARG;
  if (offsets == nullptr || (T > 0 && (ids == nullptr || pos == nullptr))) return GEMVTILE_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMax32 || T > kMax32 / k) return GEMVTILE_ERR_UNSUPPORTED;
  const int64_t need = gemvtile_route_sort_workspace(T, k, E);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GEMVTILE_ERR_INVALID_ARG;
  if (misaligned(offsets, 4) || misaligned(ids, 4) || misaligned(pos, 4) || (need > 0 && misaligned(workspace, 16)))
    return GEMVTILE_ERR_UNSUPPORTED;
  return to_status(gt::launch_route_sort(ids, offsets, pos, static_cast<int *>(workspace), T * k, static_cast<int>(E),
                                         static_cast<hipStream_t>(stream)));
}

int route_gather_fp8(const void *X, const float *scale, const int32_t *pos, void *Xs, float *scales, int64_t T, int64_t k,
                     int64_t R, int64_t K, void *stream) {
  return run_gather(true, X, scale, pos, Xs, scales, T, k, R, K, stream);
}

#define GT_16BIT(fmt, dtype)                                                                                                  \
  int quantize_fp4_##fmt(const void *x, void *q, void *scale, int64_t N, int64_t K, void *stream) {                           \
    return run_quantize_fp4(dtype, x, q, scale, N, K, stream);                                                                \
  }                                                                                                                           \
  int gemv_fp4_##fmt(const void *x, const void *W, const void *scale_W, void *y, int64_t M, int64_t N, int64_t K,             \
                     void *stream) {                                                                                          \
    return run_gemv_fp4(dtype, x, W, scale_W, y, M, N, K, stream);                                                            \
  }                                                                                                                           \
  int rmsnorm_##fmt(const void *x, const void *residual, const void *weight, void *h, void *y, float *rstd, int64_t T,        \
                    int64_t C, double eps, void *stream) {                                                                    \
    return run_rmsnorm(dtype, false, x, residual, weight, h, y, nullptr, nullptr, rstd, T, C, eps, stream);                   \
  }                                                                                                                           \
  int rmsnorm_fp8_##fmt(const void *x, const void *residual, const void *weight, void *h, void *y, void *q, float *scale,     \
                        float *rstd, int64_t T, int64_t C, double eps, void *stream) {                                        \
    return run_rmsnorm(dtype, true, x, residual, weight, h, y, q, scale, rstd, T, C, eps, stream);                            \
  }                                                                                                                           \
  int rmsnorm_grad_##fmt(const void *dy, const void *dh, const void *h, const void *weight, const float *rstd, void *dx,      \
                         float *dweight, int64_t T, int64_t C, void *workspace, int64_t workspace_bytes, void *stream) {      \
    return run_rmsnorm_grad(dtype, dy, dh, h, weight, rstd, dx, dweight, T, C, workspace, workspace_bytes, stream);           \
  }                                                                                                                           \
  int route_gather_##fmt(const void *X, const int32_t *pos, void *Xs, int64_t T, int64_t k, int64_t R, int64_t K,             \
                         void *stream) {                                                                                      \
    return run_gather(false, X, nullptr, pos, Xs, nullptr, T, k, R, K, stream);                                               \
  }                                                                                                                           \
  int route_combine_##fmt(const void *D, const int32_t *pos, const float *weights, void *Y, int64_t T, int64_t k, int64_t R,  \
                          int64_t K, void *stream) {                                                                          \
    return run_combine(dtype, D, pos, weights, Y, T, k, R, K, stream);                                                        \
  }                                                                                                                           \
  int route_combine_grad_##fmt(const void *dY, const void *D, const int32_t *pos, const float *weights, void *dD,             \
                               float *dweights, int64_t T, int64_t k, int64_t R, int64_t K, void *stream) {                   \
    return run_combine_grad(dtype, dY, D, pos, weights, dD, dweights, T, k, R, K, stream);                                    \
  }
GT_16BIT(f16, gt::kF16)
GT_16BIT(bf16, gt::kBF16)
#undef GT_16BIT

#define GT_LOGITS(fmt, dtype)                                                                                                 \
  int route_topk_##fmt(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E, int64_t k,  \
                       int64_t groups, int64_t top_groups, int group_best, int score, int norm, float scale, void *stream) {  \
    return run_topk(dtype, logits, bias, ids, weights, T, E, k, groups, top_groups, group_best, score, norm, scale, stream);  \
  }                                                                                                                           \
  int route_topk_grad_##fmt(const void *logits, const int32_t *ids, const float *dweights, void *dlogits, int64_t T,          \
                            int64_t E, int64_t k, int score, int norm, float scale, void *stream) {                           \
    return run_topk_grad(dtype, logits, ids, dweights, dlogits, T, E, k, score, norm, scale, stream);                         \
  }
GT_LOGITS(f16, gt::kF16)
GT_LOGITS(bf16, gt::kBF16)
GT_LOGITS(f32, gt::kF32)
#undef GT_LOGITS

}  // extern "C"
