// C ABI of the operators that pick weights by token: argument checks, then the
// launchers of group.cu, moe.cu and lora.cu. See include/wq.h for the contract of
// each call.
#include "wq.h"
#include "wq_internal.h"

#include <cmath>

namespace wq {
namespace {

wq_status check_choices(int64_t T, int k) {
  if (T < 0 || T > kMaxDim) return fail(WQ_EINVAL, "T must be in 0..2^31-1 (got %lld)", (long long)T);
  if (k < 1 || k > kMaxTopK) return fail(WQ_EINVAL, "k must be in 1..%d (got %d)", kMaxTopK, k);
  if (T > kMaxDim / k) return fail(WQ_EINVAL, "T * k must be below 2^31 (got %lld * %d)", (long long)T, k);
  return WQ_OK;
}

wq_status check_experts(int64_t E) {
  if (E < 1 || E > kMaxGroups) return fail(WQ_EINVAL, "E must be in 1..%d (got %lld)", kMaxGroups, (long long)E);
  return WQ_OK;
}

// R sorted rows: none only where no token is (what moe_sort gives for none).
wq_status check_rows(int64_t R, int64_t T) { return R == 0 && T == 0 ? WQ_OK : check_size(R, "R"); }

wq_status check_stride(int64_t stride, int64_t least, const char* name) {
  if (stride < least || stride > kMaxDim)
    return fail(WQ_EINVAL, "%s must be in %lld..2^31-1 (got %lld)", name, (long long)least, (long long)stride);
  return WQ_OK;
}

wq_status check_route(const RouteArgs& a) {
  if (a.type != WQ_LOGITS_BF16 && a.type != WQ_LOGITS_F32)
    return fail(WQ_EINVAL, "logits_type must be WQ_LOGITS_BF16 or WQ_LOGITS_F32 (got %d)", a.type);
  WQ_TRY(check_choices(a.T, a.k));
  WQ_TRY(check_experts(a.E));
  if (a.k > a.E) return fail(WQ_EINVAL, "k must be at most E (got %d and %lld)", a.k, (long long)a.E);
  if (a.score != WQ_SCORE_SOFTMAX && a.score != WQ_SCORE_SIGMOID)
    return fail(WQ_EINVAL, "score must be WQ_SCORE_SOFTMAX or WQ_SCORE_SIGMOID (got %d)", a.score);
  if (!std::isfinite(a.scale)) return fail(WQ_EINVAL, "scale must be finite");
  WQ_TRY(check_stride(a.ld, a.E, "ld"));
  return WQ_OK;
}

wq_status check_16bit(const void* p, const char* name) {
  if (p == nullptr) return fail(WQ_EINVAL, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 1u) != 0) return fail(WQ_EINVAL, "%s is not 2-byte aligned", name);
  return WQ_OK;
}

// Whether two 2-byte matrices of `rows` rows share a value; side by side in rows of
// one stride (columns of one buffer) they do not.
bool share_values(const void* p, int64_t p_stride, int64_t p_cols, const void* q, int64_t q_stride, int64_t q_cols,
                  int64_t rows) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t a_end = a + 2 * ((rows - 1) * p_stride + p_cols), b_end = b + 2 * ((rows - 1) * q_stride + q_cols);
  if (a >= b_end || b >= a_end) return false;
  if (p_stride != q_stride || ((a ^ b) & 1) != 0) return true;
  const int64_t apart = static_cast<int64_t>(a < b ? b - a : a - b) / 2 % p_stride;  // from the lower one's row
  const int64_t lower = a < b ? p_cols : q_cols, higher = a < b ? q_cols : p_cols;
  return apart < lower || apart + higher > p_stride;
}

}  // namespace
}  // namespace wq

using namespace wq;

extern "C" {

wq_status moe_route(const void* logits, int logits_type, int64_t ld, int64_t T, int64_t E, int k, int score,
                    int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  clear_error();
  const RouteArgs a{logits, logits_type, ld, T, E, k, score, renormalize, scale};
  WQ_TRY(check_route(a));
  if (T == 0) return WQ_OK;
  WQ_PTR(logits);
  WQ_PTR32(ids);
  WQ_PTR32(weights);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_moe_route(c, a, ids, weights), "moe_route launch");
}

wq_status moe_route_grad(const void* logits, int logits_type, int64_t ld, int64_t T, int64_t E, int k, int score,
                         int renormalize, float scale, const int32_t* ids, const float* dweights, void* dlogits,
                         void* stream) {
  clear_error();
  const RouteArgs a{logits, logits_type, ld, T, E, k, score, renormalize, scale};
  WQ_TRY(check_route(a));
  if (T == 0) return WQ_OK;
  WQ_PTR(logits);
  WQ_PTR32(ids);
  WQ_PTR32(dweights);
  WQ_PTR(dlogits);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_moe_route_grad(c, a, ids, dweights, dlogits), "moe_route_grad launch");
}

wq_status moe_sort(const wq_bf16* x, int64_t x_stride, int64_t T, int64_t D, const int32_t* ids, int k, int64_t E,
                   wq_bf16* out, int32_t* offsets, int32_t* slots, int32_t* bad_count, void* stream) {
  clear_error();
  WQ_TRY(check_choices(T, k));
  WQ_TRY(check_experts(E));
  const bool rows = x != nullptr || out != nullptr;
  if (rows && T > 0) {
    WQ_TRY(check_size(D, "D"));
    WQ_TRY(check_stride(x_stride, D, "x_stride"));
  }
  if (T > 0) {
    if (rows) {
      WQ_PTR(x);
      WQ_PTR(out);
    }
    WQ_PTR32(ids);
    WQ_PTR32(slots);
  }
  WQ_PTR32(offsets);
  WQ_OPT32(bad_count);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const ChoiceRows r{slots, nullptr, T, T * k, rows ? D : 1, k};
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(launch_moe_sort(c, r, ids, E, x, rows ? x_stride : 1, out, offsets, slots, bad_count),
                  "moe_sort launch");
}

wq_status moe_combine(const wq_bf16* y, int64_t R, const int32_t* slots, const float* weights,
                      const wq_bf16* residual, int64_t T, int64_t D, int k, wq_bf16* out, void* stream) {
  clear_error();
  WQ_TRY(check_choices(T, k));
  WQ_TRY(check_size(D, "D"));
  WQ_TRY(check_rows(R, T));
  if (T == 0) return WQ_OK;
  WQ_PTR(y);
  WQ_PTR32(slots);
  WQ_OPT32(weights);
  if (residual != nullptr) WQ_PTR(residual);
  WQ_PTR(out);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const ChoiceRows r{slots, weights, T, R, D, k};
  return launched(launch_moe_combine(c, r, y, residual, out), "moe_combine launch");
}

wq_status moe_combine_grad(const wq_bf16* dout, const wq_bf16* y, int64_t R, const int32_t* slots,
                           const float* weights, int64_t T, int64_t D, int k, wq_bf16* dy, float* dweights,
                           void* stream) {
  clear_error();
  WQ_TRY(check_choices(T, k));
  WQ_TRY(check_size(D, "D"));
  WQ_TRY(check_rows(R, T));
  if (T == 0) return WQ_OK;
  WQ_PTR(dout);
  WQ_PTR(y);
  WQ_PTR32(slots);
  WQ_PTR32(weights);
  WQ_PTR(dy);
  WQ_PTR32(dweights);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const ChoiceRows r{slots, weights, T, R, D, k};
  return launched(launch_moe_combine_grad(c, r, dout, y, dy, dweights), "moe_combine_grad launch");
}

size_t lora_workspace_bytes(int64_t M, int64_t n, int64_t r) {
  if (M < 1 || M > kMaxDim || n < 1 || n > kMaxGroups || r < 1 || r > kMaxRank) return 0;
  return lora_ws_bytes(M, n, r);
}

wq_status lora_gemm(const wq_bf16* x, int64_t x_stride, int64_t M, int64_t K, const wq_bf16* A, const wq_bf16* B,
                    int64_t n, int64_t r, int64_t N, const int32_t* adapter, const float* scale, const wq_bf16* base,
                    int64_t base_stride, wq_bf16* y, int64_t y_stride, void* workspace, size_t ws_bytes,
                    void* stream) {
  clear_error();
  if (M < 0 || M > kMaxDim) return fail(WQ_EINVAL, "M must be in 0..2^31-1 (got %lld)", (long long)M);
  WQ_TRY(check_size(K, "K"));
  WQ_TRY(check_size(N, "N"));
  if (K % 8 != 0) return fail(WQ_EINVAL, "K must be a multiple of 8 (got %lld)", (long long)K);
  if (n < 1 || n > kMaxGroups) return fail(WQ_EINVAL, "n must be in 1..%d (got %lld)", kMaxGroups, (long long)n);
  if (r < 8 || r > kMaxRank || r % 8 != 0)
    return fail(WQ_EUNSUPPORTED, "r must be a multiple of 8 in 8..%d (got %lld)", kMaxRank, (long long)r);
  if (M == 0) return WQ_OK;
  WQ_TRY(check_stride(x_stride, K, "x_stride"));
  if (x_stride % 8 != 0) return fail(WQ_EINVAL, "x_stride must be a multiple of 8 (got %lld)", (long long)x_stride);
  WQ_TRY(check_stride(base_stride, N, "base_stride"));
  WQ_TRY(check_stride(y_stride, N, "y_stride"));
  WQ_PTR(x);
  WQ_PTR(A);
  WQ_PTR(B);
  WQ_PTR32(adapter);
  WQ_OPT32(scale);
  WQ_TRY(check_16bit(base, "base"));
  WQ_TRY(check_16bit(y, "y"));
  if (y == base && y_stride != base_stride)
    return fail(WQ_EINVAL, "y is base: y_stride must be base_stride (got %lld and %lld)", (long long)y_stride,
                (long long)base_stride);
  if (y != base && share_values(base, base_stride, N, y, y_stride, N, M))
    return fail(WQ_EINVAL, "y must be base or must not overlap it");
  if (share_values(x, x_stride, K, y, y_stride, N, M)) return fail(WQ_EINVAL, "y must not overlap x");
  WQ_TRY(check_space(workspace, ws_bytes, lora_ws_bytes(M, n, r), "workspace"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const LoraArgs a{x, x_stride, M, K, N, n, r, A, B, adapter, scale, base, base_stride, y, y_stride, workspace};
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(launch_lora(c, a), "lora_gemm launch");
}

}  // extern "C"
