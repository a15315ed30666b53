// C ABI of the serving operators: argument checks, then the launchers of
// kv_append.cu, kv_attn.cu, kv_pages.cu and logprobs.cu. See include/wq.h for
// the contract of each call.
#include "wq.h"
#include "wq_internal.h"

#include <cmath>

namespace wq {
namespace {

wq_status check_opt32(const void* p, const char* name) {
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return fail(WQ_EINVAL, "%s is not 4-byte aligned", name);
  return WQ_OK;
}

// A device array of 32-bit values: non-NULL and 4-byte aligned (a caller's
// slice of a larger array, so no more than that).
wq_status check_32(const void* p, const char* name) {
  if (p == nullptr) return fail(WQ_EINVAL, "%s is NULL", name);
  return check_opt32(p, name);
}
#define WQ_PTR32(p) WQ_TRY(check_32((p), #p))
#define WQ_OPT32(p) WQ_TRY(check_opt32((p), #p))

wq_status check_cache(const KvCache& a) {
  if (a.type != WQ_KV_BF16 && a.type != WQ_KV_E4M3)
    return fail(WQ_EINVAL, "kv_type must be WQ_KV_BF16 or WQ_KV_E4M3 (got %d)", a.type);
  WQ_TRY(check_size(a.P, "P"));
  WQ_TRY(check_size(a.Hkv, "Hkv"));
  WQ_TRY(check_size(a.S, "S"));
  WQ_TRY(check_size(a.W, "W"));
  if (a.D != 64 && a.D != 96 && a.D != 128 && a.D != 192 && a.D != 256)
    return fail(WQ_EUNSUPPORTED, "D must be 64, 96, 128, 192 or 256 (got %lld)", (long long)a.D);
  if (a.Hkv > kMaxDim / a.S / a.D / 2)
    return fail(WQ_EINVAL, "a page must have fewer than 2^31 values (Hkv = %lld, S = %lld, D = %lld)",
                (long long)a.Hkv, (long long)a.S, (long long)a.D);
  if (a.W > kMaxDim / a.S)
    return fail(WQ_EINVAL, "W * S must be below 2^31 (got %lld * %lld)", (long long)a.W, (long long)a.S);
  WQ_PTR(a.kv);
  if (a.type == WQ_KV_E4M3) {
    WQ_PTR32(a.k_scale);
    WQ_PTR32(a.v_scale);
  } else if (a.k_scale != nullptr || a.v_scale != nullptr) {
    return fail(WQ_EINVAL, "k_scale and v_scale are for e4m3 caches");
  }
  return WQ_OK;
}

wq_status check_row_stride(int64_t stride, int64_t least, const char* name) {
  if (stride < least || stride % 8 != 0 || stride > kMaxDim)
    return fail(WQ_EINVAL, "%s must be a multiple of 8 in %lld..2^31-1 (got %lld)", name, (long long)least,
                (long long)stride);
  return WQ_OK;
}

wq_status check_space(const void* p, size_t bytes, size_t need, const char* name) {
  if (need == 0) return WQ_OK;
  if (p == nullptr) return fail(WQ_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(WQ_EINVAL, "%s is not 16-byte aligned", name);
  if (bytes < need) return fail(WQ_EINVAL, "%s too small: %zu < %zu bytes", name, bytes, need);
  return WQ_OK;
}

wq_status check_pool(const PagePool& p) {
  WQ_TRY(check_size(p.L, "L"));
  WQ_TRY(check_size(p.P, "P"));
  if (p.page_bytes < 16 || p.page_bytes % 16 != 0 || p.page_bytes > (int64_t{1} << 33))
    return fail(WQ_EINVAL, "page_bytes must be a multiple of 16 in 16..2^33 (got %lld)", (long long)p.page_bytes);
  WQ_PTR(p.kv);
  return WQ_OK;
}

wq_status check_tables(const SeqTables& t) {
  WQ_TRY(check_size(t.B, "B"));
  WQ_TRY(check_size(t.W, "W"));
  WQ_TRY(check_size(t.S, "S"));
  WQ_TRY(check_size(t.P, "P"));
  if (t.W > kMaxDim / t.S)
    return fail(WQ_EINVAL, "W * S must be below 2^31 (got %lld * %lld)", (long long)t.W, (long long)t.S);
  WQ_PTR32(t.table);
  WQ_PTR32(t.lens);
  WQ_PTR32(t.ref);
  return WQ_OK;
}

wq_status launched(cudaError_t e, const char* where) { return e == cudaSuccess ? WQ_OK : cuda_fail(e, where); }

}  // namespace
}  // namespace wq

using namespace wq;

extern "C" {

wq_status kv_append(const wq_bf16* k, const wq_bf16* v, int64_t k_stride, int64_t v_stride, int64_t T,
                    const int32_t* seq, const int32_t* pos, const int32_t* block_table, int64_t B, int64_t W,
                    void* kv, int kv_type, int64_t P, int64_t Hkv, int64_t S, int64_t D, const float* k_scale,
                    const float* v_scale, int32_t* bad_count, void* stream) {
  clear_error();
  const KvCache a{kv, kv_type, P, Hkv, S, D, k_scale, v_scale, block_table, B, W};
  if (T < 0 || T > kMaxDim) return fail(WQ_EINVAL, "T must be in 0..2^31-1 (got %lld)", (long long)T);
  WQ_TRY(check_size(B, "B"));
  WQ_TRY(check_cache(a));
  if (seq == nullptr && T > B)
    return fail(WQ_EINVAL, "without seq there is at most one token per sequence (T = %lld, B = %lld)", (long long)T,
                (long long)B);
  if (T == 0) return WQ_OK;
  WQ_TRY(check_row_stride(k_stride, Hkv * D, "k_stride"));
  WQ_TRY(check_row_stride(v_stride, Hkv * D, "v_stride"));
  WQ_PTR(k);
  WQ_PTR(v);
  WQ_OPT32(seq);
  WQ_PTR32(pos);
  WQ_PTR32(block_table);
  WQ_OPT32(bad_count);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_kv_append(c, a, k, v, k_stride, v_stride, T, seq, pos, bad_count), "kv_append launch");
}

size_t kv_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B < 1 || Hkv < 1 || Hq < Hkv || D < 1) return 0;
  return kv_attn_ws_bytes(B, Hq, Hkv, D);
}

wq_status kv_attn_decode(const wq_bf16* q, int64_t q_stride, const void* kv, int kv_type,
                         const int32_t* block_table, const int32_t* lens, int64_t B, int64_t W, int64_t P,
                         int64_t Hq, int64_t Hkv, int64_t S, int64_t D, const float* k_scale, const float* v_scale,
                         float sm_scale, int64_t window, wq_bf16* out, float* lse, int32_t* bad_count,
                         void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  const KvCache a{const_cast<void*>(kv), kv_type, P, Hkv, S, D, k_scale, v_scale, block_table, B, W};
  if (B < 0 || B > kMaxDim) return fail(WQ_EINVAL, "B must be in 0..2^31-1 (got %lld)", (long long)B);
  WQ_TRY(check_cache(a));
  WQ_TRY(check_size(Hq, "Hq"));
  if (Hq % Hkv != 0)
    return fail(WQ_EINVAL, "Hq must be a multiple of Hkv (got %lld and %lld)", (long long)Hq, (long long)Hkv);
  if (!std::isfinite(sm_scale)) return fail(WQ_EINVAL, "sm_scale must be finite");
  if (window < 0) return fail(WQ_EINVAL, "window must not be negative (got %lld)", (long long)window);
  if (B == 0) return WQ_OK;
  if (B > kMaxDim / Hq) return fail(WQ_EINVAL, "B * Hq must be below 2^31");
  WQ_TRY(check_row_stride(q_stride, Hq * D, "q_stride"));
  WQ_PTR(q);
  WQ_PTR32(block_table);
  WQ_PTR32(lens);
  WQ_PTR(out);
  WQ_OPT32(lse);
  WQ_OPT32(bad_count);
  WQ_TRY(check_space(workspace, ws_bytes, kv_attn_ws_bytes(B, Hq, Hkv, D), "workspace"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(launch_kv_attn(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad_count, workspace),
                  "kv_attn_decode launch");
}

size_t kv_pages_scratch_bytes(int64_t n, int64_t B, int64_t W, int64_t P) {
  if (n < 0 || B < 1 || W < 1 || P < 1) return 0;
  return kv_pages_scratch(n, B, W, P);
}

wq_status kv_pages_copy(void* kv, int64_t L, int64_t P, int64_t page_bytes, const int32_t* src, const int32_t* dst,
                        int64_t n, int32_t* bad_count, void* stream) {
  clear_error();
  const PagePool p{kv, L, P, page_bytes};
  WQ_TRY(check_pool(p));
  if (n < 0 || n > kMaxDim) return fail(WQ_EINVAL, "n must be in 0..2^31-1 (got %lld)", (long long)n);
  if (n == 0) return WQ_OK;
  WQ_PTR32(src);
  WQ_PTR32(dst);
  WQ_OPT32(bad_count);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_pages_copy(c, p, src, dst, n, bad_count), "kv_pages_copy launch");
}

wq_status kv_pages_fork(void* kv, int64_t L, int64_t P, int64_t page_bytes, const int32_t* block_table,
                        const int32_t* lens, const int32_t* ref, int64_t B, int64_t W, int64_t S,
                        const int32_t* parent, const int32_t* child, int64_t n, int32_t* table_out,
                        int32_t* lens_out, int32_t* ref_out, int32_t* granted, void* scratch, size_t scratch_bytes,
                        void* stream) {
  clear_error();
  const PagePool p{kv, L, P, page_bytes};
  const SeqTables t{block_table, lens, ref, B, W, S, P};
  WQ_TRY(check_pool(p));
  WQ_TRY(check_tables(t));
  if (n < 0 || n > B) return fail(WQ_EINVAL, "n must be in 0..B (got %lld)", (long long)n);
  WQ_PTR32(table_out);
  WQ_PTR32(lens_out);
  WQ_PTR32(ref_out);
  if (n > 0) {
    WQ_PTR32(parent);
    WQ_PTR32(child);
    WQ_PTR32(granted);
  }
  WQ_TRY(check_space(scratch, scratch_bytes, kv_pages_scratch(n, B, W, P), "scratch"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(
      launch_pages_fork(c, p, t, parent, child, n, table_out, lens_out, ref_out, granted, scratch),
      "kv_pages_fork launch");
}

wq_status kv_pages_reserve(const int32_t* block_table, const int32_t* lens, const int32_t* new_lens,
                           const int32_t* ref, int64_t B, int64_t W, int64_t S, int64_t P, int32_t* table_out,
                           int32_t* ref_out, int32_t* granted, void* scratch, size_t scratch_bytes, void* stream) {
  clear_error();
  const SeqTables t{block_table, lens, ref, B, W, S, P};
  WQ_TRY(check_tables(t));
  WQ_PTR32(new_lens);
  WQ_PTR32(table_out);
  WQ_PTR32(ref_out);
  WQ_PTR32(granted);
  WQ_TRY(check_space(scratch, scratch_bytes, kv_pages_scratch(B, B, W, P), "scratch"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_pages_reserve(c, t, new_lens, table_out, ref_out, granted, scratch),
                  "kv_pages_reserve launch");
}

wq_status kv_pages_free(const int32_t* block_table, const int32_t* lens, const int32_t* ref, int64_t B, int64_t W,
                        int64_t S, int64_t P, const int32_t* seqs, int64_t n, int32_t* lens_out, int32_t* ref_out,
                        int32_t* bad_count, void* stream) {
  clear_error();
  const SeqTables t{block_table, lens, ref, B, W, S, P};
  WQ_TRY(check_tables(t));
  if (n < 0 || n > B) return fail(WQ_EINVAL, "n must be in 0..B (got %lld)", (long long)n);
  if (n > 0) WQ_PTR32(seqs);
  WQ_PTR32(lens_out);
  WQ_PTR32(ref_out);
  WQ_OPT32(bad_count);
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  return launched(launch_pages_free(c, t, seqs, n, lens_out, ref_out, bad_count), "kv_pages_free launch");
}

wq_status kv_pages_compact(void* kv, int64_t L, int64_t P, int64_t page_bytes, const int32_t* block_table,
                           const int32_t* lens, const int32_t* ref, int64_t B, int64_t W, int64_t S,
                           int32_t* table_out, int32_t* ref_out, int32_t* remap, int32_t* n_live, void* scratch,
                           size_t scratch_bytes, void* stream) {
  clear_error();
  const PagePool p{kv, L, P, page_bytes};
  const SeqTables t{block_table, lens, ref, B, W, S, P};
  WQ_TRY(check_pool(p));
  WQ_TRY(check_tables(t));
  WQ_PTR32(table_out);
  WQ_PTR32(ref_out);
  WQ_PTR32(remap);
  WQ_PTR32(n_live);
  WQ_TRY(check_space(scratch, scratch_bytes, kv_pages_scratch(0, B, W, P), "scratch"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(launch_pages_compact(c, p, t, table_out, ref_out, remap, n_live, scratch),
                  "kv_pages_compact launch");
}

size_t token_logprobs_workspace_bytes(int64_t T, int64_t V, int top_k) {
  if (T < 1 || V < 1 || top_k < 0 || top_k > kMaxTopK) return 0;
  return logprobs_ws_bytes(T, V, top_k);
}

wq_status token_logprobs(const void* logits, int logits_type, int64_t ld, int64_t T, int64_t V, const int32_t* ids,
                         float temperature, int top_k, float* logprob, int32_t* rank, float* entropy,
                         float* top_logprobs, int32_t* top_ids, int32_t* bad_count, void* workspace, size_t ws_bytes,
                         void* stream) {
  clear_error();
  if (logits_type != WQ_LOGITS_BF16 && logits_type != WQ_LOGITS_F32)
    return fail(WQ_EINVAL, "logits_type must be WQ_LOGITS_BF16 or WQ_LOGITS_F32 (got %d)", logits_type);
  if (T < 0 || T > kMaxDim) return fail(WQ_EINVAL, "T must be in 0..2^31-1 (got %lld)", (long long)T);
  WQ_TRY(check_size(V, "V"));
  if (ld < V || ld > kMaxDim) return fail(WQ_EINVAL, "ld must be in V..2^31-1 (got %lld)", (long long)ld);
  if (top_k < 0 || top_k > kMaxTopK || top_k > V)
    return fail(WQ_EINVAL, "top_k must be in 0..min(%d, V) (got %d)", kMaxTopK, top_k);
  if (!(temperature >= 1e-30f && temperature <= 1e30f))
    return fail(WQ_EINVAL, "temperature must be in 1e-30..1e30 (got %g)", static_cast<double>(temperature));
  if (T == 0) return WQ_OK;
  WQ_PTR(logits);
  if (ids != nullptr) {
    WQ_PTR32(ids);
    WQ_PTR32(logprob);
    WQ_PTR32(rank);
  }
  WQ_OPT32(entropy);
  if (top_k > 0) {
    WQ_PTR32(top_logprobs);
    WQ_PTR32(top_ids);
  }
  WQ_OPT32(bad_count);
  WQ_TRY(check_space(workspace, ws_bytes, logprobs_ws_bytes(T, V, top_k), "workspace"));
  Ctx c{};
  WQ_TRY(get_ctx(stream, &c));
  const LogprobArgs a{logits, logits_type, ld, T, V, ids, temperature, top_k, logprob, rank, entropy, top_logprobs,
                      top_ids, bad_count, workspace};
  const std::lock_guard<std::mutex> order(launch_order());
  return launched(launch_logprobs(c, a), "token_logprobs launch");
}

}  // extern "C"
