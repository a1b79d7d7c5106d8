// C ABI layer of the operators for several answers to one prompt (microscaled 4-bit
// products, attention over shared prefixes, sampling): argument checks (no HIP
// call), dispatch.
#include <stdint.h>

#include "../../include/biloco.h"
#include "api_checks.h"
#include "biloco_internal.h"

using namespace biloco;

namespace {

constexpr int32_t kMostK = 1 << 20;
constexpr int32_t kMostRows = 1 << 30;        // of a product's operands: their tiles' ends stay 32-bit numbers
constexpr int32_t kMostLogits = 1 << 20;      // of weights up to 2^44, whose sums are to fit 64 bits

biloco_status check_k(int32_t K) {
    if (K < 32 || K % 32 != 0) return BILOCO_ERR_INVALID_VALUE;
    return K > kMostK ? BILOCO_ERR_UNSUPPORTED : BILOCO_OK;
}
biloco_status check_mx(int32_t M, int32_t K, const void *x, int64_t x_stride, const void *codes, const void *scales) {
    if (M < 0) return BILOCO_ERR_INVALID_VALUE;
    const biloco_status st = check_k(K);
    if (st != BILOCO_OK) return st;
    if (!mxfp4_rows_fit(M, K)) return BILOCO_ERR_UNSUPPORTED;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales))
        return BILOCO_ERR_INVALID_VALUE;
    return check_stride(x_stride, K);
}
Span codes_span(const void *p, int64_t rows, int64_t K) { return {p, (size_t)(rows * (K / 2))}; }
Span scales_span(const void *p, int64_t rows, int64_t K) { return {p, (size_t)(rows * (K / 32))}; }

// x: rows to quantise, or NULL for a's codes and scales.
biloco_status gemm(const uint16_t *x, int64_t x_stride, const uint8_t *a_codes, const uint8_t *a_scales,
                   const uint8_t *w_codes, const uint8_t *w_scales, int32_t M, int32_t N, int32_t K, void *y,
                   int64_t y_stride, int32_t y_fp32, void *workspace, size_t workspace_bytes, bool quant,
                   hipStream_t stream) {
    if (M < 0 || N < 1) return BILOCO_ERR_INVALID_VALUE;
    biloco_status st = check_k(K);
    if (st != BILOCO_OK) return st;
    if (M > kMostRows || N > kMostRows || !mxfp4_fits(M, N, K)) return BILOCO_ERR_UNSUPPORTED;
    if ((quant ? !x : !a_codes || !a_scales) || !w_codes || !w_scales || !y) return BILOCO_ERR_INVALID_VALUE;
    const void *ptrs[] = {x, a_codes, a_scales, w_codes, w_scales, y, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    if (quant) st = check_stride(x_stride, K);
    if (st != BILOCO_OK) return st;
    if (y_stride < N) return BILOCO_ERR_INVALID_VALUE;
    if (y_stride > kMaxStride) return BILOCO_ERR_UNSUPPORTED;
    if (M == 0) return BILOCO_OK;
    const size_t need = mxfp4_plan_bytes(M, N, K, quant);
    if (need > 0 && !workspace) return BILOCO_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return BILOCO_ERR_WORKSPACE_TOO_SMALL;
    const Span out[] = {rows(y, M, y_stride, N, y_fp32 ? 4 : 2), {workspace, need}};
    const Span in[] = {rows(x, M, x_stride, K, 2), codes_span(a_codes, M, K), scales_span(a_scales, M, K),
                       codes_span(w_codes, N, K), scales_span(w_scales, N, K)};
    if (overlaps(out[0], out[1])) return BILOCO_ERR_INVALID_VALUE;
    for (const Span &o : out)
        for (const Span &i : in)
            if (overlaps(o, i)) return BILOCO_ERR_INVALID_VALUE;
    const MxGemmArgs a{x, x_stride, a_codes, a_scales, w_codes, w_scales, M, N, K, y, y_stride, y_fp32 != 0, workspace};
    return launch_gemm_mxfp4(a, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

}  // namespace

extern "C" {

biloco_status biloco_quant_mxfp4(const void *x, int64_t x_stride, int32_t x_fp32, int32_t M, int32_t K, uint8_t *codes,
                                 uint8_t *scales, hipStream_t stream) {
    const biloco_status st = check_mx(M, K, x, x_stride, codes, scales);
    if (st != BILOCO_OK) return st;
    const Span in = rows(x, M, x_stride, K, x_fp32 ? 4 : 2), c = codes_span(codes, M, K), s = scales_span(scales, M, K);
    if (overlaps(in, c) || overlaps(in, s) || overlaps(c, s)) return BILOCO_ERR_INVALID_VALUE;
    if (M == 0) return BILOCO_OK;
    return launch_quant_mxfp4(x, x_stride, x_fp32 != 0, M, K, codes, scales, stream) == hipSuccess ? BILOCO_OK
                                                                                                 : BILOCO_ERR_HIP;
}

biloco_status biloco_dequant_mxfp4(const uint8_t *codes, const uint8_t *scales, int32_t M, int32_t K, void *out,
                                   int64_t out_stride, int32_t out_fp32, hipStream_t stream) {
    const biloco_status st = check_mx(M, K, out, out_stride, codes, scales);
    if (st != BILOCO_OK) return st;
    const Span o = rows(out, M, out_stride, K, out_fp32 ? 4 : 2);
    if (overlaps(o, codes_span(codes, M, K)) || overlaps(o, scales_span(scales, M, K))) return BILOCO_ERR_INVALID_VALUE;
    if (M == 0) return BILOCO_OK;
    return launch_dequant_mxfp4(codes, scales, M, K, out, out_stride, out_fp32 != 0, stream) == hipSuccess
               ? BILOCO_OK
               : BILOCO_ERR_HIP;
}

biloco_status biloco_gemm_mxfp4_workspace_bytes(int32_t M, int32_t N, int32_t K, size_t *bytes) {
    if (!bytes || M < 0 || N < 1) return BILOCO_ERR_INVALID_VALUE;
    const biloco_status st = check_k(K);
    if (st != BILOCO_OK) return st;
    if (M > kMostRows || N > kMostRows || !mxfp4_fits(M, N, K)) return BILOCO_ERR_UNSUPPORTED;
    *bytes = M == 0 ? 0 : mxfp4_ws_bytes(M, N, K);
    return BILOCO_OK;
}

biloco_status biloco_gemm_mxfp4(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                                const uint8_t *w_scales, int32_t M, int32_t N, int32_t K, void *y, int64_t y_stride,
                                int32_t y_fp32, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return gemm(nullptr, 0, a_codes, a_scales, w_codes, w_scales, M, N, K, y, y_stride, y_fp32, workspace,
                workspace_bytes, false, stream);
}

biloco_status biloco_gemm_mxfp4_quant(const uint16_t *x, int64_t x_stride, const uint8_t *w_codes,
                                      const uint8_t *w_scales, int32_t M, int32_t N, int32_t K, void *y,
                                      int64_t y_stride, int32_t y_fp32, void *workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    return gemm(x, x_stride, nullptr, nullptr, w_codes, w_scales, M, N, K, y, y_stride, y_fp32, workspace,
                workspace_bytes, true, stream);
}

biloco_status biloco_attn_shared_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads,
                                                 int32_t head_dim, int32_t max_q_len, int32_t max_kv_len,
                                                 int32_t n_groups, int32_t max_shared_len, size_t *bytes) {
    if (!bytes || n_groups < 1 || max_shared_len < 0) return BILOCO_ERR_INVALID_VALUE;
    if (n_groups > 65535 || max_shared_len > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    const biloco_status st = check_attn_sizes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len);
    if (st != BILOCO_OK) return st;
    if (!attn_shared_fits(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len, n_groups, max_shared_len))
        return BILOCO_ERR_UNSUPPORTED;
    *bytes = attn_shared_ws_bytes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len, n_groups, max_shared_len);
    return BILOCO_OK;
}

biloco_status biloco_attn_shared(const uint8_t *k_codes, const uint8_t *v_codes, const uint8_t *k_scales,
                                 const uint8_t *v_scales, int32_t num_pages, int32_t kv_heads, int32_t page_size,
                                 int32_t head_dim, const uint16_t *q, int64_t q_stride, int32_t q_heads,
                                 const int32_t *q_start, const int32_t *kv_len, const int32_t *block_table,
                                 int32_t max_pages, int32_t B, int32_t T, int32_t max_q_len, int32_t max_kv_len,
                                 const int32_t *group_start, const int32_t *shared_len, int32_t n_groups,
                                 int32_t max_shared_len, float scale, int32_t window, int32_t sinks, uint16_t *o,
                                 int64_t o_stride, float *lse, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
    size_t need = 0;
    biloco_status st = check_cache(num_pages, kv_heads, page_size, head_dim);
    if (st == BILOCO_OK) st = check_batch(B, T, max_q_len, max_pages, page_size);
    if (st == BILOCO_OK)
        st = biloco_attn_shared_workspace_bytes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len, n_groups,
                                                max_shared_len, &need);
    if (st != BILOCO_OK) return st;
    const AttnArgs a{k_codes, v_codes, k_scales, v_scales, num_pages, kv_heads, page_size, head_dim,
                     q, q_stride, q_heads, q_start, kv_len, block_table, max_pages, B, T,
                     max_q_len, max_kv_len, scale, window, sinks, o, o_stride, lse, workspace};
    st = check_attn(a, need, workspace_bytes, {{group_start, (size_t)(n_groups + 1) * 4}, {shared_len, (size_t)n_groups * 4}});
    if (st != BILOCO_OK || B == 0 || T == 0) return st;
    const SharedAttnArgs s{group_start, shared_len, n_groups, max_shared_len, nullptr, nullptr};
    return launch_attn_shared(a, s, workspace_bytes, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

biloco_status biloco_sample_workspace_bytes(int32_t rows, int32_t V, size_t *bytes) {
    if (!bytes || rows < 0 || V < 1) return BILOCO_ERR_INVALID_VALUE;
    if (V >= kMostLogits) return BILOCO_ERR_UNSUPPORTED;
    *bytes = rows == 0 ? 0 : sample_ws_bytes(rows, V);
    return BILOCO_OK;
}

biloco_status biloco_sample(const void *logits, int64_t stride, int32_t fp32, int32_t n, int32_t V,
                            const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                            const float *u, int32_t *token, float *logprob, void *workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    size_t need = 0;
    const biloco_status st = biloco_sample_workspace_bytes(n, V, &need);
    if (st != BILOCO_OK) return st;
    if (stride < 0) return BILOCO_ERR_INVALID_VALUE;
    if (stride > kMaxStride) return BILOCO_ERR_UNSUPPORTED;
    if (!logits || !u || !token || (need > 0 && !workspace)) return BILOCO_ERR_INVALID_VALUE;
    const void *ptrs[] = {logits, temperature, top_k, top_p, min_p, u, token, logprob, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return BILOCO_ERR_WORKSPACE_TOO_SMALL;
    const size_t per_row = (size_t)n * 4;
    const Span out[] = {{token, per_row}, {logprob, per_row}, {workspace, need}};
    const Span in[] = {rows(logits, n, stride, V, fp32 ? 4 : 2), {temperature, per_row}, {top_k, per_row},
                       {top_p, per_row}, {min_p, per_row}, {u, per_row}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(out[i], out[j])) return BILOCO_ERR_INVALID_VALUE;
        for (const Span &s : in)
            if (overlaps(out[i], s)) return BILOCO_ERR_INVALID_VALUE;
    }
    if (n == 0) return BILOCO_OK;
    const SampleArgs a{logits, stride, fp32 != 0, n, V, temperature, top_k, top_p, min_p, u, token, logprob, workspace};
    return launch_sample(a, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

}  // extern "C"
