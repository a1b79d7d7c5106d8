// C ABI layer of the decoder-layer operators (cache append, attention over
// the cache, norms around a block): argument checks (no HIP call), dispatch.
#include <math.h>
#include <stdint.h>

#include "../../include/biloco.h"
#include "biloco_internal.h"

using namespace biloco;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

struct Span {
    const void *p;
    size_t n;
};

bool overlaps(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// rows of `width` elements of `size` bytes, `stride` elements apart
Span rows(const void *p, int64_t n, int64_t stride, int64_t width, size_t size) {
    return {p, n > 0 ? (size_t)((n - 1) * stride + width) * size : 0};
}

// Rows of a and of b (the same number of each, `stride` bytes apart in both)
// that lie between one another without meeting: b's columns are within the gap
// that follows each of a's rows.
bool between(const void *a, size_t a_width, const void *b, size_t b_width, size_t stride) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    const size_t at = b0 >= a0 ? (b0 - a0) % stride : (stride - (a0 - b0) % stride) % stride;
    return at >= a_width && at + b_width <= stride;
}

// Token strides are bounded so that every byte offset fits 62 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 30;

biloco_status check_stride(int64_t stride, int64_t width) {
    if (stride < width || stride % 8 != 0) return BILOCO_ERR_INVALID_VALUE;
    return stride > kMaxStride ? BILOCO_ERR_UNSUPPORTED : BILOCO_OK;
}

// The sizes every call on a cache shares.
biloco_status check_cache(int32_t num_pages, int32_t kv_heads, int32_t page_size, int32_t head_dim) {
    if (num_pages < 1 || kv_heads < 1 || page_size < 1 || head_dim < 1)
        return BILOCO_ERR_INVALID_VALUE;
    if (head_dim != 64 && head_dim != 128) return BILOCO_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return BILOCO_ERR_UNSUPPORTED;
    if (kv_heads > 1024) return BILOCO_ERR_UNSUPPORTED;
    return BILOCO_OK;
}

// Tokens of a sequence that its table row can name: positions and what is
// added to them in the kernels stay within 32 bits.
constexpr int64_t kMostTokens = (int64_t)1 << 30;

biloco_status check_batch(int32_t B, int32_t T, int32_t max_q_len, int32_t max_pages, int32_t page_size) {
    if (B < 0 || T < 0 || max_q_len < 1 || max_pages < 1) return BILOCO_ERR_INVALID_VALUE;
    if (B > 65535 || (int64_t)max_pages * page_size > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    return BILOCO_OK;
}

}  // namespace

extern "C" {

biloco_status biloco_kv_append(uint8_t *k_codes, uint8_t *v_codes, uint8_t *k_scales,
                               uint8_t *v_scales, int32_t num_pages, int32_t kv_heads,
                               int32_t page_size, int32_t head_dim, const uint16_t *q,
                               int64_t q_stride, const uint16_t *k, int64_t k_stride,
                               const uint16_t *v, int64_t v_stride, int32_t q_heads,
                               const int32_t *positions, int32_t axes, const uint8_t *pair_axis,
                               const float *cos_sin, int32_t n_pos, int32_t rot_dim,
                               int32_t interleaved, const int32_t *q_start, const int32_t *kv_len,
                               const int32_t *block_table, int32_t max_pages, int32_t B, int32_t T,
                               int32_t max_q_len, uint16_t *q_out, int64_t q_out_stride,
                               hipStream_t stream) {
    biloco_status st = check_cache(num_pages, kv_heads, page_size, head_dim);
    if (st == BILOCO_OK) st = check_batch(B, T, max_q_len, max_pages, page_size);
    if (st != BILOCO_OK) return st;
    if (q_heads < 0 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0)
        return BILOCO_ERR_INVALID_VALUE;
    if (q_heads > 4096 || rot_dim % 16 != 0) return BILOCO_ERR_UNSUPPORTED;
    if (rot_dim > 0 && (axes < 1 || n_pos < 1)) return BILOCO_ERR_INVALID_VALUE;
    if (rot_dim > 0 && axes > 4) return BILOCO_ERR_UNSUPPORTED;
    if (!k_codes || !v_codes || !k_scales || !v_scales || !k || !v || !q_start || !kv_len ||
        !block_table)
        return BILOCO_ERR_INVALID_VALUE;
    if (q_heads > 0 && (!q || !q_out)) return BILOCO_ERR_INVALID_VALUE;
    if (rot_dim > 0 && (!positions || !cos_sin)) return BILOCO_ERR_INVALID_VALUE;
    const void *ptrs[] = {k_codes, v_codes, k_scales, v_scales, q, k, v, positions, cos_sin,
                          q_start, kv_len, block_table, q_out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)kv_heads * head_dim;
    st = check_stride(k_stride, kw);
    if (st == BILOCO_OK) st = check_stride(v_stride, kw);
    if (st == BILOCO_OK && q_heads > 0) st = check_stride(q_stride, qw);
    if (st == BILOCO_OK && q_heads > 0) st = check_stride(q_out_stride, qw);
    if (st != BILOCO_OK) return st;

    KvAppendArgs a{k_codes, v_codes, k_scales, v_scales, num_pages, kv_heads, page_size, head_dim,
                   q, k, v, q_stride, k_stride, v_stride, q_heads, positions, axes, {0},
                   cos_sin, n_pos, rot_dim, interleaved != 0, q_start, kv_len, block_table,
                   max_pages, B, T, max_q_len, q_out, q_out_stride};
    if (pair_axis)
        for (int i = 0; i < rot_dim / 2; ++i) {
            if (pair_axis[i] >= axes) return BILOCO_ERR_INVALID_VALUE;
            a.axis_bits[i / 32] |= (uint64_t)pair_axis[i] << (2 * (i % 32));
        }

    const size_t cache = (size_t)num_pages * kv_heads * page_size * head_dim;
    const size_t nscale = (size_t)num_pages * kv_heads;
    const Span out[] = {{k_codes, cache}, {v_codes, cache}, {k_scales, nscale}, {v_scales, nscale},
                        rows(q_heads ? q_out : nullptr, T, q_out_stride, qw, 2)};
    const Span in[] = {rows(k, T, k_stride, kw, 2), rows(v, T, v_stride, kw, 2),
                       {positions, rot_dim ? (size_t)axes * T * 4 : 0},
                       {cos_sin, rot_dim ? (size_t)n_pos * rot_dim * 4 : 0},
                       {q_start, (size_t)(B + 1) * 4}, {kv_len, (size_t)B * 4},
                       {block_table, (size_t)B * max_pages * 4}};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(out[i], out[j])) return BILOCO_ERR_INVALID_VALUE;
        // rows of q, k and v of one product lie between one another, and q_out may
        // be q itself: k's and v's columns are then not to be q's
        for (int j = 0; j < 7; ++j) {
            const int64_t stride = j == 0 ? k_stride : v_stride;
            const bool apart = i == 4 && j < 2 && q_out == q && stride == q_out_stride &&
                               between(q_out, (size_t)qw * 2, in[j].p, (size_t)kw * 2, (size_t)stride * 2);
            if (!apart && overlaps(out[i], in[j])) return BILOCO_ERR_INVALID_VALUE;
        }
    }
    if (q_heads > 0) {
        const Span qs = rows(q, T, q_stride, qw, 2);
        if (q_out == q ? q_out_stride != q_stride : overlaps(out[4], qs))
            return BILOCO_ERR_INVALID_VALUE;
        for (int i = 0; i < 4; ++i)
            if (overlaps(out[i], qs)) return BILOCO_ERR_INVALID_VALUE;
    }
    if (B == 0 || T == 0) return BILOCO_OK;
    return launch_kv_append(a, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

biloco_status biloco_attn_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim, int32_t max_q_len, int32_t max_kv_len,
                                          size_t *bytes) {
    if (!bytes || max_kv_len < 0 || q_heads < 1) return BILOCO_ERR_INVALID_VALUE;
    if (max_kv_len > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    biloco_status st = check_cache(1, kv_heads, 16, head_dim);
    if (st == BILOCO_OK) st = check_batch(B, T, max_q_len, 1, 1);
    if (st != BILOCO_OK) return st;
    if (q_heads % kv_heads != 0) return BILOCO_ERR_INVALID_VALUE;
    if (q_heads > 4096 || (int64_t)T * q_heads > INT32_MAX) return BILOCO_ERR_UNSUPPORTED;
    *bytes = attn_ws_bytes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len);
    return BILOCO_OK;
}

biloco_status biloco_attn_paged(const uint8_t *k_codes, const uint8_t *v_codes,
                                const uint8_t *k_scales, const uint8_t *v_scales,
                                int32_t num_pages, int32_t kv_heads, int32_t page_size,
                                int32_t head_dim, const uint16_t *q, int64_t q_stride,
                                int32_t q_heads, const int32_t *q_start, const int32_t *kv_len,
                                const int32_t *block_table, int32_t max_pages, int32_t B, int32_t T,
                                int32_t max_q_len, int32_t max_kv_len, float scale, int32_t window,
                                int32_t sinks, uint16_t *o, int64_t o_stride, float *lse,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
    size_t need = 0;
    biloco_status st = check_cache(num_pages, kv_heads, page_size, head_dim);
    if (st == BILOCO_OK) st = check_batch(B, T, max_q_len, max_pages, page_size);
    if (st == BILOCO_OK)
        st = biloco_attn_workspace_bytes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len,
                                         &need);
    if (st != BILOCO_OK) return st;
    if (!(scale > 0.0f) || !isfinite(scale) || window < 0 || sinks < 0)
        return BILOCO_ERR_INVALID_VALUE;
    if (window > kMostTokens || sinks > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    if (!k_codes || !v_codes || !k_scales || !v_scales || !q || !q_start || !kv_len ||
        !block_table || !o || (need > 0 && !workspace))
        return BILOCO_ERR_INVALID_VALUE;
    const void *ptrs[] = {k_codes, v_codes, k_scales, v_scales, q, q_start, kv_len, block_table,
                          o, lse, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    const int64_t qw = (int64_t)q_heads * head_dim;
    st = check_stride(q_stride, qw);
    if (st == BILOCO_OK) st = check_stride(o_stride, qw);
    if (st != BILOCO_OK) return st;
    if (workspace_bytes < need) return BILOCO_ERR_WORKSPACE_TOO_SMALL;
    const size_t cache = (size_t)num_pages * kv_heads * page_size * head_dim;
    const size_t nscale = (size_t)num_pages * kv_heads;
    const Span out[] = {rows(o, T, o_stride, qw, 2), {lse, (size_t)T * q_heads * 4},
                        {workspace, need}};
    const Span in[] = {{k_codes, cache}, {v_codes, cache}, {k_scales, nscale}, {v_scales, nscale},
                       rows(q, T, q_stride, qw, 2), {q_start, (size_t)(B + 1) * 4},
                       {kv_len, (size_t)B * 4}, {block_table, (size_t)B * max_pages * 4}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(out[i], out[j])) return BILOCO_ERR_INVALID_VALUE;
        for (const Span &s : in)
            if (overlaps(out[i], s)) return BILOCO_ERR_INVALID_VALUE;
    }
    if (B == 0 || T == 0) return BILOCO_OK;
    const AttnArgs a{k_codes, v_codes, k_scales, v_scales, num_pages, kv_heads, page_size, head_dim,
                     q, q_stride, q_heads, q_start, kv_len, block_table, max_pages, B, T,
                     max_q_len, max_kv_len, scale, window, sinks, o, o_stride, lse, workspace};
    return launch_attn(a, workspace_bytes, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

biloco_status biloco_norm_gate_residual(const uint16_t *x, int64_t x_stride, const uint16_t *post_w,
                                        const uint16_t *gate, int64_t gate_stride, float res_scale,
                                        const void *res, int64_t res_stride, int32_t res_fp32,
                                        const uint16_t *pre_w, float eps, float w_offset, int32_t T,
                                        int32_t C, void *res_out, int64_t res_out_stride,
                                        uint16_t *h, int64_t h_stride, uint8_t *a_codes,
                                        uint8_t *a_scales, hipStream_t stream) {
    if (T < 0 || C < 1 || !(eps >= 0.0f)) return BILOCO_ERR_INVALID_VALUE;
    if (C > 32768) return BILOCO_ERR_UNSUPPORTED;
    if (!x || !res || !pre_w || !res_out || !h || (a_codes == nullptr) != (a_scales == nullptr))
        return BILOCO_ERR_INVALID_VALUE;
    if (a_codes && C % 16 != 0) return BILOCO_ERR_INVALID_VALUE;
    if (a_codes && C % 32 != 0) return BILOCO_ERR_UNSUPPORTED;
    const void *ptrs[] = {x, post_w, gate, res, pre_w, res_out, h, a_codes, a_scales};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    const int64_t strides[] = {x_stride, res_stride, res_out_stride, h_stride};
    for (int64_t s : strides) {
        if (s < C) return BILOCO_ERR_INVALID_VALUE;
        if (s > kMaxStride) return BILOCO_ERR_UNSUPPORTED;
    }
    if (gate && gate_stride != 0 && gate_stride < C) return BILOCO_ERR_INVALID_VALUE;
    if (gate && gate_stride > kMaxStride) return BILOCO_ERR_UNSUPPORTED;
    const size_t rs = res_fp32 ? 4 : 2;
    const Span out[] = {rows(res_out, T, res_out_stride, C, rs), rows(h, T, h_stride, C, 2),
                        {a_codes, (size_t)T * C / 2}, {a_scales, (size_t)T * C / 16}};
    const Span in[] = {rows(x, T, x_stride, C, 2), {post_w, (size_t)C * 2},
                       rows(gate, gate_stride ? T : 1, gate_stride, C, 2), {pre_w, (size_t)C * 2}};
    const Span rin = rows(res, T, res_stride, C, rs);
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(out[i], out[j])) return BILOCO_ERR_INVALID_VALUE;
        for (const Span &s : in)
            if (overlaps(out[i], s)) return BILOCO_ERR_INVALID_VALUE;
        if (i > 0 && overlaps(out[i], rin)) return BILOCO_ERR_INVALID_VALUE;
    }
    if (res_out == res ? res_out_stride != res_stride : overlaps(out[0], rin))
        return BILOCO_ERR_INVALID_VALUE;
    if (T == 0) return BILOCO_OK;
    const NormArgs a{x, x_stride, post_w, gate, gate_stride, res_scale, res, res_stride,
                     res_fp32 != 0, pre_w, eps, w_offset, T, C, res_out, res_out_stride, h,
                     h_stride, a_codes, a_scales};
    return launch_norm(a, stream) == hipSuccess ? BILOCO_OK : BILOCO_ERR_HIP;
}

}  // extern "C"
