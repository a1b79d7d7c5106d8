// Argument checks that the C ABI's layers share (host only, no HIP call).
#pragma once
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/biloco.h"
#include "biloco_internal.h"

namespace biloco {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

struct Span {
    const void *p;
    size_t n;
};

inline bool overlaps(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// rows of `width` elements of `size` bytes, `stride` elements apart
inline Span rows(const void *p, int64_t n, int64_t stride, int64_t width, size_t size) {
    return {p, n > 0 ? (size_t)((n - 1) * stride + width) * size : 0};
}

// Rows of a and of b (the same number of each, `stride` bytes apart in both)
// that lie between one another without meeting: b's columns are within the gap
// that follows each of a's rows.
inline bool between(const void *a, size_t a_width, const void *b, size_t b_width, size_t stride) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    const size_t at = b0 >= a0 ? (b0 - a0) % stride : (stride - (a0 - b0) % stride) % stride;
    return at >= a_width && at + b_width <= stride;
}

// Token strides are bounded so that every byte offset fits 62 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 30;

inline biloco_status check_stride(int64_t stride, int64_t width) {
    if (stride < width || stride % 8 != 0) return BILOCO_ERR_INVALID_VALUE;
    return stride > kMaxStride ? BILOCO_ERR_UNSUPPORTED : BILOCO_OK;
}

// The sizes every call on a cache shares.
inline biloco_status check_cache(int32_t num_pages, int32_t kv_heads, int32_t page_size, int32_t head_dim) {
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

inline biloco_status check_batch(int32_t B, int32_t T, int32_t max_q_len, int32_t max_pages, int32_t page_size) {
    if (B < 0 || T < 0 || max_q_len < 1 || max_pages < 1) return BILOCO_ERR_INVALID_VALUE;
    if (B > 65535 || (int64_t)max_pages * page_size > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    return BILOCO_OK;
}

// The sizes that shape attention's launches.
inline biloco_status check_attn_sizes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                      int32_t max_q_len, int32_t max_kv_len) {
    if (max_kv_len < 0 || q_heads < 1) return BILOCO_ERR_INVALID_VALUE;
    if (max_kv_len > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    biloco_status st = check_cache(1, kv_heads, 16, head_dim);
    if (st == BILOCO_OK) st = check_batch(B, T, max_q_len, 1, 1);
    if (st != BILOCO_OK) return st;
    if (q_heads % kv_heads != 0) return BILOCO_ERR_INVALID_VALUE;
    if (q_heads > 4096 || (int64_t)T * q_heads > INT32_MAX) return BILOCO_ERR_UNSUPPORTED;
    return BILOCO_OK;
}

// Everything else about a call of attention; `more`: arrays that a kind of it reads besides.
inline biloco_status check_attn(const AttnArgs &a, size_t need, size_t workspace_bytes, std::initializer_list<Span> more) {
    if (!(a.scale > 0.0f) || !isfinite(a.scale) || a.window < 0 || a.sinks < 0) return BILOCO_ERR_INVALID_VALUE;
    if (a.window > kMostTokens || a.sinks > kMostTokens) return BILOCO_ERR_UNSUPPORTED;
    const void *needed[] = {a.kc, a.vc, a.ks, a.vs, a.q, a.q_start, a.kv_len, a.table, a.o};
    for (const void *p : needed)
        if (!p || !aligned16(p)) return BILOCO_ERR_INVALID_VALUE;
    for (const Span &s : more)
        if (!s.p || !aligned16(s.p)) return BILOCO_ERR_INVALID_VALUE;
    if ((need > 0 && !a.ws) || !aligned16(a.lse) || !aligned16(a.ws)) return BILOCO_ERR_INVALID_VALUE;
    const int64_t qw = (int64_t)a.q_heads * a.dim;
    biloco_status st = check_stride(a.q_stride, qw);
    if (st == BILOCO_OK) st = check_stride(a.o_stride, qw);
    if (st != BILOCO_OK) return st;
    if (workspace_bytes < need) return BILOCO_ERR_WORKSPACE_TOO_SMALL;
    const size_t cache = (size_t)a.num_pages * a.kv_heads * a.page * a.dim;
    const size_t nscale = (size_t)a.num_pages * a.kv_heads;
    const Span out[] = {rows(a.o, a.T, a.o_stride, qw, 2), {a.lse, (size_t)a.T * a.q_heads * 4}, {a.ws, need}};
    const Span in[] = {{a.kc, cache}, {a.vc, cache}, {a.ks, nscale}, {a.vs, nscale},
                       rows(a.q, a.T, a.q_stride, qw, 2), {a.q_start, (size_t)(a.B + 1) * 4},
                       {a.kv_len, (size_t)a.B * 4}, {a.table, (size_t)a.B * a.max_pages * 4}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(out[i], out[j])) return BILOCO_ERR_INVALID_VALUE;
        for (const Span &s : in)
            if (overlaps(out[i], s)) return BILOCO_ERR_INVALID_VALUE;
        for (const Span &s : more)
            if (overlaps(out[i], s)) return BILOCO_ERR_INVALID_VALUE;
    }
    return BILOCO_OK;
}

}  // namespace
}  // namespace biloco
