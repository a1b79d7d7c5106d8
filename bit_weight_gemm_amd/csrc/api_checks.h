// Argument checks that the C ABI's layers share (host only, no HIP call).
#pragma once
#include <stdint.h>

#include "../../include/biloco.h"

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

}  // namespace
}  // namespace biloco
