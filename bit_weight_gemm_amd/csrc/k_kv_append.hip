// Append of new keys and values to the paged 8-bit cache, with the position
// rotation of q and k on the way.
//
//   (a, b) -> (a c - b s, b c + a s)          per pair of channels, fp32
//   code = E4M3(x / 2^(e - 127)),  e the smallest byte >= 1 with
//   max|x| <= 448 * 2^(e - 127) over a page's new tokens of one head (never
//   below the page's present byte while it holds earlier tokens)
//
// A power of two costs E4M3 no precision (it only moves the exponent), makes
// the division exact and lets a page's earlier codes move to a larger scale
// without a second rounding, except where they fall below E4M3's normal range
// (less than 2^-14 of the page's largest value).
//
// One launch with two kinds of workgroup: rows of q (a token each), and
// (page, head, k or v) items, because a page's scale needs all its new tokens
// at once.  An item is one wave where at most a few tokens are new (decode)
// and four waves otherwise.  Bound by memory traffic: q is read and written
// once, k and v are read once and held in registers while their maximum is
// found.  Measured on MI355X: 13399 tokens with three axes 111.5 us, 4.74 TB/s
// (an addition of two large arrays reaches 6.1); 32 tokens of as many sequences, 64/8
// heads, 5.1 to 5.8 us, which is the launch.
#include "biloco_device.h"
#include "biloco_internal.h"

namespace biloco {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x8_t __attribute__((ext_vector_type(8), aligned(16)));

namespace {

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(d[i] << 16);
        x[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d[i] = (uint32_t)f32_to_bf16_rne(x[2 * i]) | ((uint32_t)f32_to_bf16_rne(x[2 * i + 1]) << 16);
    return make_uint4(d[0], d[1], d[2], d[3]);
}

// Cosines and sines of the eight pairs 8 * seg .. 8 * seg + 7 at token t.
struct Turn {
    f32x8_t c, s;
};
__device__ __forceinline__ Turn load_turn(const KvAppendArgs &a, int seg, int t) {
    const uint32_t bits = (uint32_t)((seg < 4 ? a.axis_bits[0] : a.axis_bits[1]) >> (16 * (seg & 3))) & 0xFFFFu;
    const int half = a.rot >> 1;
    const uint32_t first = bits & 3u;
    Turn w;
    if (bits == first * 0x5555u) {      // one axis for the eight pairs
        const int p = a.positions[(int64_t)first * a.T + t];
        const bool in = (uint32_t)p < (uint32_t)a.n_pos;
        const float *row = a.cos_sin + (int64_t)(in ? p : 0) * a.rot + 8 * seg;
        w.c = *reinterpret_cast<const f32x8_t *>(row);
        w.s = *reinterpret_cast<const f32x8_t *>(row + half);
        w.c = in ? w.c : (f32x8_t)__builtin_nanf("");
        w.s = in ? w.s : (f32x8_t)__builtin_nanf("");
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = a.positions[(int64_t)((bits >> (2 * i)) & 3u) * a.T + t];
            const bool in = (uint32_t)p < (uint32_t)a.n_pos;
            const float *row = a.cos_sin + (int64_t)(in ? p : 0) * a.rot + 8 * seg + i;
            const float c = row[0], s = row[half];
            w.c[i] = in ? c : __builtin_nanf("");
            w.s[i] = in ? s : __builtin_nanf("");
        }
    }
    return w;
}

// Sixteen channels of one head as two runs of eight: in a rotated segment
// pair i is (x[i], y[i]) when the halves are apart, and (x[2i], x[2i + 1]),
// (y[2i - 8], y[2i - 7]) when pairs are neighbours.  Offsets of the two runs:
__device__ __forceinline__ int run0(const KvAppendArgs &a, int seg) {
    return (!a.interleaved && 16 * seg < a.rot ? 8 : 16) * seg;
}
__device__ __forceinline__ int run1(const KvAppendArgs &a, int seg) {
    return run0(a, seg) + (!a.interleaved && 16 * seg < a.rot ? a.rot >> 1 : 8);
}

// Products and sums are rounded one by one (no fused multiply-add), so that a
// rotated value, and with it a code, does not depend on the compiler.
__device__ __forceinline__ void turn(bool interleaved, const Turn &w, float (&x)[8], float (&y)[8]) {
#pragma clang fp contract(off)
    const f32x8_t c = w.c, s = w.s;
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = x[i], q = y[i];
            x[i] = p * c[i] - q * s[i];
            y[i] = q * c[i] + p * s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1], u = y[2 * i], z = y[2 * i + 1];
            x[2 * i] = p * c[i] - q * s[i];
            x[2 * i + 1] = q * c[i] + p * s[i];
            y[2 * i] = u * c[i + 4] - z * s[i + 4];
            y[2 * i + 1] = z * c[i + 4] + u * s[i + 4];
        }
    }
}

// Magnitude bits, for the scale.  A value above 448 * 2^119, the largest that
// every code times its scale stays finite for, becomes NaN and does not count.
constexpr uint32_t kLargest = 0x7F600000u;
__device__ __forceinline__ uint32_t finite_mag(float &x) {
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    x = m <= kLargest ? x : __builtin_nanf("");
    return m <= kLargest ? m : 0u;
}
__device__ __forceinline__ uint32_t wave_umax64(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}
// Smallest byte e >= 1 with amax <= 1.75 * 2^8 * 2^(e - 127); at most 246.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
    const int e = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
    return max(e, 1);
}
__device__ __forceinline__ float pow2_bits(int field) {      // 2^(field - 127); 0 below
    return field > 0 ? __uint_as_float((uint32_t)field << 23) : 0.0f;
}
// Four fp32 values, already divided by the scale, as four E4M3 codes (round
// to nearest even; NaN becomes a NaN code).
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x2, x3, w, true);
    return (uint32_t)w;
}
// Four codes times f (a power of two below 1).
__device__ __forceinline__ uint32_t lower4(uint32_t w, float f) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return codes4(a[0] * f, a[1] * f, b[0] * f, b[1] * f);
}
__device__ __forceinline__ uint4 lower16(uint4 w, float f) {
    return make_uint4(lower4(w.x, f), lower4(w.y, f), lower4(w.z, f), lower4(w.w, f));
}

// Item maximum over NW waves.
template <int NW>
__device__ __forceinline__ uint32_t item_max(uint32_t m, uint32_t *lds) {
    m = wave_umax64(m);
    if constexpr (NW > 1) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
        __syncthreads();
        m = lds[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) m = max(m, lds[i]);
    }
    return m;
}

// The part of one page that a call writes: slots [lo, hi) take the tokens of
// rows t0 .. t0 + hi - lo - 1; slots below lo hold earlier tokens.
struct PagePart {
    int64_t page;
    int lo, hi;
    int64_t t0;
};

template <int D, int NW, int PASSES>
__device__ __forceinline__ void append_k(const KvAppendArgs &a, const PagePart &pp, int h, int tid, uint32_t *lds) {
    constexpr int SEGS = D / 16, TP = 64 * NW / SEGS;
    const int seg = tid % SEGS, row = tid / SEGS, n = pp.hi - pp.lo;
    const int o0 = run0(a, seg), o1 = run1(a, seg);
    uint8_t *codes = a.kc + (pp.page * a.kv_heads + h) * ((int64_t)a.page * D);
    uint8_t *scale = a.ks + pp.page * a.kv_heads + h;
    const int old = pp.lo > 0 ? (int)*scale : 0;
    float x[PASSES][8], y[PASSES][8];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = p * TP + row;
        if (i < n) {
            const uint16_t *src = a.k + (pp.t0 + i) * a.k_stride + (int64_t)h * D;
            unpack8(*reinterpret_cast<const uint4 *>(src + o0), x[p]);
            unpack8(*reinterpret_cast<const uint4 *>(src + o1), y[p]);
            if (16 * seg < a.rot) {
                turn(a.interleaved, load_turn(a, seg, (int)(pp.t0 + i)), x[p], y[p]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, max(finite_mag(x[p][j]), finite_mag(y[p][j])));
        }
    }
    const int e = max(scale_byte(item_max<NW>(m, lds)), old);
    const float r = pow2_bits(254 - e);
    if (e > old && pp.lo > 0) {
        const float f = pow2_bits(127 + old - e);
        uint4 *w = reinterpret_cast<uint4 *>(codes);
        for (int i = tid; i < pp.lo * (D / 16); i += 64 * NW) w[i] = lower16(w[i], f);
    }
    if (tid == 0 && e != old) *scale = (uint8_t)e;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = p * TP + row;
        if (i < n) {
            uint8_t *dst = codes + (pp.lo + i) * D;
            uint2 u, w;
            u.x = codes4(x[p][0] * r, x[p][1] * r, x[p][2] * r, x[p][3] * r);
            u.y = codes4(x[p][4] * r, x[p][5] * r, x[p][6] * r, x[p][7] * r);
            w.x = codes4(y[p][0] * r, y[p][1] * r, y[p][2] * r, y[p][3] * r);
            w.y = codes4(y[p][4] * r, y[p][5] * r, y[p][6] * r, y[p][7] * r);
            *reinterpret_cast<uint2 *>(dst + o0) = u;
            *reinterpret_cast<uint2 *>(dst + o1) = w;
        }
    }
}

// Bytes of a four-slot word that [lo, hi) covers, slots counted from the
// word's first.
__device__ __forceinline__ uint32_t byte_mask(int lo, int hi) {
    const uint32_t upto_hi = hi >= 4 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << (8 * hi)) - 1u;
    const uint32_t upto_lo = lo >= 4 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << (8 * lo)) - 1u;
    return upto_hi & ~upto_lo;
}

// A lane owns two channels of a group of eight tokens: eight 4-byte loads
// (a wave reads whole rows of a head) and one 16-byte store.  A group that is
// only partly new is read first and written back whole, by the one lane that
// owns it.
template <int D, int NW, int PASSES>
__device__ __forceinline__ void append_v(const KvAppendArgs &a, const PagePart &pp, int h, int tid, uint32_t *lds) {
    constexpr int LPG = D / 2, GP = 64 * NW / LPG;
    const int ch = tid % LPG, grp = tid / LPG;
    const int g0 = pp.lo >> 3, g1 = (pp.hi + 7) >> 3;
    uint4 *codes = reinterpret_cast<uint4 *>(a.vc + (pp.page * a.kv_heads + h) * ((int64_t)a.page * D));
    uint8_t *scale = a.vs + pp.page * a.kv_heads + h;
    const int old = pp.lo > 0 ? (int)*scale : 0;
    const uint16_t *src = a.v + pp.t0 * a.v_stride + (int64_t)h * D + 2 * ch;
    float x[PASSES][8], y[PASSES][8];      // channel 2 ch, channel 2 ch + 1
    uint4 kept[PASSES];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int g = g0 + p * GP + grp;
        kept[p] = make_uint4(0, 0, 0, 0);
        if (g < g1) {
            if (8 * g < pp.lo || 8 * g + 8 > pp.hi) kept[p] = codes[g * LPG + ch];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int slot = 8 * g + j;
                uint32_t w = 0;
                if (slot >= pp.lo && slot < pp.hi)
                    w = *reinterpret_cast<const uint32_t *>(src + (int64_t)(slot - pp.lo) * a.v_stride);
                x[p][j] = __uint_as_float(w << 16);
                y[p][j] = __uint_as_float(w & 0xFFFF0000u);
                m = max(m, max(finite_mag(x[p][j]), finite_mag(y[p][j])));
            }
        }
    }
    const int e = max(scale_byte(item_max<NW>(m, lds)), old);
    const float r = pow2_bits(254 - e);
    const bool grows = e > old && pp.lo > 0;
    const float f = pow2_bits(127 + old - e);
    if (grows)      // groups of earlier tokens only
        for (int i = tid; i < g0 * LPG; i += 64 * NW) codes[i] = lower16(codes[i], f);
    if (tid == 0 && e != old) *scale = (uint8_t)e;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int g = g0 + p * GP + grp;
        if (g < g1) {
            uint32_t w[4];      // channel 0: slots 0-3, 4-7; channel 1 likewise
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *t = (k < 2 ? x[p] : y[p]) + 4 * (k & 1);
                w[k] = codes4(t[0] * r, t[1] * r, t[2] * r, t[3] * r);
            }
            if (8 * g < pp.lo || 8 * g + 8 > pp.hi) {
                const uint32_t was[4] = {kept[p].x, kept[p].y, kept[p].z, kept[p].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = 8 * g + 4 * (k & 1);      // slot of the word's first byte
                    const uint32_t fresh = byte_mask(pp.lo - at, pp.hi - at);
                    const uint32_t before = byte_mask(0, pp.lo - at);
                    uint32_t rest = was[k];
                    if (grows) rest = (lower4(rest, f) & before) | (rest & ~before);
                    w[k] = (w[k] & fresh) | (rest & ~fresh);
                }
            }
            codes[g * LPG + ch] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Workgroups [0, q_blocks): a token's q rows.  The others: (page, head, k or
// v) items in the order (sequence, page, head, k/v), 4 / NW a workgroup.
template <int D, int NW, int PASSES>
__global__ void __launch_bounds__(256)
kv_append_kernel(const KvAppendArgs a, int q_blocks, int parts, int64_t items) {
    constexpr int SEGS = D / 16;
    __shared__ uint32_t lds[4];
    if ((int)blockIdx.x < q_blocks) {
        const int t = (int)blockIdx.x, seg = threadIdx.x % SEGS;
        const bool turns = 16 * seg < a.rot;
        Turn w8{};
        if (turns) w8 = load_turn(a, seg, t);
        const int o0 = run0(a, seg), o1 = run1(a, seg);
        for (int h = threadIdx.x / SEGS; h < a.q_heads; h += 256 / SEGS) {
            const uint16_t *src = a.q + (int64_t)t * a.q_stride + h * D;
            uint16_t *dst = a.q_out + (int64_t)t * a.q_out_stride + h * D;
            uint4 u = *reinterpret_cast<const uint4 *>(src + o0), w = *reinterpret_cast<const uint4 *>(src + o1);
            if (turns) {
                float x[8], y[8];
                unpack8(u, x);
                unpack8(w, y);
                turn(a.interleaved, w8, x, y);
                u = pack8(x);
                w = pack8(y);
            }
            *reinterpret_cast<uint4 *>(dst + o0) = u;
            *reinterpret_cast<uint4 *>(dst + o1) = w;
        }
        return;
    }
    const int tid = threadIdx.x % (64 * NW);
    int64_t item = (int64_t)(blockIdx.x - q_blocks) * (4 / NW) + threadIdx.x / (64 * NW);
    if (item >= items) return;      // whole waves (NW = 1) or none
    const int which = (int)(item & 1);
    item >>= 1;
    const int h = (int)(item % a.kv_heads);
    item /= a.kv_heads;
    const int b = (int)(item / parts), part = (int)(item % parts);
    // the sequence's rows, kept inside the batch, and the page's share of them
    const int first = min(max(a.q_start[b], 0), a.T), last = min(max(a.q_start[b + 1], first), a.T);
    // row i of n is token len - n + i; the first rows of more new tokens than
    // the sequence has are no tokens
    const int len = max(a.kv_len[b], 0), n = min(last - first, len), past = len - n;
    const int col = past / a.page + part;
    if (n == 0 || col >= a.max_pages) return;      // uniform over the item
    PagePart pp;
    const int64_t s0 = (int64_t)col * a.page;
    pp.lo = (int)max((int64_t)past - s0, (int64_t)0);
    pp.hi = (int)min((int64_t)past + n - s0, (int64_t)a.page);
    if (pp.lo >= pp.hi) return;
    pp.t0 = last - n + (s0 + pp.lo - past);
    pp.page = a.table[(int64_t)b * a.max_pages + col];
    if (pp.page < 0 || pp.page >= a.num_pages) return;
    if (which == 0) append_k<D, NW, PASSES>(a, pp, h, tid, lds);
    else append_v<D, NW, PASSES + 1>(a, pp, h, tid, lds);
}

template <int D, int NW, int PASSES>
hipError_t launch(const KvAppendArgs &a, hipStream_t stream) {
    const int q_blocks = a.q_heads > 0 ? a.T : 0;
    const int span = a.max_q < a.T ? a.max_q : a.T;
    // pages that `span` tokens can touch wherever they start
    const int64_t touched = ((int64_t)span + a.page - 2) / a.page + 1;
    const int parts = (int)(touched < a.max_pages ? touched : a.max_pages);
    const int64_t items = (int64_t)a.B * parts * a.kv_heads * 2;
    const int64_t grid = q_blocks + (items + 4 / NW - 1) / (4 / NW);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((kv_append_kernel<D, NW, PASSES>), dim3((unsigned)grid), dim3(256), 0, stream, a, q_blocks,
                       parts, items);
    return hipGetLastError();
}

// The fewest waves whose registers hold the tokens of a page that can be new
// at once: one wave holds 8 (head of 128) or 16 (64) a pass.
template <int D>
hipError_t launch_dim(const KvAppendArgs &a, hipStream_t stream) {
    constexpr int TP = 1024 / D;
    int most = a.max_q < a.T ? a.max_q : a.T;
    if (most > a.page) most = a.page;
    if (most <= TP) return launch<D, 1, 1>(a, stream);
    if (most <= 2 * TP) return launch<D, 1, 2>(a, stream);
    if (most <= 4 * TP) return launch<D, 4, 1>(a, stream);
    if (most <= 8 * TP) return launch<D, 4, 2>(a, stream);
    return launch<D, 4, 4>(a, stream);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t stream) {
    return a.dim == 64 ? launch_dim<64>(a, stream) : launch_dim<128>(a, stream);
}

}  // namespace biloco
