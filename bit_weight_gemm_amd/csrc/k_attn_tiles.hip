// Attention over the paged 8-bit cache, many query rows per key/value head
// (prompts and their chunks).
//
// A workgroup takes 128 rows of one key/value head (a wave 32) and walks the
// 64-token chunks they see, as bf16 in LDS (each code is made wide once for the
// 128 rows), the next chunk on its way in registers meanwhile.  As in the kernel
// for few rows the products are S^T = K Q^T and O^T = V^T P^T, here as 32 x 32
// tiles, so that a lane holds successive tokens of one row (l & 31) and the
// weights go from the first product to the second without leaving their
// registers:
//   A row 8a + 4h + b of token tile t is token 32 t + 16 (a >> 1) + 8 h + 4 (a & 1) + b,
//   so C register 4a + b of lane half h is that token, and registers 8c .. 8c + 7
//   are the eight tokens 32 t + 16 c + 8 h + (0 .. 7), an operand of the second
//   product and a group of the cache's value order.
// Per 64 tokens a wave of 128 channels issues 32 matrix instructions of 32 cycles
// and about 410 others (227 vector ones, 32 of them exponentials at a quarter of the
// rate, 44 of LDS, 141 scalar); no single part has been shown to bound it.  Measured on
// MI355X: 840 to 900 TFLOP/s at 128 channels and 720 to 760 at 64 where all tiles are
// alike (128 rows behind 16384 tokens, three or four workgroups a CU), 782 to 826
// TFLOP/s (220 to 208 us) for a causal prompt of 4096 tokens and 40 heads; an
// 8192-cubed library product reaches 1340 to 1430.  256 rows a workgroup: 226 us (waves
// of both halves of a SIMD meet at one barrier); 32-token buffers with three waves a
// SIMD: 275 us (registers spill, twice the barriers).
#include "attn_device.h"

namespace biloco {

namespace {

using namespace attn;

constexpr int kTileRows = 128, kWaves = 4;
constexpr int kWantItems = 512;      // workgroups that fill the chip (two a CU)

__device__ __forceinline__ f32x16a_t mfma32(u32x4_t a, u32x4_t b, f32x16a_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8a_t, a),
                                                   __builtin_bit_cast(bf16x8a_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16a_t zero16() {
    f32x16a_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.0f;
    return z;
}

// Codes wait in LDS as bf16, scale included: keys as [channel / 8][token][8],
// values as [token / 8][channel][8], so that the 16-byte reads of both products
// run over neighbouring addresses.  The rows of keys are 32 bytes longer than
// their 64 tokens, which spreads the banks that a wave's writes meet.
template <int D>
struct TileLds {
    static constexpr int kRow = 8 * kChunk + 16;
    alignas(16) uint16_t k[2][D / 8 * kRow];
    alignas(16) uint16_t v[2][kChunk * D];
    uint16_t nan[2][kChunk * D / 16];      // NaN codes of each 16 bytes of v's codes, valid where odd is set
    int odd[2][kWaves];
};

// A chunk's way into LDS.  A thread moves 16 bytes N times: of K's token
// tid / (D / 16) + 32 i, and of V's token group tid / (D / 2) + 4 i.  The
// tokens of a wave lie within 16 aligned ones, so its pages are uniform.
template <int D>
struct Loader {
    static constexpr int N = D / 64;
    u32x4_t k[N], v[N];
    uint32_t kscale[N], vscale[N];
    int id[N];

    // The pages of the chunk at j0, one chunk ahead of their use.
    __device__ __forceinline__ void look_up(const int *table, int shift, int last, int j0) {
        const int wave = uniform((int)(threadIdx.x >> 6));
#pragma unroll
        for (int i = 0; i < N; ++i) id[i] = table[min(j0 + 32 * i + (N == 2 ? 8 : 16) * wave, last) >> shift];
    }
    __device__ __forceinline__ void load(const AttnArgs &a, int shift, int h, int j0) {
        const int tid = threadIdx.x, wave = uniform(tid >> 6);
        const auto block = [&](int id) {
            return (int64_t)((uint32_t)id < (uint32_t)a.num_pages ? id : 0) * a.kv_heads + h;
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t at = block(uniform(id[i]));
            const int slot = (j0 + 32 * i + (N == 2 ? 8 : 16) * wave) & (a.page - 1);      // of the wave's first token
            const int64_t from = ((at << shift) + slot) * D;
            k[i] = *reinterpret_cast<const u32x4_t *>(a.kc + from + 16 * (tid & 63));
            v[i] = *reinterpret_cast<const u32x4_t *>(a.vc + from + 16 * (tid & 63));
            kscale[i] = a.ks[at];
            vscale[i] = a.vs[at];
        }
    }
    // Part i of 4 N of a chunk that all rows see whole.
    __device__ __forceinline__ void store_part(TileLds<D> &lds, int buf, int i) const {
        const int tid = threadIdx.x, j = i >> 2;
        const u32x4_t w = i & 2 ? v[j] : k[j];
        const float s = scale_of(i & 2 ? vscale[j] : kscale[j]);
        uint16_t *to = i & 2 ? &lds.v[buf][16 * (tid + 256 * j) + 8 * (i & 1)]
                             : &lds.k[buf][(2 * (tid % (D / 16)) + (i & 1)) * TileLds<D>::kRow + 8 * (tid / (D / 16) + 32 * j)];
        *reinterpret_cast<u32x4_t *>(to) = i & 1 ? widen8(w.z, w.w, s) : widen8(w.x, w.y, s);
    }
    // In a chunk that not every row of the tile (positions p_min to p_max) sees
    // whole, tokens that no row sees can hold anything: their codes become zero
    // and their scale 1.  NaN codes are taken out of the values and noted apart
    // (see mark_nan).
    __device__ __forceinline__ void store(const AttnArgs &a, TileLds<D> &lds, int buf, int j0, int p_min, int p_max) {
        const int tid = threadIdx.x;
        bool odd = false;
        if (!all_see(a, p_min, p_max, j0)) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t bits = any_sees8(a, p_min, p_max, j0 + 8 * (tid / (D / 2) + 4 * i));
                const uint32_t m0 = spread4(bits), m1 = spread4(bits >> 4);
                v[i] &= u32x4_t{m0, m1, m0, m1};
                if (bits == 0) vscale[i] = 127;
                const u32x4_t bad = nan_bytes(v[i]);
                v[i] &= ~bad;
                const u32x4_t four = ((bad & 0x08040201u) * 0x01010101u) >> 24;      // a bit a byte
                const uint32_t all = four.x | (four.y << 4) | (four.z << 8) | (four.w << 12);
                lds.nan[buf][tid + 256 * i] = (uint16_t)all;
                any |= all;
            }
            odd = __ballot(any != 0) != 0;
        }
        if ((tid & 63) == 0) lds.odd[buf][tid >> 6] = odd;
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) store_part(lds, buf, i);
    }
};

template <int D>
struct Rows32 {
    u32x4_t q[D / 16];
    f32x16a_t o[D / 32];
    float m, l;      // m: of scale * log2(e) * s
    int p, p_min, p_max;

    __device__ __forceinline__ void init(const AttnArgs &a, const Seq &s, int h, int r0, int rows) {
        const int lane = threadIdx.x & 63, G = a.q_heads / a.kv_heads;
        const int row = min(r0 + (lane & 31), rows - 1), i = row / G;
        p = s.past + i;
        p_min = s.past + min(r0, rows - 1) / G;
        p_max = s.past + min(r0 + 31, rows - 1) / G;
        const uint16_t *src = a.q + (int64_t)(s.first + i) * a.q_stride + (int64_t)(h * G + row - i * G) * D + 8 * (lane >> 5);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) q[c] = *reinterpret_cast<const u32x4_t *>(src + 16 * c);
#pragma unroll
        for (int n = 0; n < D / 32; ++n) o[n] = zero16();
        m = -__builtin_inff();
        l = 0.0f;
    }

    // Scores of the chunk's token tile t.
    __device__ __forceinline__ f32x16a_t scores(const TileLds<D> &lds, int buf, int t) const {
        const int lane = threadIdx.x & 63, r = lane & 31;
        const int token = 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3);
        const uint16_t *k = &lds.k[buf][(lane >> 5) * TileLds<D>::kRow + 8 * (32 * t + token)];
        f32x16a_t sc = zero16();
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            sc = mfma32(*reinterpret_cast<const u32x4_t *>(k + 2 * c * TileLds<D>::kRow), q[c], sc);
        return sc;
    }

    // Hides what a row does not see of the 32 tokens at j0.
    __device__ __forceinline__ void hide(const AttnArgs &a, f32x16a_t &sc, int j0) const {
        const int h = (threadIdx.x & 63) >> 5, lo = low_of(a, p);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = j0 + 16 * (i >> 3) + 8 * h + (i & 7);
            sc[i] = sees(a, p, lo, j) ? sc[i] : -__builtin_inff();
        }
    }

    __device__ __forceinline__ float top_of(const f32x16a_t &sc, float c2) const {
        float mx = sc[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
        return fmaxf(mx, __shfl_xor(mx, 32, 64)) * c2;
    }
    // The sums move to a new maximum only when it is much larger (the weights
    // stay below 2^8 of a row's present one's).
    __device__ __forceinline__ void follow(float mx) {
        if (__ballot(mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx);
            const float alpha = mn == -__builtin_inff() ? 1.0f : exp2a(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int n = 0; n < D / 32; ++n) o[n] *= alpha;
        }
    }
    // Scores to weights, rounded to bf16 for the product (2^-8 of each at
    // most); their sum is taken before that.  What the rounding leaves as a second
    // term, as in the kernel for few rows, brings o's error to that of its own rounding
    // (from 1.3 to 1.4 times that, root mean square) and takes half as many matrix
    // instructions again, which that kernel has time for and this one has not: 259 us
    // for 210 on a prompt of 4096 tokens, 441 for 348 on chunks of 64 channels.
    __device__ __forceinline__ void weigh(f32x16a_t &sc, float c2, u32x4_t (&pt)[2]) {
        const float base = m == -__builtin_inff() ? 0.0f : m;      // a row that sees nothing yet
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sc[i] = exp2a(__builtin_fmaf(sc[i], c2, -base));
            sum += sc[i];
        }
        l += sum;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            pt[c] = u32x4_t{narrow2a(sc[8 * c], sc[8 * c + 1]), narrow2a(sc[8 * c + 2], sc[8 * c + 3]),
                            narrow2a(sc[8 * c + 4], sc[8 * c + 5]), narrow2a(sc[8 * c + 6], sc[8 * c + 7])};
    }

    __device__ __forceinline__ void gather(const TileLds<D> &lds, int buf, int t, const u32x4_t (&pt)[2]) {
        const int lane = threadIdx.x & 63;
        const uint16_t *v = &lds.v[buf][8 * ((4 * t + (lane >> 5)) * D + (lane & 31))];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
                o[n] = mfma32(*reinterpret_cast<const u32x4_t *>(v + 16 * c * D + 256 * n), pt[c], o[n]);
    }

    // One tile on, in the order in which it is to be issued: between two matrix
    // instructions as much of the vector work as fits their time.  Scores s of
    // tile t in `buf` become weights while the next tile's scores (tile t1 in
    // `buf1`) are computed; the values of tile t are gathered while the next
    // scores' maximum is taken and, with `advance`, the next chunk's codes become
    // bf16 in LDS.  Returns the next scores' maximum.
    template <bool ADVANCE>
    __device__ __forceinline__ float tile(TileLds<D> &lds, int buf, int t, int buf1, int t1, f32x16a_t &s, f32x16a_t &next,
                                          float c2, const Loader<D> &ld) {
        constexpr int M = D / 16, E = 16 / M;      // matrix instructions of each product; scores between two
        const int lane = threadIdx.x & 63, r = lane & 31;
        const int token = 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3);
        const uint16_t *k = &lds.k[buf1][(lane >> 5) * TileLds<D>::kRow + 8 * (32 * t1 + token)];
        const uint16_t *v = &lds.v[buf][8 * ((4 * t + (lane >> 5)) * D + (lane & 31))];
        const auto key = [&](int i) { return *reinterpret_cast<const u32x4_t *>(k + 2 * i * TileLds<D>::kRow); };
        const auto value = [&](int i) {
            return *reinterpret_cast<const u32x4_t *>(v + 16 * (i / (D / 32)) * D + 256 * (i % (D / 32)));
        };
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f;
        u32x4_t pt[2], f[M];
        f[0] = key(0);
        f[1] = key(1);
        next = zero16();
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (i + 2 < M) f[i + 2] = key(i + 2);
            next = mfma32(f[i], q[i], next);
#pragma unroll
            for (int j = E * i; j < E * i + E; ++j) {
                s[j] = exp2a(__builtin_fmaf(s[j], c2, -base));
                sum += s[j];
                if (j & 1) pt[j >> 3][(j >> 1) & 3] = narrow2a(s[j - 1], s[j]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        l += sum;
        f[0] = value(0);
        f[1] = value(1);
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (i + 2 < M) f[i + 2] = value(i + 2);
            o[i % (D / 32)] = mfma32(f[i], pt[i / (D / 32)], o[i % (D / 32)]);
            if constexpr (ADVANCE) ld.store_part(lds, buf ^ 1, i);
#pragma unroll
            for (int j = E * i; j < E * i + E; ++j) mx = fmaxf(mx, next[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        return fmaxf(mx, __shfl_xor(mx, 32, 64)) * c2;
    }

    // NaN values, taken out of the product: a row that sees one gets NaN in its
    // channel, by a product of what is visible with what is NaN (above 0 if any).
    __device__ __forceinline__ void mark_nan(const AttnArgs &a, const TileLds<D> &lds, int buf, int j0) {
        const int lane = threadIdx.x & 63, h = lane >> 5;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
            f32x16a_t x = zero16();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t mine = sees8(a, p, j0 + 16 * c + 8 * h);
                const uint32_t bad = lds.nan[buf][(2 * c + h) * (D / 2) + 16 * n + ((lane & 31) >> 1)] >> (8 * (lane & 1));
                x = mfma32(widen8(spread4(bad) & kOnes, spread4(bad >> 4) & kOnes, 1.0f),
                           widen8(spread4(mine) & kOnes, spread4(mine >> 4) & kOnes, 1.0f), x);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][i] = x[i] > 0.0f ? __builtin_nanf("") : o[n][i];
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// A piece of an item's tokens, split by split: [rows][D] sums, then maxima
// and sums of the weights.
template <int D>
__device__ __forceinline__ float *tile_part(const AttnArgs &a, int64_t item, int splits, int split) {
    return static_cast<float *>(a.ws) + (item * splits + split) * kTileRows * (D + 2);
}

__device__ __forceinline__ int64_t tiles_of(const AttnArgs &a, const Seq &s) {
    return (s.n * (a.q_heads / a.kv_heads) + kTileRows - 1) / kTileRows;
}

// Workgroups: row tile (the last first: under causality the longest),
// split, key/value head.  Heads run fastest, so the tiles of one head meet in
// one XCD's L2 where the number of heads is a multiple of 8.
template <int D>
__global__ void __launch_bounds__(256, 2)
attn_tiles_kernel(const AttnArgs a, int which, int tiles, int splits) {
    __shared__ TileLds<D> lds;
    const int h = (int)(blockIdx.x % a.kv_heads), rest = (int)(blockIdx.x / a.kv_heads);
    const int split = rest % splits, at = tiles - 1 - rest / splits;
    int64_t before = 0;
    const int b = uniform(find_seq(a.B, at, before, [&](int i) { return tiles_of(a, seq_of(a, i, which)); }));
    if (b < 0) return;
    const Seq s = seq_uniform(a, b, which);
    const int G = a.q_heads / a.kv_heads, rows = s.n * G, r0 = (at - (int)uniform(before)) * kTileRows;
    const int shift = 31 - __clz(a.page), last = s.hi - 1;
    const int *table = a.table + (int64_t)b * a.max_pages;
    const int p_min = s.past + r0 / G, p_max = s.past + (min(r0 + kTileRows, rows) - 1) / G;
    const Span64 span = span_of(a, p_min, p_max);
    const int each = (span.nc + splits - 1) / splits;
    const int c0 = min(split * each, span.nc), c1 = min(c0 + each, span.nc);
    const int wave = uniform((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const float c2 = a.scale * kLog2e;

    Rows32<D> w;
    w.init(a, s, h, r0 + 32 * wave, rows);
    if (c0 < c1) {
        // Two 32-token tiles a chunk.  The scores of a tile are computed while
        // the one before goes through its exponentials, its maximum while that
        // one's values are gathered.
        const auto whole = [&](int c) { return all_see(a, p_min, p_max, span.start(c)); };
        Loader<D> ld;
        // chunk c on its way, and the pages of the one after it
        const auto request = [&](int c) {
            ld.load(a, shift, h, span.start(min(c, c1 - 1)));
            ld.look_up(table, shift, last, span.start(min(c + 1, c1 - 1)));
        };
        ld.look_up(table, shift, last, span.start(c0));
        request(c0);
        ld.store(a, lds, 0, span.start(c0), p_min, p_max);
        request(c0 + 1);
        __syncthreads();
        f32x16a_t s0 = w.scores(lds, 0, 0), s1;
        if (!whole(c0)) w.hide(a, s0, span.start(c0));
        w.follow(w.top_of(s0, c2));
        int c = c0;
        while (true) {
            // Nothing to hide here and next.  With 64 channels the plain order below
            // is faster: it leaves registers for three waves a SIMD instead of two
            // (chunks of 2048 behind up to 10000 tokens: 343 us, 357 this way).
            while (D == 128 && c + 1 < c1 && whole(c) && whole(c + 1)) {
                const int buf = (c - c0) & 1;
                __syncthreads();      // the other buffer has been read
                if ((threadIdx.x & 63) == 0) lds.odd[buf ^ 1][wave] = 0;
                w.follow(w.template tile<true>(lds, buf, 0, buf, 1, s0, s1, c2, ld));
                request(c + 2);
                __syncthreads();      // the next chunk is in place
                w.follow(w.template tile<false>(lds, buf, 1, buf ^ 1, 0, s1, s0, c2, ld));
                ++c;
            }
            const int buf = (c - c0) & 1, j0 = span.start(c);
            u32x4_t pt[2];
            __syncthreads();
            if (c + 1 < c1) {
                ld.store(a, lds, buf ^ 1, span.start(c + 1), p_min, p_max);
                request(c + 2);
            }
            if (lds.odd[buf][0] | lds.odd[buf][1] | lds.odd[buf][2] | lds.odd[buf][3]) w.mark_nan(a, lds, buf, j0);
            w.weigh(s0, c2, pt);
            s1 = w.scores(lds, buf, 1);
            if (!all_see(a, w.p_min, w.p_max, j0)) w.hide(a, s1, j0 + 32);
            w.gather(lds, buf, 0, pt);
            w.follow(w.top_of(s1, c2));
            __syncthreads();
            w.weigh(s1, c2, pt);
            if (c + 1 < c1) {
                s0 = w.scores(lds, buf ^ 1, 0);
                if (!all_see(a, w.p_min, w.p_max, span.start(c + 1))) w.hide(a, s0, span.start(c + 1));
            }
            w.gather(lds, buf, 1, pt);
            if (++c == c1) break;
            w.follow(w.top_of(s0, c2));
        }
    }

    const float l = w.l + __shfl_xor(w.l, 32, 64);
    const int row = r0 + 32 * wave + (lane & 31), half = lane >> 5;
    if (row >= rows) return;
    if (splits > 1) {
        float *part = tile_part<D>(a, (int64_t)at * a.kv_heads + h, splits, split);
        float *dst = part + (row - r0) * D + 4 * half;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4a_t *>(dst + 32 * n + 8 * j) =
                    f32x4a_t{w.o[n][4 * j], w.o[n][4 * j + 1], w.o[n][4 * j + 2], w.o[n][4 * j + 3]};
        if (half == 0) {
            part[kTileRows * D + 2 * (row - r0)] = w.m;
            part[kTileRows * D + 2 * (row - r0) + 1] = l;
        }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = row / G, g = row - i * G;
    const int64_t t = s.first + i;
    uint16_t *dst = a.o + t * a.o_stride + (int64_t)(h * G + g) * D + 4 * half;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2 *>(dst + 32 * n + 8 * j) =
                make_uint2(narrow2a(w.o[n][4 * j] * inv, w.o[n][4 * j + 1] * inv),
                           narrow2a(w.o[n][4 * j + 2] * inv, w.o[n][4 * j + 3] * inv));
    if (a.lse && half == 0) a.lse[t * a.q_heads + h * G + g] = (w.m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Joins the pieces of a row: a wave a row.
template <int D>
__global__ void __launch_bounds__(256)
attn_tiles_join_kernel(const AttnArgs a, int which, int splits) {
    const int64_t item = blockIdx.x / (kTileRows / 4);
    const int h = (int)(item % a.kv_heads), at = (int)(item / a.kv_heads);
    int64_t before = 0;
    const int b = uniform(find_seq(a.B, at, before, [&](int i) { return tiles_of(a, seq_of(a, i, which)); }));
    if (b < 0) return;
    const Seq s = seq_uniform(a, b, which);
    const int G = a.q_heads / a.kv_heads, lane = threadIdx.x & 63;
    const int row = (int)(blockIdx.x % (kTileRows / 4)) * 4 + (int)(threadIdx.x >> 6);
    const int whole = (at - (int)uniform(before)) * kTileRows + row;
    if (whole >= s.n * G) return;
    float m = -__builtin_inff(), l = 0.0f, acc[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = 0.0f;
    for (int i = 0; i < splits; ++i) {
        const float *part = tile_part<D>(a, item, splits, i);
        const float pm = part[kTileRows * D + 2 * row], pl = part[kTileRows * D + 2 * row + 1];
        const float top = fmaxf(m, pm), base = top == -__builtin_inff() ? 0.0f : top;
        const float f0 = exp2a(m - base), f1 = exp2a(pm - base);
        m = top;
        l = l * f0 + pl * f1;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = acc[j] * f0 + part[row * D + (D / 64) * lane + j] * f1;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = whole / G, g = whole - i * G;
    const int64_t t = s.first + i;
    uint16_t *dst = a.o + t * a.o_stride + (int64_t)(h * G + g) * D + (D / 64) * lane;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) dst[j] = f32_to_bf16_rne(acc[j] * inv);
    if (a.lse && lane == 0) a.lse[t * a.q_heads + h * G + g] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int D>
hipError_t launch(const AttnArgs &a, int which, hipStream_t stream) {
    const TilesPlan p = attn_tiles_plan(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_kv, a.window, a.sinks);
    const int64_t grid = (int64_t)p.tiles * p.splits * a.kv_heads;
    const int64_t join = (int64_t)p.tiles * a.kv_heads * (kTileRows / 4);
    if (grid > 0x7FFFFFFF || join > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_tiles_kernel<D>), dim3((unsigned)grid), dim3(256), 0, stream, a, which, p.tiles, p.splits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((attn_tiles_join_kernel<D>), dim3((unsigned)join), dim3(256), 0, stream, a, which, p.splits);
    return hipGetLastError();
}

}  // namespace

// Tiles: the kernel's sequences have more than kMostRows rows each, so there
// are at most rows / (kMostRows + 1) of them, and each ends at most one tile early.
// The token axis is split where the tiles alone leave CUs idle, into pieces of at
// least four of the chunks that a tile sees.  Behind 32768 tokens with a window of
// 1024 (64/8 heads of 128), 16 and 32 new ones: 20.6 and 21.9 us, in pieces of one
// chunk 22.3 and 27.5, of four chunks of the whole context 40.9 and 31.9.
TilesPlan attn_tiles_plan(int B, int T, int q_heads, int kv_heads, int dim, int max_kv, int window, int sinks) {
    TilesPlan p;
    const int64_t rows = (int64_t)T * (q_heads / kv_heads);
    const int64_t most = rows / (kMostRows + 1), seqs = most < B ? most : B;
    p.tiles = (int)((rows + (kTileRows - 1) * seqs) / kTileRows);
    const int64_t items = (int64_t)p.tiles * kv_heads;
    int64_t chunks = ((int64_t)max_kv + kChunk - 1) / kChunk;
    if (window > 0) {
        const int64_t tokens = kTileRows / (q_heads / kv_heads) + 1;      // of a tile's rows
        const int64_t seen = ((int64_t)window + tokens + 2 * kChunk) / kChunk + ((int64_t)sinks + kChunk - 1) / kChunk;
        if (seen < chunks) chunks = seen;
    }
    const int64_t pieces = (chunks + 3) / 4;
    int64_t splits = items > 0 ? (kWantItems + items - 1) / items : 1;
    if (splits > pieces) splits = pieces;
    p.splits = splits < 1 ? 1 : (int)splits;
    p.ws_bytes = p.splits == 1 ? 0 : (size_t)items * p.splits * kTileRows * (dim + 2) * sizeof(float);
    return p;
}

// The most that a plan of these sizes or of smaller ones asks for: fewer rows can
// have more pieces, so the plan's own bytes do not grow with the call.  Items below
// kWantItems are split, into fewer than kWantItems + items pieces in all.
size_t attn_tiles_most_bytes(int B, int T, int q_heads, int kv_heads, int dim, int max_kv) {
    const TilesPlan p = attn_tiles_plan(B, T, q_heads, kv_heads, dim, max_kv, 0, 0);
    const int64_t all = (int64_t)p.tiles * kv_heads, items = all < kWantItems ? all : kWantItems - 1;
    const int64_t pieces = ((int64_t)max_kv + 4 * kChunk - 1) / (4 * kChunk);
    if (pieces <= 1) return 0;
    const int64_t most = items * pieces < items + kWantItems - 1 ? items * pieces : items + kWantItems - 1;
    return (size_t)most * kTileRows * (dim + 2) * sizeof(float);
}

hipError_t launch_attn_tiles(const AttnArgs &a, int which, hipStream_t stream) {
    return a.dim == 64 ? launch<64>(a, which, stream) : launch<128>(a, which, stream);
}

}  // namespace biloco
