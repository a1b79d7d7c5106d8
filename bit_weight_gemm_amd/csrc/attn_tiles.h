// The parts of attention over many query rows per key/value head (k_attn_tiles.hip says
// how a workgroup works): chunks on their way into LDS, 32 rows a wave, the walk over chunks.
#pragma once
#include "attn_device.h"

namespace biloco {
namespace attn {

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

// Bit j: some row of the tile sees token t0 + j.  Rows of one sequence follow one another,
// so what they see has no gaps.
__device__ __forceinline__ uint32_t tile_sees8(const AttnArgs &a, int p_min, int p_max, int t0) {
    return any_sees8(a, p_min, p_max, t0);
}

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
    template <class A>
    __device__ __forceinline__ void store(const A &a, TileLds<D> &lds, int buf, int j0, int p_min, int p_max) {
        const int tid = threadIdx.x;
        bool odd = false;
        if (!all_see(a, p_min, p_max, j0)) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t bits = tile_sees8(a, p_min, p_max, j0 + 8 * (tid / (D / 2) + 4 * i));
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

// Weights go into the product with v rounded to bf16 (2^-8 of each at most), or as two
// bf16 terms, the second one what that rounding left (together within 2^-16), as in the
// kernel for few rows; their sum is taken before that.  The second term brings o's error
// to that of its own rounding (from 1.3 to 1.4 times that, root mean square) and takes half
// as many matrix instructions again: on sequences of many rows 259 us for 210 on a prompt of
// 4096 tokens, 441 for 348 on chunks of 64 channels, so the paged call has one term there.
// The call with shared tokens has two for all of its rows, so that none of its results is
// less exact than the paged call's of few rows: four answers behind 608 tokens 19.2 us for
// 18.1, 64 behind 16384 84 for 77; four sequences of 128 tokens behind 8192 203 for 166.
template <int D, int TERMS>
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
        start(a.q + (int64_t)(s.first + i) * a.q_stride + (int64_t)(h * G + row - i * G) * D + 8 * (lane >> 5));
    }
    // The lane's part of its row's query.
    __device__ __forceinline__ void start(const uint16_t *src) {
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
    template <class A>
    __device__ __forceinline__ void hide(const A &a, f32x16a_t &sc, int j0) const {
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
    // Two weights as pair i of terms.
    __device__ __forceinline__ static void pack(u32x4_t (&pt)[TERMS][2], int i, float w0, float w1) {
        const uint32_t w = narrow2a(w0, w1);
        pt[0][i >> 2][i & 3] = w;
        if constexpr (TERMS == 2)
            pt[1][i >> 2][i & 3] = narrow2a(w0 - __uint_as_float(w << 16), w1 - __uint_as_float(w & 0xFFFF0000u));
    }
    // Scores to weights.
    __device__ __forceinline__ void weigh(f32x16a_t &sc, float c2, u32x4_t (&pt)[TERMS][2]) {
        const float base = m == -__builtin_inff() ? 0.0f : m;      // a row that sees nothing yet
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sc[i] = exp2a(__builtin_fmaf(sc[i], c2, -base));
            sum += sc[i];
        }
        l += sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) pack(pt, i, sc[2 * i], sc[2 * i + 1]);
    }

    __device__ __forceinline__ void gather(const TileLds<D> &lds, int buf, int t, const u32x4_t (&pt)[TERMS][2]) {
        const int lane = threadIdx.x & 63;
        const uint16_t *v = &lds.v[buf][8 * ((4 * t + (lane >> 5)) * D + (lane & 31))];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t *>(v + 16 * c * D + 256 * n);
#pragma unroll
                for (int e = 0; e < TERMS; ++e) o[n] = mfma32(w, pt[e][c], o[n]);
            }
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
        u32x4_t pt[TERMS][2], f[M];
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
                if (j & 1) pack(pt, j >> 1, s[j - 1], s[j]);
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
#pragma unroll
            for (int e = 0; e < TERMS; ++e) o[i % (D / 32)] = mfma32(f[i], pt[e][i / (D / 32)], o[i % (D / 32)]);
            if constexpr (ADVANCE) ld.store_part(lds, buf ^ 1, i);
#pragma unroll
            for (int j = E * i; j < E * i + E; ++j) mx = fmaxf(mx, next[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        return fmaxf(mx, __shfl_xor(mx, 32, 64)) * c2;
    }

    // NaN values, taken out of the product: a row that sees one gets NaN in its
    // channel, by a product of what is visible with what is NaN (above 0 if any).
    template <class A>
    __device__ __forceinline__ void mark_nan(const A &a, const TileLds<D> &lds, int buf, int j0) {
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

// What a workgroup works on: chunks [c0, c1) of `span`, seen by rows at positions p_min
// to p_max, through a block table row whose last token is `last`.
template <class A>
struct TileWork {
    A a;
    const int *table;
    int last, h, c0, c1, p_min, p_max;
    Span64 span;
    int at, split;      // tile, piece of its chunks
    int r0, rows;       // first of its rows, how many there are
    Seq s;              // the sequence, where it is one
};

// What the kernels of both calls do: K::begin gives a workgroup its rows and its work (false:
// there is none), K::end takes what the rows have gathered.  In one function, since the
// walk over chunks as a function of its own costs the compiler 32 registers' moves a
// turn (chunks of 64 channels 356 -> 380 us).
template <int D, class K>
__device__ __forceinline__ void tile_rows(const K &k, int splits, TileLds<D> &lds, typename K::Lds &more) {
    Rows32<D, K::kTerms> w;
    TileWork<typename K::Args> t{k.args()};
    if (!k.begin(w, t, more, splits)) return;
    const auto &a = t.a;
    const int *table = t.table;
    const int last = t.last, h = t.h, c0 = t.c0, c1 = t.c1, p_min = t.p_min, p_max = t.p_max;
    const Span64 span = t.span;
    const int shift = 31 - __clz(a.page), wave = uniform((int)(threadIdx.x >> 6));
    const float c2 = a.scale * kLog2e;
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
            u32x4_t pt[K::kTerms][2];
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
    k.end(w, t, w.l + __shfl_xor(w.l, 32, 64), splits);
}

template <int D, class K>
__global__ void __launch_bounds__(256, 2)
attn_tiles_kernel(const K k, int splits) {
    __shared__ TileLds<D> lds;
    __shared__ typename K::Lds more;
    tile_rows<D>(k, splits, lds, more);
}

// A row's sums as a piece of them: [kTileRows][D], then maxima and sums of the weights.
// blind: nothing in their place.
template <int D, int TERMS>
__device__ __forceinline__ void leave(const Rows32<D, TERMS> &w, float l, float *part, int row, bool blind = false) {
    const int half = (threadIdx.x & 63) >> 5;
    float *dst = part + row * D + 4 * half;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4a_t *>(dst + 32 * n + 8 * j) =
                blind ? f32x4a_t{0, 0, 0, 0} : f32x4a_t{w.o[n][4 * j], w.o[n][4 * j + 1], w.o[n][4 * j + 2], w.o[n][4 * j + 3]};
    if (half == 0) {
        part[kTileRows * D + 2 * row] = blind ? -__builtin_inff() : w.m;
        part[kTileRows * D + 2 * row + 1] = blind ? 0.0f : l;
    }
}

}  // namespace attn
}  // namespace biloco
