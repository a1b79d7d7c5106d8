// Attention over the paged 8-bit cache, many query rows per key/value head
// (prompts and their chunks).
//
// A workgroup takes 128 rows of one key/value head (a wave 32) and walks the
// 64-token chunks they see, codes staged in LDS, the next chunk's under way in
// registers meanwhile.  As in the kernel for few rows the products are
// S^T = K Q^T and O^T = V^T P^T, here as 32 x 32 tiles, so that a lane holds
// successive tokens of one row (l & 31) and the weights go from the first
// product to the second without leaving their registers:
//   A row 8a + 4h + b of token tile t is token 32 t + 16 (a >> 1) + 8 h + 4 (a & 1) + b,
//   so C register 4a + b of lane half h is that token, and registers 8c .. 8c + 7
//   are the eight tokens 32 t + 16 c + 8 h + (0 .. 7), an operand of the second
//   product and a group of the cache's value order.
// Bound by the vector ALUs next to the matrix cores: the exponentials, and the
// conversion of codes to bf16 in every wave.
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

template <int D>
struct TileLds {
    alignas(16) uint8_t k[2][kChunk * D];       // codes, rows of tokens (k_slot)
    alignas(16) uint16_t v[2][kChunk * D];      // bf16 [token / 8][channel][8]
    int ks[2][8];                               // scale bytes, per eight tokens
    uint16_t nan[2][kChunk * D / 16];      // NaN codes of each 16 bytes of v's codes, valid where odd is set
    int odd[2][kWaves];
};

// 16-byte slot of a token's row of K in LDS: rotated so that the 16 tokens
// that one phase of a 16-byte read takes lie in different banks.
template <int D>
__device__ __forceinline__ int k_slot(int token, int slot) {
    return token * D + 16 * (slot ^ (D == 128 ? (token >> 1) & 7 : (token >> 2) & 3));
}

// A chunk's way into LDS.  A thread moves 16 bytes N times: of K's token
// tid / (D / 16) + 32 i, and of V's token group tid / (D / 2) + 4 i.  The
// tokens of a wave lie within 16 aligned ones, so its pages are uniform.
template <int D>
struct Loader {
    static constexpr int N = D / 64;
    u32x4_t k[N], v[N];
    uint32_t scale[N], kscale;      // of the value group; of eight keys (the first eight threads)
    int id[N], kid;

    // The pages of the chunk at j0, one chunk ahead of their use.
    __device__ __forceinline__ void look_up(const int *table, int shift, int last, int j0) {
        const int wave = uniform((int)(threadIdx.x >> 6));
#pragma unroll
        for (int i = 0; i < N; ++i) id[i] = table[min(j0 + 32 * i + (N == 2 ? 8 : 16) * wave, last) >> shift];
        kid = table[min(j0 + 8 * (int)(threadIdx.x & 7), last) >> shift];
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
            scale[i] = a.vs[at];
        }
        if (wave == 0) kscale = a.ks[block(kid)];
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
                if (bits == 0) scale[i] = 127;
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
        for (int i = 0; i < N; ++i) {
            *reinterpret_cast<u32x4_t *>(&lds.k[buf][k_slot<D>(tid / (D / 16) + 32 * i, tid % (D / 16))]) = k[i];
            const float s = scale_of(scale[i]);
            u32x4_t *to = reinterpret_cast<u32x4_t *>(&lds.v[buf][16 * (tid + 256 * i)]);
            to[0] = widen8(v[i].x, v[i].y, s);
            to[1] = widen8(v[i].z, v[i].w, s);
        }
        if (tid < 8) lds.ks[buf][tid] = (int)kscale;
    }
};

template <int D>
struct Rows32 {
    u32x4_t q[D / 32][2];
    f32x16a_t o[D / 32];
    float m, l;      // m: of scale * log2(e) * s
    int p, p_min, p_max;

    __device__ __forceinline__ void init(const AttnArgs &a, const Seq &s, int h, int r0, int rows) {
        const int lane = threadIdx.x & 63, G = a.q_heads / a.kv_heads;
        const int row = min(r0 + (lane & 31), rows - 1), i = row / G;
        p = s.past + i;
        p_min = s.past + min(r0, rows - 1) / G;
        p_max = s.past + min(r0 + 31, rows - 1) / G;
        const uint16_t *src = a.q + (int64_t)(s.first + i) * a.q_stride + (int64_t)(h * G + row - i * G) * D + 16 * (lane >> 5);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) q[c][t] = *reinterpret_cast<const u32x4_t *>(src + 32 * c + 8 * t);
#pragma unroll
        for (int n = 0; n < D / 32; ++n) o[n] = zero16();
        m = -__builtin_inff();
        l = 0.0f;
    }

    __device__ __forceinline__ void scores(const TileLds<D> &lds, int buf, f32x16a_t (&sc)[2]) const {
        const int lane = threadIdx.x & 63, r = lane & 31;
        const int token = 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sc[t] = zero16();
            const float s = scale_of(lds.ks[buf][4 * t + (token >> 3)]);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t *>(&lds.k[buf][k_slot<D>(32 * t + token, 2 * c + (lane >> 5))]);
                sc[t] = mfma32(widen8(w.x, w.y, s), q[c][0], sc[t]);
                sc[t] = mfma32(widen8(w.z, w.w, s), q[c][1], sc[t]);
                if (c & 1) __builtin_amdgcn_sched_barrier(0);      // bounds the registers of codes made wide
            }
        }
    }

    // Scores to weights (at most 2^8 times a row's present maximum's: the
    // sums are moved to a new maximum only when it is that much larger).
    __device__ __forceinline__ void weigh(f32x16a_t (&sc)[2], float c2, u32x4_t (&pt)[4]) {
        float mx = fmaxf(sc[0][0], sc[1][0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, fmaxf(sc[0][i], sc[1][i]));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64)) * c2;
        if (__ballot(mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx);
            const float alpha = mn == -__builtin_inff() ? 1.0f : exp2a(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int n = 0; n < D / 32; ++n) o[n] *= alpha;
        }
        const float base = m == -__builtin_inff() ? 0.0f : m;      // a row that sees nothing yet
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sc[t][i] = exp2a(__builtin_fmaf(sc[t][i], c2, -base));
                sum += sc[t][i];
            }
        l += sum;
        // Rounded to bf16 (2^-8 of each at most); their sum l is kept as it was.
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x16a_t &x = sc[c >> 1];
            const int i = 8 * (c & 1);
            pt[c] = u32x4_t{narrow2a(x[i], x[i + 1]), narrow2a(x[i + 2], x[i + 3]), narrow2a(x[i + 4], x[i + 5]),
                            narrow2a(x[i + 6], x[i + 7])};
        }
    }

    __device__ __forceinline__ void gather(const TileLds<D> &lds, int buf, const u32x4_t (&pt)[4]) {
        const int lane = threadIdx.x & 63, h = lane >> 5;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t *>(&lds.v[buf][8 * ((2 * c + h) * D + 32 * n + (lane & 31))]);
                o[n] = mfma32(w, pt[c], o[n]);
            }
        }
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

    __device__ __forceinline__ void step(const AttnArgs &a, const TileLds<D> &lds, int buf, int j0, float c2) {
        f32x16a_t sc[2];
        u32x4_t pt[4];
        scores(lds, buf, sc);
        if (!all_see(a, p_min, p_max, j0)) {
            const int h = (threadIdx.x & 63) >> 5, lo = low_of(a, p);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = j0 + 32 * t + 16 * (i >> 3) + 8 * h + (i & 7);
                    sc[t][i] = sees(a, p, lo, j) ? sc[t][i] : -__builtin_inff();
                }
        }
        weigh(sc, c2, pt);
        if (lds.odd[buf][0] | lds.odd[buf][1] | lds.odd[buf][2] | lds.odd[buf][3]) mark_nan(a, lds, buf, j0);
        gather(lds, buf, pt);
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
        Loader<D> ld;
        ld.look_up(table, shift, last, span.start(c0));
        ld.load(a, shift, h, span.start(c0));
        if (c0 + 1 < c1) ld.look_up(table, shift, last, span.start(c0 + 1));
        ld.store(a, lds, 0, span.start(c0), p_min, p_max);
        __syncthreads();
        for (int c = c0; c < c1; ++c) {
            const int buf = (c - c0) & 1, j0 = span.start(c);
            if (c + 1 < c1) {
                ld.load(a, shift, h, span.start(c + 1));
                if (c + 2 < c1) ld.look_up(table, shift, last, span.start(c + 2));
            }
            w.step(a, lds, buf, j0, c2);
            if (c + 1 < c1) ld.store(a, lds, buf ^ 1, span.start(c + 1), p_min, p_max);
            __syncthreads();
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
    const TilesPlan p = attn_tiles_plan(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_kv);
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

// Tiles: every sequence ends at most one of them early.  The token axis is
// split where the tiles alone leave CUs idle, into pieces of at least four
// chunks.
TilesPlan attn_tiles_plan(int B, int T, int q_heads, int kv_heads, int dim, int max_kv) {
    TilesPlan p;
    const int64_t rows = (int64_t)T * (q_heads / kv_heads);
    p.tiles = (int)(rows / kTileRows + B);
    const int64_t items = (rows + kTileRows - 1) / kTileRows * kv_heads;
    const int pieces = (max_kv + 4 * kChunk - 1) / (4 * kChunk);
    int64_t splits = (kWantItems + items - 1) / items;
    if (splits > pieces) splits = pieces;
    p.splits = splits < 1 ? 1 : (int)splits;
    p.ws_bytes = p.splits == 1 ? 0 : (size_t)p.tiles * kv_heads * p.splits * kTileRows * (dim + 2) * sizeof(float);
    return p;
}

hipError_t launch_attn_tiles(const AttnArgs &a, int which, hipStream_t stream) {
    return a.dim == 64 ? launch<64>(a, which, stream) : launch<128>(a, which, stream);
}

}  // namespace biloco
