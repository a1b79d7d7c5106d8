// Attention over the paged 8-bit cache, few query rows per key/value head
// (decode, drafted tokens).
//
//   s = scale q.k,  w = softmax over the visible tokens,  o = sum w v
//
// One pass over the cache with the running maximum m and sum l of a softmax
// (in powers of two).  The G = q_heads / kv_heads query heads that share a
// key/value head, times the new tokens, are the rows of one product, so a
// cached token is read once for all of them.
//
// A wave takes 64 tokens at a time and needs no shared memory for it:
//   S^T = K Q^T     A = K (16 tokens x 32 channels), B = Q^T: lane l holds row
//                   l & 15 and, with the token order below, eight successive
//                   tokens of it for every 32
//   O^T = V^T P^T   B = P^T straight from those registers; A = V^T from the
//                   cache's order of eight tokens per channel
// K's and V's codes become bf16 (exact, the block's scale included) by the
// conversion instruction that takes a power of two.  The tokens of tile (kk, f)
// of a chunk: A row m is token 32 kk + 8 (m >> 2) + 4 f + (m & 3), so C row
// 4 q4 + i of the tiles f = 0, 1 are tokens 32 kk + 8 q4 + 4 f + i.  Channels
// are taken in the order in which a lane's 16-byte load brings them: channel
// 64 c + 16 q4 + 8 s + j is slot 8 q4 + j of step (c, s).
#include "attn_device.h"

namespace biloco {

namespace {

using namespace attn;

constexpr int kSplitGrid = 512;    // workgroups of a call that splits the token axis

template <int D>
struct Stage {
    u32x4_t k[2][2][D / 64];      // [kk][f][c]
    u32x4_t v[2][D / 32];         // [kk][nb]
    float ks[2];
    uint32_t vs[2];
};
// Pages of the next chunk's tokens, asked for one chunk ahead of their use.
struct Pages {
    int k[2], v[2];
};

// One piece: units [u0, u1) of item (b, h, tile), by the whole workgroup.
template <int D, int R>
struct Piece {
    const AttnArgs &a;
    const Seq s;
    const int b, h, tile, G, lane, wave, q4, rows, shift;
    int p_min, p_max;
    u32x4_t q[R][D / 64][2];
    f32x4a_t o[R][D / 16];
    float m[R], l[R];
    int p[R];

    __device__ __forceinline__ Piece(const AttnArgs &a_, const Seq &s_, int b_, int h_, int tile_)
        : a(a_), s(s_), b(b_), h(h_), tile(tile_), G(a_.q_heads / a_.kv_heads), lane(threadIdx.x & 63),
          wave(__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6))), q4((threadIdx.x & 63) >> 4),
          rows(s_.n * (a_.q_heads / a_.kv_heads)), shift(31 - __clz(a_.page)) {
        const int r0 = tile * 16 * R;
        p_min = s.past + r0 / G;
        p_max = s.past + (min(r0 + 16 * R, rows) - 1) / G;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = min(r0 + 16 * r + (lane & 15), rows - 1);
            const int i = row / G, g = row - i * G;
            p[r] = s.past + i;
            const uint16_t *src = a.q + (int64_t)(s.first + i) * a.q_stride + (int64_t)(h * G + g) * D;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    q[r][c][t] = *reinterpret_cast<const u32x4_t *>(src + 64 * c + 16 * q4 + 8 * t);
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[r][n] = f32x4a_t{0, 0, 0, 0};
        }
    }

    __device__ __forceinline__ int start_of(int c) const { return s.c.start(c); }

    // Page of token j (a token past the last one reads the last one's page).
    __device__ __forceinline__ int page_of(int j) const {
        return a.table[(int64_t)b * a.max_pages + (min(j, s.hi - 1) >> shift)];
    }
    __device__ __forceinline__ int64_t block_of(int id) const {
        return (int64_t)((uint32_t)id < (uint32_t)a.num_pages ? id : 0) * a.kv_heads + h;
    }
    __device__ __forceinline__ void look_up(Pages &g, int chunk) const {
        const int j0 = start_of(chunk);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            g.k[kk] = page_of(j0 + 32 * kk + 8 * ((lane & 15) >> 2));
            g.v[kk] = page_of(j0 + 32 * kk + 8 * q4);
        }
    }
    __device__ __forceinline__ void load_k(Stage<D> &st, const Pages &g, int chunk) const {
        const int mrow = lane & 15, j = (start_of(chunk) + 8 * (mrow >> 2)) & (a.page - 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int64_t bk = block_of(g.k[kk]);
            const int slot = (j + 32 * kk) & (a.page - 1);
            const uint8_t *k = a.kc + (((bk << shift) + slot + (mrow & 3)) * D + 16 * q4);
            st.ks[kk] = scale_of(a.ks[bk]);
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    st.k[kk][f][c] = *reinterpret_cast<const u32x4_t *>(k + 4 * f * D + 64 * c);
        }
    }
    __device__ __forceinline__ void load_v(Stage<D> &st, const Pages &g, int chunk) const {
        const int j = (start_of(chunk) + 8 * q4) & (a.page - 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int64_t bv = block_of(g.v[kk]);
            const int slot = (j + 32 * kk) & (a.page - 1);
            const uint8_t *v = a.vc + (((bv << shift) + slot) * D + 16 * (lane & 15));
            st.vs[kk] = a.vs[bv];
#pragma unroll
            for (int n = 0; n < D / 32; ++n) st.v[kk][n] = *reinterpret_cast<const u32x4_t *>(v + 256 * n);
        }
    }

    // One chunk; the next one's keys are asked for as soon as this one's are
    // used up, its values likewise.
    __device__ __forceinline__ void step(Stage<D> &st, Pages &g, int chunk, int next, bool more) {
        const int j0 = start_of(chunk);
        const bool full = all_see(a, p_min, p_max, j0);
        bool odd = false;
        if (!full) {
            // Tokens that no row sees can hold anything: zero codes, scale 1.
            // What only some rows see must not reach the others as 0 * NaN.
            uint32_t bad = 0;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const uint32_t bits = any_sees8(a, p_min, p_max, j0 + 32 * kk + 8 * q4);
                const uint32_t m0 = spread4(bits), m1 = spread4(bits >> 4);
                if (bits == 0) st.vs[kk] = 127;
#pragma unroll
                for (int n = 0; n < D / 32; ++n) {
                    st.v[kk][n] &= u32x4_t{m0, m1, m0, m1};
                    const u32x4_t t = nan_bytes(st.v[kk][n]);
                    bad |= t.x | t.y | t.z | t.w;
                }
            }
            odd = __ballot(bad != 0) != 0;
        }
        f32x4a_t sc[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[r][t] = f32x4a_t{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const u32x4_t w = st.k[kk][f][c];
                    const u32x4_t a0 = widen8(w.x, w.y, st.ks[kk]), a1 = widen8(w.z, w.w, st.ks[kk]);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        sc[r][2 * kk + f] = mfma16(a0, q[r][c][0], sc[r][2 * kk + f]);
                        sc[r][2 * kk + f] = mfma16(a1, q[r][c][1], sc[r][2 * kk + f]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        if (more) load_k(st, g, next);
        const float c2 = a.scale * kLog2e;
        u32x4_t pt[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[r][t][i] *= c2;
                    mx = fmaxf(mx, sc[r][t][i]);
                }
            if (!full) {      // the maximum is that of the visible
                const int lo = low_of(a, p[r]);
                mx = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1) + i;
                        sc[r][t][i] = sees(a, p[r], lo, j) ? sc[r][t][i] : -__builtin_inff();
                        mx = fmaxf(mx, sc[r][t][i]);
                    }
            }
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float mn = fmaxf(m[r], mx);
            const float base = mn == -__builtin_inff() ? 0.0f : mn;      // a row that sees nothing yet
            const float alpha = exp2a(m[r] - base);
            m[r] = mn;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[r][t][i] = exp2a(sc[r][t][i] - base);
                    sum += sc[r][t][i];
                }
            l[r] = l[r] * alpha + sum;
            if (__ballot(alpha != 1.0f)) {
#pragma unroll
                for (int n = 0; n < D / 16; ++n) o[r][n] *= alpha;
            }
            // The weights are rounded to bf16 (at most 2^-8 of each, to either
            // side); their sum l is kept as it was.
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                pt[r][kk] = u32x4_t{narrow2a(sc[r][2 * kk][0], sc[r][2 * kk][1]),
                                    narrow2a(sc[r][2 * kk][2], sc[r][2 * kk][3]),
                                    narrow2a(sc[r][2 * kk + 1][0], sc[r][2 * kk + 1][1]),
                                    narrow2a(sc[r][2 * kk + 1][2], sc[r][2 * kk + 1][3])};
        }
        if (odd) take_out_nan(st, j0);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t w = st.v[kk][n];
                const float s1 = scale_of(st.vs[kk]);
                const u32x4_t a0 = widen8(w.x, w.y, s1), a1 = widen8(w.z, w.w, s1);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    o[r][2 * n] = mfma16(a0, pt[r][kk], o[r][2 * n]);
                    o[r][2 * n + 1] = mfma16(a1, pt[r][kk], o[r][2 * n + 1]);
                }
                if (n & 1) __builtin_amdgcn_sched_barrier(0);      // bounds the registers of codes made wide
            }
        if (more) load_v(st, g, next);
    }

    // Where a partly visible chunk holds NaN values: they are taken out of the
    // product, and a row that sees one gets NaN in that channel, by a product
    // of what is visible with what is NaN (a sum of ones, above 0 if any).
    __device__ __forceinline__ void take_out_nan(Stage<D> &st, int j0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const uint32_t bits = sees8(a, p[r], j0 + 32 * kk + 8 * q4);
                const u32x4_t seen = widen8(spread4(bits) & kOnes, spread4(bits >> 4) & kOnes, 1.0f);
#pragma unroll
                for (int n = 0; n < D / 32; ++n) {
                    const u32x4_t w = nan_bytes(st.v[kk][n]) & kOnes;
                    const f32x4a_t zero{0, 0, 0, 0};
                    const f32x4a_t t0 = mfma16(widen8(w.x, w.y, 1.0f), seen, zero);
                    const f32x4a_t t1 = mfma16(widen8(w.z, w.w, 1.0f), seen, zero);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (t0[i] > 0.0f) o[r][2 * n][i] = __builtin_nanf("");
                        if (t1[i] > 0.0f) o[r][2 * n + 1][i] = __builtin_nanf("");
                    }
                    if (r == R - 1) st.v[kk][n] &= ~nan_bytes(st.v[kk][n]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
    }

    // The wave's share of units [u0, u1).
    __device__ __forceinline__ void run(int u0, int u1) {
        const int c1 = min(u1 * kWaves, s.c.nc);
        int c = u0 * kWaves + wave;
        if (c >= c1) return;
        Stage<D> st;
        Pages g;
        look_up(g, c);
        load_k(st, g, c);
        load_v(st, g, c);
        if (c + kWaves < c1) look_up(g, c + kWaves);
        while (true) {
            const int next = c + kWaves;
            const bool more = next < c1;
            step(st, g, c, next, more);
            if (!more) return;
            if (next + kWaves < c1) look_up(g, next + kWaves);
            c = next;
        }
    }

    // Joins the four waves' rows and writes them: as they are to be (whole
    // item) or as a partial (o, m, l) with o relative to the maximum m.
    __device__ __forceinline__ void finish(float (*lo)[16][D + 4], float (*lm)[16][2], float *part_o, float *part_ml) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r > 0) __syncthreads();      // the tile before has been read
            float sum = l[r] + __shfl_xor(l[r], 16, 64);
            sum += __shfl_xor(sum, 32, 64);
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                // lane: channels 32 n + 8 q4 + 2 i + parity of row lane & 15
                float *dst = &lo[wave][lane & 15][32 * n + 8 * q4];
                *reinterpret_cast<f32x4a_t *>(dst) =
                    f32x4a_t{o[r][2 * n][0], o[r][2 * n + 1][0], o[r][2 * n][1], o[r][2 * n + 1][1]};
                *reinterpret_cast<f32x4a_t *>(dst + 4) =
                    f32x4a_t{o[r][2 * n][2], o[r][2 * n + 1][2], o[r][2 * n][3], o[r][2 * n + 1][3]};
            }
            if (lane < 16) {
                lm[wave][lane][0] = m[r];
                lm[wave][lane][1] = sum;
            }
            __syncthreads();
            const int row = threadIdx.x >> 4, ch = (threadIdx.x & 15) * (D / 16);
            const int at = tile * 16 * R + 16 * r + row;
            if (at < rows) {
                float top = -__builtin_inff();
#pragma unroll
                for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lm[w][row][0]);
                const float base = top == -__builtin_inff() ? 0.0f : top;
                float all = 0.0f, acc[D / 16];
#pragma unroll
                for (int j = 0; j < D / 16; ++j) acc[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float f = exp2a(lm[w][row][0] - base);
                    all += f * lm[w][row][1];
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) acc[j] += f * lo[w][row][ch + j];
                }
                if (part_o) {
                    float *dst = part_o + (16 * r + row) * D + ch;
#pragma unroll
                    for (int j = 0; j < D / 16; j += 4)
                        *reinterpret_cast<f32x4a_t *>(dst + j) = f32x4a_t{acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
                    if (ch == 0) {
                        part_ml[2 * (16 * r + row)] = top;
                        part_ml[2 * (16 * r + row) + 1] = all;
                    }
                } else {
                    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
                    const int i = at / G, g = at - i * G;
                    const int64_t t = s.first + i;
                    uint16_t *dst = a.o + t * a.o_stride + (int64_t)(h * G + g) * D + ch;
#pragma unroll
                    for (int j = 0; j < D / 16; j += 4)
                        *reinterpret_cast<uint2 *>(dst + j) = make_uint2(narrow2a(acc[j] * inv, acc[j + 1] * inv),
                                                                         narrow2a(acc[j + 2] * inv, acc[j + 3] * inv));
                    if (a.lse && ch == 0)
                        a.lse[t * a.q_heads + h * G + g] = (top + __builtin_amdgcn_logf(all)) * kLn2;
                }
            }
        }
    }
};

// Where a workgroup's partials lie: slot 0 holds a piece that continues an
// item, slot 1 one that begins an item without ending it.
template <int D, int R>
__device__ __forceinline__ float *part_of(const AttnArgs &a, int wg, int slot) {
    return static_cast<float *>(a.ws) + (int64_t)(2 * wg + slot) * (16 * R) * (D + 2);
}

// Work is a flat list of units: sequence, key/value head, row tile, unit.
__device__ __forceinline__ int64_t seq_units(const AttnArgs &a, const Seq &s) {
    return (int64_t)s.units * s.tiles * a.kv_heads;
}

// direct: a workgroup an item (sequence, head, row tile).  Otherwise the flat
// list of units is cut into equal shares, one a workgroup.
template <int D, int R>
__global__ void __launch_bounds__(256, D * R <= 128 ? 2 : 1)
attn_rows_kernel(const AttnArgs a, int which, int direct, int max_tiles) {
    __shared__ float lo[kWaves][16][D + 4];
    __shared__ float lm[kWaves][16][2];
    int64_t u = 0, end = 1, before = 0;
    int b, item;
    Seq s;
    if (direct) {
        const int tile = (int)(blockIdx.x % max_tiles), h = (int)(blockIdx.x / max_tiles % a.kv_heads);
        b = (int)(blockIdx.x / max_tiles / a.kv_heads);
        s = seq_uniform(a, b, 16 * R, which);
        if (tile >= s.tiles) return;
        item = h * s.tiles + tile;
        u = (int64_t)item * s.units;
        end = u + s.units;
    } else {
        const auto units = [&](int i) { return seq_units(a, seq_of(a, i, 16 * R, which)); };
        int64_t total = 0;
        for (int i = threadIdx.x & 63; i < a.B; i += 64) total += units(i);
        total = uniform(wave_sum64(total));
        const int64_t share = (total + gridDim.x - 1) / gridDim.x;
        u = (int64_t)blockIdx.x * share;
        end = min(u + share, total);
        if (u >= end) return;
        b = uniform(find_seq(a.B, u, before, units));
        before = uniform(before);
        s = seq_uniform(a, b, 16 * R, which);
    }
    while (true) {
        item = (int)((u - before) / s.units);
        const int u0 = (int)(u - before - (int64_t)item * s.units);
        const int u1 = (int)min((int64_t)s.units, u0 + (end - u));
        Piece<D, R> pc(a, s, b, item / s.tiles, item % s.tiles);
        pc.run(u0, u1);
        float *part = u0 == 0 && u1 == s.units ? nullptr : part_of<D, R>(a, blockIdx.x, u0 == 0);
        pc.finish(lo, lm, part, part ? part + 16 * R * D : nullptr);
        u += u1 - u0;
        if (u >= end) return;
        __syncthreads();      // lo and lm are free again
        while (u >= before + seq_units(a, s)) {      // ends: u < total
            before += seq_units(a, s);
            s = seq_uniform(a, ++b, 16 * R, which);
        }
    }
}

// Joins the pieces of one row of an item that several workgroups shared.
template <int D, int R>
__global__ void __launch_bounds__(256)
attn_join_kernel(const AttnArgs a, int which, int shares, int max_tiles) {
    __shared__ float lo[kWaves][D];
    __shared__ float ll[kWaves][2];
    const int row = (int)(blockIdx.x % (16 * R)), item = (int)(blockIdx.x / (16 * R));
    const int tile = item % max_tiles, h = item / max_tiles % a.kv_heads, b = item / max_tiles / a.kv_heads;
    const Seq s = seq_of(a, b, 16 * R, which);
    const int G = a.q_heads / a.kv_heads;
    if (tile >= s.tiles || (int64_t)tile * 16 * R + row >= (int64_t)s.n * G) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t before = 0, total = 0;
    for (int i = lane; i < a.B; i += 64) {
        const int64_t n = seq_units(a, seq_of(a, i, 16 * R, which));
        total += n;
        before += i < b ? n : 0;
    }
    total = wave_sum64(total);
    before = wave_sum64(before);
    const int64_t share = (total + shares - 1) / shares;
    const int64_t u0 = before + (int64_t)(h * s.tiles + tile) * s.units, u1 = u0 + s.units;
    const int w0 = (int)(u0 / share), w1 = (int)((u1 - 1) / share);
    if (w0 == w1) return;      // the item was one workgroup's
    float m = -__builtin_inff(), l = 0.0f, acc[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = 0.0f;
    for (int w = w0 + wave; w <= w1; w += kWaves) {
        const float *part = part_of<D, R>(a, w, w == w0 && u0 >= (int64_t)w * share);
        const float pm = part[16 * R * D + 2 * row], pl = part[16 * R * D + 2 * row + 1];
        const float top = fmaxf(m, pm), base = top == -__builtin_inff() ? 0.0f : top;
        const float f0 = exp2a(m - base), f1 = exp2a(pm - base);
        m = top;
        l = l * f0 + pl * f1;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = acc[j] * f0 + part[row * D + (D / 64) * lane + j] * f1;
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) lo[wave][(D / 64) * lane + j] = acc[j];
    if (lane == 0) {
        ll[wave][0] = m;
        ll[wave][1] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D) return;
    float top = -__builtin_inff(), all = 0.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ll[w][0]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = exp2a(ll[w][0] - base);
        all += f * ll[w][1];
        sum += f * lo[w][threadIdx.x];
    }
    const int at = tile * 16 * R + row, i = at / G, g = at - i * G;
    const int64_t t = s.first + i;
    a.o[t * a.o_stride + (int64_t)(h * G + g) * D + threadIdx.x] =
        f32_to_bf16_rne(all == 0.0f ? 0.0f : sum * (1.0f / all));
    if (a.lse && threadIdx.x == 0) a.lse[t * a.q_heads + h * G + g] = (top + __builtin_amdgcn_logf(all)) * kLn2;
}

struct Plan {
    int R, max_tiles, direct, grid;
    int64_t items;
    bool rows, tiles;      // which kernels the call needs
    size_t rows_bytes, tiles_bytes;
};

// What the host can know: at most this many rows, tiles and units.  A batch
// of more tokens than its longest sequence has may hold sequences of few and
// of many rows: both kernels are then launched, each taking its own.
Plan plan_of(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv) {
    Plan p;
    const int G = q_heads / kv_heads;
    const int64_t most = (int64_t)(max_q < T ? max_q : T) * G;
    p.tiles = most > kMostRows;
    p.rows = !p.tiles || B > 1;
    const int64_t rows = p.tiles ? (most < kMostRows ? most : kMostRows) : most;
    p.R = rows <= 16 ? 1 : 2;
    p.max_tiles = (int)((rows + 16 * p.R - 1) / (16 * p.R));
    p.items = (int64_t)B * kv_heads * p.max_tiles;
    const int units = (max_kv + kChunk * kWaves - 1) / (kChunk * kWaves);
    p.direct = units <= 3;
    p.grid = p.direct ? 0 : kSplitGrid;
    p.rows_bytes = p.rows ? (size_t)p.grid * 2 * (16 * p.R) * (dim + 2) * sizeof(float) : 0;
    p.tiles_bytes = p.tiles ? attn_tiles_plan(B, T, q_heads, kv_heads, dim, max_kv).ws_bytes : 0;
    return p;
}

template <int D, int R>
hipError_t launch(const AttnArgs &a, const Plan &p, hipStream_t stream) {
    if (p.items * 16 * R > 0x7FFFFFFF) return hipErrorInvalidValue;
    const int which = p.tiles ? kFewRows : kAllSeqs;
    hipLaunchKernelGGL((attn_rows_kernel<D, R>), dim3((unsigned)(p.direct ? p.items : p.grid)), dim3(256), 0, stream,
                       a, which, p.direct, p.max_tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.direct) return e;
    hipLaunchKernelGGL((attn_join_kernel<D, R>), dim3((unsigned)(p.items * 16 * R)), dim3(256), 0, stream, a, which,
                       p.grid, p.max_tiles);
    return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const AttnArgs &a, const Plan &p, hipStream_t stream) {
    return p.R == 1 ? launch<D, 1>(a, p, stream) : launch<D, 2>(a, p, stream);
}

}  // namespace

size_t attn_ws_bytes(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv) {
    if (B == 0 || T == 0) return 0;
    const Plan p = plan_of(B, T, q_heads, kv_heads, dim, max_q, max_kv);
    return p.rows_bytes + p.tiles_bytes;
}

hipError_t launch_attn(const AttnArgs &a, hipStream_t stream) {
    const Plan p = plan_of(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_q, a.max_kv);
    if (p.tiles) {      // first: the longest workgroups
        AttnArgs t = a;
        t.ws = static_cast<char *>(a.ws) + p.rows_bytes;
        const hipError_t e = launch_attn_tiles(t, p.rows ? kManyRows : kAllSeqs, stream);
        if (e != hipSuccess || !p.rows) return e;
    }
    return a.dim == 64 ? launch_dim<64>(a, p, stream) : launch_dim<128>(a, p, stream);
}

}  // namespace biloco
