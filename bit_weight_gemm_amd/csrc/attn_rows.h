// The parts of attention over few query rows per key/value head (k_attn.hip says how a
// wave works): loads, rows and their sums, joins in LDS, the split call's workspace.
#pragma once
#include "attn_device.h"

namespace biloco {
namespace attn {

constexpr int kSplitLog = 2, kSplitWaves = 1 << kSplitLog, kPieces = 512, kSizes = 4;      // two workgroups a CU
constexpr int kWholeWaves = 8;

template <int D>
struct Stage {
    u32x4_t k[2][2][D / 64];      // [kk][f][c]
    u32x4_t v[2][D / 32];         // [kk][nb]
    float ks[2];
    uint32_t vs[2];
};
// Pages of a chunk's tokens, asked for one chunk ahead of their use.
struct Pages {
    int k[2], v[2];
};

// Where a wave reads: block table row, head, page arithmetic.
struct Where {
    const int *table;
    int h, shift, lane, q4;
    __device__ __forceinline__ Where(const AttnArgs &a, int b, int h_)
        : table(a.table + (int64_t)b * a.max_pages), h(h_), shift(31 - __clz(a.page)), lane(threadIdx.x & 63),
          q4((threadIdx.x & 63) >> 4) {}

    // Pages of the chunk at j0; `last` is the last column to look at (tokens
    // past the last one read some page of the sequence, or page 0).
    __device__ __forceinline__ void look_up(Pages &g, int j0, int last) const {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            g.k[kk] = table[min((j0 + 32 * kk + 8 * ((lane & 15) >> 2)) >> shift, last)];
            g.v[kk] = table[min((j0 + 32 * kk + 8 * q4) >> shift, last)];
        }
    }
    __device__ __forceinline__ int64_t block_of(const AttnArgs &a, int id) const {
        return (int64_t)((uint32_t)id < (uint32_t)a.num_pages ? id : 0) * a.kv_heads + h;
    }
    template <int D>
    __device__ __forceinline__ void load_k(const AttnArgs &a, Stage<D> &st, const Pages &g, int j0) const {
        const int mrow = lane & 15, j = (j0 + 8 * (mrow >> 2)) & (a.page - 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int64_t bk = block_of(a, g.k[kk]);
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
    template <int D>
    __device__ __forceinline__ void load_v(const AttnArgs &a, Stage<D> &st, const Pages &g, int j0) const {
        const int j = (j0 + 8 * q4) & (a.page - 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int64_t bv = block_of(a, g.v[kk]);
            const int slot = (j + 32 * kk) & (a.page - 1);
            const uint8_t *v = a.vc + (((bv << shift) + slot) * D + 16 * (lane & 15));
            st.vs[kk] = a.vs[bv];
#pragma unroll
            for (int n = 0; n < D / 32; ++n) st.v[kk][n] = *reinterpret_cast<const u32x4_t *>(v + 256 * n);
        }
    }
};

// Sixteen rows of one item and what they have gathered: row r of the lanes
// l & 15 == r.
template <int D>
struct Rows16 {
    u32x4_t q[D / 64][2];
    f32x4a_t o[D / 16];
    float m, l;      // m: of scale * log2(e) * s
    int p, p_min, p_max;

    __device__ __forceinline__ Rows16(const AttnArgs &a, const Seq &s, int h, int r0, int rows) {
        const int lane = threadIdx.x & 63, G = a.q_heads / a.kv_heads;
        const int row = min(r0 + (lane & 15), rows - 1), i = row / G;
        p = s.past + i;
        p_min = s.past + min(r0, rows - 1) / G;
        p_max = s.past + min(r0 + 15, rows - 1) / G;
        const uint16_t *src = a.q + (int64_t)(s.first + i) * a.q_stride + (int64_t)(h * G + row - i * G) * D + 16 * (lane >> 4);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) q[c][t] = *reinterpret_cast<const u32x4_t *>(src + 64 * c + 8 * t);
        m = -__builtin_inff();
        l = 0.0f;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) o[n] = f32x4a_t{0, 0, 0, 0};
    }

    // The scores of the chunk whose keys are in st.
    __device__ __forceinline__ void scores(const Stage<D> &st, f32x4a_t (&sc)[4]) const {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            sc[t] = f32x4a_t{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const u32x4_t w = st.k[t >> 1][t & 1][c];
                sc[t] = mfma16(widen8(w.x, w.y, st.ks[t >> 1]), q[c][0], sc[t]);
                sc[t] = mfma16(widen8(w.z, w.w, st.ks[t >> 1]), q[c][1], sc[t]);
            }
            if (t & 1) __builtin_amdgcn_sched_barrier(0);      // bounds the registers of codes made wide
        }
    }

    // Scores to weights, relative to the running maximum.
    template <class A>
    __device__ __forceinline__ void weigh(const A &a, f32x4a_t (&sc)[4], bool whole, int j0, u32x4_t (&pt)[2][2]) {
        const int q4 = (threadIdx.x & 63) >> 4;
        const float c2 = a.scale * kLog2e;
        if (__builtin_expect(!whole, 0)) {
            const int lo = low_of(a, p);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[t][i] = sees(a, p, lo, j0 + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1) + i) ? sc[t][i] : -__builtin_inff();
        }
        float mx = sc[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i >> 2][i & 3]);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64)) * c2;
        const float mn = fmaxf(m, mx);
        const float base = mn == -__builtin_inff() ? 0.0f : mn;      // a row that sees nothing yet
        const float alpha = exp2a(m - base);
        m = mn;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[t][i] = exp2a(__builtin_fmaf(sc[t][i], c2, -base));
                sum += sc[t][i];
            }
        l = l * alpha + sum;
        if (__ballot(alpha != 1.0f)) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[n] *= alpha;
        }
        // Each weight as the sum of two bf16, its rounding and what that left
        // (together within 2^-16 of it): the matrix cores have time for a second
        // product here, and o then carries its own rounding only.
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const uint32_t w = narrow2a(sc[t][i], sc[t][i + 1]);
                pt[t >> 1][0][2 * (t & 1) + i / 2] = w;
                pt[t >> 1][1][2 * (t & 1) + i / 2] = narrow2a(sc[t][i] - __uint_as_float(w << 16),
                                                              sc[t][i + 1] - __uint_as_float(w & 0xFFFF0000u));
            }
    }

    // Where not every row sees the whole chunk: tokens that no row sees can
    // hold anything, so their codes become zero and their scale 1.  NaN values are
    // taken out of the product too, and a row that sees one gets NaN in its
    // channel, by a product of what is visible with what is NaN (above 0 if any).
    template <class A>
    __device__ __forceinline__ void clean(const A &a, Stage<D> &st, int j0) {
        const int q4 = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const uint32_t bits = any_sees8(a, p_min, p_max, j0 + 32 * kk + 8 * q4);
            const uint32_t m0 = spread4(bits), m1 = spread4(bits >> 4);
            if (bits == 0) st.vs[kk] = 127;
#pragma unroll
            for (int n = 0; n < D / 32; ++n) st.v[kk][n] &= u32x4_t{m0, m1, m0, m1};
        }
        if (p_min == p_max) return;      // rows of one token see the same
        uint32_t any = 0;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t t = nan_bytes(st.v[kk][n]);
                any |= t.x | t.y | t.z | t.w;
            }
        if (__builtin_expect(__ballot(any != 0) == 0, 1)) return;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const uint32_t bits = sees8(a, p, j0 + 32 * kk + 8 * q4);
            const u32x4_t seen = widen8(spread4(bits) & kOnes, spread4(bits >> 4) & kOnes, 1.0f);
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t bad = nan_bytes(st.v[kk][n]), w = bad & kOnes;
                const f32x4a_t zero{0, 0, 0, 0};
                const f32x4a_t t0 = mfma16(widen8(w.x, w.y, 1.0f), seen, zero);
                const f32x4a_t t1 = mfma16(widen8(w.z, w.w, 1.0f), seen, zero);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[2 * n][i] = t0[i] > 0.0f ? __builtin_nanf("") : o[2 * n][i];
                    o[2 * n + 1][i] = t1[i] > 0.0f ? __builtin_nanf("") : o[2 * n + 1][i];
                }
                st.v[kk][n] &= ~bad;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    __device__ __forceinline__ void gather(const Stage<D> &st, const u32x4_t (&pt)[2][2]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const u32x4_t w = st.v[kk][n];
                const float s = scale_of(st.vs[kk]);
                const u32x4_t a0 = widen8(w.x, w.y, s), a1 = widen8(w.z, w.w, s);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[2 * n] = mfma16(a0, pt[kk][e], o[2 * n]);
                    o[2 * n + 1] = mfma16(a1, pt[kk][e], o[2 * n + 1]);
                }
                if (n & 1) __builtin_amdgcn_sched_barrier(0);
            }
    }

    // Chunks c, c + step, ... below c1; the next one's keys are asked for as
    // soon as this one's are used up, its values likewise.  With `loaded`, st
    // holds chunk c already.
    template <class A>
    __device__ __forceinline__ void run(const A &a, const Where &w, const Seq &s, Stage<D> &st, bool loaded, int c,
                                        int c1, int step) {
        if (c >= c1) return;
        const int last = (s.hi - 1) >> w.shift;
        Pages g;
        if (!loaded) {
            w.look_up(g, s.c.start(c), last);
            w.load_k(a, st, g, s.c.start(c));
            w.load_v(a, st, g, s.c.start(c));
        }
        if (c + step < c1) w.look_up(g, s.c.start(c + step), last);
        while (true) {
            const int j0 = s.c.start(c), next = c + step;
            const bool more = next < c1, whole = all_see(a, p_min, p_max, j0);
            f32x4a_t sc[4];
            u32x4_t pt[2][2];
            scores(st, sc);
            if (more) w.load_k(a, st, g, s.c.start(next));
            weigh(a, sc, whole, j0, pt);
            if (__builtin_expect(!whole, 0)) clean(a, st, j0);
            gather(st, pt);
            if (!more) return;
            w.load_v(a, st, g, s.c.start(next));
            if (next + step < c1) w.look_up(g, s.c.start(next + step), last);
            c = next;
        }
    }
};

template <int D, int WAVES>
struct JoinLds {
    float o[WAVES][16][D + 4];
    float ml[WAVES][16][2];
};

// Joins the waves' sums row by row and writes them: as they are to be (whole
// item) or as a partial (o relative to the maximum m, then m and l).
template <int D, int WAVES>
__device__ __forceinline__ void finish(const AttnArgs &a, const Seq &s, const Rows16<D> &x, JoinLds<D, WAVES> &lds, int h,
                                       int rows, int row_groups, float *part, int part_rows) {
    constexpr int CH = D / (4 * WAVES);      // channels a thread joins
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q4 = lane >> 4, G = a.q_heads / a.kv_heads;
    float sum = x.l + __shfl_xor(x.l, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {
        // lane: channels 32 n + 8 q4 + 2 i + parity of row lane & 15
        float *dst = &lds.o[wave][lane & 15][32 * n + 8 * q4];
        const f32x4a_t u = x.o[2 * n], v = x.o[2 * n + 1];
        *reinterpret_cast<f32x4a_t *>(dst) = f32x4a_t{u[0], v[0], u[1], v[1]};
        *reinterpret_cast<f32x4a_t *>(dst + 4) = f32x4a_t{u[2], v[2], u[3], v[3]};
    }
    if (lane < 16) {
        lds.ml[wave][lane][0] = x.m;
        lds.ml[wave][lane][1] = sum;
    }
    __syncthreads();
    const int row = threadIdx.x / (4 * WAVES), ch = (threadIdx.x % (4 * WAVES)) * CH;
    for (int t = 0; t < row_groups; ++t) {
        const int at = 16 * t + row;
        if (at >= rows) return;
        float top = -__builtin_inff();
        for (int w = t; w < WAVES; w += row_groups) top = fmaxf(top, lds.ml[w][row][0]);
        const float base = top == -__builtin_inff() ? 0.0f : top;
        float all = 0.0f, acc[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) acc[j] = 0.0f;
        for (int w = t; w < WAVES; w += row_groups) {
            const float f = exp2a(lds.ml[w][row][0] - base);
            all += f * lds.ml[w][row][1];
#pragma unroll
            for (int j = 0; j < CH; ++j) acc[j] += f * lds.o[w][row][ch + j];
        }
        if (part) {
#pragma unroll
            for (int j = 0; j < CH; ++j) part[at * D + ch + j] = acc[j];
            if (ch == 0) {
                part[part_rows * D + 2 * at] = top;
                part[part_rows * D + 2 * at + 1] = all;
            }
        } else {
            const float inv = all == 0.0f ? 0.0f : 1.0f / all;
            const int i = at / G, g = at - i * G;
            const int64_t tok = s.first + i;
            uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + tok * a.o_stride + (int64_t)(h * G + g) * D + ch);
#pragma unroll
            for (int j = 0; j < CH; j += 2) dst[j / 2] = narrow2a(acc[j] * inv, acc[j + 1] * inv);
            if (a.lse && ch == 0) a.lse[tok * a.q_heads + h * G + g] = (top + __builtin_amdgcn_logf(all)) * kLn2;
        }
    }
}

// Rows of a sequence, and 1 << row_shift groups of waves that take 16 of them
// each: by the sequence's own rows, not the batch's most, so that waves which
// would have no rows take chunks instead.
__device__ __forceinline__ int rows_of(const AttnArgs &a, const Seq &s, int most_rows) {
    return min(s.n * (a.q_heads / a.kv_heads), most_rows);
}
__host__ __device__ __forceinline__ int row_shift_of(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : 2; }

// What the workgroup of an item's first piece leaves for the join: itself,
// and how many pieces the item has (1: it is done).
struct Begun {
    int wg, pieces;
};

// The split call's workspace: a Begun per item, then a partial a workgroup.
__host__ __device__ __forceinline__ int64_t part_floats(int dim, int rows) { return (int64_t)rows * (dim + 2); }
__host__ __device__ __forceinline__ int64_t begun_slots(int64_t items) { return (items + 1) / 2 * 2; }      // 16 bytes
__device__ __forceinline__ float *part_of(const AttnArgs &a, int dim, int rows, int wg) {
    return reinterpret_cast<float *>(static_cast<Begun *>(a.ws) + begun_slots((int64_t)a.B * a.kv_heads)) +
           wg * part_floats(dim, rows);
}

// A workgroup a piece of an item: equal pieces of as many units (chunks that
// its waves take side by side) as spread all items over kPieces workgroups, or a
// few more.  At most kPieces + items pieces, the grid's size; the workgroups that
// are left over end at once.  K::of(b): the call's arguments for sequence b.  An item
// that is one piece is written as it is to be, unless it is part of a longer one.
template <int D, class K>
__device__ __forceinline__ void split_rows(const K &k, int which, int most_rows, int wg, JoinLds<D, kSplitWaves> &lds) {
    const AttnArgs &a = k.a;
    const int wave = uniform((int)(threadIdx.x >> 6));
    const auto shift_of = [&](const Seq &s) { return row_shift_of(rows_of(a, s, most_rows)); };
    // a sequence with rows has at least one unit, to write its rows in
    const auto units = [&](const Seq &s) {
        const int by = kSplitLog - shift_of(s);      // chunks side by side, as a power of two
        return s.n > 0 ? max((s.c.nc + (1 << by) - 1) >> by, 1) : 0;
    };
    int64_t total = 0, before;
    for (int i = threadIdx.x & 63; i < a.B; i += 64) total += (int64_t)units(seq_of(k.of(i), i, which)) * a.kv_heads;
    const int64_t each = max((uniform(wave_sum64(total)) + kPieces - 1) / kPieces, (int64_t)1);
    const int even = (int)min(each, (int64_t)1 << 24);      // no item has more units
    // Each item's last piece can be short, and a workgroup above kPieces waits for
    // another to end.  So sizes up to twice the even share: the smallest with no
    // more pieces than that (944 units: 528 pieces of two or 384 of three, 27.9 and
    // 24.3 us with the join).
    float count[kSizes] = {};      // compared with kPieces only, so exact where it matters
    for (int i = threadIdx.x & 63; i < a.B; i += 64) {
        const uint32_t u = (uint32_t)units(seq_of(k.of(i), i, which));
#pragma unroll
        for (int z = 0; z < kSizes; ++z) count[z] += (float)((u + even + z - 1) / (uint32_t)(even + z));
    }
    int more = 0;
#pragma unroll
    for (int z = kSizes - 1; z >= 0; --z)
        if (wave_sum_dpp(count[z]) * (float)a.kv_heads <= (float)kPieces) more = z;
    const int size = even + (uniform(more) <= even ? uniform(more) : 0);
    const auto pieces = [&](const Seq &s) { return (int)(((uint32_t)units(s) + size - 1) / (uint32_t)size); };
    const int b = uniform(find_seq(a.B, wg, before,
                                   [&](int i) { return (int64_t)pieces(seq_of(k.of(i), i, which)) * a.kv_heads; }));
    if (b < 0) return;
    const auto &part = k.of(b);
    const Seq s = seq_uniform(part, b, which);
    const int n = uniform(pieces(s)), at = (int)(wg - uniform(before));
    const int h = uniform(at / n), u0 = uniform((at - h * n) * size);
    const int rows = rows_of(a, s, most_rows), row_shift = shift_of(s), lanes = kSplitWaves >> row_shift;
    const int mine = 16 * (wave & ((1 << row_shift) - 1));
    const Where w(a, b, h);
    Rows16<D> x(a, s, h, mine, rows);
    Stage<D> st;
    if (mine < rows)
        x.run(part, w, s, st, false, u0 * lanes + (wave >> row_shift), min((u0 + size) * lanes, s.c.nc), lanes);
    if (u0 == 0 && threadIdx.x == 0) static_cast<Begun *>(a.ws)[b * a.kv_heads + h] = Begun{wg, n};
    finish<D, kSplitWaves>(a, s, x, lds, h, rows, 1 << row_shift,
                           n == 1 && !K::kPart ? nullptr : part_of(a, D, most_rows, wg), most_rows);
}

template <int D, class K>
__global__ void __launch_bounds__(64 * kSplitWaves, 2)
attn_split_kernel(const K k, int which, int most_rows) {
    __shared__ JoinLds<D, kSplitWaves> lds;
    split_rows<D>(k, which, most_rows, (int)blockIdx.x, lds);
}

}  // namespace attn
}  // namespace biloco
