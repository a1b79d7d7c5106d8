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
// A wave takes 16 rows and 64 tokens at a time and needs no shared memory for it:
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
//
// The waves of a workgroup take different chunks of one item (sequence,
// key/value head) and join their sums in LDS at its end; where there
// are more than 16 rows, groups of them take different rows of the same chunks
// (the second read of a chunk is a cache hit).  A workgroup takes a whole item,
// or, where that would leave the chip idle, a piece of one; pieces are joined by
// a second launch.
//
// Bound by the cache's bytes where contexts are long, by the chain lookup -> load
// -> two products -> join where they are short.  Measured on MI355X (a kernel that
// only reads reaches 7.2 TB/s): one sequence of 131071 tokens, 64/8 heads, 55.7 us,
// 4.82 TB/s with the join (5.3 before it); 32 sequences of 1 to 8192 tokens, 40/40
// heads, 93 us, 4.03 TB/s (the longest items end last); one of 613 tokens, 8.5 us.
#include "attn_device.h"

namespace biloco {

namespace {

using namespace attn;

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
    __device__ __forceinline__ void weigh(const AttnArgs &a, f32x4a_t (&sc)[4], bool whole, int j0, u32x4_t (&pt)[2][2]) {
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
    __device__ __forceinline__ void clean(const AttnArgs &a, Stage<D> &st, int j0) {
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
    __device__ __forceinline__ void run(const AttnArgs &a, const Where &w, const Seq &s, Stage<D> &st, bool loaded, int c,
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

// A workgroup an item.  The first chunk's pages, keys and values are asked
// for before the sequence's length is known where it is chunk 0 on (no window),
// in the order of the batch's most rows.
template <int D>
__global__ void __launch_bounds__(64 * kWholeWaves, 2)
attn_whole_kernel(const AttnArgs a, int which, int most_rows) {
    __shared__ JoinLds<D, kWholeWaves> lds;
    const int h = (int)(blockIdx.x % a.kv_heads), b = (int)(blockIdx.x / a.kv_heads);
    const int wave = uniform((int)(threadIdx.x >> 6));
    const int most_shift = row_shift_of(most_rows), c = wave >> most_shift;
    const Where w(a, b, h);
    Stage<D> st;
    const bool early = a.window == 0;
    if (early) {
        Pages g;
        w.look_up(g, c * kChunk, a.max_pages - 1);
        w.load_k(a, st, g, c * kChunk);
        w.load_v(a, st, g, c * kChunk);
    }
    const Seq s = seq_uniform(a, b, which);
    if (s.n == 0) return;
    const int rows = rows_of(a, s, most_rows), row_shift = row_shift_of(rows);
    const int mine = 16 * (wave & ((1 << row_shift) - 1));
    Rows16<D> x(a, s, h, mine, rows);
    if (mine < rows)
        x.run(a, w, s, st, early && row_shift == most_shift, wave >> row_shift, s.c.nc, kWholeWaves >> row_shift);
    finish<D, kWholeWaves>(a, s, x, lds, h, rows, 1 << row_shift, nullptr, 0);
}

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
// are left over end at once.
template <int D>
__global__ void __launch_bounds__(64 * kSplitWaves, 2)
attn_split_kernel(const AttnArgs a, int which, int most_rows) {
    __shared__ JoinLds<D, kSplitWaves> lds;
    const int wave = uniform((int)(threadIdx.x >> 6));
    const auto shift_of = [&](const Seq &s) { return row_shift_of(rows_of(a, s, most_rows)); };
    // a sequence with rows has at least one unit, to write its rows in
    const auto units = [&](const Seq &s) {
        const int by = kSplitLog - shift_of(s);      // chunks side by side, as a power of two
        return s.n > 0 ? max((s.c.nc + (1 << by) - 1) >> by, 1) : 0;
    };
    int64_t total = 0, before;
    for (int i = threadIdx.x & 63; i < a.B; i += 64) total += (int64_t)units(seq_of(a, i, which)) * a.kv_heads;
    const int64_t each = max((uniform(wave_sum64(total)) + kPieces - 1) / kPieces, (int64_t)1);
    const int even = (int)min(each, (int64_t)1 << 24);      // no item has more units
    // Each item's last piece can be short, and a workgroup above kPieces waits for
    // another to end.  So sizes up to twice the even share: the smallest with no
    // more pieces than that (944 units: 528 pieces of two or 384 of three, 27.9 and
    // 24.3 us with the join).
    float count[kSizes] = {};      // compared with kPieces only, so exact where it matters
    for (int i = threadIdx.x & 63; i < a.B; i += 64) {
        const uint32_t u = (uint32_t)units(seq_of(a, i, which));
#pragma unroll
        for (int k = 0; k < kSizes; ++k) count[k] += (float)((u + even + k - 1) / (uint32_t)(even + k));
    }
    int more = 0;
#pragma unroll
    for (int k = kSizes - 1; k >= 0; --k)
        if (wave_sum_dpp(count[k]) * (float)a.kv_heads <= (float)kPieces) more = k;
    const int size = even + (uniform(more) <= even ? uniform(more) : 0);
    const auto pieces = [&](const Seq &s) { return (int)(((uint32_t)units(s) + size - 1) / (uint32_t)size); };
    const int b = uniform(find_seq(a.B, blockIdx.x, before,
                                   [&](int i) { return (int64_t)pieces(seq_of(a, i, which)) * a.kv_heads; }));
    if (b < 0) return;
    const Seq s = seq_uniform(a, b, which);
    const int n = uniform(pieces(s)), at = (int)(blockIdx.x - uniform(before));
    const int h = uniform(at / n), u0 = uniform((at - h * n) * size);
    const int rows = rows_of(a, s, most_rows), row_shift = shift_of(s), lanes = kSplitWaves >> row_shift;
    const int mine = 16 * (wave & ((1 << row_shift) - 1));
    const Where w(a, b, h);
    Rows16<D> x(a, s, h, mine, rows);
    Stage<D> st;
    if (mine < rows)
        x.run(a, w, s, st, false, u0 * lanes + (wave >> row_shift), min((u0 + size) * lanes, s.c.nc), lanes);
    if (u0 == 0 && threadIdx.x == 0) static_cast<Begun *>(a.ws)[b * a.kv_heads + h] = Begun{(int)blockIdx.x, n};
    finish<D, kSplitWaves>(a, s, x, lds, h, rows, 1 << row_shift,
                           n == 1 ? nullptr : part_of(a, D, most_rows, blockIdx.x), most_rows);
}

// Joins the pieces of the rows of items that several workgroups shared: WAYS
// waves a row, each taking every WAYS-th piece; 4 / WAYS rows of one item a
// workgroup.
template <int D, int WAYS>
__global__ void __launch_bounds__(256)
attn_join_kernel(const AttnArgs a, int which, int most_rows, int items) {
    __shared__ float lo[WAYS][D];
    __shared__ float ll[WAYS][2];
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int item = (int)(blockIdx.x % items), row = (int)(blockIdx.x / items) * (4 / WAYS) + wave / WAYS;
    const int b = item / a.kv_heads, h = item % a.kv_heads, G = a.q_heads / a.kv_heads;
    const Begun x = static_cast<const Begun *>(a.ws)[item];      // written if the sequence has rows
    const Seq s = seq_of(a, b, which);
    if (row >= min(s.n * G, most_rows) || x.pieces < 2) return;      // with four ways: the whole workgroup
    const int wg = uniform(x.wg), pieces = uniform(x.pieces);
    float m = -__builtin_inff(), l = 0.0f, acc[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = 0.0f;
    // o of pieces k .. k + 7 from i0 on (past the last one: the last one)
    const auto fetch = [&](float (&v)[8][D / 64], int i0, int k, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float *part = part_of(a, D, most_rows, wg + i0 + WAYS * min(k + e, n - 1)) + row * D + (D / 64) * lane;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) v[e][j] = part[j];
        }
    };
    for (int i0 = wave % WAYS; i0 < pieces; i0 += 64 * WAYS) {
        // up to 64 pieces: a lane each their maximum, sum and weight; the first
        // eight pieces' o is on its way meanwhile
        const int i = i0 + WAYS * lane, n = min((pieces - i0 + WAYS - 1) / WAYS, 64);
        float v[8][D / 64];
        fetch(v, i0, 0, n);
        float pm = -__builtin_inff(), pl = 0.0f;
        if (i < pieces) {
            const float *ml = part_of(a, D, most_rows, wg + i) + most_rows * D + 2 * row;
            pm = ml[0];
            pl = ml[1];
        }
        float top = fmaxf(m, pm);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        const float base = top == -__builtin_inff() ? 0.0f : top, f0 = exp2a(m - base), f = exp2a(pm - base);
        m = top;
        l = l * f0 + wave_sum_dpp(pl * f);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] *= f0;
        for (int k = 0; k < n; k += 8) {
            if (k > 0) fetch(v, i0, k, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), min(k + e, n - 1)));
#pragma unroll
                for (int j = 0; j < D / 64; ++j) acc[j] = k + e < n ? __builtin_fmaf(g, v[e][j], acc[j]) : acc[j];
            }
        }
    }
    if constexpr (WAYS > 1) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) lo[wave][(D / 64) * lane + j] = acc[j];
        if (lane == 0) {
            ll[wave][0] = m;
            ll[wave][1] = l;
        }
        __syncthreads();
        if (wave > 0) return;
        float top = m;
#pragma unroll
        for (int w = 1; w < WAYS; ++w) top = fmaxf(top, ll[w][0]);
        const float base = top == -__builtin_inff() ? 0.0f : top, f0 = exp2a(m - base);
        m = top;
        l *= f0;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] *= f0;
#pragma unroll
        for (int w = 1; w < WAYS; ++w) {
            const float f = exp2a(ll[w][0] - base);
            l += f * ll[w][1];
#pragma unroll
            for (int j = 0; j < D / 64; ++j) acc[j] += f * lo[w][(D / 64) * lane + j];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = row / G, g = row - i * G;
    const int64_t t = s.first + i;
    uint16_t *dst = a.o + t * a.o_stride + (int64_t)(h * G + g) * D + (D / 64) * lane;
    if constexpr (D == 128) *reinterpret_cast<uint32_t *>(dst) = narrow2a(acc[0] * inv, acc[1] * inv);
    else *dst = f32_to_bf16_rne(acc[0] * inv);
    if (a.lse && lane == 0) a.lse[t * a.q_heads + h * G + g] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Whether a workgroup takes a whole item: it takes `turns` of 8 waves in turn,
// against an even share of all chunks over the chip's 2048 waves and, for the list
// and the join, about as long as two more (four of 64 channels).  The host knows the longest sequence
// only, and the others may be short: the longest is not to take more than eight
// times a CU's share if all were as long (items / 256 items), or, where waves form four
// groups that read a chunk each, twice.
// Measured, us whole | split, joins included, for 32 and 128 sequences (64/8 heads) and
// 32 (40/40), lengths all of the longest (=) or spread evenly in their logarithm (~):
//   longest   32, 64/8 (256 items)     128, 64/8 (1024)         32, 40/40 (1280)
//    2048     = 24 | 29,  ~ 16 | 14    = 101 | 106, ~ 39 | 39   = 122 | 123, ~ 41 | 38
//    4096     = 42 | 49,  ~ 27 | 18    = 187 | 191, ~ 43 | 44   = 227 | 230, ~ 51 | 48
//    8192     = 95 | 101, ~ 46 | 24    = 356 | 363, ~ 69 | 67   = 441 | 449, ~ 77 | 93
//   16384     = 182 | 191, ~ 85 | 35   = 699 | 709, ~ 139 | 126 = 881 | 897, ~ 168 | 182
//   32768     = 358 | 366, ~ 185 | 83  = 1408 | 1421, ~ 208 | 197   = 1787 | 1823, ~ 312 | 338
// One sequence of 512, 1024, 1536 and 2048 tokens (1 to 4 turns), 40/40: 7.5 | 11.2,
// 10.3 | 11.0, 12.8 | 11.6, 15.6 | 12.8; of 64 channels 6.0 | 9.7, 7.7 | 9.9, 8.6 | 9.9,
// 10.2 | 11.2.  40 rows, 128 sequences, 64/8 heads: 2048
// = 196 | 189, ~ 82 | 78; 8192 = 701 | 677, ~ 190 | 167.
int64_t free_turns(int dim) { return dim == 64 ? 4 : 2; }
int64_t turns_of(int64_t chunks, int row_shift) { return ((chunks << row_shift) + kWholeWaves - 1) / kWholeWaves; }
int64_t items_a_turn(int row_shift) { return row_shift < 2 ? 32 : 128; }
bool whole_items(int64_t items, int64_t chunks, int row_shift, int dim) {
    const int64_t turns = turns_of(chunks, row_shift), most = items / items_a_turn(row_shift);
    const int64_t shared = ((items * chunks) << row_shift) / (kPieces * kSplitWaves) + free_turns(dim);
    return turns <= shared && (turns <= free_turns(dim) || turns <= most);
}

// The most workspace that pieces of items need, for a call of these sizes or
// of smaller ones: up to free_turns no number of items is split; above, only fewer items
// than the 256 at which `shared` passes `turns`, or than turns * items_a_turn.
size_t split_bytes(int64_t items, int dim, int rows) {
    return begun_slots(items) * sizeof(Begun) + (items + kPieces) * part_floats(dim, rows) * sizeof(float);
}
size_t most_split_bytes(int64_t items, int64_t chunks, int row_shift, int dim, int rows) {
    constexpr int64_t kShared = kPieces * kSplitWaves / kWholeWaves;
    const int64_t turns = turns_of(chunks, row_shift);
    if (turns <= free_turns(dim)) return 0;
    int64_t most = turns * items_a_turn(row_shift);
    if (most < kShared) most = kShared;
    return split_bytes(items < most ? items : most - 1, dim, rows);
}

struct Plan {
    int row_shift, most_rows;
    int64_t items;
    bool rows, tiles;      // which kernels the call needs
    bool whole;            // a workgroup an item
    size_t bytes;          // of workspace that the launches use, one after the other
    size_t most_bytes;     // at least that, whatever the window, for this call and every smaller one
};

// What the host can know: at most this many rows, tiles and chunks.  A batch
// may hold sequences of few and of many rows: both kernels are then launched,
// each taking its own, unless the shortest sequence that T allows has many.
Plan plan_of(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv, int window, int sinks) {
    Plan p;
    const int64_t G = q_heads / kv_heads, longest = max_q < T ? max_q : T;
    p.tiles = longest * G > kMostRows;
    p.rows = !p.tiles || (T - (B - 1) * longest) * G <= kMostRows;
    const int64_t rows = longest * G < kMostRows ? longest * G : kMostRows;
    p.row_shift = row_shift_of((int)rows);
    p.most_rows = (int)rows;
    p.items = (int64_t)B * kv_heads;      // at most 2^26
    const int64_t chunks = (max_kv + kChunk - 1) / kChunk;
    p.whole = whole_items(p.items, chunks, p.row_shift, dim);
    p.most_bytes = most_split_bytes(p.items, chunks, p.row_shift, dim, p.most_rows);
    if (window > 0) {
        const int64_t seen = ((int64_t)window + longest + 2 * kChunk) / kChunk + ((int64_t)sinks + kChunk - 1) / kChunk;
        p.whole = p.whole || whole_items(p.items, seen < chunks ? seen : chunks, p.row_shift, dim);
    }
    p.bytes = p.rows && !p.whole ? split_bytes(p.items, dim, p.most_rows) : 0;
    if (p.tiles) {
        const size_t now = attn_tiles_plan(B, T, q_heads, kv_heads, dim, max_kv, window, sinks).ws_bytes;
        const size_t most = attn_tiles_most_bytes(B, T, q_heads, kv_heads, dim, max_kv);
        p.bytes = p.bytes < now ? now : p.bytes;
        p.most_bytes = p.most_bytes < most ? most : p.most_bytes;
    }
    return p;
}

template <int D>
hipError_t launch(const AttnArgs &a, const Plan &p, hipStream_t stream) {
    const int which = p.tiles ? kFewRows : kAllSeqs;
    if (p.whole) {
        if (p.items > 0x7FFFFFFF) return hipErrorInvalidValue;
        hipLaunchKernelGGL((attn_whole_kernel<D>), dim3((unsigned)p.items), dim3(64 * kWholeWaves), 0, stream, a, which,
                           p.most_rows);
        return hipGetLastError();
    }
    if (p.items + kPieces > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_split_kernel<D>), dim3((unsigned)(p.items + kPieces)), dim3(64 * kSplitWaves), 0, stream, a,
                       which, p.most_rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // few rows: four waves a row; many: a wave
    const int ways = p.items * p.most_rows <= 1024 ? 4 : 1;
    const int64_t grid = p.items * ((p.most_rows + 4 / ways - 1) / (4 / ways));
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (ways == 4)
        hipLaunchKernelGGL((attn_join_kernel<D, 4>), dim3((unsigned)grid), dim3(256), 0, stream, a, which, p.most_rows,
                           (int)p.items);
    else
        hipLaunchKernelGGL((attn_join_kernel<D, 1>), dim3((unsigned)grid), dim3(256), 0, stream, a, which, p.most_rows,
                           (int)p.items);
    return hipGetLastError();
}

}  // namespace

size_t attn_ws_bytes(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv) {
    if (B == 0 || T == 0) return 0;
    return plan_of(B, T, q_heads, kv_heads, dim, max_q, max_kv, 0, 0).most_bytes;
}

// The launches for many and for few rows follow one another on the stream and
// use the same workspace.
hipError_t launch_attn(const AttnArgs &a, size_t ws_bytes, hipStream_t stream) {
    const Plan p = plan_of(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_q, a.max_kv, a.window, a.sinks);
    if (p.bytes > ws_bytes) return hipErrorInvalidValue;
    if (p.tiles) {      // first: the longest workgroups
        const hipError_t e = launch_attn_tiles(a, p.rows ? kManyRows : kAllSeqs, stream);
        if (e != hipSuccess || !p.rows) return e;
    }
    return a.dim == 64 ? launch<64>(a, p, stream) : launch<128>(a, p, stream);
}

}  // namespace biloco
