// Attention over the paged 8-bit cache for a batch whose sequences share their first
// tokens in groups.
//
// A row's softmax over all its tokens is joined from two parts, o = sum_i e^(m_i - m) o_i
// over the same of l_i: the group's shared tokens, and the sequence's own ones.
//   shared  a workgroup takes 128 rows of a group (rows of several sequences) and walks
//           the shared tokens' chunks as the kernel for many rows does, so that a
//           shared token is read and made wide once for 128 rows, not once a sequence
//   own     the kernel for few rows, from the first own token on
// A row's position is its own sequence's, so that masks by position (causality, window,
// first tokens) hold in both parts.  Sequences of more than kMostRows rows make tiles by
// themselves and share nothing: the kernel for many rows takes them whole, here with
// weights of two terms, so that all of the call's results are of one exactness.
#include "attn_rows.h"
#include "attn_tiles.h"

namespace biloco {

namespace {

using namespace attn;

constexpr int kWantItems = 512;      // workgroups that fill the chip (two a CU)

// Where the sequences' rows lie in the groups' tiles; made by one workgroup first.
struct Tables {
    int *before;      // [B + 1] new tokens of the sequences before (of few rows), T at most
    int *tile;        // [groups + 1] tiles of the groups before
    int *from;        // [B] the first own token
    int *row;         // [B] the first row among the tiles' rows, or -1: nothing is shared
};
__host__ __device__ __forceinline__ size_t table_ints(int64_t B, int64_t groups) {
    return (size_t)((3 * B + groups + 2 + 3) / 4 * 4);
}
__device__ __forceinline__ Tables tables_of(const SharedAttnArgs &s, int B) {
    Tables t;
    t.before = static_cast<int *>(s.tables);
    t.tile = t.before + B + 1;
    t.from = t.tile + s.groups + 1;
    t.row = t.from + B;
    return t;
}

struct Group {
    int b0, b1, upto;      // its sequences, its shared tokens
};
__device__ __forceinline__ Group group_at(const AttnArgs &a, const SharedAttnArgs &s, int g) {
    Group x;
    x.b0 = min(max(s.group_start[g], 0), a.B);
    x.b1 = min(max(s.group_start[g + 1], x.b0), a.B);
    x.upto = (int)min((int64_t)max(s.shared_len[g], 0), (int64_t)a.max_pages * a.page);
    return x;
}

constexpr int kTableThreads = 1024;
// Sums that stop at a cap below 2^31, as those of lists that are not in order have to: these
// can claim every row for each second sequence.
__device__ __forceinline__ int capped(int a, int b, int cap) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)cap); }
// Exclusive sums over the workgroup of numbers from 0 to `cap`, behind `carry`, which
// becomes the whole sum.
__device__ __forceinline__ int sums_before(int v, int cap, int (&tmp)[kTableThreads / 64], int &carry) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int in = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(in, o, 64);
        if (lane >= o) in = capped(in, t, cap);
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = in;
    __syncthreads();
    const int up = __shfl_up(in, 1, 64);
    int before = carry;
    for (int i = 0; i < kTableThreads / 64; ++i) {
        if (i == wave) before = capped(carry, lane > 0 ? up : 0, cap);
        carry = capped(carry, tmp[i], cap);
    }
    return before;
}

__global__ void __launch_bounds__(kTableThreads)
attn_shared_tables_kernel(const AttnArgs a, const SharedAttnArgs s, int which, int tiles) {
    __shared__ int tmp[kTableThreads / 64];
    const Tables t = tables_of(s, a.B);
    const int G = a.q_heads / a.kv_heads;
    int carry = 0;
    for (int at = 0; at < a.B; at += kTableThreads) {
        const int b = at + threadIdx.x, n = b < a.B ? seq_of(a, b, which).n : 0;
        const int mine = sums_before(n, a.T, tmp, carry);
        if (b < a.B) t.before[b] = mine;
    }
    if (threadIdx.x == 0) t.before[a.B] = carry;
    __threadfence_block();
    __syncthreads();
    carry = 0;
    for (int at = 0; at < s.groups; at += kTableThreads) {
        const int g = at + threadIdx.x;
        int n = 0;
        if (g < s.groups) {
            const Group x = group_at(a, s, g);
            const int64_t rows = (int64_t)(t.before[x.b1] - t.before[x.b0]) * G;
            n = x.upto > 0 ? (int)min((rows + kTileRows - 1) / kTileRows, (int64_t)tiles) : 0;
        }
        const int mine = sums_before(n, tiles, tmp, carry);
        if (g < s.groups) t.tile[g] = mine;
    }
    if (threadIdx.x == 0) t.tile[s.groups] = carry;
    __threadfence_block();
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += kTableThreads) {
        int lo = 0, hi = s.groups - 1;      // the last group that begins at or before b
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s.group_start[mid] <= b) lo = mid;
            else hi = mid - 1;
        }
        const Group x = group_at(a, s, lo);
        const int64_t row = (int64_t)t.tile[lo] * kTileRows + (int64_t)(t.before[b] - t.before[x.b0]) * G;
        const int64_t end = row + (int64_t)(t.before[b + 1] - t.before[b]) * G;
        const bool in = x.upto > 0 && b >= x.b0 && b < x.b1 && end <= (int64_t)t.tile[lo + 1] * kTileRows;
        t.from[b] = in ? x.upto : 0;
        t.row[b] = in ? (int)row : -1;
    }
}

template <int D>
__device__ __forceinline__ float *shared_part(const SharedAttnArgs &s, int64_t item, int splits, int split) {
    return static_cast<float *>(s.parts) + (item * splits + split) * kTileRows * (D + 2);
}

// A tile's rows are of several sequences: where their positions lie further apart than a
// window, there are tokens between them that none of them sees (`gaps`).
struct SharedArgs : PartArgs {
    const int *pos;      // of the tile's rows
    int rows;
    bool gaps, blind;    // blind: the lane's row sees none of the shared tokens
    __device__ __forceinline__ explicit SharedArgs(const AttnArgs &a) : PartArgs(a, 0, 0), pos(nullptr), rows(0), gaps(false), blind(false) {}
};
__device__ __forceinline__ uint32_t tile_sees8(const SharedArgs &a, int p_min, int p_max, int t0) {
    const uint32_t bits = any_sees8(a, p_min, p_max, t0);
    if (__builtin_expect(!a.gaps || bits == 0, 1)) return bits;
    uint32_t some = 0;
#pragma unroll 1      // out of the walk's way: unrolled, groups with drafts take 43.5 us for 43.1
    for (int r = 0; r < a.rows; ++r) some |= sees8(a, a.pos[r], t0);
    return some;
}

// A workgroup takes 128 rows of a group, whose tokens and positions it first lists.  Rows
// that see none of the shared tokens (idle slots, windows that begin behind them) go along
// at another row's position, so that they do not mask the others' chunks, and leave nothing.
struct SharedTiles {
    using Args = SharedArgs;
    static constexpr int kTerms = 2;
    struct Lds {
        int token[kTileRows], pos[kTileRows];
    };
    AttnArgs a;
    SharedAttnArgs s;
    int which;

    __device__ __forceinline__ SharedArgs args() const { return SharedArgs(a); }
    __device__ __forceinline__ bool sees_any(int pos, int upto) const {
        return pos >= 0 && (low_of(a, pos) < upto || a.sinks > 0);
    }
    __device__ __forceinline__ static int lowest(int v) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) v = min(v, __shfl_xor(v, o, 64));
        return uniform(v);
    }
    template <int D>
    __device__ __forceinline__ bool begin(Rows32<D, kTerms> &w, TileWork<SharedArgs> &t, Lds &lds, int splits) const {
        const Tables tab = tables_of(s, a.B);
        t.h = (int)(blockIdx.x % a.kv_heads);
        const int rest = (int)(blockIdx.x / a.kv_heads);
        t.split = rest % splits;
        t.at = rest / splits;
        if (t.at >= scalar_load(tab.tile + s.groups)) return false;
        int g = 0, last_g = s.groups - 1;      // the last group whose tiles begin at or before this one
        while (g < last_g) {
            const int mid = (g + last_g + 1) / 2;
            if (scalar_load(tab.tile + mid) <= t.at) g = mid;
            else last_g = mid - 1;
        }
        const Group x = group_at(a, s, g);
        const int G = a.q_heads / a.kv_heads, r0 = (t.at - scalar_load(tab.tile + g)) * kTileRows;
        const int first = scalar_load(tab.before + x.b0);
        t.rows = min((scalar_load(tab.before + x.b1) - first) * G - r0, kTileRows);
        for (int b = x.b0 + threadIdx.x; b < x.b1; b += 256) {
            const Seq q = seq_of(a, b, which);
            // rows of its first row and behind its last one in the tile
            const int at0 = (tab.before[b] - first) * G - r0, at1 = (tab.before[b + 1] - first) * G - r0;
            for (int r = max(at0, 0); r < min(at1, kTileRows); ++r) {
                const int i = (r - at0) / G;
                lds.token[r] = q.first + i;
                lds.pos[r] = q.past + i;
            }
        }
        __syncthreads();
        const int wave = uniform((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
        const int p0 = lds.pos[min(lane, t.rows - 1)], p1 = lds.pos[min(lane + 64, t.rows - 1)];
        const bool s0 = sees_any(p0, x.upto), s1 = sees_any(p1, x.upto);
        t.p_min = lowest(min(s0 ? p0 : 0x7FFFFFFF, s1 ? p1 : 0x7FFFFFFF));
        t.p_max = -lowest(min(s0 ? -p0 : 1, s1 ? -p1 : 1));      // -1: none sees any
        const int row = min(32 * wave + (lane & 31), t.rows - 1), gi = (r0 + row) % G;
        t.a.blind = !sees_any(lds.pos[row], x.upto);
        w.p = t.a.blind ? t.p_max : lds.pos[row];
        w.p_min = lowest(w.p);
        w.p_max = -lowest(-w.p);
        w.start(a.q + (int64_t)lds.token[row] * a.q_stride + (int64_t)(t.h * G + gi) * D + 8 * (lane >> 5));
        t.a.upto = x.upto;
        t.a.pos = lds.pos;
        t.a.rows = t.rows;
        t.a.gaps = a.window > 0 && t.p_min < x.upto - 1 && t.p_max - a.window > t.p_min;
        t.last = x.upto - 1;
        t.table = a.table + (int64_t)x.b0 * a.max_pages;
        t.span = t.p_max < 0 ? Span64{0, 0, 0} : span_of(t.a, t.p_min, t.p_max);
        const int each = (t.span.nc + splits - 1) / splits;
        t.c0 = min(t.split * each, t.span.nc);
        t.c1 = min(t.c0 + each, t.span.nc);
        return true;
    }
    template <int D>
    __device__ __forceinline__ void end(const Rows32<D, kTerms> &w, const TileWork<SharedArgs> &t, float l, int splits) const {
        const int row = 32 * (int)(threadIdx.x >> 6) + (int)(threadIdx.x & 31);
        if (row < t.rows) leave(w, l, shared_part<D>(s, (int64_t)t.at * a.kv_heads + t.h, splits, t.split), row, t.a.blind);
    }
};

// A sequence's own tokens.
struct OwnRows {
    static constexpr bool kPart = true;
    AttnArgs a;
    SharedAttnArgs s;
    __device__ __forceinline__ PartArgs of(int b) const { return PartArgs(a, tables_of(s, a.B).from[b], 0x7FFFFFFF); }
};

// Both in one launch, the tiles' workgroups first; neither waits for the other.  Four answers
// behind 608 shared tokens, groups with drafts and many answers: 20.1, 43.1 and 86 us.  With
// weights of one term they took 18.1, 39.2 and 77, and as two launches 25.5, 48.5 and 82.
template <int D>
__global__ void __launch_bounds__(256, 2)
attn_shared_kernel(const AttnArgs a, const SharedAttnArgs s, int which, int most_rows, int tiles, int splits) {
    union Lds {
        struct {
            TileLds<D> chunks;
            SharedTiles::Lds rows;
        } tiles;
        JoinLds<D, kSplitWaves> join;
    };
    __shared__ Lds lds;
    if ((int)blockIdx.x < tiles) tile_rows<D>(SharedTiles{a, s, which}, splits, lds.tiles.chunks, lds.tiles.rows);
    else split_rows<D>(OwnRows{a, s}, which, most_rows, (int)blockIdx.x - tiles, lds.join);
}

// Joins a row's parts: a wave a row.
template <int D>
__global__ void __launch_bounds__(256)
attn_shared_join_kernel(const AttnArgs a, const SharedAttnArgs sh, int which, int most_rows, int items, int splits) {
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int item = (int)(blockIdx.x % items), row = (int)(blockIdx.x / items) * 4 + wave;
    const int b = item / a.kv_heads, h = item % a.kv_heads, G = a.q_heads / a.kv_heads;
    const Tables tab = tables_of(sh, a.B);
    const Begun x = static_cast<const Begun *>(a.ws)[item];      // written if the sequence has rows
    const Seq s = seq_of(a, b, which);
    if (row >= min(s.n * G, most_rows)) return;
    float m = -__builtin_inff(), l = 0.0f, acc[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = 0.0f;
    const auto take = [&](const float *o, const float *ml) {
        const float pm = ml[0], pl = ml[1];
        const float top = fmaxf(m, pm), base = top == -__builtin_inff() ? 0.0f : top;
        const float f0 = exp2a(m - base), f1 = exp2a(pm - base);
        m = top;
        l = l * f0 + pl * f1;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = acc[j] * f0 + o[(D / 64) * lane + j] * f1;
    };
    for (int i = 0; i < x.pieces; ++i) {
        const float *part = part_of(a, D, most_rows, x.wg + i);
        take(part + row * D, part + most_rows * D + 2 * row);
    }
    const int first = tab.row[b];
    if (first >= 0) {
        const int at = first + row, r = at % kTileRows;
        for (int i = 0; i < splits; ++i) {
            const float *part = shared_part<D>(sh, (int64_t)(at / kTileRows) * a.kv_heads + h, splits, i);
            take(part + r * D, part + kTileRows * D + 2 * r);
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

struct SharedPlan {
    bool rows, tiles;      // sequences of few rows; of many
    int most_rows, shared_tiles, splits;
    int64_t items, tile_grid, join_grid;      // workgroups for the shared tokens, and for the join
    size_t table_bytes, own_bytes;
    size_t bytes, most_bytes;      // for this call; for it and every smaller one
};

// A multiple of 16: the shared parts behind them are written 16 bytes at a time.
size_t own_bytes(int64_t items, int dim, int rows) {
    const size_t n = begun_slots(items) * sizeof(Begun) + (size_t)((items + kPieces) * part_floats(dim, rows)) * sizeof(float);
    return (n + 15) / 16 * 16;
}

// Sequences of many rows, if the host cannot exclude them, are taken first, in the same
// workspace.
SharedPlan plan_of(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv, int groups, int max_shared,
                   int window, int sinks) {
    SharedPlan p;
    const int64_t G = q_heads / kv_heads, longest = max_q < T ? max_q : T;
    p.tiles = longest * G > kMostRows;
    p.rows = !p.tiles || (T - (B - 1) * longest) * G <= kMostRows;
    p.most_rows = (int)(longest * G < kMostRows ? longest * G : kMostRows);
    p.items = (int64_t)B * kv_heads;
    const int64_t parts = groups < B ? groups : B;
    p.shared_tiles = (int)(((int64_t)T * G + (kTileRows - 1) * parts) / kTileRows);
    const int64_t wgs = (int64_t)p.shared_tiles * kv_heads;
    const int64_t most = ((int64_t)max_shared + 4 * kChunk - 1) / (4 * kChunk);      // pieces of at least four chunks
    int64_t splits = wgs > 0 ? (kWantItems + wgs - 1) / wgs : 1;
    if (splits > most) splits = most;
    p.splits = splits < 1 ? 1 : (int)splits;
    p.tile_grid = wgs * p.splits;
    p.join_grid = p.items * ((p.most_rows + 3) / 4);
    p.table_bytes = table_ints(B, groups) * sizeof(int);
    p.own_bytes = own_bytes(p.items, dim, p.most_rows);
    const size_t part = (size_t)kTileRows * (dim + 2) * sizeof(float);
    p.bytes = p.table_bytes + p.own_bytes + (size_t)wgs * p.splits * part;
    const int64_t cut = wgs + kWantItems - 1, all = wgs * (most < 1 ? 1 : most);
    p.most_bytes = p.table_bytes + p.own_bytes + (size_t)(cut < all ? cut : all) * part;
    if (p.tiles) {
        const size_t now = attn_tiles_plan(B, T, q_heads, kv_heads, dim, max_kv, window, sinks).ws_bytes;
        const size_t bound = attn_tiles_most_bytes(B, T, q_heads, kv_heads, dim, max_kv);
        if (p.bytes < now) p.bytes = now;
        if (p.most_bytes < bound) p.most_bytes = bound;
    }
    return p;
}

template <int D>
hipError_t launch(const AttnArgs &a, SharedAttnArgs s, const SharedPlan &p, hipStream_t stream) {
    const int which = p.tiles ? kFewRows : kAllSeqs;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    AttnArgs own = a;
    s.tables = ws;
    own.ws = ws + p.table_bytes;
    s.parts = ws + p.table_bytes + p.own_bytes;
    const int64_t tiles = p.tile_grid, pieces = p.items + kPieces, join = p.join_grid;
    hipLaunchKernelGGL(attn_shared_tables_kernel, dim3(1), dim3(kTableThreads), 0, stream, own, s, which, p.shared_tiles);
    static_assert(kSplitWaves == 4, "both kinds of workgroups in one grid");
    hipLaunchKernelGGL((attn_shared_kernel<D>), dim3((unsigned)(tiles + pieces)), dim3(256), 0, stream, own, s, which,
                       p.most_rows, (int)tiles, p.splits);
    hipLaunchKernelGGL((attn_shared_join_kernel<D>), dim3((unsigned)join), dim3(256), 0, stream, own, s, which, p.most_rows,
                       (int)p.items, p.splits);
    return hipGetLastError();
}

}  // namespace

bool attn_shared_fits(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv, int groups, int max_shared) {
    if (B == 0 || T == 0) return true;
    const SharedPlan p = plan_of(B, T, q_heads, kv_heads, dim, max_q, max_kv, groups, max_shared, 0, 0);
    return fits_grid(p.tile_grid + p.items + kPieces, 256) && fits_grid(p.join_grid, 256);
}

size_t attn_shared_ws_bytes(int B, int T, int q_heads, int kv_heads, int dim, int max_q, int max_kv, int groups,
                            int max_shared) {
    if (B == 0 || T == 0) return 0;
    return plan_of(B, T, q_heads, kv_heads, dim, max_q, max_kv, groups, max_shared, 0, 0).most_bytes;
}

hipError_t launch_attn_shared(const AttnArgs &a, const SharedAttnArgs &s, size_t ws_bytes, hipStream_t stream) {
    const SharedPlan p = plan_of(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_q, a.max_kv, s.groups, s.max_shared, a.window,
                                 a.sinks);
    if (p.bytes > ws_bytes) return hipErrorInvalidValue;
    if (p.tiles) {
        const hipError_t e = launch_attn_tiles(a, p.rows ? kManyRows : kAllSeqs, 2, stream);
        if (e != hipSuccess || !p.rows) return e;
    }
    return a.dim == 64 ? launch<64>(a, s, p, stream) : launch<128>(a, s, p, stream);
}

}  // namespace biloco
