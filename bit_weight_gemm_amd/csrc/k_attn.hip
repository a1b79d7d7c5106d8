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
#include "attn_rows.h"

namespace biloco {

namespace {

using namespace attn;

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

// Items of the whole batch.
struct PagedRows {
    static constexpr bool kPart = false;
    AttnArgs a;
    __device__ __forceinline__ const AttnArgs &of(int) const { return a; }
};

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
        if (!fits_grid(p.items, 64 * kWholeWaves)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((attn_whole_kernel<D>), dim3((unsigned)p.items), dim3(64 * kWholeWaves), 0, stream, a, which,
                           p.most_rows);
        return hipGetLastError();
    }
    if (!fits_grid(p.items + kPieces, 64 * kSplitWaves)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((attn_split_kernel<D, PagedRows>), dim3((unsigned)(p.items + kPieces)), dim3(64 * kSplitWaves), 0,
                       stream, PagedRows{a}, which, p.most_rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // few rows: four waves a row; many: a wave
    const int ways = p.items * p.most_rows <= 1024 ? 4 : 1;
    const int64_t grid = p.items * ((p.most_rows + 4 / ways - 1) / (4 / ways));
    if (!fits_grid(grid, 256)) return hipErrorInvalidConfiguration;
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
        const hipError_t e = launch_attn_tiles(a, p.rows ? kManyRows : kAllSeqs, 1, stream);
        if (e != hipSuccess || !p.rows) return e;
    }
    return a.dim == 64 ? launch<64>(a, p, stream) : launch<128>(a, p, stream);
}

}  // namespace biloco
