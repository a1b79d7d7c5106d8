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
#include "attn_tiles.h"

namespace biloco {

namespace {

using namespace attn;

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
template <int TERMS>
struct PagedTiles {
    using Args = AttnArgs;
    static constexpr int kTerms = TERMS;
    struct Lds {};
    AttnArgs a;
    int which, tiles;

    __device__ __forceinline__ const AttnArgs &args() const { return a; }
    template <int D>
    __device__ __forceinline__ bool begin(Rows32<D, kTerms> &w, TileWork<AttnArgs> &t, Lds &, int splits) const {
        t.h = (int)(blockIdx.x % a.kv_heads);
        const int rest = (int)(blockIdx.x / a.kv_heads);
        t.split = rest % splits;
        t.at = tiles - 1 - rest / splits;
        int64_t before = 0;
        const int b = uniform(find_seq(a.B, t.at, before, [&](int i) { return tiles_of(a, seq_of(a, i, which)); }));
        if (b < 0) return false;
        t.s = seq_uniform(a, b, which);
        const int G = a.q_heads / a.kv_heads;
        t.rows = t.s.n * G;
        t.r0 = (t.at - (int)uniform(before)) * kTileRows;
        t.last = t.s.hi - 1;
        t.table = a.table + (int64_t)b * a.max_pages;
        t.p_min = t.s.past + t.r0 / G;
        t.p_max = t.s.past + (min(t.r0 + kTileRows, t.rows) - 1) / G;
        t.span = span_of(a, t.p_min, t.p_max);
        const int each = (t.span.nc + splits - 1) / splits;
        t.c0 = min(t.split * each, t.span.nc);
        t.c1 = min(t.c0 + each, t.span.nc);
        w.init(a, t.s, t.h, t.r0 + 32 * uniform((int)(threadIdx.x >> 6)), t.rows);
        return true;
    }
    template <int D>
    __device__ __forceinline__ void end(const Rows32<D, kTerms> &w, const TileWork<AttnArgs> &t, float l, int splits) const {
        const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6)), G = a.q_heads / a.kv_heads;
        const int row = t.r0 + 32 * wave + (lane & 31), half = lane >> 5;
        if (row >= t.rows) return;
        if (splits > 1) {
            leave(w, l, tile_part<D>(a, (int64_t)t.at * a.kv_heads + t.h, splits, t.split), row - t.r0);
            return;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int i = row / G, g = row - i * G;
        const int64_t tok = t.s.first + i;
        uint16_t *dst = a.o + tok * a.o_stride + (int64_t)(t.h * G + g) * D + 4 * half;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint2 *>(dst + 32 * n + 8 * j) =
                    make_uint2(narrow2a(w.o[n][4 * j] * inv, w.o[n][4 * j + 1] * inv),
                               narrow2a(w.o[n][4 * j + 2] * inv, w.o[n][4 * j + 3] * inv));
        if (a.lse && half == 0) a.lse[tok * a.q_heads + t.h * G + g] = (w.m + __builtin_amdgcn_logf(l)) * kLn2;
    }
};

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

template <int D, int TERMS>
hipError_t launch(const AttnArgs &a, int which, hipStream_t stream) {
    const TilesPlan p = attn_tiles_plan(a.B, a.T, a.q_heads, a.kv_heads, a.dim, a.max_kv, a.window, a.sinks);
    const int64_t grid = (int64_t)p.tiles * p.splits * a.kv_heads;
    const int64_t join = (int64_t)p.tiles * a.kv_heads * (kTileRows / 4);
    if (!fits_grid(grid, 256) || (p.splits > 1 && !fits_grid(join, 256))) return hipErrorInvalidConfiguration;
    const PagedTiles<TERMS> k{a, which, p.tiles};
    hipLaunchKernelGGL((attn_tiles_kernel<D, PagedTiles<TERMS>>), dim3((unsigned)grid), dim3(256), 0, stream, k, p.splits);
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

hipError_t launch_attn_tiles(const AttnArgs &a, int which, int terms, hipStream_t stream) {
    if (terms == 2) return a.dim == 64 ? launch<64, 2>(a, which, stream) : launch<128, 2>(a, which, stream);
    return a.dim == 64 ? launch<64, 1>(a, which, stream) : launch<128, 1>(a, which, stream);
}

}  // namespace biloco
