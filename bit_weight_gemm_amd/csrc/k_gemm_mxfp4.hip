// y = A W^T of microscaled 4-bit operands on the scaled matrix instructions of gfx950,
// which take E2M1 codes and one scale byte for 32 of them as they are.
//
//   y[m][n] = sum over blocks b of 2^(sa[m][b] + sw[n][b] - 254) sum_k a[m][k] w[n][k]
//
// Sums are fp32 (the instruction adds a block's exact sum).  A scale byte of 255 makes
// its row NaN.
#include <type_traits>

#include "mx_device.h"
#include "mx_plan.h"

namespace biloco {

namespace {

using namespace mx;

// Operands, outputs and sizes of a call.
struct Mx {
    const uint8_t *ac, *as, *wc, *ws;
    const uint16_t *x;      // or rows to be quantised in place of ac and as
    int64_t xs;
    int M, N, K;
    int spitch;      // bytes from one row of scales to the next (many rows)
    void *y;
    int64_t ys;
    float *part;      // sums of the pieces of K, [piece][M][N], or NULL
    int pieces;
};

__device__ __forceinline__ i32x8m_t frag(const u32x4_t &v) {
    return i32x8m_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
template <int SA, int SB = SA>
__device__ __forceinline__ f32x4m_t mfma16(const u32x4_t &a, const u32x4_t &b, f32x4m_t c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(a), frag(b), c, 4, 4, SA, (int)sa, SB, (int)sb);
}
template <int S>
__device__ __forceinline__ f32x16m_t mfma32(const u32x4_t &a, const u32x4_t &b, f32x16m_t c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(a), frag(b), c, 4, 4, S, (int)sa, S, (int)sb);
}
__device__ __forceinline__ uint32_t load4(const uint8_t *p) {      // at any address
    uint32_t v;
    __builtin_memcpy(&v, p, 4);
    return v;
}
template <class T>
__device__ __forceinline__ T rounded(float v) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(uint16_t, (__bf16)v);      // to nearest, ties to even
    else return v;
}

// ---------------------------------------------------------------- few rows
// A workgroup takes 16 NT rows of W (the instructions' first operand, so that a lane's
// results are successive n of one m) and all rows of A (16 MT of them); its waves take
// chunks of 512 k in turn and join their sums in LDS.  In a chunk the lanes l >> 4 == g
// take the blocks 4 g .. 4 g + 3, one a step, so that a lane's four scale bytes are one
// dword and each step's byte is the instruction's selector.
template <int NT, int MT>
struct Chunk {
    u32x4_t w[NT][4], a[MT][4];
    uint32_t ws[NT], as[MT];

    // Chunk c whole, or its first blocks: codes of blocks past the last become zero
    // and their scales 1.
    __device__ __forceinline__ void load(const uint8_t *const (&wr)[NT], const uint8_t *const (&wsr)[NT],
                                         const uint8_t *const (&ar)[MT], const uint8_t *const (&asr)[MT], int c, int blocks) {
        const int g = (threadIdx.x & 63) >> 4, b0 = 16 * c + 4 * g;
        if (16 * c + 16 <= blocks) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                ws[i] = load4(wsr[i] + b0);
#pragma unroll
                for (int s = 0; s < 4; ++s) w[i][s] = *reinterpret_cast<const u32x4_t *>(wr[i] + 16 * (int64_t)(b0 + s));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                as[i] = load4(asr[i] + b0);
#pragma unroll
                for (int s = 0; s < 4; ++s) a[i][s] = *reinterpret_cast<const u32x4_t *>(ar[i] + 16 * (int64_t)(b0 + s));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) part(wr[i], wsr[i], b0, blocks, w[i], ws[i]);
#pragma unroll
        for (int i = 0; i < MT; ++i) part(ar[i], asr[i], b0, blocks, a[i], as[i]);
    }
    __device__ __forceinline__ static void part(const uint8_t *r, const uint8_t *sr, int b0, int blocks, u32x4_t (&v)[4], uint32_t &sc) {
        sc = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = b0 + s < blocks;
            const int b = in ? b0 + s : blocks - 1;
            v[s] = *reinterpret_cast<const u32x4_t *>(r + 16 * (int64_t)b);
            if (!in) v[s] = u32x4_t{0, 0, 0, 0};
            sc |= (in ? (uint32_t)sr[b] : 127u) << (8 * s);
        }
    }
    __device__ __forceinline__ void add(f32x4m_t (&acc)[NT][MT]) const {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                acc[i][j] = mfma16<0>(w[i][0], a[j][0], acc[i][j], ws[i], as[j]);
                acc[i][j] = mfma16<1>(w[i][1], a[j][1], acc[i][j], ws[i], as[j]);
                acc[i][j] = mfma16<2>(w[i][2], a[j][2], acc[i][j], ws[i], as[j]);
                acc[i][j] = mfma16<3>(w[i][3], a[j][3], acc[i][j], ws[i], as[j]);
            }
    }
};

template <int NT, int MT, int WAVES, class T>
__global__ void __launch_bounds__(64 * WAVES)
mxfp4_rows_kernel(const Mx p) {
    __shared__ f32x4m_t sums[WAVES][NT * MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n0 = (int)blockIdx.x * 16 * NT, blocks = p.K / 32, chunks = (blocks + 15) / 16;
    const int64_t pitch = p.K / 2;
    const uint8_t *wr[NT], *wsr[NT], *ar[MT], *asr[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t r = min(n0 + 16 * i + (lane & 15), p.N - 1);
        wr[i] = p.wc + r * pitch;
        wsr[i] = p.ws + r * blocks;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t r = min(16 * i + (lane & 15), p.M - 1);
        ar[i] = p.ac + r * pitch;
        asr[i] = p.as + r * blocks;
    }
    f32x4m_t acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = f32x4m_t{0, 0, 0, 0};
    Chunk<NT, MT> x;
    for (int c = wave; c < chunks; c += WAVES) {
        x.load(wr, wsr, ar, asr, c, blocks);
        x.add(acc);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) sums[wave][i * MT + j][lane] = acc[i][j];
    __syncthreads();
    // element e: n = e mod 16 NT, m = e div 16 NT; lane (n & 15) / 4 * 16 + (m & 15) holds it
    const float *flat = reinterpret_cast<const float *>(sums);
    for (int e = threadIdx.x; e < 16 * NT * min(16 * MT, p.M); e += 64 * WAVES) {
        const int n = e % (16 * NT), m = e / (16 * NT);
        if (n0 + n >= p.N) continue;
        const int at = (((n >> 4) * MT + (m >> 4)) * 64 + ((n & 15) >> 2) * 16 + (m & 15)) * 4 + (n & 3);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += flat[w * NT * MT * 256 + at];
        static_cast<T *>(p.y)[m * p.ys + n0 + n] = rounded<T>(v);
    }
}

// Rows of A that fit into LDS: a workgroup a CU holds them there, quantised by itself where
// they come as bf16, and its waves walk along W by themselves, 16 rows of it in chunks of
// 512 k, with kAhead chunks under way.  A workgroup's chunks, tile after tile, are one list,
// of which each wave takes an equal run; a tile belongs to the wave that begins it, and those
// that go on with it leave their sums in LDS.
// Step s of a chunk multiplies blocks 4 s + g in lanes l >> 4 == g, so that a load brings 64
// bytes in a row of each of 16 rows (16 bytes out of 64, four times and non-temporal: 122 us
// for the logits below, with plain loads 95, since L1 does not hold the lines that long).
// Blocks of a row of A lie an odd number of 16-byte slots apart from row to row, so that
// sixteen rows' reads of one block meet all banks.
// Bound by reading W, of which as many bytes are under way as the registers hold: 32 rows to
// 100001 columns of 5120 take 75 us, 3.7 TB/s (a plain read of W 51, 5.5 TB/s; the kernel
// above 110), one row to 13824 of 5120 10.0 us (11.0).  12 waves with four
// chunks under way 75.6 and 10.6, eight with six 83 and 10.3; rows quantised by a launch of
// their own 78.5 and 11.9.
constexpr int kAhead = 2, kHeldWaves = 16, kHeldThreads = 64 * kHeldWaves;
constexpr size_t kHeldLds = 160 * 1024;
struct Held {
    int chunks, pitch, spitch;      // chunks a row; from row to row: slots of codes, bytes of scales
    size_t sums, bytes;             // where the sums lie (behind A), and all of it
};
__host__ __device__ __forceinline__ Held held_of(int M, int K) {
    Held h;
    h.chunks = K / 512;
    h.pitch = 16 * h.chunks + 1;
    h.spitch = 16 * h.chunks + 4;
    h.sums = ((size_t)M * (16 * (size_t)h.pitch + h.spitch) + 15) / 16 * 16;
    h.bytes = h.sums + (size_t)kHeldWaves * (M > 16 ? 2 : 1) * 64 * 16;
    return h;
}

template <int MT, class T>
__global__ void __launch_bounds__(kHeldThreads)
mxfp4_held_kernel(const Mx p, int tiles) {
    extern __shared__ u32x4_t held_lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), g = lane >> 4;
    const Held h = held_of(p.M, p.K);
    const int blocks = p.K / 32;
    uint8_t *scales = reinterpret_cast<uint8_t *>(held_lds + p.M * h.pitch);
    f32x4m_t *sums = reinterpret_cast<f32x4m_t *>(reinterpret_cast<uint8_t *>(held_lds) + h.sums);
    // this workgroup's tiles of 16 columns, and this wave's run of their chunks
    const int wgs = (int)gridDim.x, each = tiles / wgs, rest = tiles % wgs, b = (int)blockIdx.x;
    const int t0 = b * each + min(b, rest), list = (each + (b < rest)) * h.chunks;
    const auto begins = [&](int w) { return w * (list / kHeldWaves) + min(w, list % kHeldWaves); };
    const int c0 = begins(wave), c1 = begins(wave + 1);

    u32x4_t w[kAhead][4], ws[kAhead];
    int at = t0 + c0 / h.chunks, ac = c0 % h.chunks;      // the tile and chunk to ask for next
    // By buffer loads: rows past the last and, without a request, chunks past the run (`left`
    // counts down to it) read as zeros, codes and scales, which add nothing.
    int left = c1 - c0;
    const int row = (lane & 15) * blocks;
    const auto ask = [&](int i) __attribute__((always_inline)) {
        const int64_t base = 16 * (int64_t)at * blocks + 16 * ac;
        const int here = left > 0 ? min(16, p.N - 16 * at) * blocks - 16 * ac : 0;      // blocks from there on
        const auto wr = buffer_of(p.wc + 16 * base, 16 * (int64_t)here);
        ws[i] = load16(buffer_of(p.ws + base, here), row);
#pragma unroll
        for (int s = 0; s < 4; ++s) w[i][s] = load16(wr, 16 * (row + g) + 64 * s);
        --left;
        if (++ac == h.chunks) {
            ac = 0;
            ++at;
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ask(i);

    // A into LDS, each row by as many waves as there are for it,
    // four chunks of a row at a time.  Of a chunk's scale bytes those of blocks g, 4 + g, ..
    // make up dword g.
    const int share = max(kHeldWaves / (p.M > 8 ? 16 : p.M > 4 ? 8 : p.M > 2 ? 4 : p.M), 1);
    for (int m = wave / share; m < p.M; m += kHeldWaves / share)
        for (int k = wave % share; k < h.chunks; k += 4 * share) {
            uint8_t *sc = scales + m * h.spitch;
            if (p.x) {
                u32x4_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)      // eight elements a lane
                    v[i] = *reinterpret_cast<const u32x4_t *>(p.x + m * p.xs + 8 * (64 * min(k + i * share, h.chunks - 1) + lane));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = k + i * share;
                    if (kk >= h.chunks) break;
                    uint32_t most = amax8(v[i]);
                    most = max(most, (uint32_t)__shfl_xor((int)most, 1, 64));
                    most = max(most, (uint32_t)__shfl_xor((int)most, 2, 64));
                    const uint32_t byte = scale_byte(most), c = codes8(v[i], scale_value(min(byte, 254u)));
                    reinterpret_cast<uint32_t *>(held_lds)[4 * m * h.pitch + 64 * kk + lane] = byte == 255u ? 0u : c;
                    if ((lane & 3) == 0) sc[16 * kk + (lane >> 2 & 3) * 4 + (lane >> 4)] = (uint8_t)byte;
                }
            } else if (lane < 16) {
                u32x4_t v[4];
                uint8_t e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {      // a block a lane
                    const int64_t j = (int64_t)m * blocks + 16 * min(k + i * share, h.chunks - 1) + lane;
                    v[i] = *reinterpret_cast<const u32x4_t *>(p.ac + 16 * j);
                    e[i] = p.as[j];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = k + i * share;
                    if (kk >= h.chunks) break;
                    held_lds[m * h.pitch + 16 * kk + lane] = v[i];
                    sc[16 * kk + (lane & 3) * 4 + (lane >> 2)] = e[i];
                }
            }
        }
    __syncthreads();
    int arow[MT], srow[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int m = min(16 * j + (lane & 15), p.M - 1);
        arow[j] = m * h.pitch + g;
        srow[j] = m * h.spitch + 4 * g;
    }
    f32x4m_t acc[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[j] = f32x4m_t{0, 0, 0, 0};
    int tile = t0 + c0 / h.chunks, c = c0 % h.chunks;
    bool leads = c != 0;      // the tile was begun by another wave
    const auto leave = [&] {
#pragma unroll
        for (int j = 0; j < MT; ++j) sums[(wave * MT + j) * 64 + lane] = acc[j];
    };
    const auto store = [&] {
        const int n = 16 * tile + 4 * g;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int m = 16 * j + (lane & 15);
            if (m >= p.M) continue;
            T *y = static_cast<T *>(p.y) + m * p.ys + n;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) y[e] = rounded<T>(acc[j][e]);
        }
    };
    for (int u = c0; u < c1; u += kAhead)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const u32x4_t e = ws[i] >> (uint32_t)(8 * g);
            const bool in = u + i < c1;
            const int k = in ? c : 0;      // past the run: zeros times any of A
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const u32x4_t *a = held_lds + arow[j] + 16 * k;
                const uint32_t as = *reinterpret_cast<const uint32_t *>(scales + srow[j] + 16 * k);
                acc[j] = mfma16<0, 0>(w[i][0], a[0], acc[j], e.x, as);
                acc[j] = mfma16<0, 1>(w[i][1], a[4], acc[j], e.y, as);
                acc[j] = mfma16<0, 2>(w[i][2], a[8], acc[j], e.z, as);
                acc[j] = mfma16<0, 3>(w[i][3], a[12], acc[j], e.w, as);
            }
            ask(i);
            __builtin_amdgcn_sched_barrier(0);      // the next chunk's reads of A would only take registers here
            c += in;
            if (c == h.chunks) {
                if (leads) leave();
                else store();
                leads = false;
                c = 0;
                ++tile;
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[j] = f32x4m_t{0, 0, 0, 0};
            }
        }
    if (leads) leave();      // the tile does not end here either
    __syncthreads();
    if (leads || c == 0) return;
    for (int v = wave + 1; v < kHeldWaves && begins(v) < (tile + 1 - t0) * h.chunks; ++v)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[j] += sums[(v * MT + j) * 64 + lane];
    store();
}

// ---------------------------------------------------------------- many rows
// A workgroup of WM x WN waves takes BM rows of A and BN of W.  Stages of 128 k go
// straight from memory to LDS, four of them under way: all workgroups of an XCD walk along
// K together, so every stage waits for lines that none of them has touched yet.
// Rows of a stage are 64 bytes in LDS, a quarter of the banks; block j of row r lies in slot
// j ^ (r >> 2 & 3), so that sixteen successive rows' reads of one block meet all banks.
// Lanes of half h multiply blocks 2 h and 2 h + 1 of a stage, one a step; their scale
// bytes are half a dword.  Scales come by 32 a row, for eight stages (a load of a dword a
// row costs as many requests to L2 as two stages' codes: one a stage 249 us for the last size
// below where four at a time took 205).
// Bound by the matrix instructions and what holds them up: 4096 x 8192 x 8192 takes 171 to
// 175 us of its own, 3.2 PFLOP/s, and 190 to 203 with the quantisation; the instruction alone on random
// operands 90 us (6.1 PFLOP/s, from registers) or 103 (from LDS).  Two buffers of 256 k
// instead 200 us with it where this one took 205; eight waves then 194, but their registers spill.
constexpr int kStages = 4;      // in LDS; the scales of kGroup of them come together

template <int BM, int BN>
struct StageLds {
    alignas(16) uint8_t x[(BM + BN) * 64];
};
// Scales of a group of stages, a row's 32 bytes in the order of its blocks.
template <int BM, int BN>
struct ScaleLds {
    alignas(16) uint8_t x[(BM + BN) * 32];
};

// Waits until at most N of the wave's loads are under way, and for its LDS reads and writes.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);
}
// 16 or 4 bytes a lane straight into LDS.
__device__ __forceinline__ void bring16(const uint8_t *from, int bytes, uint32_t off, uint8_t *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(from, bytes), (__attribute__((address_space(3))) void *)to, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void bring4(const uint8_t *from, int bytes, uint32_t off, uint8_t *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(from, bytes), (__attribute__((address_space(3))) void *)to, 4, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int BM, int BN, int WM, int WN>
struct Tile {
    static constexpr int THREADS = 64 * WM * WN, MT = BM / (32 * WM), NT = BN / (32 * WN);
    static constexpr int STEP = THREADS / 4, LOADS = (BM + BN) / STEP;      // rows that the threads bring at a time
    static constexpr int SROWS = THREADS / 8, SCALES = (BM + BN) / SROWS;       // likewise of scales
    using Stage = StageLds<BM, BN>;
    f32x16m_t acc[NT][MT];
    const uint8_t *a, *w, *sa, *sw;     // the tile's first rows
    int m, n, blocks, spitch;           // rows that are there, blocks a row, bytes from one row of scales to the next
    uint32_t from, sfrom;               // byte offsets of a thread's first codes and scales

    // The wave's first row of A and of W.
    __device__ __forceinline__ static int m_of() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) % WM * (32 * MT); }
    __device__ __forceinline__ static int n_of() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) / WM * (32 * NT); }
    // The block of a stage that a thread brings.
    __device__ __forceinline__ static int mine() { return (threadIdx.x & 3) ^ (threadIdx.x >> 4 & 3); }

    struct Scales {
        uint32_t a[MT], w[NT];      // of a stage, the lane's two in the low half
    };

    __device__ __forceinline__ void init(const Mx &p, int m0, int n0) {
        const uint32_t pitch = p.K / 2;
        blocks = p.K / 32;
        spitch = p.spitch;
        from = threadIdx.x / 4 * 16 * blocks + 16 * mine();
        sfrom = threadIdx.x / 8 * spitch + 4 * (threadIdx.x & 7);
        m = min(BM, p.M - m0);
        n = min(BN, p.N - n0);
        a = p.ac + (int64_t)m0 * pitch;
        sa = p.as + (int64_t)m0 * spitch;
        w = p.wc + (int64_t)n0 * pitch;
        sw = p.ws + (int64_t)n0 * spitch;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    }

    // Stage t on its way into LDS in LOADS parts.  Buffer loads: rows past the last come as
    // zeros.  So do blocks past a row's last, in A by an offset that is past everything; in W
    // they are whatever follows, which A's zeros make nothing of.
    struct Request {
        const uint8_t *a, *w;
        int bytes_a, bytes_w;      // up to the tile's end
        uint8_t *to;
        uint32_t from_a, from_w;
    };
    __device__ __forceinline__ Request request(Stage &lds, int t) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        const int64_t at = 64 * (int64_t)t, pitch = 16 * (int64_t)blocks;
        return Request{a + at, w + at, (int)max(m * pitch - at, (int64_t)0), (int)max(n * pitch - at, (int64_t)0), &lds.x[1024 * wave],
                       4 * t + mine() < blocks ? from : (uint32_t)kOob, from};
    }
    __device__ __forceinline__ void load(const Request &r, int i) const {
        const bool is_a = STEP * i < BM;
        const uint32_t pitch = 16 * blocks, off = is_a ? r.from_a + STEP * i * pitch : r.from_w + (STEP * i - BM) * pitch;
        bring16(is_a ? r.a : r.w, is_a ? r.bytes_a : r.bytes_w, off, r.to + 16 * THREADS * i);
    }
    // Part i of SCALES of the scales of group t: a dword a lane, since rows of them begin at
    // multiples of four bytes.  Past a row's end they are zeros (2^-127), in both, lest the
    // next row's NaN come in.
    __device__ __forceinline__ void load_scales(ScaleLds<BM, BN> &lds, int t, int i) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        const bool is_a = SROWS * i < BM;
        const int64_t at = 32 * (int64_t)t, pitch = spitch;
        bring4((is_a ? sa : sw) + at, (int)((is_a ? m : n) * pitch - at), 32 * t + 4 * (int)(threadIdx.x & 7) < blocks ? sfrom + (SROWS * i - (is_a ? 0 : BM)) * spitch : (uint32_t)kOob,
               &lds.x[4 * THREADS * i + 256 * wave]);
    }
    // Dwords of its stage q.
    __device__ __forceinline__ static uint32_t scale_at(const ScaleLds<BM, BN> &lds, int r, int q) {
        const int lane = threadIdx.x & 63;
        return *reinterpret_cast<const uint32_t *>(&lds.x[32 * (r + (lane & 31)) + 4 * q]);
    }
    __device__ __forceinline__ void get_scales(const ScaleLds<BM, BN> &lds, int q, Scales &sc) const {
#pragma unroll
        for (int i = 0; i < MT; ++i) sc.a[i] = scale_at(lds, m_of() + 32 * i, q);
#pragma unroll
        for (int i = 0; i < NT; ++i) sc.w[i] = scale_at(lds, BM + n_of() + 32 * i, q);
    }
    // Dwords as read, to the lane's two bytes.
    __device__ __forceinline__ static void halve(Scales &sc) {
        const int shift = (threadIdx.x & 63) >> 5 << 4;
#pragma unroll
        for (int i = 0; i < MT; ++i) sc.a[i] >>= shift;
#pragma unroll
        for (int i = 0; i < NT; ++i) sc.w[i] >>= shift;
    }
    // Operands of a step of a stage.
    struct Frags {
        u32x4_t a[MT], w[NT];
    };
    template <int S>
    __device__ __forceinline__ static u32x4_t at(const Stage &lds, int r) {
        const int lane = threadIdx.x & 63, j = 2 * (lane >> 5) + S, row = r + (lane & 31);
        return *reinterpret_cast<const u32x4_t *>(&lds.x[row * 64 + 16 * (j ^ (row >> 2 & 3))]);
    }
    template <int S>
    __device__ __forceinline__ void read(const Stage &lds, Frags &f, int i) const {
        if (i < MT) f.a[i] = at<S>(lds, m_of() + 32 * i);
        if (i < NT) f.w[i] = at<S>(lds, BM + n_of() + 32 * i);
    }
    // Step S by groups of MT products, and between them reads of the operands of the step
    // after it (step 1 - S of `lds`) and, in the second step, the parts of a request (all
    // at once they hold up the wave).  Nothing moves over a group's end: left alone, the
    // compiler reads all operands first or multiplies behind the next wait.
    template <int S, class More>
    __device__ __forceinline__ void step(const Frags &f, const Scales &sc, const Stage &lds, Frags &next, const Request *r, More more) {
        constexpr int EACH = LOADS / NT;
        static_assert(MT <= NT && LOADS % NT == 0, "a group a fragment, as many parts of the request in each");
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (2 * i < NT) {      // early: the next step begins with them
                read<1 - S>(lds, next, 2 * i);
                read<1 - S>(lds, next, 2 * i + 1);
            }
            if (r)
#pragma unroll
                for (int k = 0; k < EACH; ++k) load(*r, EACH * i + k);
            more(i);
#pragma unroll
            for (int k = 0; k < MT; ++k) acc[i][k] = mfma32<S>(f.a[k], f.w[i], acc[i][k], sc.a[k], sc.w[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Tile `at` of mt x nt: each of the 8 XCDs (workgroups go round them) takes a run of
// tiles, in blocks of 8 rows of A's tiles, so that its L2 holds what its tiles share.
__device__ __forceinline__ void tile_of(int at, int mt, int nt, int &m, int &n) {
    const int all = mt * nt, each = all / 8, rest = all % 8, x = at % 8;
    const int t = x * each + min(x, rest) + at / 8;
    const int group = t / (8 * nt), first = group * 8, rows = min(8, mt - first), in = t - group * 8 * nt;
    m = first + in % rows;
    n = in / rows;
}

template <int BM, int BN, int WM, int WN, class T>
__global__ void __launch_bounds__(64 * WM * WN)
mxfp4_tiles_kernel(const Mx p, int mtiles) {
    __shared__ StageLds<BM, BN> lds0, lds1, lds2, lds3;      // apart: the compiler knows which the loads go to
    __shared__ ScaleLds<BM, BN> scales0, scales1;
    using X = Tile<BM, BN, WM, WN>;
    const int piece = (int)(blockIdx.x % p.pieces), at = (int)(blockIdx.x / p.pieces);
    int m0, n0;
    tile_of(at, mtiles, (p.N + BN - 1) / BN, m0, n0);
    m0 *= BM;
    n0 *= BN;
    const int groups = (p.K / 32 + 4 * kGroup - 1) / (4 * kGroup);      // of stages
    const int each = (groups + p.pieces - 1) / p.pieces;
    const int g0 = min(piece * each, groups), g1 = min(g0 + each, groups);
    X x;
    x.init(p, m0, n0);
    if (g0 < g1) {
        constexpr int L = X::LOADS, SC = X::SCALES / 4;      // the next group's scales come in four of the stages
        static_assert(SC % X::NT == 0 || X::NT % SC == 0, "spread over a step's groups");
        const int last = kGroup * g1 - 1;
        typename X::Scales now, then;
        typename X::Frags f, g;
        const auto bring = [&](StageLds<BM, BN> &lds, int t) {
            const auto r = x.request(lds, t);
#pragma unroll
            for (int i = 0; i < L; ++i) x.load(r, i);
        };
#pragma unroll
        for (int i = 0; i < X::SCALES; ++i) x.load_scales(scales0, g0, i);
        bring(lds0, kGroup * g0);
        bring(lds1, kGroup * g0 + 1);
        bring(lds2, kGroup * g0 + 2);
        bring(lds3, kGroup * g0 + 3);
        wait_loads<3 * L>();
        meet();
        x.get_scales(scales0, 0, now);
        X::halve(now);
#pragma unroll
        for (int i = 0; i < X::NT; ++i) x.template read<0>(lds0, f, i);
        const auto nothing = [](int) __attribute__((always_inline)) {};
        // Stage q of group u in `here`, the next one in `next`.  Between its two steps the
        // wave's loads of the next stage are done (of later ones: two stages' codes, and the
        // scales that the two stages before asked for), and all waves have read the last of
        // `here`, which takes the fourth stage from now.  Past the last one it is asked for
        // again: a branch would let the compiler move the products.
        const auto stage = [&](auto q, StageLds<BM, BN> &here, const StageLds<BM, BN> &next, int u,
                               const ScaleLds<BM, BN> &mine, ScaleLds<BM, BN> &coming) __attribute__((always_inline)) {
            constexpr int Q = decltype(q)::value;
            constexpr int LATER = 2 * L + SC * ((Q >= 1 && Q <= 4) + (Q >= 2 && Q <= 5));
            x.template step<0>(f, now, here, g, nullptr, nothing);
            wait_loads<LATER>();
            meet();
            const auto r = x.request(here, min(kGroup * u + Q + kStages, last));
            if constexpr (Q + 1 < kGroup) x.get_scales(mine, Q + 1, then);
            else x.get_scales(coming, 0, then);
            x.template step<1>(g, now, next, f, &r, [&](int i) __attribute__((always_inline)) {
                if constexpr (Q < 4) {
#pragma unroll
                    for (int k = 0; k < SC; ++k)
                        if (k % X::NT == i) x.load_scales(coming, min(u + 1, g1 - 1), SC * Q + k);
                }
            });
            now = then;
            X::halve(now);
        };
        const auto group = [&](int u, const ScaleLds<BM, BN> &mine, ScaleLds<BM, BN> &coming) __attribute__((always_inline)) {
            stage(std::integral_constant<int, 0>(), lds0, lds1, u, mine, coming);
            stage(std::integral_constant<int, 1>(), lds1, lds2, u, mine, coming);
            stage(std::integral_constant<int, 2>(), lds2, lds3, u, mine, coming);
            stage(std::integral_constant<int, 3>(), lds3, lds0, u, mine, coming);
            stage(std::integral_constant<int, 4>(), lds0, lds1, u, mine, coming);
            stage(std::integral_constant<int, 5>(), lds1, lds2, u, mine, coming);
            stage(std::integral_constant<int, 6>(), lds2, lds3, u, mine, coming);
            stage(std::integral_constant<int, 7>(), lds3, lds0, u, mine, coming);
        };
        int u = g0;
        for (; u + 1 < g1; u += 2) {
            group(u, scales0, scales1);
            group(u + 1, scales1, scales0);
        }
        for (; u < g1; ++u) group(u, scales0, scales1);      // once at most; as a plain branch it costs the compiler registers
        wait_loads<0>();
    }
    // a lane holds one n of 16 m
    const int lane = threadIdx.x & 63, m1 = m0 + X::m_of() + 4 * (lane >> 5), n1 = n0 + X::n_of() + (lane & 31);
#pragma unroll
    for (int k = 0; k < X::MT; ++k)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int m = m1 + 32 * k + 8 * (e >> 2) + (e & 3);
            if (m >= p.M) continue;
            float *part = p.part + ((int64_t)piece * p.M + m) * p.N;
            T *y = static_cast<T *>(p.y) + m * p.ys;
#pragma unroll
            for (int i = 0; i < X::NT; ++i) {
                const int n = n1 + 32 * i;
                if (n >= p.N) continue;
                if (p.part) part[n] = x.acc[i][k][e];
                else y[n] = rounded<T>(x.acc[i][k][e]);
            }
        }
}

template <class T>
__global__ void __launch_bounds__(256)
mxfp4_join_kernel(const Mx p) {
    const int64_t n = (int64_t)p.M * p.N;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        float v = 0.0f;
        for (int i = 0; i < p.pieces; ++i) v += p.part[i * n + e];
        const int64_t m = e / p.N;
        static_cast<T *>(p.y)[m * p.ys + (e - m * p.N)] = rounded<T>(v);
    }
}

// Rows of scales to rows that begin at multiples of four bytes, zeros at their ends.
__global__ void __launch_bounds__(256)
mxfp4_scales_kernel(const uint8_t *__restrict__ a, int M, const uint8_t *__restrict__ w, int N, int blocks, uint32_t *__restrict__ out) {
    const int dwords = (blocks + 3) / 4;
    const int64_t n = ((int64_t)M + N) * dwords;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t row = e / dwords;
        const int j = (int)(e - row * dwords);
        const uint8_t *from = row < M ? a + row * blocks : w + (row - M) * blocks;
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * j + i < blocks) v |= (uint32_t)from[4 * j + i] << (8 * i);
        out[e] = v;
    }
}

// Every workgroup quantises all of A, which pays where it has much of W to read or A is
// short.  M rows of K to N, held against streamed, on twelve weights in turn (one row to 13824
// on three, which stay in the last cache, 10.0 and 11.0): 1 x 5120 to 5120 8.0 and 8.0 us, 8 rows 9.4
// and 9.0, 32 rows 15.0 and 10.9; to 13824 1 row 12.0 and 12.9, 8 rows 13.5 and 14.9, 32 rows
// 20.0 and 20.5; 8192 to 8192 1 row 11.5 and 13.2, 16 rows 16.8 and 15.9.
bool held(int M, int N, int K) {
    return M <= kRows && (M <= 4 || N >= 48 * kCUs) && K % 512 == 0 && held_of(M, K).bytes <= kHeldLds;
}
// Of A's and W's rows of scales in multiples of four bytes, where they are not so already.
size_t padded_bytes(int64_t M, int64_t N, int K) {
    const int64_t blocks = K / 32;
    return M <= kRows || blocks % 4 == 0 ? 0 : (size_t)((M + N) * ((blocks + 3) / 4 * 4) + 255) / 256 * 256;
}
size_t codes_bytes(int64_t M, int64_t K) { return ((size_t)(M * (K / 2)) + 255) / 256 * 256; }
size_t scales_bytes(int64_t M, int64_t K) { return ((size_t)(M * (K / 32)) + 255) / 256 * 256; }

// Columns of a launch: 2^27 take more threads (512 for 16 of them) than it can count.
constexpr int64_t kMostColumns = 1 << 26;
template <int NT, int MT, int WAVES>
void rows_launch(const Mx &all, bool fp32, hipStream_t stream) {
    for (int64_t n0 = 0; n0 < all.N; n0 += kMostColumns) {
        Mx p = all;
        p.N = (int)(all.N - n0 < kMostColumns ? all.N - n0 : kMostColumns);
        p.wc += n0 * (p.K / 2);
        p.ws += n0 * (p.K / 32);
        p.y = static_cast<char *>(p.y) + n0 * (fp32 ? 4 : 2);
        const unsigned grid = (unsigned)((p.N + 16 * NT - 1) / (16 * NT));
        if (fp32) hipLaunchKernelGGL((mxfp4_rows_kernel<NT, MT, WAVES, float>), dim3(grid), dim3(64 * WAVES), 0, stream, p);
        else hipLaunchKernelGGL((mxfp4_rows_kernel<NT, MT, WAVES, uint16_t>), dim3(grid), dim3(64 * WAVES), 0, stream, p);
    }
}
template <int MT, class T>
hipError_t held_launch(const Mx &p, hipStream_t stream) {
    const int lds = (int)held_of(p.M, p.K).bytes, tiles = (p.N + 15) / 16;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(mxfp4_held_kernel<MT, T>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)kHeldLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mxfp4_held_kernel<MT, T>), dim3(tiles < kCUs ? tiles : kCUs), dim3(kHeldThreads), lds, stream, p, tiles);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN>
hipError_t tiles_launch(const Mx &p, bool fp32, hipStream_t stream) {
    const int mt = (p.M + BM - 1) / BM;
    const int64_t grid = (int64_t)mt * ((p.N + BN - 1) / BN) * p.pieces;
    if (!fits_grid(grid, 64 * WM * WN)) return hipErrorInvalidValue;
    const dim3 threads(64 * WM * WN);
    if (fp32) hipLaunchKernelGGL((mxfp4_tiles_kernel<BM, BN, WM, WN, float>), dim3((unsigned)grid), threads, 0, stream, p, mt);
    else hipLaunchKernelGGL((mxfp4_tiles_kernel<BM, BN, WM, WN, uint16_t>), dim3((unsigned)grid), threads, 0, stream, p, mt);
    return hipGetLastError();
}

}  // namespace

bool mxfp4_fits(int M, int N, int K) {
    if (M == 0) return true;
    const MxPlan p = plan_of(M, N, K);
    const int64_t b = p.rows ? 1 : p.bm, tiles = p.rows ? 1 : ((M + b - 1) / b) * ((N + b - 1) / b);
    return mxfp4_rows_fit(M, K) && fits_grid(tiles * p.pieces, 256);
}
size_t mxfp4_plan_bytes(int M, int N, int K, bool quant) {
    return plan_of(M, N, K).part_bytes + padded_bytes(M, N, K) + (quant ? codes_bytes(M, K) + scales_bytes(M, K) : 0);
}
// For every call of up to M rows: only where there are fewer than kWant tiles of 128
// is K cut, into at most 3/2 kWant pieces of tiles in all.
size_t mxfp4_ws_bytes(int M, int N, int K) {
    size_t most = 0;
    for (int64_t m = 128;; m += 128) {
        const int64_t at = m < M ? m : M;
        const MxPlan p = plan_of((int)at, N, K);
        if (p.part_bytes > most) most = p.part_bytes;
        if (m >= M || (!p.rows && ((at + 127) / 128) * ((N + 127) / 128) >= kWant)) break;
    }
    return most + padded_bytes(M, N, K) + codes_bytes(M, K) + scales_bytes(M, K);
}

hipError_t launch_gemm_mxfp4(const MxGemmArgs &a, hipStream_t stream) {
    const MxPlan plan = plan_of(a.M, a.N, a.K);
    const uint8_t *ac = a.a_codes, *as = a.a_scales;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const bool holds = held(a.M, a.N, a.K), own = a.x && holds;
    if (a.x && !own) {
        uint8_t *c = ws, *s = ws + codes_bytes(a.M, a.K);
        ws = s + scales_bytes(a.M, a.K);
        const hipError_t e = launch_quant_mxfp4(a.x, a.x_stride, false, a.M, a.K, c, s, stream);
        if (e != hipSuccess) return e;
        ac = c;
        as = s;
    }
    const uint8_t *wsc = a.w_scales;
    int pitch = a.K / 32;
    if (const size_t n = padded_bytes(a.M, a.N, a.K)) {
        const int64_t dwords = (int64_t)(n / 4), grid = (dwords + 255) / 256;
        hipLaunchKernelGGL(mxfp4_scales_kernel, dim3((unsigned)(grid < 4096 ? grid : 4096)), dim3(256), 0, stream, as, a.M, wsc, a.N,
                           pitch, reinterpret_cast<uint32_t *>(ws));
        pitch = (pitch + 3) / 4 * 4;
        as = ws;
        wsc = ws + (int64_t)a.M * pitch;
        ws += n;
    }
    const Mx p{ac, as, a.w_codes, wsc, own ? a.x : nullptr, a.x_stride, a.M, a.N, a.K, pitch, a.y, a.y_stride,
               plan.pieces > 1 ? reinterpret_cast<float *>(ws) : nullptr, plan.pieces};
    if (holds) {
        if (a.M <= 16) return a.y_fp32 ? held_launch<1, float>(p, stream) : held_launch<1, uint16_t>(p, stream);
        return a.y_fp32 ? held_launch<2, float>(p, stream) : held_launch<2, uint16_t>(p, stream);
    }
    if (plan.rows) {
        if (a.M <= 16) rows_launch<1, 1, 8>(p, a.y_fp32, stream);
        else rows_launch<2, 2, 8>(p, a.y_fp32, stream);
        return hipGetLastError();
    }
    const hipError_t e = plan.bm == 256 ? tiles_launch<256, 256, 2, 2>(p, a.y_fp32, stream)
                                          : tiles_launch<128, 128, 2, 2>(p, a.y_fp32, stream);
    if (e != hipSuccess || plan.pieces == 1) return e;
    const int64_t n = ((int64_t)a.M * a.N + 255) / 256;
    const unsigned grid = (unsigned)(n < 4096 ? n : 4096);
    if (a.y_fp32) hipLaunchKernelGGL((mxfp4_join_kernel<float>), dim3(grid), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((mxfp4_join_kernel<uint16_t>), dim3(grid), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace biloco
