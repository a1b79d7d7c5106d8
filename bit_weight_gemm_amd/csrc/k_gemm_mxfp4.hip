// y = A W^T of microscaled 4-bit operands on the scaled matrix instructions of gfx950,
// which take E2M1 codes and one scale byte for 32 of them as they are.
//
//   y[m][n] = sum over blocks b of 2^(sa[m][b] + sw[n][b] - 254) sum_k a[m][k] w[n][k]
//
// Sums are fp32 (the instruction adds a block's exact sum).  A scale byte of 255 makes
// its row NaN.
#include "mx_device.h"

namespace biloco {

namespace {

using namespace mx;

// Operands, outputs and sizes of a call.
struct Mx {
    const uint8_t *ac, *as, *wc, *ws;
    int M, N, K;
    void *y;
    int64_t ys;
    float *part;      // sums of the pieces of K, [piece][M][N], or NULL
    int pieces;
};

__device__ __forceinline__ i32x8m_t frag(const u32x4_t &v) {
    return i32x8m_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
template <int S>
__device__ __forceinline__ f32x4m_t mfma16(const u32x4_t &a, const u32x4_t &b, f32x4m_t c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(a), frag(b), c, 4, 4, S, (int)sa, S, (int)sb);
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
    if constexpr (sizeof(T) == 2) return f32_to_bf16_rne(v);
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

// ---------------------------------------------------------------- many rows
// A workgroup of four waves takes BM rows of A and BN of W, a wave a quarter; stages of
// 256 k go straight from memory to LDS, the next one while this one is multiplied.
// Rows of a stage are 128 bytes in LDS, half of the banks; block j of row r lies in slot
// j ^ (r >> 1 & 7), so that sixteen successive rows' reads of one block meet all banks.
// Lanes of half h multiply blocks 4 h .. 4 h + 3 of a stage, one a step, whose four scale
// bytes are one dword.  Four stages are taken together, 1024 k: stage s has blocks 4 s ..
// of the first 16 for h = 0 and of the others for h = 1, so that a lane's scales of four
// stages are 16 bytes.  (A load of a dword a row costs as many requests to L2 as a stage's
// codes: with one a stage 249 us for 4096 rows of 8192 to 8192.)
template <int BM, int BN>
struct StageLds {
    alignas(16) uint8_t x[(BM + BN) * 128];
};

template <int BM, int BN>
struct Tile {
    static constexpr int MT = BM / 64, NT = BN / 64, LOADS = (BM + BN) / 32;
    f32x16m_t acc[NT][MT];
    uint32_t from[LOADS];                   // byte offsets of a wave's pieces from the tile's rows
    uint32_t afrom[MT], wfrom[NT];          // of its scales
    const uint8_t *a, *w, *sa, *sw;         // the tile's first rows

    struct Scales {
        u32x4_t a[MT], w[NT];               // a dword a stage
    };

    __device__ __forceinline__ void init(const Mx &p, int m0, int n0) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const uint32_t pitch = p.K / 2, blocks = p.K / 32;
        a = p.ac + (int64_t)m0 * pitch;
        sa = p.as + (int64_t)m0 * blocks;
        w = p.wc + (int64_t)n0 * pitch;
        sw = p.ws + (int64_t)n0 * blocks;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = 32 * i + tid / 8;
            const bool is_a = 32 * i < BM;
            from[i] = (uint32_t)(is_a ? min(row, p.M - 1 - m0) : min(row - BM, p.N - 1 - n0)) * pitch;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
            afrom[i] = (uint32_t)min((wave & 1) * (BM / 2) + 32 * i + (lane & 31), p.M - 1 - m0) * blocks;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            wfrom[i] = (uint32_t)min((wave >> 1) * (BN / 2) + 32 * i + (lane & 31), p.N - 1 - n0) * blocks;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    }
    // The block of a stage that a thread brings.
    __device__ __forceinline__ static int mine() { return (threadIdx.x & 7) ^ (threadIdx.x >> 4 & 7); }

    // Stage s of the four at 1024 t, on its way into LDS.
    __device__ __forceinline__ void request(StageLds<BM, BN> &lds, int t, int s) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), j = mine();
        const uint32_t in = 256 * (j >> 2) + 16 * (j & 3);
        const uint8_t *ga = a + 512 * (int64_t)t + 64 * s, *gw = w + 512 * (int64_t)t + 64 * s;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)((32 * i < BM ? ga : gw) + from[i] + in),
                                             (__attribute__((address_space(3))) void *)&lds.x[4096 * i + 1024 * wave], 16, 0, 0);
    }
    __device__ __forceinline__ void scales(int t, Scales &sc) const {
        const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int i = 0; i < MT; ++i) __builtin_memcpy(&sc.a[i], sa + 32 * (int64_t)t + 16 * h + afrom[i], 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) __builtin_memcpy(&sc.w[i], sw + 32 * (int64_t)t + 16 * h + wfrom[i], 16);
    }
    // Eight blocks from b0 on, of which those past the last are zeros with scale 1: through
    // registers.
    __device__ __forceinline__ void request_part(StageLds<BM, BN> &lds, int b0, int blocks) const {
        const int tid = threadIdx.x, b = b0 + mine();
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            u32x4_t v{0, 0, 0, 0};
            if (b < blocks) v = *reinterpret_cast<const u32x4_t *>((32 * i < BM ? a : w) + from[i] + 16 * (int64_t)b);
            *reinterpret_cast<u32x4_t *>(&lds.x[4096 * i + 16 * tid]) = v;
        }
    }
    __device__ __forceinline__ static uint32_t scales_of(const uint8_t *p, int b0, int blocks) {
        uint32_t v = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) v |= (b0 + s < blocks ? (uint32_t)p[b0 + s] : 127u) << (8 * s);
        return v;
    }
    __device__ __forceinline__ void scales_part(int b0, int blocks, Scales &sc) const {
        const int b = b0 + 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
        for (int i = 0; i < MT; ++i) sc.a[i].x = scales_of(sa + afrom[i], b, blocks);
#pragma unroll
        for (int i = 0; i < NT; ++i) sc.w[i].x = scales_of(sw + wfrom[i], b, blocks);
    }

    // Operands of step S of a stage.
    struct Frags {
        u32x4_t a[MT], w[NT];
    };
    template <int S>
    __device__ __forceinline__ void read(const StageLds<BM, BN> &lds, Frags &f) const {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), j = 4 * (lane >> 5) + S;
        const int ra = (wave & 1) * (BM / 2) + (lane & 31), rw = BM + (wave >> 1) * (BN / 2) + (lane & 31);
#pragma unroll
        for (int i = 0; i < MT; ++i) f.a[i] = *reinterpret_cast<const u32x4_t *>(&lds.x[(ra + 32 * i) * 128 + 16 * (j ^ (ra >> 1 & 7))]);
#pragma unroll
        for (int i = 0; i < NT; ++i) f.w[i] = *reinterpret_cast<const u32x4_t *>(&lds.x[(rw + 32 * i) * 128 + 16 * (j ^ (rw >> 1 & 7))]);
    }
    // Step S of stage Q; R of the next step's operands are read meanwhile.
    template <int S, int Q, int R>
    __device__ __forceinline__ void products(const Frags &f, const Scales &sc) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < MT; ++k) acc[i][k] = mfma32<S>(f.a[k], f.w[i], acc[i][k], sc.a[k][Q], sc.w[i][Q]);
        // reads between the first products, and nothing moves over the step's end: left
        // alone, the compiler reads all operands first or multiplies behind the wait for
        // the next stage
#pragma unroll
        for (int i = 0; i < R; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // an LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // a matrix instruction
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    template <int Q>
    __device__ __forceinline__ void multiply(const StageLds<BM, BN> &lds, const Scales &sc) {
        Frags f, g;
        read<0>(lds, f);
        __builtin_amdgcn_sched_barrier(0);
        read<1>(lds, g);
        products<0, Q, MT + NT>(f, sc);
        read<2>(lds, f);
        products<1, Q, MT + NT>(g, sc);
        read<3>(lds, g);
        products<2, Q, MT + NT>(f, sc);
        products<3, Q, 0>(g, sc);
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

template <int BM, int BN, class T>
__global__ void __launch_bounds__(256)
mxfp4_tiles_kernel(const Mx p, int mtiles) {
    __shared__ StageLds<BM, BN> lds0, lds1;
    using X = Tile<BM, BN>;
    const int piece = (int)(blockIdx.x % p.pieces), at = (int)(blockIdx.x / p.pieces);
    int m0, n0;
    tile_of(at, mtiles, (p.N + BN - 1) / BN, m0, n0);
    m0 *= BM;
    n0 *= BN;
    const int blocks = p.K / 32, fours = blocks / 32;      // blocks, and stages by four
    const int each = (fours + p.pieces - 1) / p.pieces;
    const int t0 = min(piece * each, fours), t1 = min(t0 + each, fours);
    X x;
    x.init(p, m0, n0);
    typename X::Scales sc, next;
    if (t0 < t1) {
        x.request(lds0, t0, 0);
        x.scales(t0, next);
    }
    for (int t = t0; t < t1; ++t) {
        // the last turn asks for its own stage again: a branch here would let the
        // compiler move the products behind the loads' end
        const int u = min(t + 1, t1 - 1);
        __syncthreads();      // the requested stage is in place, the other buffer has been read
        sc = next;
        x.request(lds1, t, 1);
        x.template multiply<0>(lds0, sc);
        __syncthreads();
        x.request(lds0, t, 2);
        x.template multiply<1>(lds1, sc);
        __syncthreads();
        x.request(lds1, t, 3);
        x.template multiply<2>(lds0, sc);
        __syncthreads();
        x.request(lds0, u, 0);
        x.scales(u, next);
        x.template multiply<3>(lds1, sc);
    }
    if (piece == p.pieces - 1)      // what is left of K, stage by stage
        for (int b = 32 * fours; b < blocks; b += 8) {
            __syncthreads();
            x.request_part(lds0, b, blocks);
            x.scales_part(b, blocks, sc);
            __syncthreads();
            x.template multiply<0>(lds0, sc);
        }
    // a lane holds one n of 16 m
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int m1 = m0 + (wave & 1) * (BM / 2) + 4 * (lane >> 5), n1 = n0 + (wave >> 1) * (BN / 2) + (lane & 31);
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

constexpr int kRows = 32;              // rows of A up to which W is streamed
constexpr int kWant = 256;             // workgroups that the pieces of K are to make

struct MxPlan {
    bool rows;
    int bm, bn, pieces;
    size_t part_bytes;
};
MxPlan plan_of(int M, int N, int K) {
    MxPlan p{M <= kRows, 0, 0, 1, 0};
    if (p.rows) return p;
    const auto tiles = [&](int b) { return (int64_t)((M + b - 1) / b) * ((N + b - 1) / b); };
    p.bm = p.bn = tiles(256) >= 256 ? 256 : 128;
    const int64_t n = tiles(p.bm);
    int64_t pieces = n >= kWant ? 1 : (2 * kWant) / n;
    const int64_t most = K / 1024;      // at least four stages a piece
    if (pieces > most) pieces = most;
    p.pieces = pieces < 1 ? 1 : (int)pieces;
    if (p.pieces > 1) p.part_bytes = (size_t)p.pieces * M * N * 4;
    return p;
}
size_t codes_bytes(int64_t M, int64_t K) { return ((size_t)(M * (K / 2)) + 255) / 256 * 256; }
size_t scales_bytes(int64_t M, int64_t K) { return ((size_t)(M * (K / 32)) + 255) / 256 * 256; }

template <int NT, int MT, int WAVES>
void rows_launch(const Mx &p, bool fp32, hipStream_t stream) {
    const unsigned grid = (unsigned)((p.N + 16 * NT - 1) / (16 * NT));
    if (fp32) hipLaunchKernelGGL((mxfp4_rows_kernel<NT, MT, WAVES, float>), dim3(grid), dim3(64 * WAVES), 0, stream, p);
    else hipLaunchKernelGGL((mxfp4_rows_kernel<NT, MT, WAVES, uint16_t>), dim3(grid), dim3(64 * WAVES), 0, stream, p);
}
template <int BM, int BN>
hipError_t tiles_launch(const Mx &p, bool fp32, hipStream_t stream) {
    const int mt = (p.M + BM - 1) / BM;
    const int64_t grid = (int64_t)mt * ((p.N + BN - 1) / BN) * p.pieces;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (fp32) hipLaunchKernelGGL((mxfp4_tiles_kernel<BM, BN, float>), dim3((unsigned)grid), dim3(256), 0, stream, p, mt);
    else hipLaunchKernelGGL((mxfp4_tiles_kernel<BM, BN, uint16_t>), dim3((unsigned)grid), dim3(256), 0, stream, p, mt);
    return hipGetLastError();
}

}  // namespace

size_t mxfp4_plan_bytes(int M, int N, int K, bool quant) {
    return plan_of(M, N, K).part_bytes + (quant ? codes_bytes(M, K) + scales_bytes(M, K) : 0);
}
// For every call of up to M rows: only where there are fewer than kWant tiles of 128
// is K cut, into at most 2 kWant pieces of tiles in all.
size_t mxfp4_ws_bytes(int M, int N, int K) {
    size_t most = 0;
    for (int64_t m = 128;; m += 128) {
        const int64_t at = m < M ? m : M;
        const MxPlan p = plan_of((int)at, N, K);
        if (p.part_bytes > most) most = p.part_bytes;
        if (m >= M || (!p.rows && ((at + 127) / 128) * ((N + 127) / 128) >= kWant)) break;
    }
    return most + codes_bytes(M, K) + scales_bytes(M, K);
}

hipError_t launch_gemm_mxfp4(const MxGemmArgs &a, hipStream_t stream) {
    const MxPlan plan = plan_of(a.M, a.N, a.K);
    const uint8_t *ac = a.a_codes, *as = a.a_scales;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    if (a.x) {
        uint8_t *c = ws, *s = ws + codes_bytes(a.M, a.K);
        ws = s + scales_bytes(a.M, a.K);
        const hipError_t e = launch_quant_mxfp4(a.x, a.x_stride, false, a.M, a.K, c, s, stream);
        if (e != hipSuccess) return e;
        ac = c;
        as = s;
    }
    const Mx p{ac, as, a.w_codes, a.w_scales, a.M, a.N, a.K, a.y, a.y_stride,
               plan.pieces > 1 ? reinterpret_cast<float *>(ws) : nullptr, plan.pieces};
    if (plan.rows) {
        if (a.M <= 16) rows_launch<1, 1, 8>(p, a.y_fp32, stream);
        else rows_launch<2, 2, 8>(p, a.y_fp32, stream);
        return hipGetLastError();
    }
    const hipError_t e = plan.bm == 256 ? tiles_launch<256, 256>(p, a.y_fp32, stream) : tiles_launch<128, 128>(p, a.y_fp32, stream);
    if (e != hipSuccess || plan.pieces == 1) return e;
    const int64_t n = ((int64_t)a.M * a.N + 255) / 256;
    const unsigned grid = (unsigned)(n < 4096 ? n : 4096);
    if (a.y_fp32) hipLaunchKernelGGL((mxfp4_join_kernel<float>), dim3(grid), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((mxfp4_join_kernel<uint16_t>), dim3(grid), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace biloco
