// A token for each row of logits: softmax at a temperature, cut to the top k, to the
// smallest set of mass p, to weights of at least m of the largest, drawn with a given
// number u.
//
//   y_i = (top - x_i) log2(e) / T,  w_i = 2^-y_i in steps of 2^-44
//   order: x descending, equal ones by index; key (x, index) of the last one kept by k,
//   then by p; among the kept with w_i >= m: the first i with sum_{j <= i} w_j > u sum w
//
// Weights are 64-bit whole numbers, so every sum is exact and no order of adding changes
// a result.  Nothing is sorted: a histogram over y (counts and weights of 2048 equal
// parts) says which part holds a border, and only the elements of such parts are
// compared with one another.  Few elements up to the border: all that follows is done on
// their list in LDS.  Many: the draw takes one more pass over the row.
#include "biloco_device.h"
#include "biloco_internal.h"

namespace biloco {

namespace {

constexpr int kMostSlices = 16;
constexpr int kThreads = 1024, kWavesS = kThreads / 64, kBins = 2048, kList = 1024;
constexpr int kOneShift = 44;                    // w = 1 is 1 << 44
constexpr double kMostY = 45.0;                  // from here on a weight rounds to 0
constexpr float kLargest = 3.402823466e38f;
constexpr double kLog2eD = 1.4426950408889634, kLn2D = 0.6931471805599453;
typedef unsigned long long u64;

struct Best {      // of a row or a part of it
    float top, low;      // largest and smallest above -inf; -inf and inf where there is none
    int at;              // the first of the largest
};

struct Shared {
    uint32_t count[kBins];
    u64 mass[kBins];
    u64 key[kList], w[kList];
    u64 sum[kWavesS], sum2[kWavesS];
    Best best[kWavesS];
    uint32_t n, pick, lo, hi;
    u64 at, upto, all;
    int first;
    double exp[64];      // 2^(j / 64)
};

// A row as 16-byte blocks: the first may begin before it, the last end behind it.  Blocks are
// aligned and hold something of the row, so that no page but its own is touched.
template <class T>
struct Row {
    static constexpr int E = 16 / sizeof(T);
    const T *x;
    const u32x4_t *p;
    int before, V, blocks;
    __device__ __forceinline__ Row(const T *x_, int V_) : x(x_), V(V_) {
        const uintptr_t a = (uintptr_t)x;
        p = reinterpret_cast<const u32x4_t *>(a & ~(uintptr_t)15);
        before = (int)((a & 15) / sizeof(T));
        blocks = (before + V + E - 1) / E;
    }
    // NaN is -inf.
    __device__ __forceinline__ static float tidy(float v) { return fmaxf(v, -__builtin_inff()); }
    // Element e of a block.
    __device__ __forceinline__ static float value(const u32x4_t &w, int e) {
        if constexpr (sizeof(T) == 4) return tidy(__uint_as_float(w[e]));
        else return tidy(__uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16));
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return tidy(x[i]);
        else return tidy(bf16_to_f32(x[i]));
    }
    __device__ __forceinline__ int index(int b, int e) const { return b * E + e - before; }
    // Block b, with NaN for what lies outside the row.
    __device__ __forceinline__ u32x4_t block(int b) const {
        u32x4_t w = p[min(b, blocks - 1)];
        if (b == 0 || b >= blocks - 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = index(b, e);
                if (i >= 0 && i < V) continue;
                if constexpr (sizeof(T) == 4) w[e] = 0x7FC00000u;
                else w[e >> 1] = e & 1 ? w[e >> 1] | 0x7FC00000u : w[e >> 1] | 0x7FC0u;
            }
        }
        return w;
    }
    // f(index of the first, values) of four elements at a time of blocks [b0, b1), each
    // wave a run of them.
    template <class F>
    __device__ __forceinline__ void each(int b0, int b1, F f) const {
        const int wave = threadIdx.x >> 6, per = ((b1 - b0 + kWavesS - 1) / kWavesS + 63) & ~63;
        run(min(b0 + wave * per, b1), min(b0 + wave * per + per, b1), f);
    }
    // The same of one wave's blocks.  Elements outside the row come as -inf.
    template <class F>
    __device__ __forceinline__ void run(int b0, int b1, F f) const {
        constexpr int U = 2;      // loads under way beside the one in use
        const int lane = threadIdx.x & 63;
        u32x4_t w[U];
#pragma unroll
        for (int k = 0; k < U; ++k) w[k] = block(b0 + lane + 64 * k < b1 ? b0 + lane + 64 * k : blocks);
        for (int b = b0 + lane; b - lane < b1; b += 64 * U)
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const u32x4_t v = w[k];
                const int next = b + 64 * (k + U);
                if (next - lane < b1) w[k] = block(next < b1 ? next : blocks);
                if (b + 64 * k - lane < b1)
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const float x[4] = {value(v, e), value(v, e + 1), value(v, e + 2), value(v, e + 3)};
                        f(index(b + 64 * k, e), x);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
    }
};

// v of another lane by a data-parallel move; 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved(u64 v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_scan_u64(u64 v) {      // inclusive
    v += moved<0x111, 0xF>(v);      // within rows of 16 lanes
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);      // from row to row
    v += moved<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ u64 wave_sum_u64(u64 v) {
    v = wave_scan_u64(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
    return (u64)hi << 32 | lo;
}
// Sum over the workgroup, to every thread.
__device__ __forceinline__ u64 group_sum(u64 v, u64 (&tmp)[kWavesS]) {
    v = wave_sum_u64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    u64 all = 0;
#pragma unroll
    for (int i = 0; i < kWavesS; ++i) all += tmp[i];
    return all;
}
// Exclusive sums over the threads.
__device__ __forceinline__ u64 group_before(u64 v, u64 (&tmp)[kWavesS]) {
    const u64 in = wave_scan_u64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) tmp[threadIdx.x >> 6] = in;
    __syncthreads();
    u64 b = in - v;
    for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) b += tmp[i];
    return b;
}

__device__ __forceinline__ uint32_t key_of(float x) {      // -0 is 0
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 full_key(float x, int i) { return (u64)key_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)i); }

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// What a request asks of a row, and the row's scale.
struct Ask {
    double c;            // log2(e) / T
    double p;            // p >= 1: no cut
    u64 m;               // least weight
    float top;
    double most;         // the top, or the largest number for an infinite one
    float far;           // logits further than this below the top have no weight
    float parts;         // histogram's parts to a logit
    uint32_t k;          // 0: no cut
    bool first;          // the first of the largest

    __device__ __forceinline__ void set(const SampleArgs &a, int row) {
        double t = a.temperature ? (double)a.temperature[row] : 1.0;
        p = a.top_p ? (double)a.top_p[row] : 1.0;
        const double mp = a.min_p ? (double)a.min_p[row] : 0.0;
        const int kk = a.top_k ? a.top_k[row] : 0;
        k = kk > 0 && kk < a.V ? (uint32_t)kk : 0;
        if (!(p < 1.0)) p = 1.0;
        m = (u64)ceil((mp > 0.0 ? fmin(mp, 1.0) : 0.0) * (double)(1ull << kOneShift));
        first = !(t > 0.0);
        if (first) t = 1.0;
        c = kLog2eD / t;
    }
    // By k or p: the histogram is needed.
    __device__ __forceinline__ bool cut() const { return !first && (k > 0 || p < 1.0); }
    __device__ __forceinline__ void scale(const Best &b) {
        top = b.top;
        most = (double)fminf(top, kLargest);
        // Infinite at the highest temperatures; 0 where only infinite logits have weight.
        far = b.top == __builtin_inff() ? 0.0f : (float)((kMostY + 1.0) / c);
        parts = (float)(kBins - 1) / fmaxf(fminf(b.top - b.low, far), 1e-30f);      // inf - inf: far
    }
    // Whether x may have weight.
    __device__ __forceinline__ bool near(float x) const { return x > -__builtin_inff() && !(top - x > far); }
    __device__ __forceinline__ int bin_of(float x) const { return min((int)((top - x) * parts), kBins - 1); }
    // 2^-y in steps of 2^-44 of N logits that are near(); of others anything.  -y = n + j / 64 + g
    // with whole n and j, |g| <= 1/128: 2^(j / 64) from a table, 2^g by the polynomial
    // through Chebyshev's points, within 2^-48 relative.  Several at once, since one is a
    // chain of dependent instructions.
    template <int N>
    __device__ __forceinline__ void weights(const Shared &s, const float (&x)[N], u64 (&w)[N]) const {
        constexpr double kRound = 6755399441055744.0 / 64.0;      // 1.5 2^52 / 64: sums round to 64ths
        double d[N], t[N], g[N], v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = most - (double)fminf(x[i], kLargest);      // inf - inf: 0
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = __builtin_fma(d[i], -c, kRound);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = __builtin_fma(d[i], -c, kRound - t[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.009618140880813336;
            v[i] = __builtin_fma(v[i], g[i], 0.05550421039181774);
            v[i] = __builtin_fma(v[i], g[i], 0.24022650695892073);
            v[i] = __builtin_fma(v[i], g[i], 0.6931471805583931);
            v[i] = __builtin_fma(v[i], g[i], 1.0);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = (int)(uint32_t)__builtin_bit_cast(u64, t[i]);      // 64 n + j
            const double p = v[i] * s.exp[k & 63];
            const u64 scaled = __builtin_bit_cast(u64, p) + ((u64)(uint32_t)((k >> 6) + kOneShift) << 52);
            const double whole = __builtin_bit_cast(double, scaled) + 4503599627370496.0;      // 2^52: rounds
            w[i] = __builtin_bit_cast(u64, whole) & 0xFFFFFFFFFFFFFull;
        }
    }
    __device__ __forceinline__ u64 weight(const Shared &s, float x) const {
        const float one[1] = {x};
        u64 w[1];
        weights(s, one, w);
        return w[0];
    }
};

// ---------------------------------------------------------------- steps of a row
template <class T>
__device__ __forceinline__ Best best_of(const Row<T> &r, int b0, int b1, Shared &s) {
    float top = -__builtin_inff(), low = __builtin_inff();
    int at = 0x7FFFFFFF;
    r.each(b0, b1, [&](int i, const float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            at = x[e] > top ? i + e : at;      // a lane's elements come in the order of their index
            top = fmaxf(top, x[e]);
            low = fminf(low, x[e] > -__builtin_inff() ? x[e] : low);
        }
    });
    const auto join = [&](float t, float l, int i) {
        at = t > top ? i : t == top ? min(at, i) : at;
        top = fmaxf(top, t);
        low = fminf(low, l);
    };
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) join(__shfl_xor(top, o, 64), __shfl_xor(low, o, 64), __shfl_xor(at, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.best[threadIdx.x >> 6] = Best{top, low, at};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWavesS; ++i) join(s.best[i].top, s.best[i].low, s.best[i].at);
    return Best{top, low, at};
}

__device__ __forceinline__ void clear(Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.count[i] = 0;
        s.mass[i] = 0;
    }
    __syncthreads();
}

template <class T, class Part>
__device__ __forceinline__ void count_parts(const Row<T> &r, int b0, int b1, const Ask &q, Shared &s, Part part) {
    r.each(b0, b1, [&](int, const float (&x)[4]) {
        int at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = q.near(x[e]) ? part(x[e]) : -1;
        if ((at[0] & at[1] & at[2] & at[3]) == -1) return;
        u64 w[4];
        q.weights(s, x, w);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at[e] >= 0) {
                atomicAdd(&s.count[at[e]], 1u);
                atomicAdd(&s.mass[at[e]], w[e]);
            }
    });
    __syncthreads();
}
template <class T>
__device__ __forceinline__ void histogram(const Row<T> &r, int b0, int b1, const Ask &q, Shared &s) {
    count_parts(r, b0, b1, q, s, [&](float x) { return q.bin_of(x); });
}

struct Upto {
    uint32_t count;
    u64 mass;
};
// The first bin b at which reached(sums through b) holds, and the sums before it; -1
// where it holds nowhere.  reached() does not go back as the sums grow.
template <class F>
__device__ __forceinline__ int first_bin(Shared &s, Upto &before, F reached) {
    constexpr int N = kBins / kThreads;
    uint32_t c[N];
    u64 m[N], cs = 0, ms = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = s.count[threadIdx.x * N + i];
        m[i] = s.mass[threadIdx.x * N + i];
        cs += c[i];
        ms += m[i];
    }
    u64 cb = group_before(cs, s.sum), mb = group_before(ms, s.sum2);
    if (threadIdx.x == 0) s.pick = 0xFFFFFFFFu;
    __syncthreads();
    const bool had = threadIdx.x > 0 && reached(Upto{(uint32_t)cb, mb});
    u64 c0 = cb, m0 = mb;
    int mine = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool now = reached(Upto{(uint32_t)(cb + c[i]), mb + m[i]});
        if (mine < 0 && !had && now) {
            mine = threadIdx.x * N + i;
            c0 = cb;
            m0 = mb;
        }
        cb += c[i];
        mb += m[i];
    }
    if (mine >= 0) {      // one thread
        s.pick = mine;
        s.at = m0;
        s.lo = (uint32_t)c0;
    }
    __syncthreads();
    before = Upto{s.lo, s.at};
    const int b = (int)s.pick;
    __syncthreads();
    return b;
}

// The elements of a row with weight for which in(x) holds, in the list while it has room;
// their number, and their smallest and largest keys.
template <class T, class F>
__device__ __forceinline__ uint32_t gather(const Row<T> &r, const Ask &q, Shared &s, F in) {
    if (threadIdx.x == 0) {
        s.n = 0;
        s.lo = 0xFFFFFFFFu;
        s.hi = 0;
    }
    __syncthreads();
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    r.each(0, r.blocks, [&](int i, const float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (q.near(x[e]) && in(x[e])) {
                const uint32_t k = key_of(x[e]);
                lo = min(lo, k);
                hi = max(hi, k);
                const uint32_t at = atomicAdd(&s.n, 1u);
                if (at < kList) s.key[at] = full_key(x[e], i + e);
            }
    });
    if (hi >= lo) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
    }
    __syncthreads();
    return s.n;
}

// The workgroup's (key, w), a thread one, in descending order of the keys of the first
// `n` threads (the others' keys are taken as 0).
__device__ __forceinline__ void sort_down(Shared &s, uint32_t n, u64 &key, u64 &w) {
    const int tid = threadIdx.x;
    if (tid >= (int)n) key = 0;
    for (int size = 2; size < 2 * (int)n; size *= 2)
        for (int d = size / 2; d > 0; d /= 2) {
            u64 k2, w2;
            if (d >= 64) {
                __syncthreads();
                s.key[tid] = key;
                s.w[tid] = w;
                __syncthreads();
                k2 = s.key[tid ^ d];
                w2 = s.w[tid ^ d];
            } else {
                k2 = __shfl_xor(key, d, 64);
                w2 = __shfl_xor(w, d, 64);
            }
            const bool down = (tid & size) == 0, upper = (tid & d) == 0;      // upper: keeps the larger where down
            if ((k2 > key) == (down == upper) && k2 != key) {
                key = k2;
                w = w2;
            }
        }
    __syncthreads();
}
// The listed elements in order, with their weights.
__device__ __forceinline__ void sort_list(const Ask &q, Shared &s, uint32_t n) {
    u64 key = threadIdx.x < n ? s.key[threadIdx.x] : 0, w = 0;
    if (threadIdx.x < n) w = q.weight(s, value_of((uint32_t)(key >> 32)));
    sort_down(s, n, key, w);
    s.key[threadIdx.x] = key;
    s.w[threadIdx.x] = w;
    __syncthreads();
}
// Of the list in order, the element at which reached(sums through it) begins to hold.
// s.at and s.upto: its key, and the mass through it; s.n: its place.
template <class F>
__device__ __forceinline__ void first_listed(Shared &s, uint32_t n, const Upto &base, F reached) {
    const uint32_t i = threadIdx.x;
    const u64 w = i < n ? s.w[i] : 0;
    const u64 before = base.mass + group_before(w, s.sum);
    if (i < n && reached(Upto{base.count + i + 1, before + w}) && (i == 0 || !reached(Upto{base.count + i, before}))) {
        s.at = s.key[i];
        s.upto = before + w;
        s.lo = i;
    }
    __syncthreads();
}

// The element of a bin at which reached() begins to hold, where more than the list's
// room lie in it: its keys are cut into parts until the list takes one, or until they
// are one key, whose elements count by index.
template <class T, class F>
__device__ __forceinline__ void border(const Row<T> &r, const Ask &q, Shared &s, int bin, Upto base, F reached) {
    uint32_t n = gather(r, q, s, [&](float x) { return q.bin_of(x) == bin; });
    uint32_t lo = s.lo, hi = s.hi;
    while (n > kList && lo < hi) {
        const int shift = max(32 - __clz(hi - lo) - 11, 0);      // parts below kBins
        __syncthreads();
        clear(s);
        count_parts(r, 0, r.blocks, q, s, [&](float x) {
            const uint32_t k = key_of(x);
            return k >= lo && k <= hi ? (int)((hi - k) >> shift) : -1;
        });
        Upto b;
        const uint32_t part = first_bin(s, b, [&](const Upto &t) { return reached(Upto{base.count + t.count, base.mass + t.mass}); });
        base.count += b.count;
        base.mass += b.mass;
        const uint32_t top = hi - (part << shift), width = (1u << shift) - 1;
        const uint32_t bottom = max(lo, top >= width ? top - width : 0u);
        n = gather(r, q, s, [&](float x) { return key_of(x) >= bottom && key_of(x) <= top; });
        lo = s.lo;
        hi = s.hi;
    }
    if (n <= kList) {
        sort_list(q, s, n);
        first_listed(s, n, base, reached);
        return;
    }
    // one key: the number of its elements that are wanted, then the last one's index
    const u64 w = q.weight(s, value_of(lo));
    uint32_t a = 1, b = n;      // the fewest for which reached() holds
    while (a < b) {
        const uint32_t mid = a + (b - a) / 2;
        if (reached(Upto{base.count + mid, base.mass + mid * w})) b = mid;
        else a = mid + 1;
    }
    const uint32_t key = lo;
    int b0 = 0, b1 = r.blocks;
    uint32_t want = a;
    while (b1 - b0 > 0) {
        const int wave = threadIdx.x >> 6, per = ((b1 - b0 + kWavesS - 1) / kWavesS + 63) & ~63;
        if (b1 - b0 <= 64) {      // a wave of blocks, one a lane
            if (wave == 0) {
                const int at = b0 + (threadIdx.x & 63);
                uint32_t c = 0;
                r.run(b0, b1, [&](int, const float (&x)[4]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) c += key_of(x[e]) == key;
                });
                const uint32_t in = (uint32_t)wave_scan_u64(c);
                if (in >= want && in - c < want) {
                    uint32_t left = want - (in - c);
                    const u32x4_t v = r.block(at);
#pragma unroll
                    for (int e = 0; e < Row<T>::E; ++e) {
                        const float x = Row<T>::value(v, e);
                        if (key_of(x) == key && --left == 0) s.at = full_key(x, r.index(at, e));
                    }
                }
            }
            break;
        }
        u64 c = 0;
        r.each(b0, b1, [&](int, const float (&x)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c += key_of(x[e]) == key;
        });
        c = wave_sum_u64(c);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) s.sum[wave] = c;
        __syncthreads();
        int g = 0;
        while (g < kWavesS - 1 && want > s.sum[g]) want -= (uint32_t)s.sum[g++];
        const int from = min(b0 + g * per, b1);
        b1 = min(from + per, b1);
        b0 = from;
    }
    __syncthreads();
    if (threadIdx.x == 0) s.upto = base.mass + a * w;
    __syncthreads();
}

// What is kept of a row: keys from tau on, by weight from q.m on.
struct Kept {
    u64 tau;
    float least;      // the value of tau
    __device__ __forceinline__ explicit Kept(u64 t) : tau(t), least(t ? value_of((uint32_t)(t >> 32)) : -__builtin_inff()) {}
    __device__ __forceinline__ bool may(const Ask &q, float x) const { return x >= least && q.near(x); }
    // of one that may be
    __device__ __forceinline__ bool is(float x, int i) const { return x > least || (uint32_t)i <= 0xFFFFFFFFu - (uint32_t)tau || tau == 0; }
};

// Sums of the kept weights (and, with ALL, of every weight) of four elements.
template <bool ALL>
__device__ __forceinline__ void add_kept(const Ask &q, const Shared &s, const Kept &k, int i, const float (&x)[4], u64 &mine, u64 &total) {
    bool may[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) may[e] = k.may(q, x[e]);
    if (!(may[0] | may[1] | may[2] | may[3])) return;
    u64 w[4];
    q.weights(s, x, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[e] = may[e] ? w[e] : 0;
        if constexpr (ALL) total += w[e];
        mine += w[e] >= q.m && k.is(x[e], i + e) ? w[e] : 0;
    }
}

// The sums over blocks [b0, b1), to every thread; s.sum: the kept ones of each wave's run.
template <class T>
__device__ __forceinline__ void masses(const Row<T> &r, const Ask &q, Shared &s, const Kept &k, int b0, int b1, u64 &kept, u64 &all) {
    u64 mine = 0, total = 0;
    r.each(b0, b1, [&](int i, const float (&x)[4]) { add_kept<true>(q, s, k, i, x, mine, total); });
    all = group_sum(total, s.sum2);
    kept = group_sum(mine, s.sum);
}

// The first index at which the kept weights' sum passes `target`, among blocks [b0, b1),
// before which they come to `before`: parts in turn, each a sixteenth of the one before.
// known: s.sum holds those of the first sixteen.
template <class T>
__device__ __forceinline__ int draw(const Row<T> &r, const Ask &q, Shared &s, const Kept &k, int b0, int b1, u64 before, double target,
                                    bool known) {
#pragma unroll 1
    while (b1 - b0 > kThreads) {
        const int wave = threadIdx.x >> 6, per = ((b1 - b0 + kWavesS - 1) / kWavesS + 63) & ~63;
        if (!known) {
            u64 mine = 0, none = 0;
            r.each(b0, b1, [&](int i, const float (&x)[4]) { add_kept<false>(q, s, k, i, x, mine, none); });
            mine = wave_sum_u64(mine);
            __syncthreads();
            if ((threadIdx.x & 63) == 0) s.sum[wave] = mine;
            __syncthreads();
        }
        known = false;
        // the last part that holds anything where no sum passes the target (u at or above 1)
        int g = -1, last = 0;
        u64 at = before, last_at = before, g_at = before;
        for (int i = 0; i < kWavesS; ++i) {
            if (s.sum[i] != 0) {
                last = i;
                last_at = at;
                if (g < 0 && (double)(at + s.sum[i]) > target) {
                    g = i;
                    g_at = at;
                }
            }
            at += s.sum[i];
        }
        before = g < 0 ? last_at : g_at;
        const int from = min(b0 + (g < 0 ? last : g) * per, b1);
        b1 = min(from + per, b1);
        b0 = from;
    }
    // a block a thread
    const int b = b0 + threadIdx.x;
    const u32x4_t v = r.block(b < b1 ? b : r.blocks);
    u64 w[Row<T>::E], mine = 0;
#pragma unroll
    for (int e0 = 0; e0 < Row<T>::E; e0 += 4) {
        const float x[4] = {Row<T>::value(v, e0), Row<T>::value(v, e0 + 1), Row<T>::value(v, e0 + 2), Row<T>::value(v, e0 + 3)};
        u64 four[4];
        q.weights(s, x, four);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool is = k.may(q, x[e]) && four[e] >= q.m && k.is(x[e], r.index(b, e0 + e));
            w[e0 + e] = is ? four[e] : 0;
            mine += w[e0 + e];
        }
    }
    if (threadIdx.x == 0) {
        s.pick = 0xFFFFFFFFu;
        s.hi = 0;
    }
    u64 at = before + group_before(mine, s.sum);
    const bool passes = mine != 0 && (double)(at + mine) > target;
    int hit = 0, held = 0;
#pragma unroll
    for (int e = 0; e < Row<T>::E; ++e) {
        const bool was = (double)at > target;
        at += w[e];
        if (w[e] != 0) held = r.index(b, e);
        if (w[e] != 0 && !was && (double)at > target) hit = r.index(b, e);
    }
    // the first that passes lies in the first block that does; none: the last one held
    if (passes) atomicMin(&s.pick, (uint32_t)threadIdx.x);
    if (mine != 0) atomicMax(&s.hi, (uint32_t)held);
    __syncthreads();
    if (s.pick == 0xFFFFFFFFu) return (int)s.hi;
    if (threadIdx.x == s.pick) s.lo = (uint32_t)hit;
    __syncthreads();
    return (int)s.lo;
}

// The same on the list in order: its first `kept` elements, in the order of their index.
__device__ __forceinline__ int draw_listed(const Ask &q, Shared &s, double u, uint32_t kept) {
    u64 w = threadIdx.x < kept ? s.w[threadIdx.x] : 0;
    if (w < q.m) w = 0;
    const double target = u * (double)group_sum(w, s.sum);
    u64 key = (uint32_t)s.key[threadIdx.x];      // 2^32 - 1 - index
    if (threadIdx.x == 0) {
        s.pick = 0xFFFFFFFFu;
        s.hi = 0;
    }
    sort_down(s, kept, key, w);
    const u64 upto = group_before(w, s.sum) + w;
    if (w != 0) {
        const uint32_t i = 0xFFFFFFFFu - (uint32_t)key;
        if ((double)upto > target) atomicMin(&s.pick, i);
        atomicMax(&s.hi, i);      // u at or above 1: the last one
    }
    __syncthreads();
    return (int)(s.pick == 0xFFFFFFFFu ? s.hi : s.pick);
}

__device__ __forceinline__ double number_of(const SampleArgs &a, int row) { return a.u[row] >= 0.0f ? (double)a.u[row] : 0.0; }      // NaN: 0

template <class T>
__device__ __forceinline__ void answer(const SampleArgs &a, int row, const Row<T> &r, const Ask &q, int token, u64 all) {
    if (threadIdx.x != 0) return;
    a.token[row] = token;
    if (!a.logprob) return;
    const float x = r.at(token);
    const double y = x == q.top ? 0.0 : ((double)q.top - (double)x) * q.c;
    a.logprob[row] = (float)(-y * kLn2D - log((double)all * (1.0 / (double)(1ull << kOneShift))));
}

// Of a row whose histogram is in s: true if the row is answered, else the least kept key.
// s.all: the sum of every weight.
template <class T>
__device__ __forceinline__ bool cut_row(const SampleArgs &a, int row, const Row<T> &r, const Ask &q, Shared &s, u64 &tau) {
    u64 m = 0;
    for (int i = threadIdx.x; i < kBins; i += kThreads) m += s.mass[i];
    m = group_sum(m, s.sum);
    if (threadIdx.x == 0) s.all = m;
    tau = 0;
    uint32_t n = 0;
    bool listed = false;
    // the border by k, then that by p of what k has left
    bool by_k = q.k > 0;
    double target = q.p * (double)m;
    const auto reached = [&](const Upto &t) { return by_k ? t.count >= q.k : t.count > 0 && (double)t.mass >= target; };
#pragma unroll 1
    for (int step = 0;; ++step) {
        int bin = 0;
        if (!listed) {
            Upto base;
            bin = first_bin(s, base, reached);
            // every element up to the border's bin in the list, if it has room
            listed = step == 0 && bin >= 0 && base.count + s.count[bin] <= kList;
            if (listed) {
                n = gather(r, q, s, [&](float x) { return q.bin_of(x) <= bin; });
                sort_list(q, s, n);
            } else if (bin >= 0) {
                border(r, q, s, bin, base, reached);
            }
        }
        if (listed) first_listed(s, n, Upto{0, 0}, reached);
        if (bin >= 0) {      // else all that have weight are kept
            tau = max(tau, s.at);
            if (listed) n = s.lo + 1;
        }
        if (!by_k || !(q.p < 1.0)) break;
        by_k = false;
        target = q.p * (double)(bin >= 0 ? s.upto : s.all);
        if (!listed) {      // the search for k's border has used the histogram's room
            __syncthreads();
            clear(s);
            histogram(r, 0, r.blocks, q, s);
        }
    }
    if (listed) answer(a, row, r, q, draw_listed(q, s, number_of(a, row), n), s.all);
    return listed;
}

template <class T>
__device__ __forceinline__ Row<T> row_of(const SampleArgs &a, int row) {
    return Row<T>(static_cast<const T *>(a.logits) + row * a.stride, a.V);
}
__device__ __forceinline__ bool none_left(const SampleArgs &a, int row, const Best &b) {
    if (b.top > -__builtin_inff()) return false;
    if (threadIdx.x == 0) {
        a.token[row] = -1;
        if (a.logprob) a.logprob[row] = -__builtin_inff();
    }
    return true;
}

__device__ __forceinline__ void fill_table(Shared &s) {
    if (threadIdx.x < 64) s.exp[threadIdx.x] = exp2((double)threadIdx.x / 64.0);
}

// A workgroup a row.
template <class T>
__global__ void __launch_bounds__(kThreads)
sample_row_kernel(const SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.x;
    const Row<T> r = row_of<T>(a, row);
    Ask q;
    q.set(a, row);
    fill_table(s);
    clear(s);
    const Best b = best_of(r, 0, r.blocks, s);
    if (none_left(a, row, b)) return;
    q.scale(b);
    if (q.first && !a.logprob) return answer(a, row, r, q, b.at, 0);
    // across the passes these wait in LDS
    if (threadIdx.x == 0) s.first = b.at;
    u64 tau = 0;
    if (q.cut()) {
        histogram(r, 0, r.blocks, q, s);
        if (cut_row(a, row, r, q, s, tau)) return;
    }
    const Kept k(tau);
    u64 kept, sum;
    masses(r, q, s, k, 0, r.blocks, kept, sum);
    if (threadIdx.x == 0 && !q.cut()) s.all = sum;
    const int token = q.first ? s.first : draw(r, q, s, k, 0, r.blocks, 0, number_of(a, row) * (double)kept, true);
    answer(a, row, r, q, token, s.all);
}

// Few rows: a row in slices, a workgroup each, in up to five launches:
//   best     largest logit of each slice
//   sums     histogram of each slice, or where nothing is cut its sums
//   cut      (a workgroup a row) the histogram's border; short lists are answered here
//   keep     sums of what is kept of each slice, of rows whose list is not short
//   pick     (a workgroup a row) the slice that holds the draw, and the token in it
struct Slice {
    u64 kept, all;
    Best best;
};
struct RowState {
    u64 tau, all;
    int done;
};
struct Work {
    Slice *slice;       // [rows][S]
    RowState *row;      // [rows]
    u64 *mass;          // [rows][S][kBins]
    uint32_t *count;    // likewise
};
__host__ __device__ __forceinline__ size_t part_bytes(size_t n) { return (n + 15) / 16 * 16; }
__host__ __device__ __forceinline__ size_t work_bytes(size_t rows, size_t slices) {
    return part_bytes(slices * sizeof(Slice)) + part_bytes(rows * sizeof(RowState)) + slices * kBins * 12;
}
__device__ __forceinline__ Work work_of(const SampleArgs &a, int S) {
    Work w;
    uint8_t *p = static_cast<uint8_t *>(a.ws);
    const size_t n = (size_t)a.rows * S;
    w.slice = reinterpret_cast<Slice *>(p);
    p += part_bytes(n * sizeof(Slice));
    w.row = reinterpret_cast<RowState *>(p);
    p += part_bytes(a.rows * sizeof(RowState));
    w.mass = reinterpret_cast<u64 *>(p);
    w.count = reinterpret_cast<uint32_t *>(w.mass + n * kBins);
    return w;
}
struct Blocks {
    int b0, b1;
};
__device__ __forceinline__ Blocks slice_blocks(int blocks, int i, int S) {
    const int per = ((blocks + S - 1) / S + 63) & ~63;
    return Blocks{min(i * per, blocks), min(i * per + per, blocks)};
}
// Lane l takes slice l & 15 of a row, so that their loads go out together.
__device__ __forceinline__ Best row_best(const Slice *s, int S) {
    const int i = threadIdx.x & (kMostSlices - 1);
    Best b = i < S ? s[i].best : Best{-__builtin_inff(), __builtin_inff(), 0x7FFFFFFF};
#pragma unroll
    for (int o = kMostSlices / 2; o > 0; o >>= 1) {
        const Best x{__shfl_xor(b.top, o, 64), __shfl_xor(b.low, o, 64), __shfl_xor(b.at, o, 64)};
        b.at = x.top > b.top ? x.at : x.top == b.top ? min(x.at, b.at) : b.at;
        b.top = fmaxf(b.top, x.top);
        b.low = fminf(b.low, x.low);
    }
    return b;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sample_best_kernel(const SampleArgs a, int S) {
    __shared__ Shared s;
    const int row = blockIdx.x / S, i = blockIdx.x % S;
    const Row<T> r = row_of<T>(a, row);
    const Blocks x = slice_blocks(r.blocks, i, S);
    const Best b = best_of(r, x.b0, x.b1, s);
    if (threadIdx.x == 0) work_of(a, S).slice[blockIdx.x].best = b;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sample_sums_kernel(const SampleArgs a, int S) {
    __shared__ Shared s;
    const int row = blockIdx.x / S, i = blockIdx.x % S;
    const Work w = work_of(a, S);
    const Row<T> r = row_of<T>(a, row);
    const Blocks x = slice_blocks(r.blocks, i, S);
    Ask q;
    q.set(a, row);
    fill_table(s);
    const Best b = row_best(w.slice + (size_t)row * S, S);
    q.scale(b);
    if (!(b.top > -__builtin_inff()) || (q.first && !a.logprob)) return;
    clear(s);
    if (q.cut()) {
        histogram(r, x.b0, x.b1, q, s);
        for (int k = threadIdx.x; k < kBins; k += kThreads) {
            w.mass[(size_t)blockIdx.x * kBins + k] = s.mass[k];
            w.count[(size_t)blockIdx.x * kBins + k] = s.count[k];
        }
        return;
    }
    u64 kept, all;
    masses(r, q, s, Kept(0), x.b0, x.b1, kept, all);
    if (threadIdx.x == 0) {
        w.slice[blockIdx.x].kept = kept;
        w.slice[blockIdx.x].all = all;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sample_cut_kernel(const SampleArgs a, int S) {
    __shared__ Shared s;
    const int row = blockIdx.x;
    const Work w = work_of(a, S);
    const Row<T> r = row_of<T>(a, row);
    Ask q;
    q.set(a, row);
    fill_table(s);
    const Best b = row_best(w.slice + (size_t)row * S, S);
    q.scale(b);
    u64 tau = 0;
    bool done = true;
    if (threadIdx.x == 0) s.all = 0;
    if (none_left(a, row, b)) {
    } else if (q.first && !a.logprob) {
        answer(a, row, r, q, b.at, 0);
    } else if (!q.cut()) {
        done = false;
    } else {
        for (int k = threadIdx.x; k < kBins; k += kThreads) {
            u64 m = 0;
            uint32_t c = 0;
#pragma unroll
            for (int i0 = 0; i0 < kMostSlices; i0 += 8) {
                if (i0 >= S) break;
                u64 mi[8];
                uint32_t ci[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const size_t at = ((size_t)row * S + min(i0 + i, S - 1)) * kBins + k;
                    mi[i] = w.mass[at];
                    ci[i] = w.count[at];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m += i0 + i < S ? mi[i] : 0;
                    c += i0 + i < S ? ci[i] : 0;
                }
            }
            s.mass[k] = m;
            s.count[k] = c;
        }
        __syncthreads();
        done = cut_row(a, row, r, q, s, tau);
    }
    if (threadIdx.x == 0) w.row[row] = RowState{tau, s.all, done};      // s.all by this thread
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sample_keep_kernel(const SampleArgs a, int S) {
    __shared__ Shared s;
    const int row = blockIdx.x / S, i = blockIdx.x % S;
    const Work w = work_of(a, S);
    const RowState st = w.row[row];
    Ask q;
    q.set(a, row);
    if (st.done || !q.cut()) return;
    const Row<T> r = row_of<T>(a, row);
    const Blocks x = slice_blocks(r.blocks, i, S);
    fill_table(s);
    q.scale(row_best(w.slice + (size_t)row * S, S));
    __syncthreads();
    u64 kept, all;
    masses(r, q, s, Kept(st.tau), x.b0, x.b1, kept, all);
    if (threadIdx.x == 0) w.slice[blockIdx.x].kept = kept;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sample_pick_kernel(const SampleArgs a, int S) {
    __shared__ Shared s;
    const int row = blockIdx.x;
    const Work w = work_of(a, S);
    const Slice *x = w.slice + (size_t)row * S;
    const int i = threadIdx.x & (kMostSlices - 1);
    // loads first
    const RowState st = w.row[row];
    const u64 mine = i < S ? x[i].kept : 0, every = i < S ? x[i].all : 0;
    const Best b = row_best(x, S);
    const Row<T> r = row_of<T>(a, row);
    Ask q;
    q.set(a, row);
    if (st.done) return;
    fill_table(s);
    q.scale(b);
    __syncthreads();
    u64 upto = mine, all = every;
#pragma unroll
    for (int o = 1; o < kMostSlices; o <<= 1) {
        const u64 t = __shfl_up(upto, o, kMostSlices);
        if (i >= o) upto += t;
        all += __shfl_xor(all, o, 64);
    }
    if (q.cut()) all = st.all;
    const double target = number_of(a, row) * (double)__shfl(upto, kMostSlices - 1, 64);
    // the last one that holds anything where no sum passes the target (u at or above 1)
    const uint32_t holds = (uint32_t)__ballot(mine != 0) & 0xFFFFu, past = (uint32_t)__ballot(mine != 0 && (double)upto > target) & 0xFFFFu;
    const int slice = past ? __ffs((int)past) - 1 : 31 - __clz((int)holds);
    const u64 before = __shfl(upto - mine, slice, 64);
    const Blocks y = slice_blocks(r.blocks, slice, S);
    answer(a, row, r, q, q.first ? b.at : draw(r, q, s, Kept(st.tau), y.b0, y.b1, before, target, false), all);
}

// Slices a row where the rows alone leave CUs idle: at most kMostSlices, of at least
// kLeastSlice logits each, and only if a workgroup is spared kLeastSpared logits, which is
// what the launches cost.  In slices against a workgroup a row (fp32, p 0.9): one row of 16000
// 41.6 and 31.0 us, of 32000 44.6 and 45.9 (either way within the spread of calls), of 50000 48.5 and 63.5, of 262144 89 and 247; 32
// rows of 32000 47.9 and 46.7, of 100000 66.5 and 112; 64 of 50000 58.9 and 66.6; 128 of 64000
// (two slices) 83.5 and 77.3, of 150000 147 and 157.
constexpr int kCUs = 256, kLeastSlice = 4096, kLeastSpared = 32768;
int slices_of(int rows, int V) {
    int s = kCUs / rows;
    if (s > kMostSlices) s = kMostSlices;
    if (s > V / kLeastSlice) s = V / kLeastSlice;
    return s < 2 || V - V / s < kLeastSpared ? 1 : s;
}

// Rows of a launch: more than 2^22 would take 2^32 threads, which it cannot count.
constexpr int kMostGrid = 1 << 21;
SampleArgs rows_from(const SampleArgs &a, int64_t first, size_t size) {
    SampleArgs b = a;
    b.rows = (int)(a.rows - first < kMostGrid ? a.rows - first : kMostGrid);
    b.logits = static_cast<const char *>(a.logits) + first * a.stride * (int64_t)size;
    const auto on = [&](auto *&p) { if (p) p += first; };
    on(b.temperature);
    on(b.top_k);
    on(b.top_p);
    on(b.min_p);
    on(b.u);
    on(b.token);
    on(b.logprob);
    return b;
}
template <class T>
void launch_rows(const SampleArgs &a, int S, hipStream_t stream) {
    if (S == 1) {
        for (int64_t r = 0; r < a.rows; r += kMostGrid) {
            const SampleArgs b = rows_from(a, r, sizeof(T));
            hipLaunchKernelGGL(sample_row_kernel<T>, dim3((unsigned)b.rows), dim3(kThreads), 0, stream, b);
        }
        return;
    }
    const dim3 rows((unsigned)a.rows), slices((unsigned)(a.rows * S)), threads(kThreads);
    hipLaunchKernelGGL(sample_best_kernel<T>, slices, threads, 0, stream, a, S);
    hipLaunchKernelGGL(sample_sums_kernel<T>, slices, threads, 0, stream, a, S);
    hipLaunchKernelGGL(sample_cut_kernel<T>, rows, threads, 0, stream, a, S);
    // without k and p nothing is cut
    if (a.top_k || a.top_p) hipLaunchKernelGGL(sample_keep_kernel<T>, slices, threads, 0, stream, a, S);
    hipLaunchKernelGGL(sample_pick_kernel<T>, rows, threads, 0, stream, a, S);
}

}  // namespace

// For every smaller number of rows too: slices in all are at most those of as many as fit.
size_t sample_ws_bytes(int rows, int V) {
    int most = V / kLeastSlice < kMostSlices ? V / kLeastSlice : kMostSlices;
    if (most < 2) return 0;
    const int64_t all = (int64_t)rows * most;
    return work_bytes((size_t)(rows < kCUs ? rows : kCUs), (size_t)(all < kCUs ? all : kCUs));
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
    const int S = slices_of(a.rows, a.V);
    if (a.fp32) launch_rows<float>(a, S, stream);
    else launch_rows<uint16_t>(a, S, stream);
    return hipGetLastError();
}

}  // namespace biloco
