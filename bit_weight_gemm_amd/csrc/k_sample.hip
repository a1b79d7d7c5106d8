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

constexpr int kThreads = 1024, kWavesS = kThreads / 64, kBins = 2048, kList = 1024;
constexpr int kOneShift = 44;                    // w = 1 is 1 << 44
constexpr double kMostY = 45.0;                  // from here on a weight rounds to 0
constexpr double kLog2eD = 1.4426950408889634, kLn2D = 0.6931471805599453;
typedef unsigned long long u64;

struct Best {      // of a row or a part of it
    float top, low;      // largest and smallest above -inf; -inf and inf where there is none
};

struct Shared {
    uint32_t count[kBins];
    u64 mass[kBins];
    u64 key[kList], w[kList];
    u64 sum[kWavesS], sum2[kWavesS];
    float f0[kWavesS], f1[kWavesS];
    uint32_t n, pick, lo, hi;
    u64 at, upto, all;
};

// A row as 16-byte blocks: the first may begin before it, the last end behind it.
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
    // NaN is -inf, and -0 is 0.
    __device__ __forceinline__ static float tidy(float v) { return v != v ? -__builtin_inff() : v + 0.0f; }
    // Element e of a block.
    __device__ __forceinline__ static float value(const u32x4_t &w, int e) {
        if constexpr (sizeof(T) == 4) return tidy(__uint_as_float(w[e]));
        else return tidy(__uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16));
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return tidy(x[i]);
        else return tidy(bf16_to_f32(x[i]));
    }
    // f(index, value) of the elements of blocks [b0, b1), each wave a run of them.
    template <class F>
    __device__ __forceinline__ void each(int b0, int b1, F f) const {
        const int wave = threadIdx.x >> 6, per = ((b1 - b0 + kWavesS - 1) / kWavesS + 63) & ~63;
        run(min(b0 + wave * per, b1), min(b0 + wave * per + per, b1), f);
    }
    // The same of one wave's blocks.
    template <class F>
    __device__ __forceinline__ void run(int b0, int b1, F f) const {
        constexpr int U = 4;
        const int lane = threadIdx.x & 63;
        for (int b = b0 + lane; b - lane < b1; b += 64 * U) {
            u32x4_t w[U];
#pragma unroll
            for (int k = 0; k < U; ++k) w[k] = p[min(b + 64 * k, blocks - 1)];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (b + 64 * k >= b1) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = (b + 64 * k) * E + e - before;
                    if (i >= 0 && i < V) f(i, value(w[k], e));
                }
            }
        }
    }
};

__device__ __forceinline__ u64 wave_sum_u64(u64 v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ u64 wave_scan_u64(u64 v) {      // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const u64 t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    return v;
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

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 full_key(float x, int i) { return (u64)key_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)i); }

// What a request asks of a row, and the row's scale.
struct Ask {
    double c;            // log2(e) / T
    float top;
    double bins;         // parts of y's range to a unit
    double p, m;         // p >= 1: no cut; m in weights
    uint32_t k;          // 0: no cut
    bool cut;            // by k or p: the histogram is needed

    __device__ __forceinline__ void set(const SampleArgs &a, int row) {
        double t = a.temperature ? (double)a.temperature[row] : 1.0;
        p = a.top_p ? (double)a.top_p[row] : 1.0;
        m = a.min_p ? (double)a.min_p[row] : 0.0;
        const int kk = a.top_k ? a.top_k[row] : 0;
        k = kk > 0 && kk < a.V ? (uint32_t)kk : 0;
        if (!(p < 1.0)) p = 1.0;
        m = (m > 0.0 ? fmin(m, 1.0) : 0.0) * (double)(1ull << kOneShift);
        if (!(t > 0.0)) {      // the first of the largest
            t = 1.0;
            k = 1;
            p = 1.0;
            m = 0.0;
        }
        c = kLog2eD / t;
        cut = k > 0 || p < 1.0;
    }
    __device__ __forceinline__ void scale(const Best &b) {
        top = b.top;
        const double range = ((double)b.top - (double)b.low) * c;      // NaN or inf: an infinite top
        bins = (double)(kBins - 1) / (range < kMostY ? fmax(range, 1e-30) : kMostY);
    }
    __device__ __forceinline__ double y_of(float x) const {
        const double y = fmin(((double)top - (double)x) * c, 64.0);      // also where that is inf - inf
        return x == top ? 0.0 : y;
    }
    __device__ __forceinline__ int bin_of(double y) const { return (int)fmin(y * bins, (double)(kBins - 1)); }
    // 2^-y in steps of 2^-44, y in [0, 64]: the polynomial through Chebyshev's points of
    // [-1/2, 1/2], within 2^-45 of 2^f relative.
    __device__ __forceinline__ static u64 weight(double y) {
        const double n = __builtin_rint(-y), f = -y - n;
        double v = 1.0205905320493103e-07;
        v = __builtin_fma(v, f, 1.3259645243929057e-06);
        v = __builtin_fma(v, f, 1.5252672925346873e-05);
        v = __builtin_fma(v, f, 0.00015403433751254997);
        v = __builtin_fma(v, f, 0.0013333558200793719);
        v = __builtin_fma(v, f, 0.009618129193934304);
        v = __builtin_fma(v, f, 0.05550410866465168);
        v = __builtin_fma(v, f, 0.2402265069564034);
        v = __builtin_fma(v, f, 0.6931471805599462);
        v = __builtin_fma(v, f, 1.0000000000000135);
        v = __builtin_amdgcn_ldexp(v, (int)n + kOneShift) + 4503599627370496.0;      // 2^52: rounds to whole numbers
        return __builtin_bit_cast(u64, v) & 0xFFFFFFFFFFFFFull;
    }
};

// ---------------------------------------------------------------- steps of a row
template <class T>
__device__ __forceinline__ Best best_of(const Row<T> &r, int b0, int b1, Shared &s) {
    float top = -__builtin_inff(), low = __builtin_inff();
    r.each(b0, b1, [&](int, float x) {
        top = fmaxf(top, x);
        low = x > -__builtin_inff() ? fminf(low, x) : low;
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor(top, o, 64));
        low = fminf(low, __shfl_xor(low, o, 64));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        s.f0[threadIdx.x >> 6] = top;
        s.f1[threadIdx.x >> 6] = low;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWavesS; ++i) {
        top = fmaxf(top, s.f0[i]);
        low = fminf(low, s.f1[i]);
    }
    return Best{top, low};
}

__device__ __forceinline__ void clear(Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.count[i] = 0;
        s.mass[i] = 0;
    }
    __syncthreads();
}

template <class T>
__device__ __forceinline__ void histogram(const Row<T> &r, int b0, int b1, const Ask &q, Shared &s) {
    r.each(b0, b1, [&](int, float x) {
        const double y = q.y_of(x);
        const int b = q.bin_of(y);
        atomicAdd(&s.count[b], 1u);
        atomicAdd(&s.mass[b], Ask::weight(y));
    });
    __syncthreads();
}

struct Upto {
    uint32_t count;
    u64 mass;
};
// The first bin b at which reached(sums through b) holds, and the sums before it; the
// last bin where it holds nowhere.  reached() does not go back as the sums grow.
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
    if (threadIdx.x == 0) s.pick = kBins - 1;
    __syncthreads();
    const bool had = threadIdx.x > 0 && reached(Upto{(uint32_t)cb, mb});
    u64 c0 = cb, m0 = mb;
    int mine = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool now = reached(Upto{(uint32_t)(cb + c[i]), mb + m[i]});
        const bool last = threadIdx.x == kThreads - 1 && i == N - 1;
        if (mine < 0 && !had && (now || last)) {
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
    const int b = s.pick;
    __syncthreads();
    return b;
}

// The elements of a row for which in(key, y) holds, in the list while it has room; their
// number, and their smallest and largest keys.
template <class T, class F>
__device__ __forceinline__ uint32_t gather(const Row<T> &r, const Ask &q, Shared &s, F in) {
    if (threadIdx.x == 0) {
        s.n = 0;
        s.lo = 0xFFFFFFFFu;
        s.hi = 0;
    }
    __syncthreads();
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    r.each(0, r.blocks, [&](int i, float x) {
        const double y = q.y_of(x);
        const uint32_t k = key_of(x);
        if (in(k, y)) {
            lo = min(lo, k);
            hi = max(hi, k);
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < kList) {
                s.key[at] = full_key(x, i);
                s.w[at] = Ask::weight(y);
            }
        }
    });
    if (hi >= lo) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
    }
    __syncthreads();
    return s.n;
}

// Of the listed elements, in order: the one at which reached(sums through it) begins to
// hold, and the sums through it.  s.at and s.upto: its key, and the mass.
template <class F>
__device__ __forceinline__ void first_listed(Shared &s, uint32_t n, const Upto &base, F reached) {
    __syncthreads();
    if (threadIdx.x < n) {
        const u64 k = s.key[threadIdx.x], w = s.w[threadIdx.x];
        Upto b = base;
        for (uint32_t j = 0; j < n; ++j)
            if (s.key[j] > k) {
                ++b.count;
                b.mass += s.w[j];
            }
        const Upto t{b.count + 1, b.mass + w};
        if (reached(t) && (b.count == base.count || !reached(b))) {
            s.at = k;
            s.upto = t.mass;
        }
    }
    __syncthreads();
}

// The element of a bin at which reached() begins to hold, where more than the list's
// room lie in it: its keys are cut into parts until the list takes one, or until they
// are one key, whose elements count by index.
template <class T, class F>
__device__ __forceinline__ void border(const Row<T> &r, const Ask &q, Shared &s, int bin, Upto base, F reached) {
    uint32_t n = gather(r, q, s, [&](uint32_t, double y) { return q.bin_of(y) == bin; });
    uint32_t lo = s.lo, hi = s.hi;
    while (n > kList && lo < hi) {
        const int shift = max(32 - __clz(hi - lo) - 11, 0);      // parts below kBins
        __syncthreads();
        clear(s);
        r.each(0, r.blocks, [&](int, float x) {
            const double y = q.y_of(x);
            const uint32_t k = key_of(x);
            if (k >= lo && k <= hi) {
                atomicAdd(&s.count[(hi - k) >> shift], 1u);
                atomicAdd(&s.mass[(hi - k) >> shift], Ask::weight(y));
            }
        });
        __syncthreads();
        Upto b;
        const uint32_t part = first_bin(s, b, [&](const Upto &t) { return reached(Upto{base.count + t.count, base.mass + t.mass}); });
        base.count += b.count;
        base.mass += b.mass;
        const uint32_t top = hi - (part << shift), width = (1u << shift) - 1;
        const uint32_t bottom = max(lo, top >= width ? top - width : 0u);
        n = gather(r, q, s, [&](uint32_t k, double) { return k >= bottom && k <= top; });
        lo = s.lo;
        hi = s.hi;
    }
    if (n <= kList) {
        first_listed(s, n, base, reached);
        return;
    }
    // one key: the number of its elements that are wanted, then the last one's index
    const u64 w = s.w[0];
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
                r.run(b0, b1, [&](int, float x) { c += key_of(x) == key; });
                const uint32_t in = (uint32_t)wave_scan_u64(c);
                if (in >= want && in - c < want) {
                    uint32_t left = want - (in - c);
                    const u32x4_t v = r.p[at];
#pragma unroll
                    for (int e = 0; e < Row<T>::E; ++e) {
                        const int i = at * Row<T>::E + e - r.before;
                        if (i >= 0 && i < r.V && key_of(Row<T>::value(v, e)) == key && --left == 0)
                            s.at = (u64)key << 32 | (0xFFFFFFFFu - (uint32_t)i);
                    }
                }
            }
            break;
        }
        u64 c = 0;
        r.each(b0, b1, [&](int, float x) { c += key_of(x) == key; });
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

// The first index at which the kept weights' sum passes u of them all: parts of the row
// in turn, each a sixteenth of the one before.  all: the sum of every weight.
template <class T>
__device__ __forceinline__ int draw(const Row<T> &r, const Ask &q, Shared &s, double u, u64 tau) {
    int b0 = 0, b1 = r.blocks;
    u64 before = 0;
    double target = 0.0;
#pragma unroll 1
    for (bool first = true; first || b1 - b0 > 64; first = false) {
        const int wave = threadIdx.x >> 6, per = ((b1 - b0 + kWavesS - 1) / kWavesS + 63) & ~63;
        u64 mine = 0, total = 0;
        r.each(b0, b1, [&](int i, float x) {
            const u64 w = Ask::weight(q.y_of(x));
            total += w;
            mine += full_key(x, i) >= tau && (double)w >= q.m ? w : 0ull;
        });
        mine = wave_sum_u64(mine);
        total = wave_sum_u64(total);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            s.sum[wave] = mine;
            s.sum2[wave] = total;
        }
        __syncthreads();
        if (first) {
            u64 kept = 0, all = 0;
            for (int i = 0; i < kWavesS; ++i) {
                kept += s.sum[i];
                all += s.sum2[i];
            }
            target = u * (double)kept;
            if (threadIdx.x == 0) s.all = all;
        }
        // the last part that holds anything where no sum passes u (u at or above 1)
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
    __syncthreads();
    if (threadIdx.x < 64) {
        const int b = b0 + threadIdx.x;
        u64 w[Row<T>::E], mine = 0;
        const u32x4_t v = r.p[min(b, r.blocks - 1)];
#pragma unroll
        for (int e = 0; e < Row<T>::E; ++e) {
            const int i = b * Row<T>::E + e - r.before;
            const float x = Row<T>::value(v, e);
            const u64 t = Ask::weight(q.y_of(x));
            w[e] = b < b1 && i >= 0 && i < r.V && full_key(x, i) >= tau && (double)t >= q.m ? t : 0ull;
            mine += w[e];
        }
        u64 at = before + wave_scan_u64(mine) - mine;
        int hit = 0x7FFFFFFF, held = -1;
#pragma unroll
        for (int e = 0; e < Row<T>::E; ++e) {
            at += w[e];
            const int i = b * Row<T>::E + e - r.before;
            if (w[e] != 0) {
                held = i;
                if ((double)at > target) hit = min(hit, i);
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            hit = min(hit, __shfl_xor(hit, o, 64));
            held = max(held, __shfl_xor(held, o, 64));
        }
        if (threadIdx.x == 0) s.pick = (uint32_t)(hit == 0x7FFFFFFF ? held : hit);
    }
    __syncthreads();
    return (int)s.pick;
}

// The same on the listed elements, in the order of their index.
__device__ __forceinline__ int draw_listed(const Ask &q, Shared &s, double u, u64 tau, uint32_t n) {
    const auto kept_of = [&](uint32_t j) { return s.key[j] >= tau && (double)s.w[j] >= q.m ? s.w[j] : 0ull; };
    const u64 mine = threadIdx.x < n ? kept_of(threadIdx.x) : 0ull;
    const double target = u * (double)group_sum(mine, s.sum);
    if (threadIdx.x == 0) {
        s.pick = 0xFFFFFFFFu;
        s.hi = 0;
    }
    __syncthreads();
    if (mine != 0) {
        const uint32_t at = (uint32_t)s.key[threadIdx.x];      // 2^32 - 1 - index
        u64 to = 0;
        for (uint32_t j = 0; j < n; ++j) to += (uint32_t)s.key[j] >= at ? kept_of(j) : 0ull;
        if ((double)to > target) atomicMin(&s.pick, 0xFFFFFFFFu - at);
        atomicMax(&s.hi, 0xFFFFFFFFu - at);      // u at or above 1: the last one
    }
    __syncthreads();
    return (int)(s.pick == 0xFFFFFFFFu ? s.hi : s.pick);
}

// The row's token, from its histogram in s where q.cut.
template <class T>
__device__ __forceinline__ void choose(const SampleArgs &a, int row, const Row<T> &r, const Ask &q, Shared &s) {
    const double u = a.u[row] >= 0.0f ? (double)a.u[row] : 0.0;      // NaN: 0
    u64 tau = 0, all = 0;
    uint32_t n = 0;
    bool listed = false;
    if (q.cut) {
        u64 m = 0;
        for (int i = threadIdx.x; i < kBins; i += kThreads) m += s.mass[i];
        all = group_sum(m, s.sum);
        // the border by k, then that by p of what k has left
        bool by_k = q.k > 0;
        double target = q.p * (double)all;
        const auto reached = [&](const Upto &t) { return by_k ? t.count >= q.k : t.count > 0 && (double)t.mass >= target; };
#pragma unroll 1
        for (int step = 0;; ++step) {
            if (!listed) {
                Upto base;
                const int bin = first_bin(s, base, reached);
                // every element up to the border's bin in the list, if it has room
                listed = step == 0 && base.count + s.count[bin] <= kList;
                if (listed) n = gather(r, q, s, [&](uint32_t, double y) { return q.bin_of(y) <= bin; });
                else border(r, q, s, bin, base, reached);
            }
            if (listed) first_listed(s, n, Upto{0, 0}, reached);
            tau = max(tau, s.at);
            if (!by_k || !(q.p < 1.0)) break;
            by_k = false;
            target = q.p * (double)s.upto;
            if (!listed) {      // the search for k's border has used the histogram's room
                __syncthreads();
                clear(s);
                histogram(r, 0, r.blocks, q, s);
            }
        }
    }
    int token;
    if (listed) {
        token = draw_listed(q, s, u, tau, n);
    } else {
        token = draw(r, q, s, u, tau);
        all = s.all;
    }
    if (threadIdx.x == 0) {
        a.token[row] = token;
        if (a.logprob) {
            const double y = q.y_of(r.at(token));
            a.logprob[row] = (float)(-y * kLn2D - log((double)all * (1.0 / (double)(1ull << kOneShift))));
        }
    }
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

// A workgroup a row.
template <class T>
__global__ void __launch_bounds__(kThreads)
sample_kernel(const SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.x;
    const Row<T> r = row_of<T>(a, row);
    Ask q;
    q.set(a, row);
    clear(s);
    const Best b = best_of(r, 0, r.blocks, s);
    if (none_left(a, row, b)) return;
    q.scale(b);
    if (q.cut) histogram(r, 0, r.blocks, q, s);
    choose(a, row, r, q, s);
}

}  // namespace

size_t sample_ws_bytes(int, int) { return 0; }

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
    if (a.fp32) hipLaunchKernelGGL(sample_kernel<float>, dim3((unsigned)a.rows), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(sample_kernel<uint16_t>, dim3((unsigned)a.rows), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace biloco
