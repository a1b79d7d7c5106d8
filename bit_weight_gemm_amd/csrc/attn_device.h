// Shared by the two attention kernels: the batch's sequences as lists of
// 64-token chunks, what a row sees, and the conversions of cache codes.
#pragma once
#include "biloco_device.h"
#include "biloco_internal.h"

namespace biloco {
namespace attn {

typedef __bf16 bf16x2a_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8a_t __attribute__((ext_vector_type(8)));
typedef float f32x2a_t __attribute__((ext_vector_type(2)));
typedef float f32x4a_t __attribute__((ext_vector_type(4)));
typedef float f32x16a_t __attribute__((ext_vector_type(16)));

constexpr int kChunk = 64;         // tokens a wave takes at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ f32x4a_t mfma16(u32x4_t a, u32x4_t b, f32x4a_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8a_t, a),
                                                   __builtin_bit_cast(bf16x8a_t, b), c, 0, 0, 0);
}
// Eight codes times a power of two as eight bf16.
__device__ __forceinline__ u32x4_t widen8(uint32_t lo, uint32_t hi, float s) {
    u32x4_t r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
    return r;
}
__device__ __forceinline__ uint32_t narrow2a(float a, float b) {      // round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2a_t){a, b}, bf16x2a_t));
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float exp2a(float x) { return __builtin_amdgcn_exp2f(x); }

// Rows of a sequence (new tokens times query heads of a key/value head) up to
// which the rows kernel takes it; the tiles kernel takes the others.
constexpr int kMostRows = 64;
enum { kAllSeqs = 0, kFewRows = 1, kManyRows = 2 };

// The chunks of 64 tokens that the rows at positions [p_min, p_max] need:
// `ns` chunks of first tokens, then those from `lo0` on.
struct Span64 {
    int lo0, ns, nc;
    __device__ __forceinline__ int start(int c) const { return c < ns ? c * kChunk : lo0 + (c - ns) * kChunk; }
};
__device__ __forceinline__ Span64 span_of(const AttnArgs &a, int p_min, int p_max) {
    Span64 s;
    const int lo = a.window > 0 ? max(p_min - a.window + 1, 0) : 0;
    s.lo0 = lo & ~(kChunk - 1);
    s.ns = (min(a.sinks, s.lo0) + kChunk - 1) / kChunk;
    s.nc = s.ns + (max(p_max + 1 - s.lo0, 0) + kChunk - 1) / kChunk;
    return s;
}
// What a row at position pos sees; lo = low_of(pos).  No branches.
__device__ __forceinline__ int low_of(const AttnArgs &a, int pos) { return a.window > 0 ? pos - a.window + 1 : 0; }
__device__ __forceinline__ bool sees(const AttnArgs &a, int pos, int lo, int j) {
    return (bool)((j <= pos) & ((j >= lo) | (j < a.sinks)));
}
// Bit j: some row at a position of [p_min, p_max] sees token t0 + j.
__device__ __forceinline__ uint32_t any_sees8(const AttnArgs &a, int p_min, int p_max, int t0) {
    const int lo = low_of(a, p_min);
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bits |= (uint32_t)sees(a, p_max, lo, t0 + j) << j;
    return bits;
}
__device__ __forceinline__ uint32_t sees8(const AttnArgs &a, int pos, int t0) {
    return any_sees8(a, pos, pos, t0);
}
// Every row at a position of [p_min, p_max] sees all of the chunk at j0.
__device__ __forceinline__ bool all_see(const AttnArgs &a, int p_min, int p_max, int j0) {
    return j0 + kChunk - 1 <= p_min && (a.window == 0 || p_max - j0 < a.window || j0 + kChunk <= a.sinks);
}
constexpr uint32_t kOnes = 0x38383838u;      // the code of 1, four times
// 0xFF for each NaN code (0x7F or 0xFF), else 0x00.
__device__ __forceinline__ u32x4_t nan_bytes(u32x4_t w) {
    const u32x4_t t = (w & 0x7F7F7F7Fu) + 0x01010101u;
    return ((t & 0x80808080u) >> 7) * 255u;
}
// Four 0x00 / 0xFF bytes for four bits.
__device__ __forceinline__ uint32_t spread4(uint32_t bits) {
    return ((bits & 1u) | ((bits & 2u) << 7) | ((bits & 4u) << 14) | ((bits & 8u) << 21)) * 255u;
}

// One sequence of the batch.
struct Seq {
    int first, n, past;      // first row, new tokens, position of the first one
    int hi;                  // tokens it has
    Span64 c;                // the chunks its rows need
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v), hi = (uint32_t)uniform((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ Seq seq_from(const AttnArgs &a, int start, int stop, int kv_len, int which) {
    Seq s;
    s.first = min(max(start, 0), a.T);
    s.n = min(max(stop, s.first), a.T) - s.first;
    const int rows = s.n * (a.q_heads / a.kv_heads);
    if ((which == kFewRows && rows > kMostRows) || (which == kManyRows && rows <= kMostRows)) s.n = 0;
    s.hi = (int)min((int64_t)max(kv_len, 0), (int64_t)a.max_pages * a.page);
    s.past = s.hi - s.n;
    s.c = span_of(a, s.past, s.hi - 1);
    return s;
}

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, int which) {
    return seq_from(a, a.q_start[b], a.q_start[b + 1], a.kv_len[b], which);
}
// The same for a sequence that the whole workgroup works on, through scalar
// loads into scalar registers (b is uniform).
__device__ __forceinline__ int scalar_load(const int *p) {
    return *(const __attribute__((address_space(4))) int *)(uintptr_t)p;
}
__device__ __forceinline__ Seq seq_uniform(const AttnArgs &a, int b, int which) {
    return seq_from(a, scalar_load(a.q_start + b), scalar_load(a.q_start + b + 1), scalar_load(a.kv_len + b), which);
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor((long long)v, o, 64);
    return v;
}
// The sequence that holds entry u of a list to which sequence b contributes
// count(b) entries, and the entries before it; -1 if the list is shorter.
template <class Count>
__device__ __forceinline__ int find_seq(int B, int64_t u, int64_t &before, Count count) {
    const int lane = threadIdx.x & 63;
    before = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int64_t mine = b0 + lane < B ? count(b0 + lane) : 0;
        int64_t upto = mine;      // inclusive prefix sum
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t t = __shfl_up((long long)upto, o, 64);
            if (lane >= o) upto += t;
        }
        const uint64_t past = __ballot(before + upto > u);
        if (past) {
            const int l = __ffsll((long long)past) - 1;
            before += __shfl((long long)(upto - mine), l, 64);
            return b0 + l;
        }
        before += __shfl((long long)upto, 63, 64);
    }
    return -1;
}

}  // namespace attn

// The tiles kernel (k_attn_tiles.hip): sequences of many rows.
struct TilesPlan {
    int tiles;        // row tiles of the batch, at most
    int splits;       // pieces of the token axis
    size_t ws_bytes;
};
TilesPlan attn_tiles_plan(int B, int T, int q_heads, int kv_heads, int dim, int max_kv, int window, int sinks);
size_t attn_tiles_most_bytes(int B, int T, int q_heads, int kv_heads, int dim, int max_kv);
hipError_t launch_attn_tiles(const AttnArgs &a, int which, hipStream_t stream);

}  // namespace biloco
