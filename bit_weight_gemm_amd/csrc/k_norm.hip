// The norm after a block, the block's gate and residual scale, and the norm
// before the next block, in one pass over the row:
//
//   n  = x * rsqrt(mean(x^2) + eps) * (w_offset + post_w)
//   r' = res + res_scale * gate * n
//   h  = r' * rsqrt(mean(r'^2) + eps) * (w_offset + pre_w)
//
// and, if asked for, h's FP4 quantisation (the next product's operand).
// Bound by memory traffic: each of x, gate, res is read once, r' and h are
// written once; the row stays in registers in fp32 between the two sums.
// Two reductions a row are the only exchange between waves.  Measured on MI355X:
// 6001 gated rows of 8192 channels 129 us, 5.34 TB/s (an addition of two large
// arrays reaches 6.1); 32 rows of 5120 4.3 us, which is the launch, 4.5 with codes.
// Rows that are not aligned go an element a lane: 6001 of 8191 channels 348 us, 1.13 TB/s.
#include "biloco_device.h"
#include "biloco_internal.h"

namespace biloco {

namespace {

__device__ __forceinline__ void widen8(uint4 w, float (&x)[8]) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(d[i] << 16);
        x[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
}
typedef __bf16 bf16x2n_t __attribute__((ext_vector_type(2)));
typedef float f32x2n_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t narrow2(float a, float b) {      // round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2n_t){a, b}, bf16x2n_t));
}

// Sum over a row's NW waves; `slot` is LDS of the row's own, one per sum.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float *slot) {
    v = wave_sum_dpp(v);
    if constexpr (NW > 1) {
        if ((threadIdx.x & 63) == 0) slot[(threadIdx.x >> 6) % NW] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) v += slot[i];
    }
    return v;
}

// Rows of eight-element vectors: a lane holds PER vectors, NW waves a row
// (below four waves a row, several rows a workgroup).
template <int NW, int PER, bool RES32>
__global__ void __launch_bounds__(NW < 4 ? 256 : 64 * NW)
norm_vec_kernel(const NormArgs a) {
    constexpr int ROWS = NW < 4 ? 4 / NW : 1;
    __shared__ float lds[2][NW < 4 ? 4 : NW];
    const int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / (64 * NW);
    const int tid = threadIdx.x % (64 * NW);
    if (t >= a.T) return;      // whole waves of one-wave rows
    float *slot0 = lds[0], *slot1 = lds[1];
    const int nv = a.C >> 3;
    const float rc = 1.0f / (float)a.C;
    uint4 xr[PER], gr[PER], rr[PER], rr2[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int v = p * 64 * NW + tid;
        xr[p] = gr[p] = rr[p] = rr2[p] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
            xr[p] = reinterpret_cast<const uint4 *>(a.x + t * a.x_stride)[v];
            if (a.gate) gr[p] = reinterpret_cast<const uint4 *>(a.gate + t * a.gate_stride)[v];
            if constexpr (RES32) {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.res) + t * a.res_stride);
                rr[p] = src[2 * v];
                rr2[p] = src[2 * v + 1];
            } else {
                rr[p] = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.res) + t * a.res_stride)[v];
            }
        }
    }
    float inv = 1.0f;
    if (a.post_w) {
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            float x[8];
            widen8(xr[p], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
        }
        inv = 1.0f / __builtin_sqrtf(row_sum<NW>(sum, slot0) * rc + a.eps);
    }
    float r[PER][8], sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int v = p * 64 * NW + tid;
        float x[8], w[8];
        widen8(xr[p], x);
        if (a.post_w) {
            widen8(v < nv ? reinterpret_cast<const uint4 *>(a.post_w)[v] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * (w[j] + a.w_offset);
        }
        if (a.gate) {
            widen8(gr[p], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= w[j];
        }
        if constexpr (RES32) {
            const uint32_t d[8] = {rr[p].x, rr[p].y, rr[p].z, rr[p].w, rr2[p].x, rr2[p].y, rr2[p].z, rr2[p].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(d[j]);
        } else {
            widen8(rr[p], w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[p][j] = __builtin_fmaf(a.res_scale, x[j], w[j]);
            sum = __builtin_fmaf(r[p][j], r[p][j], sum);
        }
        if (v < nv) {
            if constexpr (RES32) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.res_out) + t * a.res_out_stride);
                dst[2 * v] = make_float4(r[p][0], r[p][1], r[p][2], r[p][3]);
                dst[2 * v + 1] = make_float4(r[p][4], r[p][5], r[p][6], r[p][7]);
            } else {
                reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.res_out) + t * a.res_out_stride)[v] =
                    make_uint4(narrow2(r[p][0], r[p][1]), narrow2(r[p][2], r[p][3]), narrow2(r[p][4], r[p][5]),
                               narrow2(r[p][6], r[p][7]));
            }
        }
    }
    inv = 1.0f / __builtin_sqrtf(row_sum<NW>(sum, slot1) * rc + a.eps);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int v = p * 64 * NW + tid;
        if (v >= nv) continue;
        float w[8];
        widen8(reinterpret_cast<const uint4 *>(a.pre_w)[v], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r[p][j] * inv * (w[j] + a.w_offset);
        const uint4 h = make_uint4(narrow2(w[0], w[1]), narrow2(w[2], w[3]), narrow2(w[4], w[5]), narrow2(w[6], w[7]));
        reinterpret_cast<uint4 *>(a.h + t * a.h_stride)[v] = h;
        if (a.a_codes) {      // C % 32 == 0: both lanes of a block of 16 are here
            const uint32_t d[4] = {h.x, h.y, h.z, h.w};
            uint32_t am = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) am = max(am, max(d[j] & 0x7FFFu, (d[j] >> 16) & 0x7FFFu));
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
            const uint32_t sb = f32_to_e4m3_rne(bf16_to_f32(am) / 6.0f);
            const float s = sb ? e4m3_to_f32(sb) : 1.0f;
            const float q = sb ? 1.0f / s : 0.0f;
            uint32_t c = fp4_pair<0>(0u, d[0], s, q);
            c = fp4_pair<1>(c, d[1], s, q);
            c = fp4_pair<2>(c, d[2], s, q);
            c = fp4_pair<3>(c, d[3], s, q);
            reinterpret_cast<uint32_t *>(a.a_codes + t * (a.C / 2))[v] = c;
            if ((v & 1) == 0) a.a_scales[t * (a.C / 16) + (v >> 1)] = (uint8_t)sb;
        }
    }
}

// Element i of row t of h, an element a lane, and its code: with codes
// C % 32 == 0, so the 16 lanes of a block are all here or none is.
__device__ __forceinline__ void store_any(const NormArgs &a, int64_t t, int i, float v) {
    const uint32_t h = f32_to_bf16_rne(v);
    a.h[t * a.h_stride + i] = (uint16_t)h;
    if (!a.a_codes) return;
    uint32_t am = h & 0x7FFFu;
    am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
    am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x4E, 0xF, 0xF, false));
    am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x141, 0xF, 0xF, false));
    am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x140, 0xF, 0xF, false));
    const uint32_t sb = f32_to_e4m3_rne(bf16_to_f32(am) / 6.0f);
    const uint32_t mag = sb ? e2m1_mag_code(bf16_to_f32(h & 0x7FFFu), e4m3_to_f32(sb)) : 0u;
    const uint32_t code = mag | ((h >> 12) & 8u);
    const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)code, 0xB1, 0xF, 0xF, false);
    if ((i & 1) == 0) a.a_codes[t * (a.C / 2) + (i >> 1)] = (uint8_t)(code | (next << 4));
    if ((i & 15) == 0) a.a_scales[t * (a.C / 16) + (i >> 4)] = (uint8_t)sb;
}

// Any C, any strides: an element a lane, PER times, 64 * NW lanes a row.
template <int NW, int PER>
__global__ void __launch_bounds__(64 * NW)
norm_any_kernel(const NormArgs a) {
    __shared__ float lds[2][NW];
    const int64_t t = blockIdx.x;
    const float rc = 1.0f / (float)a.C;
    const uint16_t *gate = a.gate ? a.gate + t * a.gate_stride : nullptr;
    float x[PER], sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = p * 64 * NW + threadIdx.x;
        x[p] = i < a.C ? bf16_to_f32(a.x[t * a.x_stride + i]) : 0.0f;
        sum = __builtin_fmaf(x[p], x[p], sum);
    }
    float inv = 1.0f;
    if (a.post_w) inv = 1.0f / __builtin_sqrtf(row_sum<NW>(sum, lds[0]) * rc + a.eps);
    sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = p * 64 * NW + threadIdx.x;
        if (i < a.C) {
            if (a.post_w) x[p] = x[p] * inv * (bf16_to_f32(a.post_w[i]) + a.w_offset);
            if (gate) x[p] *= bf16_to_f32(gate[i]);
            const float res = a.res_fp32 ? static_cast<const float *>(a.res)[t * a.res_stride + i]
                                         : bf16_to_f32(static_cast<const uint16_t *>(a.res)[t * a.res_stride + i]);
            x[p] = __builtin_fmaf(a.res_scale, x[p], res);
            if (a.res_fp32) static_cast<float *>(a.res_out)[t * a.res_out_stride + i] = x[p];
            else static_cast<uint16_t *>(a.res_out)[t * a.res_out_stride + i] = f32_to_bf16_rne(x[p]);
            sum = __builtin_fmaf(x[p], x[p], sum);
        }
    }
    inv = 1.0f / __builtin_sqrtf(row_sum<NW>(sum, lds[1]) * rc + a.eps);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = p * 64 * NW + threadIdx.x;
        if (i < a.C) store_any(a, t, i, x[p] * inv * (bf16_to_f32(a.pre_w[i]) + a.w_offset));
    }
}

// The same for rows too long for registers: r' waits in LDS (160 KB a CU on
// gfx950) between the two sums.
constexpr int kLongRow = 32768, kLongThreads = 1024;
__global__ void __launch_bounds__(kLongThreads)
norm_long_kernel(const NormArgs a) {
    __shared__ float lds[2][kLongThreads / 64];
    __shared__ float row[kLongRow];
    const int64_t t = blockIdx.x;
    const float rc = 1.0f / (float)a.C;
    const uint16_t *x = a.x + t * a.x_stride;
    const uint16_t *gate = a.gate ? a.gate + t * a.gate_stride : nullptr;
    float sum = 0.0f, inv = 1.0f;
    if (a.post_w) {
        for (int i = threadIdx.x; i < a.C; i += kLongThreads) {
            const float v = bf16_to_f32(x[i]);
            sum = __builtin_fmaf(v, v, sum);
        }
        inv = 1.0f / __builtin_sqrtf(row_sum<kLongThreads / 64>(sum, lds[0]) * rc + a.eps);
    }
    sum = 0.0f;
    for (int i = threadIdx.x; i < a.C; i += kLongThreads) {
        float v = bf16_to_f32(x[i]);
        if (a.post_w) v = v * inv * (bf16_to_f32(a.post_w[i]) + a.w_offset);
        if (gate) v *= bf16_to_f32(gate[i]);
        const float res = a.res_fp32 ? static_cast<const float *>(a.res)[t * a.res_stride + i]
                                     : bf16_to_f32(static_cast<const uint16_t *>(a.res)[t * a.res_stride + i]);
        v = __builtin_fmaf(a.res_scale, v, res);
        if (a.res_fp32) static_cast<float *>(a.res_out)[t * a.res_out_stride + i] = v;
        else static_cast<uint16_t *>(a.res_out)[t * a.res_out_stride + i] = f32_to_bf16_rne(v);
        row[i] = v;      // read back by this thread only
        sum = __builtin_fmaf(v, v, sum);
    }
    inv = 1.0f / __builtin_sqrtf(row_sum<kLongThreads / 64>(sum, lds[1]) * rc + a.eps);
    for (int i = threadIdx.x; i < a.C; i += kLongThreads)
        store_any(a, t, i, row[i] * inv * (bf16_to_f32(a.pre_w[i]) + a.w_offset));
}

template <int NW, int PER>
hipError_t launch_vec(const NormArgs &a, hipStream_t stream) {
    constexpr int ROWS = NW < 4 ? 4 / NW : 1, NT = NW < 4 ? 256 : 64 * NW;
    const unsigned grid = (unsigned)(((int64_t)a.T + ROWS - 1) / ROWS);
    if (!fits_grid(grid, NT)) return hipErrorInvalidConfiguration;
    if (a.res_fp32) hipLaunchKernelGGL((norm_vec_kernel<NW, PER, true>), dim3(grid), dim3(NT), 0, stream, a);
    else hipLaunchKernelGGL((norm_vec_kernel<NW, PER, false>), dim3(grid), dim3(NT), 0, stream, a);
    return hipGetLastError();
}

template <int NW, int PER>
hipError_t launch_any(const NormArgs &a, hipStream_t stream) {
    if (!fits_grid(a.T, 64 * NW)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((norm_any_kernel<NW, PER>), dim3((unsigned)a.T), dim3(64 * NW), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// Few rows: as many waves a row as its vectors fill (the call is a chain of
// latencies).  Many rows: fewer waves with more vectors each, so that a row's
// reductions join few waves and other rows run meanwhile.
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
    const int64_t strides = a.x_stride | a.res_stride | a.res_out_stride | a.h_stride | (a.gate ? a.gate_stride : 0);
    if (a.C % 8 == 0 && strides % 8 == 0) {
        const int nv = a.C / 8;
        if (nv <= 64) return launch_vec<1, 1>(a, stream);
        if (a.T <= 512) {
            if (nv <= 256) return launch_vec<4, 1>(a, stream);
            if (nv <= 512) return launch_vec<8, 1>(a, stream);
            if (nv <= 1024) return launch_vec<16, 1>(a, stream);
        } else {
            if (nv <= 128) return launch_vec<1, 2>(a, stream);
            if (nv <= 256) return launch_vec<1, 4>(a, stream);
            if (nv <= 512) return launch_vec<4, 2>(a, stream);
            if (nv <= 1024) return launch_vec<4, 4>(a, stream);
        }
        if (nv <= 2048) return launch_vec<8, 4>(a, stream);
        return launch_vec<16, 4>(a, stream);
    }
    if (a.C <= 1024) return launch_any<4, 4>(a, stream);
    if (a.C <= 4096) return launch_any<16, 4>(a, stream);
    if (a.C <= 16384) return launch_any<16, 16>(a, stream);
    if (!fits_grid(a.T, kLongThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(norm_long_kernel, dim3((unsigned)a.T), dim3(kLongThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace biloco
