// Rows to microscaled 4-bit floats and back.
//
//   e = exponent of max |x| over 32 elements, less 2 (E2M1's largest exponent)
//   code = E2M1(x / 2^e), to nearest, ties to even, saturating at 6;  x ~ code 2^e
//
// A lane takes eight elements (16 or 32 bytes), four lanes a block; the maximum goes
// over the four by two lane permutations.  Bound by memory.
#include "mx_device.h"

namespace biloco {

namespace {

using namespace mx;

// Eight-element groups of rows: element offset of group u.
struct Groups {
    int64_t n;           // groups in all
    uint32_t per;        // a row; 0: the rows follow one another without a gap
    int64_t stride;      // elements from row to row
    __device__ __forceinline__ int64_t at(int64_t u) const {
        if (per == 0) return u * 8;
        const int64_t row = u < 0x100000000ll ? (int64_t)((uint32_t)u / per) : u / per;
        return row * stride + (u - row * per) * 8;
    }
};

template <class T, int N>
__global__ void __launch_bounds__(256)
quant_mxfp4_kernel(const T *__restrict__ x, Groups g, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int64_t u0 = (int64_t)blockIdx.x * (256 * N) + threadIdx.x;
    uint32_t amax[N];
    u32x4_t w[N];
    f32x4m_t a[N], b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t u = min(u0 + 256 * i, g.n - 1);
        if constexpr (sizeof(T) == 2) {
            w[i] = *reinterpret_cast<const u32x4_t *>(x + g.at(u));
        } else {
            const f32x4m_t *p = reinterpret_cast<const f32x4m_t *>(x + g.at(u));
            a[i] = p[0];
            b[i] = p[1];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (sizeof(T) == 2) amax[i] = amax8(w[i]);
        else amax[i] = amax8(a[i], b[i]);
        amax[i] = max(amax[i], (uint32_t)__shfl_xor((int)amax[i], 1, 64));
        amax[i] = max(amax[i], (uint32_t)__shfl_xor((int)amax[i], 2, 64));
        const uint32_t byte = scale_byte(amax[i]);
        const float s = scale_value(min(byte, 254u));
        uint32_t c;
        if constexpr (sizeof(T) == 2) c = codes8(w[i], s);
        else c = codes8(a[i], b[i], s);
        const int64_t u = u0 + 256 * i;
        if (u < g.n) {
            reinterpret_cast<uint32_t *>(codes)[u] = byte == 255u ? 0u : c;
            if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)byte;
        }
    }
}

template <class T, int N>
__global__ void __launch_bounds__(256)
dequant_mxfp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, Groups g, T *__restrict__ out) {
    const int64_t u0 = (int64_t)blockIdx.x * (256 * N) + threadIdx.x;
    uint32_t c[N], e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t u = min(u0 + 256 * i, g.n - 1);
        c[i] = reinterpret_cast<const uint32_t *>(codes)[u];
        e[i] = scales[u >> 2];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t u = u0 + 256 * i;
        const float s = scale_value(min(e[i], 254u));
        if (u >= g.n) continue;
        T *to = out + g.at(u);
        if constexpr (sizeof(T) == 2) {
            u32x4_t v;
            v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 0));
            v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 1));
            v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 2));
            v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 3));
            *reinterpret_cast<u32x4_t *>(to) = e[i] == 255u ? u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u} : v;
        } else {
            const float nan = __builtin_nanf("");
            const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 1),
                       p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 3);
            f32x4m_t lo{p0[0], p0[1], p1[0], p1[1]}, hi{p2[0], p2[1], p3[0], p3[1]};
            if (e[i] == 255u) lo = hi = f32x4m_t{nan, nan, nan, nan};
            reinterpret_cast<f32x4m_t *>(to)[0] = lo;
            reinterpret_cast<f32x4m_t *>(to)[1] = hi;
        }
    }
}

Groups groups_of(int64_t rows, int64_t K, int64_t stride) {
    Groups g;
    g.n = rows * (K / 8);
    g.per = stride == K ? 0u : (uint32_t)(K / 8);
    g.stride = stride;
    return g;
}
// Few groups: one a lane, so that they spread over more CUs (bf16 rows of 5120: 819 of them 3.5
// us, with four a lane 4.0; 1638 4.9 and 5.2; 4096 the same).
constexpr int64_t kFew = 1 << 21;
int64_t grid_of(int64_t n, int each) { return (n + 256 * each - 1) / (256 * each); }

}  // namespace

bool mxfp4_rows_fit(int64_t M, int64_t K) {
    const int64_t n = M * (K / 8);
    return fits_grid(grid_of(n, n <= kFew ? 1 : 4), 256);
}

hipError_t launch_quant_mxfp4(const void *x, int64_t stride, bool fp32, int64_t M, int64_t K, uint8_t *codes,
                              uint8_t *scales, hipStream_t stream) {
    const Groups g = groups_of(M, K, stride);
    const int each = g.n <= kFew ? 1 : 4;
    const int64_t grid = grid_of(g.n, each);
    if (!fits_grid(grid, 256)) return hipErrorInvalidValue;
    const float *xf = static_cast<const float *>(x);
    const uint16_t *xb = static_cast<const uint16_t *>(x);
    if (fp32 && each == 1) hipLaunchKernelGGL((quant_mxfp4_kernel<float, 1>), dim3((unsigned)grid), dim3(256), 0, stream, xf, g, codes, scales);
    else if (fp32) hipLaunchKernelGGL((quant_mxfp4_kernel<float, 4>), dim3((unsigned)grid), dim3(256), 0, stream, xf, g, codes, scales);
    else if (each == 1) hipLaunchKernelGGL((quant_mxfp4_kernel<uint16_t, 1>), dim3((unsigned)grid), dim3(256), 0, stream, xb, g, codes, scales);
    else hipLaunchKernelGGL((quant_mxfp4_kernel<uint16_t, 4>), dim3((unsigned)grid), dim3(256), 0, stream, xb, g, codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K, void *out,
                                int64_t stride, bool fp32, hipStream_t stream) {
    const Groups g = groups_of(M, K, stride);
    const int each = g.n <= kFew ? 1 : 4;
    const int64_t grid = grid_of(g.n, each);
    if (!fits_grid(grid, 256)) return hipErrorInvalidValue;
    float *of = static_cast<float *>(out);
    uint16_t *ob = static_cast<uint16_t *>(out);
    if (fp32 && each == 1) hipLaunchKernelGGL((dequant_mxfp4_kernel<float, 1>), dim3((unsigned)grid), dim3(256), 0, stream, codes, scales, g, of);
    else if (fp32) hipLaunchKernelGGL((dequant_mxfp4_kernel<float, 4>), dim3((unsigned)grid), dim3(256), 0, stream, codes, scales, g, of);
    else if (each == 1) hipLaunchKernelGGL((dequant_mxfp4_kernel<uint16_t, 1>), dim3((unsigned)grid), dim3(256), 0, stream, codes, scales, g, ob);
    else hipLaunchKernelGGL((dequant_mxfp4_kernel<uint16_t, 4>), dim3((unsigned)grid), dim3(256), 0, stream, codes, scales, g, ob);
    return hipGetLastError();
}

}  // namespace biloco
