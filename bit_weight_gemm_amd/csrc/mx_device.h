// Microscaled 4-bit floats: E2M1 codes, two a byte, the even element in the low
// nibble, and for 32 of them a scale byte b that stands for 2^(b - 127); 255 is NaN.
#pragma once
#include "biloco_device.h"
#include "biloco_internal.h"

namespace biloco {
namespace mx {

typedef __bf16 bf16x2m_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2m_t __attribute__((ext_vector_type(2)));
typedef float f32x4m_t __attribute__((ext_vector_type(4)));
typedef float f32x16m_t __attribute__((ext_vector_type(16)));
typedef int i32x8m_t __attribute__((ext_vector_type(8)));

constexpr uint32_t kInf = 0x7F800000u;      // magnitude bits from here on: not finite

// Scale byte of a block whose largest magnitude has these fp32 bits: that one's
// exponent less two, E2M1's largest, so that it lands in [4, 8) and saturates from 6 on.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    return amax_bits >= kInf ? 255u : (uint32_t)max((int)(amax_bits >> 23) - 2, 0);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {      // of a byte below 255
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// By value: a vector's element is no lvalue of its own for a bit cast.
__device__ __forceinline__ bf16x2m_t pair_of(uint32_t w) { return __builtin_bit_cast(bf16x2m_t, w); }
__device__ __forceinline__ u16x2m_t halves_of(uint32_t w) { return __builtin_bit_cast(u16x2m_t, w); }

// Eight elements to a dword of codes.  The conversion divides by the scale (a power
// of two: exact), rounds to nearest, ties to the even code, and saturates at 6; checked
// against that on gfx950 over all midpoints and neighbours, at scales from 2^-127 on.
__device__ __forceinline__ uint32_t codes8(const u32x4_t &w, float s) {      // bf16
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w.x), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w.y), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w.z), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w.w), s, 3);
}
__device__ __forceinline__ uint32_t codes8(const f32x4m_t &a, const f32x4m_t &b, float s) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], s, 3);
}
// Largest magnitude of eight bf16, as fp32 bits.
__device__ __forceinline__ uint32_t amax8(const u32x4_t &w) {
    const u32x4_t a = w & 0x7FFF7FFFu;
    u16x2m_t m = halves_of(a.x);
    m = __builtin_elementwise_max(m, halves_of(a.y));
    m = __builtin_elementwise_max(m, halves_of(a.z));
    m = __builtin_elementwise_max(m, halves_of(a.w));
    return (uint32_t)max(m[0], m[1]) << 16;
}
__device__ __forceinline__ uint32_t amax8(const f32x4m_t &a, const f32x4m_t &b) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(a[i]) & 0x7FFFFFFFu, __float_as_uint(b[i]) & 0x7FFFFFFFu));
    return m;
}

}  // namespace mx
}  // namespace biloco
