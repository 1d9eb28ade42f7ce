// MX4 (OCP Microscaling Formats v1.0, MXFP4) on gfx950: 32 values share one E8M0 scale 2^(s - 127),
// each value an E2M1 code, two codes per byte with element 2i in the low nibble.
#pragma once

#include "moe_common.hpp"

namespace moe {

typedef int i32x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

constexpr int MX_BLOCK = 32;
constexpr uint32_t MX_NAN = 0xFFu;      // E8M0 NaN: every value of the block is NaN

// E8M0 code -> fp32: 2^(s - 127), 2^-127 being subnormal; 0xFF is NaN.
__device__ __forceinline__ float e8m0_f32(uint32_t s)
{
    const uint32_t u = s << 23;
    return __uint_as_float(s == 0 ? 0x00400000u : (s == MX_NAN ? 0x7FC00000u : u));
}

// The scale of a block whose largest magnitude has the fp32 bits `amax`: exponent
// floor(log2(amax)) - 2 (E2M1's largest exponent), clamped at 2^-127; NaN when the block holds a
// NaN or an infinity.  amax = 0 gives 2^-127.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax)
{
    const int e = (int)(amax >> 23);
    return e == 255 ? MX_NAN : (uint32_t)(e > 2 ? e - 2 : 0);
}

// v[0..7] / 2^(s - 127) rounded to E2M1: nearest, ties to the even code, saturating at 6 (the
// conversion instruction's own rule; 2^(s-127) is a power of two, so the quotient is exact).
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8], float scale)
{
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
    return r;
}

// Eight codes times 2^(s - 127) as bf16 (exact: two significand bits).
__device__ __forceinline__ bf16x8 mx4_bf16x8(uint32_t codes, float scale)
{
    U4 r;
    r.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    r.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    r.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    r.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    return r.v;
}

}  // namespace moe
