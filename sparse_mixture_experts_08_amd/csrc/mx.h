// mx.h -- device helpers of the microscaled (OCP MX) formats: groups of 32 consecutive elements share one
// E8M0 scale, a byte c that stands for 2^(c - 127) (255: NaN).  MXFP4 holds E2M1 elements (0, .5, 1, 1.5, 2,
// 3, 4, 6 and their negatives), two to a byte with the element of the lower index in the low half; MXFP8
// holds E4M3 elements (largest 448), one to a byte.
//
// Quantisation of a group: with a = max |v|, the scale's exponent is floor(log2 a) - emax, clamped to
// [-127, 127], emax the exponent of the element type's largest value (E2M1: 2, E4M3: 8); an element is
// v / scale rounded to nearest even and saturated to the largest value.  The quotient of a power of two is
// exact, so each element is rounded once.
#pragma once

#include "moe_common.h"

namespace moe {

template <bool FP4> struct MxFmt;
template <> struct MxFmt<true> { static constexpr int emax = 2; };
template <> struct MxFmt<false> { static constexpr int emax = 8; };

// Scale code of a group whose largest |v| has the bit pattern amax (sign cleared).  As bit patterns order like
// the magnitudes, infinities and NaN above every finite value, the maximum is an integer maximum.  The
// exponent field of amax minus emax is the code; subnormal maxima and zero have field 0 and take code 0, the
// clamp of their exponents.  A group with an infinity or NaN: 255.
template <bool FP4> __device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax)
{
    const int c = (int)(amax >> 23) - MxFmt<FP4>::emax;
    return amax >= 0x7F800000u ? 255u : (uint32_t)max(c, 0);
}

// Maximum over each aligned group of four lanes, returned to all four (two DPP moves).
__device__ __forceinline__ uint32_t quad_max(uint32_t u)
{
    u = max(u, dpp_u32<0xB1>(u));                      // quad_perm [1, 0, 3, 2]
    return max(u, dpp_u32<0x4E>(u));                   // quad_perm [2, 3, 0, 1]
}

// Eight elements of a group with scale code c as E2M1 codes, in order from the low half byte.  The hardware
// conversion divides by the power of two in its scale operand's exponent field (field 0 stands for 2^-127, as
// the code 0 does), rounds to nearest even and saturates.
__device__ __forceinline__ uint32_t mx_pack_fp4(const float (&v)[8], uint32_t c)
{
    const float s = __uint_as_float(c << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
    return q;
}

// Eight elements of a group with scale code c (0 .. 246) as E4M3 codes.  The product with 2^(127 - c) is exact
// except where it is subnormal, far below the smallest E4M3 value; the clamp saturates (the conversion alone
// makes NaN of values past 448).
__device__ __forceinline__ uint2 mx_pack_fp8(const float (&v)[8], uint32_t c)
{
    const float inv = __uint_as_float((254u - c) << 23);
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; e++) t[e] = __builtin_amdgcn_fmed3f(v[e] * inv, -448.0f, 448.0f);
    return make_uint2(f32x2_to_e4m3(t[0], t[1]) | (f32x2_to_e4m3(t[2], t[3]) << 16),
                      f32x2_to_e4m3(t[4], t[5]) | (f32x2_to_e4m3(t[6], t[7]) << 16));
}

// Eight of a 128-element group's values (16 lanes hold the group) as E4M3 codes of v / s, s = f8_act_scale<true>;
// s to every lane.
__device__ __forceinline__ uint2 quant8_e4m3(const float (&v)[8], float& s)
{
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(v[e]));
    amax = row16_max(amax);
    s = f8_act_scale<true>(amax);
    float t[8];
    if (quant_div_fast(s)) {
        const float r = recip_rn(s);
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = quant_div(v[e], s, r);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = v[e] / s;
    }
    return make_uint2(f32x2_to_e4m3(t[0], t[1]) | (f32x2_to_e4m3(t[2], t[3]) << 16),
                      f32x2_to_e4m3(t[4], t[5]) | (f32x2_to_e4m3(t[6], t[7]) << 16));
}

// Bit pattern maximum of the magnitudes of eight values.
__device__ __forceinline__ uint32_t mx_amax8(const float (&v)[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) a = max(a, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return a;
}

// The eight bf16 values of a 16-byte vector.
__device__ __forceinline__ void bf16x8_to_f32(const uint4& r, float (&v)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

}  // namespace moe
