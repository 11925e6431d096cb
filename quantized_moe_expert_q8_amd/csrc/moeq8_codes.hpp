// int8 codes of fp32 values: the rule of the int8 rows (scale = max / 127, the
// code roundf of the fp32 quotient), eight values a thread, and what a row's
// maximum is taken with.
#pragma once

#include "moeq8_types.hpp"

namespace moeq8 {

constexpr int VEC = 8;                            // values a thread takes at a time: a quarter of a block

// Bits of |v|: as unsigned numbers they are in the order of the magnitudes, a
// NaN above all, so a maximum of them keeps a NaN.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL, typename V>
__device__ __forceinline__ V moved(V v) {          // v of the lane that the DPP control names, an active one
    if constexpr (sizeof(V) == 8) {
        const uint2 u = __builtin_bit_cast(uint2, v);
        return __builtin_bit_cast(V, uint2{(uint32_t)__builtin_amdgcn_mov_dpp((int)u.x, CTRL, 0xf, 0xf, false),
                                           (uint32_t)__builtin_amdgcn_mov_dpp((int)u.y, CTRL, 0xf, 0xf, false)});
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    }
}
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140;

// Codes of 8 values of scale d, packed; their sum.  d = 0 and a d that is not
// finite give zeros (the scale says which).
//
// The code of y is roundf of the correctly rounded quotient y / d.  y * rcp(d)
// differs from it by less than 2.3e-5 (v_rcp_f32 within an ulp, the quotient
// rounded by half of one, both times 127), so where it lies more than 2^-14
// from every half both round to the same integer; a vector with another value,
// about one wave's in 16, takes the division.  Adding 1.5 * 2^23 rounds to an
// integer whose low byte is the code.
__device__ __forceinline__ uint2 codes8(const float (&y)[VEC], float d, int& sum) {
    uint2 o = {0u, 0u};
    sum = 0;
    if (!(d > 0.0f && d < __builtin_inff())) return o;
    constexpr float ROUND = 12582912.0f;
    const float rd = __builtin_amdgcn_rcpf(d);
    uint32_t u[VEC];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float r = __builtin_fmaf(y[i], rd, ROUND);
        off = fmaxf(off, fabsf(__builtin_fmaf(y[i], rd, ROUND - r)));
        u[i] = __float_as_uint(r);
    }
    // below the normal range the reciprocal is not what the above takes it for
    if (__builtin_expect(off >= 0.5f - 0x1p-14f || d < 0x1p-126f, 0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // d is so coarse there that a quotient may round past 127
            const int c = (int)roundf(y[i] / d);
            u[i] = (uint32_t)(c > 127 ? 127 : (c < -127 ? -127 : c));
        }
    }
    o.x = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u) | __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
    o.y = __builtin_amdgcn_perm(u[5], u[4], 0x0c0c0400u) | __builtin_amdgcn_perm(u[7], u[6], 0x04000c0cu);
    sum = __builtin_amdgcn_sdot4((int)o.x, 0x01010101, __builtin_amdgcn_sdot4((int)o.y, 0x01010101, 0, false), false);
    return o;
}

}  // namespace moeq8
