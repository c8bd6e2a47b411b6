// MXFP8: e4m3 codes with one e8m0 scale per 32 elements along K.
#pragma once

#include "common.hpp"

namespace moe {

// The e8m0 byte of a block whose largest finite magnitude is amax: the
// smallest power of two s with amax / s <= 448 (the largest e4m3), from the
// exponent and mantissa bits of amax, so no rounding decides it. amax = m 2^e
// with m in [1, 2): 448 = 1.75 * 2^8, so s = 2^(e-8) up to m = 1.75, else
// 2^(e-7). Bytes are clamped at 0 (2^-127; an all-zero block has byte 0).
// above: the magnitude is above amax by what amax was rounded off by, which
// counts where amax is at the border itself.
__device__ __forceinline__ bool mx8_at_border(float amax) { return (__float_as_uint(amax) & 0x7fffffu) == 0x600000u; }
__device__ __forceinline__ uint32_t mx8_scale_byte(float amax, bool above = false) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u || (above && mx8_at_border(amax)) ? 1 : 0);
    return (uint32_t)(e < 0 ? 0 : e);
}

// 1 / scale of a block as a float: 2^(127 - byte), exact. byte <= 247 here,
// so the result is a normal number or (byte 0) 2^127.
__device__ __forceinline__ float mx8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// |v| if finite, else 0: a NaN or infinity becomes a NaN code by itself and
// does not choose the scale of its block's other elements.
__device__ __forceinline__ float mx8_finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

// Two values times 1 / scale -> two e4m3 codes in bits [15:0], or [31:16] of
// `old` (v_cvt_pk_fp8_f32: round to nearest even; NaN and infinities give the
// NaN code, and no finite value exceeds 448 by the choice of the scale).
template <bool HIGH>
__device__ __forceinline__ uint32_t mx8_pack(float a, float b, float inv, uint32_t old) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, (int)old, HIGH);
}

__device__ __forceinline__ uint32_t mx8_pack4(float a, float b, float c, float d, float inv) {
    return mx8_pack<true>(c, d, inv, mx8_pack<false>(a, b, inv, 0u));
}

}  // namespace moe
