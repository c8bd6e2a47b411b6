// Rows of bf16 or fp32 elements by eights: loads, stores and sums over a wave
// (the norms and the row movers).
#pragma once

#include "common.hpp"

namespace moe {
namespace rows {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double join(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wave, the same in every lane: xor by 1 and 2 inside quads, then
// mirrored halves of a row, then the rows.
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
    v += dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
    v += dpp<0x141>(v);  // row_half_mirror
    v += dpp<0x140>(v);  // row_mirror
    uint64_t b = __builtin_bit_cast(uint64_t, v);
    auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = join(lo[0], hi[0]) + join(lo[1], hi[1]);
    b = __builtin_bit_cast(uint64_t, v);
    auto lo2 = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    auto hi2 = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    return join(lo2[0], hi2[0]) + join(lo2[1], hi2[1]);
}

__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    uint32_t b = __float_as_uint(v);
    auto h = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    b = __float_as_uint(v);
    auto w = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

// Eight elements i..i+7 of a row. VEC: all of them are in the row and 16-byte
// aligned (8 bytes in q); else they are at any element's address, which one
// wide load or store takes as well, and the row's last eight may be fewer.
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef u16x8 __attribute__((aligned(2))) u16x8_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;

template <bool VEC>
__device__ __forceinline__ f32x8 load8(const void* row, bool f32, int i, int H) {
    f32x8 r;
    if (VEC || i + 8 <= H) {
        if (f32) {
            const f32x4_any* p = (const f32x4_any*)((const float*)row + i);
            const f32x4 a = VEC ? *(const f32x4*)p : p[0], b = VEC ? ((const f32x4*)p)[1] : p[1];
            r = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const u16x8_any* p = (const u16x8_any*)((const uint16_t*)row + i);
            const u16x8 u = VEC ? *(const u16x8*)p : *p;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = bf16_bits_to_f32(u[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = i + e;
            r[e] = k >= H ? 0.0f : f32 ? ((const float*)row)[k] : bf16_bits_to_f32(((const uint16_t*)row)[k]);
        }
    }
    return r;
}

template <bool VEC>
__device__ __forceinline__ void store8(void* row, bool f32, int i, int H, f32x8 v) {
    if (VEC || i + 8 <= H) {
        if (f32) {
            const f32x4 lo = __builtin_shufflevector(v, v, 0, 1, 2, 3), hi = __builtin_shufflevector(v, v, 4, 5, 6, 7);
            f32x4_any* p = (f32x4_any*)((float*)row + i);
            if constexpr (VEC) {
                __builtin_nontemporal_store(lo, (f32x4*)p);
                __builtin_nontemporal_store(hi, (f32x4*)p + 1);
            } else {
                p[0] = lo;
                p[1] = hi;
            }
        } else {
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
            u32x4_any* p = (u32x4_any*)((uint16_t*)row + i);
            if constexpr (VEC) __builtin_nontemporal_store(o, (u32x4*)p);
            else *p = o;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = i + e;
            if (k >= H) continue;
            if (f32) ((float*)row)[k] = v[e];
            else ((uint16_t*)row)[k] = f32_to_bf16_bits(v[e]);
        }
    }
}

}  // namespace rows
}  // namespace moe
