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
// wide load or store takes as well. The row's last eight may be fewer: they are
// taken four, two and one at a time, by the bits of H, which all rows share.
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef f32x2 __attribute__((aligned(4))) f32x2_any;
typedef u16x8 __attribute__((aligned(2))) u16x8_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_half;
typedef uint32_t __attribute__((aligned(2))) u32_half;

__device__ __forceinline__ float low_half(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float high_half(uint32_t d) { return __uint_as_float(d & 0xffff0000u); }

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
        const bool four = H & 4, two = H & 2, one = H & 1;
        f32x4 a = {0, 0, 0, 0};
        f32x2 b = {0, 0};
        float c = 0.0f;
        if (f32) {
            const float* p = (const float*)row + i;
            if (four) a = *(const f32x4_any*)p;
            if (two) b = *(const f32x2_any*)(p + (four ? 4 : 0));
            if (one) c = p[(four ? 4 : 0) + (two ? 2 : 0)];
        } else {
            const uint16_t* p = (const uint16_t*)row + i;
            if (four) {
                const u32x2 d = *(const u32x2_half*)p;
                a = f32x4{low_half(d[0]), high_half(d[0]), low_half(d[1]), high_half(d[1])};
            }
            if (two) {
                const uint32_t d = *(const u32_half*)(p + (four ? 4 : 0));
                b = f32x2{low_half(d), high_half(d)};
            }
            if (one) c = bf16_bits_to_f32(p[(four ? 4 : 0) + (two ? 2 : 0)]);
        }
        // Behind each other.
        const f32x4 t = two ? f32x4{b[0], b[1], c, 0.0f} : f32x4{c, 0.0f, 0.0f, 0.0f};
        const f32x4 zero = {0, 0, 0, 0};
        r = four ? __builtin_shufflevector(a, t, 0, 1, 2, 3, 4, 5, 6, 7) : __builtin_shufflevector(t, zero, 0, 1, 2, 3, 4, 5, 6, 7);
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
        const bool four = H & 4, two = H & 2;
        const f32x4 t = four ? __builtin_shufflevector(v, v, 4, 5, 6, 7) : __builtin_shufflevector(v, v, 0, 1, 2, 3);
        const float last = two ? t[2] : t[0];
        const int b = four ? 4 : 0, c = b + (two ? 2 : 0);
        if (f32) {
            float* p = (float*)row + i;
            if (four) *(f32x4_any*)p = __builtin_shufflevector(v, v, 0, 1, 2, 3);
            if (two) *(f32x2_any*)(p + b) = f32x2{t[0], t[1]};
            if (H & 1) p[c] = last;
        } else {
            uint16_t* p = (uint16_t*)row + i;
            if (four) *(u32x2_half*)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            if (two) *(u32_half*)(p + b) = pack_bf16x2(t[0], t[1]);
            if (H & 1) p[c] = f32_to_bf16_bits(last);
        }
    }
}

// The same in two halves, so that nothing waits between the loads of a row's
// several operands: fetch8 loads (what it loads for f32 and for bf16 differs,
// but no branch holds an arithmetic instruction), widen8 makes numbers of it.
// MODE kAligned as VEC; kTiny: H < 8. kAnywhere: any element's address and H >=
// 8, where the lane of the row's last elements takes the last eight, from H - 8
// on: the first skip8 of them are its neighbour's, who sums and stores them.
// (Moving the lane's own to the front instead took a wave that holds a whole row
// some half more: 32768 rows of 333, layer norm, 33 us, 22 so.)
constexpr int kAligned = 0, kAnywhere = 1, kTiny = 2;

struct Raw8 {
    u32x4 a, b;
};

template <int MODE>
__device__ __forceinline__ Raw8 fetch8(const void* row, bool f32, int i, int H) {
    Raw8 r;
    if constexpr (MODE == kTiny) {
        const f32x8 v = load8<false>(row, f32, i, H);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.a[e] = __float_as_uint(v[e]);
            r.b[e] = __float_as_uint(v[e + 4]);
        }
    } else {
        const int at = MODE == kAligned || i + 8 <= H ? i : H - 8;
        if (f32) {
            const float* p = (const float*)row + at;
            if constexpr (MODE == kAligned) {
                r.a = ((const u32x4*)p)[0];
                r.b = ((const u32x4*)p)[1];
            } else {
                r.a = __builtin_bit_cast(u32x4, *(const f32x4_any*)p);
                r.b = __builtin_bit_cast(u32x4, *(const f32x4_any*)(p + 4));
            }
        } else {
            const uint16_t* p = (const uint16_t*)row + at;
            if constexpr (MODE == kAligned) r.a = *(const u32x4*)p;
            else r.a = *(const u32x4_any*)p;
        }
    }
    return r;
}

template <int MODE>
__device__ __forceinline__ f32x8 widen8(Raw8 r, bool f32, int i, int H) {
    f32x8 v;
    if (MODE == kTiny || f32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(r.a[e]);
            v[e + 4] = __uint_as_float(r.b[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = low_half(r.a[e]);
            v[2 * e + 1] = high_half(r.a[e]);
        }
    }
    return v;
}

template <int MODE>
__device__ __forceinline__ int skip8(int i, int H) {
    return MODE == kAnywhere && i + 8 > H ? i + 8 - H : 0;
}

template <int MODE>
__device__ __forceinline__ void put8(void* row, bool f32, int i, int H, f32x8 v) {
    if (MODE != kAnywhere || i + 8 <= H) {
        store8<MODE == kAligned>(row, f32, i, H, v);
        return;
    }
    // The last H % 8 of v, one, two and four from the end.
    const bool one = H & 1, two = H & 2;
    const f32x2 b = one ? f32x2{v[5], v[6]} : f32x2{v[6], v[7]};
    const f32x4 lo = __builtin_shufflevector(v, v, 1, 2, 3, 4), l2 = __builtin_shufflevector(v, v, 2, 3, 4, 5);
    const f32x4 l3 = __builtin_shufflevector(v, v, 3, 4, 5, 6), l4 = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    const f32x4 c = one ? (two ? lo : l3) : (two ? l2 : l4);
    const int at1 = H - 1, at2 = H - (one ? 3 : 2), at4 = i;
    if (f32) {
        float* p = (float*)row;
        if (one) p[at1] = v[7];
        if (two) *(f32x2_any*)(p + at2) = b;
        if (H & 4) *(f32x4_any*)(p + at4) = c;
    } else {
        uint16_t* p = (uint16_t*)row;
        if (one) p[at1] = f32_to_bf16_bits(v[7]);
        if (two) *(u32_half*)(p + at2) = pack_bf16x2(b[0], b[1]);
        if (H & 4) *(u32x2_half*)(p + at4) = u32x2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
    }
}

}  // namespace rows
}  // namespace moe
