// Residual addition and RMS norm of token rows, with a bf16 output and an
// optional MXFP8 output:
//   s = x + residual;  v = s / sqrt(mean(s^2) + eps) * (offset + weight);
//   residual_out = s, y = bf16(v), (q, qs) = MXFP8(v).
// s is fp32 and its squares are summed in fp64. For the MXFP8 output v is the
// fp32 number nearest to the exact product with what it was rounded off by,
// and s carries what a sum with an fp32 residual was rounded off by: a code
// changes where v crosses a tie, which an error of 1e-7 does for one element
// in a million, and a scale where the block's largest crosses the border of
// two (eights of squares in fp32 were worth 0.7 us at 1531 rows of 2784, which
// take 12, and changed single codes). y and q are each rounded once from v.
//
// Bound by memory: 8 bytes an element with bf16 streams, about 9 with the
// MXFP8 output. A row is read once and stays in registers between the sum and
// the outputs. Every element is read and written by one lane, so outputs may
// be the inputs' own buffers. 16384 rows of 3584 with both outputs take 91 us,
// 5.8 TB/s (a plain copy of 1 GiB: 5.1). Streaming stores count in that
// (ordinary ones: 95 us), and four waves a row (a wave a row, with 56 elements
// a lane: 117 us with ordinary stores). Rows at any element address: 19248 of
// 2794, bf16 residual and output, 109 us (element by element: 200).
#include "common.hpp"
#include "dense.hpp"
#include "mx8.hpp"

namespace moe {

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// (s + sl) * r * w as the nearest fp32 number and the rest, for r = rh + rl
// and sl, rl at most half a step of s and rh: exact products by fma, to about
// 2^-45. NaN and infinities come from the plain product.
struct Product {
    float v, rest;
};
__device__ __forceinline__ Product product3(float s, float sl, float rh, float rl, float w) {
#pragma clang fp contract(off)  // p and v are the rounded products
    const float p = s * rh;
    const float ep = fmaf(sl, rh, fmaf(s, rl, fmaf(s, rh, -p)));
    const float v = p * w;
    const float ev = fmaf(ep, w, fmaf(p, w, -v));
    const float n = v + ev;
    const bool fine = fabsf(n) < __builtin_inff();
    return {fine ? n : v, fine ? (v - n) + ev : 0.0f};
}

// Whether z can be halfway between two e4m3 codes: ties have four mantissa bits
// in the normal range and at most three below 2^-6.
__device__ __forceinline__ bool may_tie(float z) { return (__float_as_uint(z) & 0x7ffffu) == 0u; }

// z = v * inv for its e4m3 code: a tie goes by the rest that v was rounded off
// by, one step of z towards it. (A code, or a number between code and tie, is
// rounded as before from there.)
__device__ __forceinline__ float settle(float z, float rest) {
    const int step = ((int)(__float_as_uint(z) ^ __float_as_uint(rest)) >> 31) | 1;
    return may_tie(z) && rest != 0.0f && z != 0.0f ? __uint_as_float(__float_as_uint(z) + (uint32_t)step) : z;
}

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

}  // namespace

// WAVES waves hold a row of at most WAVES * 512 * NC elements. WAVES == 1:
// four rows a workgroup.
template <int WAVES, int NC, bool VEC>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void rms_norm_kernel(NormArgs a) {
    constexpr int kLanes = WAVES * 64;
    const int tid = WAVES == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int t = WAVES == 1 ? (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)
                             : (int)blockIdx.x;
    if (WAVES == 1 && t >= a.T) return;  // whole waves; no barrier below when WAVES == 1
    const uint16_t* xr = a.x + t * a.ldx;
    const char* rr = (const char*)a.residual + t * a.ldr * (a.res_f32 ? 4 : 2);
    char* ro = (char*)a.residual_out + t * a.ldro * (a.res_f32 ? 4 : 2);
    const int H = a.H;
    // Chunk c of this lane: elements [first(c), +8).
    auto first = [&](int c) { return (c * kLanes + tid) * 8; };
    f32x8 s[NC], sl[NC];  // sl: what an fp32 residual's sum was rounded off by
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        if (i < H) {
            s[c] = load8<VEC>(xr, false, i, H);
            sl[c] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (a.residual) {
                const f32x8 x = s[c], r = load8<VEC>(rr, a.res_f32, i, H);
                s[c] = x + r;
                if (a.res_f32) {
                    const f32x8 b = s[c] - x;
                    sl[c] = (x - (s[c] - b)) + (r - b);
                }
            }
        } else {
            s[c] = sl[c] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        if (a.residual_out && i < H) store8<VEC>(ro, a.res_f32, i, H, s[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fma((double)s[c][e], (double)s[c][e], sum);
    }
    sum = wave_sum(sum);
    if constexpr (WAVES > 1) {
        __shared__ double part[WAVES];
        if ((tid & 63) == 0) part[tid >> 6] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += part[w];
    }
    const double root = 1.0 / sqrt(sum / (double)H + (double)a.eps);
    const float rh = (float)root;
    const float rl = fabsf(rh) < __builtin_inff() ? (float)(root - (double)rh) : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        if (i >= H) continue;
        f32x8 v = load8<VEC>(a.weight, a.weight_f32, i, H);
        Product p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.q) p[e] = product3(s[c][e], sl[c][e], rh, rl, a.offset + v[e]);
            else p[e] = {s[c][e] * rh * (a.offset + v[e]), 0.0f};  // bf16 needs no more
            v[e] = p[e].v;
        }
        if (a.y) store8<VEC>(a.y + t * a.ldy, false, i, H, v);
        if (a.q) {
            uint8_t* qr = a.q + t * a.ldq;
            uint8_t* sr = a.qs + t * a.ldqs;
            // A block of 32 is four lanes' chunks; H % 32 == 0, so a block is
            // inside the row for all of its lanes or none.
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, mx8_finite_abs(v[e]));
            m = fmaxf(m, dpp<0xB1>(m));
            m = fmaxf(m, dpp<0x4E>(m));
            // A maximum that rounds to the border of two scales goes by its rest
            // (the four lanes have the same m).
            float above = 0.0f;
            if (mx8_at_border(m)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    above = fabsf(v[e]) == m && p[e].rest != 0.0f && (p[e].rest > 0.0f) == (v[e] > 0.0f) ? 1.0f : above;
                above = fmaxf(above, dpp<0xB1>(above));
                above = fmaxf(above, dpp<0x4E>(above));
            }
            const uint32_t b = mx8_scale_byte(m, above > 0.0f);
            const float inv = mx8_inv_scale(b);
            u32x2 o;
            bool ties = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= inv;
                ties |= may_tie(v[e]);
            }
            if (ties) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = settle(v[e], p[e].rest);
            }
            o[0] = mx8_pack4(v[0], v[1], v[2], v[3], 1.0f);
            o[1] = mx8_pack4(v[4], v[5], v[6], v[7], 1.0f);
            if constexpr (VEC) __builtin_nontemporal_store(o, (u32x2*)(qr + i));
            else *(u32x2_any*)(qr + i) = o;
            if ((tid & 3) == 0) sr[i >> 5] = (uint8_t)b;
        }
    }
}

template <int WAVES, int NC>
static void launch(const NormArgs& a, bool vec, hipStream_t s) {
    const dim3 grid(WAVES == 1 ? (unsigned)((a.T + 3) / 4) : (unsigned)a.T), block(WAVES == 1 ? 256 : WAVES * 64);
    if (vec) hipLaunchKernelGGL((rms_norm_kernel<WAVES, NC, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_norm_kernel<WAVES, NC, false>), grid, block, 0, s, a);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
    // A launch holds fewer than 2^32 threads (1024 a row at most).
    constexpr int kMostRows = 1 << 21;
    if (a.T > kMostRows) {
        for (int t = 0; t < a.T; t += kMostRows) {
            NormArgs b = a;
            const int64_t rb = a.res_f32 ? 4 : 2;
            b.T = a.T - t < kMostRows ? a.T - t : kMostRows;
            b.x = a.x + t * a.ldx;
            if (a.residual) b.residual = (const char*)a.residual + t * a.ldr * rb;
            if (a.residual_out) b.residual_out = (char*)a.residual_out + t * a.ldro * rb;
            if (a.y) b.y = a.y + t * a.ldy;
            if (a.q) {
                b.q = a.q + t * a.ldq;
                b.qs = a.qs + t * a.ldqs;
            }
            const hipError_t e = launch_rms_norm(b, s);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    auto ok = [](const void* p, int64_t ld, int bytes) {
        return p == nullptr || ((uintptr_t)p % 16 == 0 && (ld * bytes) % 16 == 0);
    };
    const int rb = a.res_f32 ? 4 : 2;
    const bool vec = a.H % 8 == 0 && ok(a.x, a.ldx, 2) && ok(a.residual, a.ldr, rb) &&
                     ok(a.residual_out, a.ldro, rb) && ok(a.y, a.ldy, 2) && ok(a.weight, 0, 4) &&
                     (a.q == nullptr || ((uintptr_t)a.q % 8 == 0 && a.ldq % 8 == 0));
    // A wave a row while that is one load a lane, else four waves (16384 rows,
    // ordinary stores: of 256, 10.3 us against 15.3; of 512, 14.7 against 16.4;
    // of 1024, 33.4 against 33.9; of 3584, 117 against 95).
    if (a.H <= 512) launch<1, 1>(a, vec, s);
    else if (a.H <= 2048) launch<4, 1>(a, vec, s);
    else if (a.H <= 4096) launch<4, 2>(a, vec, s);
    else if (a.H <= 8192) launch<4, 4>(a, vec, s);
    else if (a.H <= 16384) launch<4, 8>(a, vec, s);
    else if (a.H <= 32768) launch<16, 4>(a, vec, s);
    else launch<16, 8>(a, vec, s);  // spills 172 bytes a lane
    return hipGetLastError();
}

}  // namespace moe
