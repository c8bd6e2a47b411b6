// The end of a dense product for four consecutive outputs of one token (the
// few-token kernels and the kernel that joins a split K), and what the tiles'
// epilogues share with it.
#pragma once

#include "common.hpp"
#include "dense.hpp"

namespace moe {
namespace dense {

// B[a] (scale A[a] x) of one token for rows col..col+3 (and N + col.. of the
// gated block), from v = scale * A[a] x: a dot product of at most a few
// hundred elements.
template <bool GATED>
__device__ __forceinline__ void lora_dot(const LoraArgs& l, int N, int64_t token, int col, f32x4 (&low)[2]) {
    const int ad = l.index[token];
    if ((unsigned)ad >= (unsigned)l.n) return;
    int rank = l.ranks ? l.ranks[ad] : l.rank;
    rank = rank < l.rank ? rank : l.rank;
    const uint16_t* b = l.b + ((int64_t)ad * (GATED ? 2 * (int64_t)N : N) + col) * l.rank;
    const float* v = l.v + token * l.vld;
    // Parts come without the scale, which multiplies their sum and so acts
    // within the rank alone, as where there is one part.
    const float scale = l.parts > 1 && l.scale ? l.scale[ad] : 1.0f;
    // Sixteen columns at a time; the first batch is loaded before the rank is
    // known (what lies beyond it is memory of v and B, but not read as numbers).
    for (int k0 = 0;;) {
        f32x4 vv[4];
        u32x4 w[GATED ? 2 : 1][4][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + 8 * h < l.rank ? k0 + 8 * h : k0;  // rank is a multiple of 8
            vv[2 * h] = *(const f32x4*)(v + k);
            vv[2 * h + 1] = *(const f32x4*)(v + k + 4);
            for (int p = 1; p < l.parts; ++p) {
                vv[2 * h] += *(const f32x4*)(v + p * l.part_stride + k);
                vv[2 * h + 1] += *(const f32x4*)(v + p * l.part_stride + k + 4);
            }
            vv[2 * h] *= scale;
            vv[2 * h + 1] *= scale;
#pragma unroll
            for (int s = 0; s < (GATED ? 2 : 1); ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) w[s][r][h] = *(const u32x4*)(b + ((int64_t)s * N + r) * l.rank + k);
        }
#pragma unroll
        for (int s = 0; s < (GATED ? 2 : 1); ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    // Columns beyond the adapter's rank are not read as numbers.
                    const uint32_t d = w[s][r][e / 8][e % 8 / 2];
                    const float f = __uint_as_float(e & 1 ? d & 0xffff0000u : d << 16);
                    if (k0 + e < rank) low[s][r] = fmaf(f, vv[e / 4][e % 4], low[s][r]);
                }
        k0 += 16;
        if (k0 >= rank) break;
    }
}

// With the hardware exp2 and reciprocal, about an ulp each (and |g| 2^-24 from
// the exponent's product): every output of it is rounded to bf16 or e4m3. The
// accurate expf and quotient are some 40 vector instructions for each of the
// 64 outputs a lane has in a tile of the gated product (4096 pairs, K = 3584,
// 8192 tokens: 353 us with them, 336 with these). Below -87 the value is under 2^-125 and
// comes out as 0.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

__device__ __forceinline__ u32x2 pack4(f32x4 v) { return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}; }

// GATED: v gate, up up (saved to a.gate_up if asked for) -> silu(gate) * up;
// else v + addend.
//
// What is rounded to bf16 before its end: h (here and in the tiles), and in the
// backward dgate, dup and h, once each. They are operands of the next product on
// the bf16 matrix cores: 16 more bits of them would be a second product and
// twice the bytes. It shows: a result is 2.4e-3 of its 2-norm off without an
// addend, 1.7e-3 if its own rounding were the only one (1.9e-3 with an addend
// of its size; gradients of one or two tokens up to 2.7e-3). The routed experts' h has the same rounding.
template <bool GATED>
__device__ __forceinline__ f32x4 finish4(const DenseArgs& a, int64_t token, int col, f32x4 v, f32x4 up) {
    if constexpr (GATED) {
        if (a.gate_up) {
            uint16_t* gu = a.gate_up + token * 2 * (int64_t)a.N + col;
            *(u32x2*)gu = pack4(v);
            *(u32x2*)(gu + a.N) = pack4(up);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = v[r] * sigmoid(v[r]) * up[r];
    } else if (a.addend) {
        const u32x2 d = *(const u32x2*)(a.addend + token * a.ldadd + col);
        v[0] += __uint_as_float(d[0] << 16);
        v[1] += __uint_as_float(d[0] & 0xffff0000u);
        v[2] += __uint_as_float(d[1] << 16);
        v[3] += __uint_as_float(d[1] & 0xffff0000u);
    }
    return v;
}

// dh of four columns -> dgate and dup (a.out, rows of [gate; up]) and h, from
// the saved gate_up.
__device__ __forceinline__ void backward4(const DenseArgs& a, int64_t token, int col, f32x4 dh) {
    const uint16_t* gu = a.gate_up + token * 2 * (int64_t)a.N + col;
    const u32x2 gb = *(const u32x2*)gu, ub = *(const u32x2*)(gu + a.N);
    f32x4 dg, du, h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float gv = __uint_as_float(e & 1 ? gb[e / 2] & 0xffff0000u : gb[e / 2] << 16);
        const float uv = __uint_as_float(e & 1 ? ub[e / 2] & 0xffff0000u : ub[e / 2] << 16);
        const float sg = sigmoid(gv), silu = gv * sg;
        dg[e] = dh[e] * uv * sg * (1.0f + gv * (1.0f - sg));
        du[e] = dh[e] * silu;
        h[e] = silu * uv;
    }
    uint16_t* o = (uint16_t*)a.out + token * a.ldo + col;
    *(u32x2*)o = pack4(dg);
    *(u32x2*)(o + a.N) = pack4(du);
    if (a.h) *(u32x2*)(a.h + token * (int64_t)a.N + col) = pack4(h);
}

__device__ __forceinline__ void store4(const DenseArgs& a, int64_t token, int col, f32x4 v) {
    if (a.out_f32) *(f32x4*)((float*)a.out + token * a.ldo + col) = v;
    else *(u32x2*)((uint16_t*)a.out + token * a.ldo + col) = pack4(v);
}

}  // namespace dense
}  // namespace moe
