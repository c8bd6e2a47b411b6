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

// Four elements of bf16 or fp32 from element `at`, 8-byte (16-byte) aligned.
__device__ __forceinline__ f32x4 load4(const void* p, int f32, int64_t at) {
    if (f32) return *(const f32x4*)((const float*)p + at);
    const u32x2 d = *(const u32x2*)((const uint16_t*)p + at);
    return f32x4{__uint_as_float(d[0] << 16), __uint_as_float(d[0] & 0xffff0000u), __uint_as_float(d[1] << 16),
                 __uint_as_float(d[1] & 0xffff0000u)};
}

constexpr float kLog2e = 1.44269504f, kSqrt2OverPi = 0.797884561f, kInvSqrt2Pi = 0.398942280f;

// Phi(-x) for x >= 0, the normal distribution's tail: erfc(x / sqrt 2) / 2 =
// exp(-x^2 / 2) P(t) with t = 1 / (1 + 0.36 x) and P the polynomial of degree 7
// with P(0) = 0 whose largest relative error is least for x in [0, 14], 8.7e-7
// (beyond, fp32 holds no more of it). z Phi(z) is off by 2e-7 at most; about 16
// vector instructions, against some 40 of the library's erff. This is P.
__device__ __forceinline__ float normal_tail_factor(float x) {
    const float t = __builtin_amdgcn_rcpf(fmaf(x, 0.36f, 1.0f));
    float p = 0.0470560603f;
    p = fmaf(p, t, -0.179763913f);
    p = fmaf(p, t, 0.180952996f);
    p = fmaf(p, t, 0.0265499931f);
    p = fmaf(p, t, 0.139719039f);
    p = fmaf(p, t, 0.141772494f);
    p = fmaf(p, t, 0.143713042f);
    return p * t;
}

// exp(-z^2 / 2)
__device__ __forceinline__ float gauss(float z) { return __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e)); }

// act(z) for four or eight outputs. The switch is uniform and outside the
// elements: silu and the tanh form are z / (1 + 2^-u), and z Phi(z) =
// max(z, 0) - |z| Phi(-|z|).
template <int V>
__device__ __forceinline__ void activate(int act, float (&z)[V]) {
    if (act == kActNone) return;
    if (act == kActRelu) {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];
    } else if (act == kActGelu) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // (Infinite times 0 is not met; a NaN comes through the factor.)
            const float tail = normal_tail_factor(fabsf(z[e])) * gauss(z[e]);
            z[e] = fmaf(-__builtin_amdgcn_fmed3f(fabsf(z[e]), 0.0f, 40.0f), tail, __builtin_amdgcn_fmed3f(z[e], 0.0f, __builtin_inff()));
        }
    } else {
        // (Below -200 the quotient is 0, which -inf must not meet.)
        constexpr float c = 2.0f * kSqrt2OverPi * kLog2e;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float u = act == kActSilu ? z[e] * kLog2e : z[e] * fmaf(z[e] * z[e], c * 0.044715f, c);
            z[e] = fmaxf(z[e], -200.0f) * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u));
        }
    }
}

// act'(z); far out it is the limit, 0 or 1, and a NaN stays one.
__device__ __forceinline__ float act_slope(int act, float z) {
    if (act == kActNone) return 1.0f;
    if (act == kActRelu) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    const float near = __builtin_amdgcn_fmed3f(z, -200.0f, 200.0f);  // what meets a 0
    if (act == kActGelu) {
        // Phi(z) + z phi(z)
        const float g = gauss(z), q = normal_tail_factor(fabsf(z)) * g;
        return fmaf(near, kInvSqrt2Pi * g, z < 0.0f ? q : 1.0f - q);
    }
    // p = 1 / (1 + exp(-u)): p + z p (1 - p) u'
    const float c = act == kActSilu ? 1.0f : 2.0f * kSqrt2OverPi, d = act == kActSilu ? 0.0f : c * 0.044715f;
    const float u = act == kActSilu ? z : z * fmaf(near * near, d, c);
    const float du = act == kActSilu ? 1.0f : fmaf(near * near, 3.0f * d, c);
    const float e = __builtin_amdgcn_exp2f(-fabsf(u) * kLog2e), r = __builtin_amdgcn_rcpf(1.0f + e);
    return fmaf(near * du, e * r * r, u < 0.0f ? e * r : r);
}

// GATED: v gate, up up (saved to a.gate_up if asked for) -> silu(gate) * up;
// else act(v + bias) (v + bias saved to a.pre if asked for) + addend.
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
    } else {
        if (a.bias) v += load4(a.bias, a.bias_f32, col);
        if (a.pre) *(u32x2*)(a.pre + token * (int64_t)a.N + col) = pack4(v);
        if (a.act) {
            float z[4] = {v[0], v[1], v[2], v[3]};
            activate<4>(a.act, z);
            v = f32x4{z[0], z[1], z[2], z[3]};
        }
        if (a.addend) v += load4(a.addend, a.addend_f32, token * a.ldadd + col);
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
