// Dense products for few tokens (decode): C[m, n] = sum_k X[m, k] W[n, k] for
// up to 64 tokens m, bound by the stream of W from HBM.
//
// A workgroup of eight waves owns 16 rows of W (for the gated block 8 gate
// rows and their 8 up rows) and all of K: wave w takes the 128-byte K chunks
// w, w + 8, ... of every row straight into the MFMA operand registers (lane
// (i, g) holds pieces g and 4 + g of row i), with the tokens' chunks, which
// all workgroups read, coming from L2. A batch of chunks is loaded before the
// first of them is multiplied, so most of a wave's bytes are one round trip.
// The waves' sums meet in LDS, always in the same order.
//
// The low-rank term of an output is a dot product of at most a few hundred
// elements that depends on the output's token: the thread that finishes the
// output computes it, while the first batch of weights is on its way.
#include "dense_tile.hpp"

namespace moe {

using namespace dense;

namespace {

constexpr int kWaves = 8;

// scale * B[a] (A[a] x) of one token for rows col..col+3 (and N + col.. of the
// gated block), from v = scale * A[a] x.
template <bool GATED>
__device__ __forceinline__ void lora_dot(const LoraArgs& l, int N, int token, int col, f32x4 (&low)[2]) {
    const int ad = l.index[token];
    if ((unsigned)ad >= (unsigned)l.n) return;
    int rank = l.ranks ? l.ranks[ad] : l.rank;
    rank = rank < l.rank ? rank : l.rank;
    const uint16_t* b = l.b + ((int64_t)ad * (GATED ? 2 * (int64_t)N : N) + col) * l.rank;
    const float* v = l.v + (int64_t)token * l.vld;
    for (int k = 0; k < rank; k += 8) {
        const f32x4 v0 = *(const f32x4*)(v + k), v1 = *(const f32x4*)(v + k + 4);
        u32x4 w[GATED ? 2 : 1][4];
#pragma unroll
        for (int s = 0; s < (GATED ? 2 : 1); ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) w[s][r] = *(const u32x4*)(b + ((int64_t)s * N + r) * l.rank + k);
#pragma unroll
        for (int s = 0; s < (GATED ? 2 : 1); ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // Columns beyond the adapter's rank are not read as numbers.
                    const uint32_t d = w[s][r][e / 2];
                    const float f = __uint_as_float(e & 1 ? d & 0xffff0000u : d << 16);
                    const float t = (e < 4 ? v0[e & 3] : v1[e & 3]);
                    if (k + e < rank) low[s][r] = fmaf(f, t, low[s][r]);
                }
    }
}

// ELT: see dense_tile.hpp. NJ: 16-token column blocks. XF32: X is fp32 and is
// quantised to MXFP8 as it is read (the second product of the MXFP8 block).
template <int ELT, int NJ, bool GATED, bool XF32, bool LORA>
__global__ __launch_bounds__(kWaves * 64) void skinny_kernel(DenseArgs a, const float* __restrict__ xf) {
    constexpr int BK = ELT == kEltBf16 ? 64 : 128;
    constexpr int ESZ = ELT == kEltBf16 ? 2 : 1;
    // Chunks in flight per wave: as many as the registers of two waves a SIMD
    // allow next to the tokens' operands.
    constexpr int U = XF32 ? (NJ <= 2 ? 2 : 1) : ELT == kEltMx8 ? (NJ <= 2 ? 4 : 2) : NJ <= 2 ? 7 : 4;
    __shared__ f32x4 red[kWaves][NJ][64];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * (GATED ? 8 : 16);
    const int kb = a.K / 32;

    const int n = GATED ? n0 + (i & 7) : n0 + i;
    const int64_t wrow = n < a.N ? (int64_t)(GATED && i >= 8 ? a.N + n : n) : -1;
    // Weights of at most 2^31 bytes (checked by the caller of the launcher).
    const rsrc_t rw = make_rsrc(a.w, kRecord);
    const uint32_t wo = wrow >= 0 ? (uint32_t)(wrow * a.ldw * ESZ) + 16u * g : kOob;
    const rsrc_t rx = make_rsrc(XF32 ? (const void*)xf : a.x, kRecord);
    uint32_t xo[NJ];
    int m[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        m[j] = 16 * j + i;
        xo[j] = m[j] < a.M ? (uint32_t)(m[j] * a.ldx * (XF32 ? 4 : ESZ)) + (XF32 ? 64u : 16u) * g : kOob;
    }
    f32x4 acc[1][NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[0][j] = f32x4{0, 0, 0, 0};

    const int nch = (a.K + BK - 1) / BK;
    const rsrc_t rws = make_rsrc(a.ws, kRecord), rxs = make_rsrc(a.xs, kRecord);
    u32x4 wv[U][2], xv[U][NJ][XF32 ? 8 : 2];
    uint32_t ws[U], xs[U][NJ];
    auto load = [&](int c0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + kWaves * u;
            const int left = a.K - c * BK;  // <= 0 past the end: everything masked
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (4 * h + g) * (16 / ESZ);
                const bool ok = k < left;
                wv[u][h] = bld16nt(rw, ok && wo != kOob ? wo + c * 128 + 64 * h : kOob);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if constexpr (XF32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            xv[u][j][4 * h + e] = bld16(rx, ok && xo[j] != kOob ? xo[j] + c * 512 + 256 * h + 16 * e : kOob);
                    } else {
                        xv[u][j][h] = bld16(rx, ok && xo[j] != kOob ? xo[j] + c * 128 + 64 * h : kOob);
                    }
                }
            }
            if constexpr (ELT == kEltMx8) {
                // Byte of block g of the chunk; blocks past the end have zero codes.
                const int b = 4 * c + g;
                ws[u] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                    rws, wrow >= 0 && b < kb ? (uint32_t)(wrow * kb) + (uint32_t)b : kOob, 0, 0);
                if constexpr (!XF32) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        xs[u][j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                            rxs, m[j] < a.M && b < kb ? (uint32_t)(m[j] * kb + b) : kOob, 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // all of the batch in flight
    };
    load(w);
    // Thread (j, token, q) finishes rows 4q..4q+3 of the tile (gated: pairs,
    // with the up rows in q + 2).
    constexpr int Q = GATED ? 2 : 4;
    const int fj = tid / (16 * Q), fq = (tid / 16) % Q, token = 16 * fj + i;
    const int col = n0 + 4 * fq;
    const bool finish = tid < NJ * 16 * Q && token < a.M && col < a.N;
    f32x4 low[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if constexpr (LORA) {
        if (finish) lora_dot<GATED>(a.lora, a.N, token, col, low);
    }
    for (int c0 = w;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if constexpr (ELT == kEltBf16) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        acc[0][j] = mfma16x16x32(__builtin_bit_cast(bf16x8, wv[u][h]), __builtin_bit_cast(bf16x8, xv[u][j][h]), acc[0][j]);
                } else {
                    i32x8 xq;
                    uint32_t sx;
                    if constexpr (XF32) {
                        // Half h of the lane is half a block (the other half
                        // is lane g ^ 1's): block 2h + g / 2 of the chunk.
                        uint32_t sb[2];
                        float inv[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float big = 0.0f;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                big = fmaxf(big, mx8_finite_abs(__uint_as_float(xv[u][j][4 * h + e / 4][e % 4])));
                            big = fmaxf(big, __shfl_xor(big, 16));
                            sb[h] = mx8_scale_byte(big);
                            inv[h] = mx8_inv_scale(sb[h]);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const u32x4 v = xv[u][j][e];
                            xq[e] = (int)mx8_pack4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]),
                                                   __uint_as_float(v[3]), inv[e / 4]);
                        }
                        // The scale operand of lane g is block g's: lanes 1
                        // and 2 hold each other's.
                        const uint32_t give = g == 0 || g == 2 ? sb[0] : sb[1];
                        const int from = g == 1 ? 32 + i : g == 2 ? 16 + i : lane;
                        sx = (uint32_t)__shfl((int)give, from);
                    } else {
                        const u32x4 lo = xv[u][j][0], hi = xv[u][j][1];
                        xq = __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                        sx = xs[u][j];
                    }
                    const u32x4 lo = wv[u][0], hi = wv[u][1];
                    const i32x8 wq = __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    acc[0][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, acc[0][j], 0, 0, 0, (int)ws[u], 0, (int)sx);
                }
            }
        }
        c0 += kWaves * U;
        if (c0 >= nch) break;
        load(c0);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) red[w][j][lane] = acc[0][j];
    __syncthreads();
    if (!finish) return;
    f32x4 v = low[0];
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += red[k][fj][16 * fq + i];
    if constexpr (GATED) {
        f32x4 up = low[1];
#pragma unroll
        for (int k = 0; k < kWaves; ++k) up += red[k][fj][16 * (fq + 2) + i];
        if (a.gate_up) {
            uint16_t* gu = a.gate_up + token * 2 * (int64_t)a.N + col;
            *(u32x2*)gu = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            *(u32x2*)(gu + a.N) = u32x2{pack_bf16x2(up[0], up[1]), pack_bf16x2(up[2], up[3])};
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = swiglu(v[r], up[r]);
    } else if (a.addend) {
        const u32x2 d = *(const u32x2*)(a.addend + token * a.ldadd + col);
        v[0] += __uint_as_float(d[0] << 16);
        v[1] += __uint_as_float(d[0] & 0xffff0000u);
        v[2] += __uint_as_float(d[1] << 16);
        v[3] += __uint_as_float(d[1] & 0xffff0000u);
    }
    if (a.out_f32) *(f32x4*)((float*)a.out + token * a.ldo + col) = v;
    else *(u32x2*)((uint16_t*)a.out + token * a.ldo + col) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

template <int ELT, int NJ, bool GATED, bool XF32>
void launch_one(const DenseArgs& a, const float* xf, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16))), block(kWaves * 64);
    if constexpr (ELT == kEltBf16) {
        if (a.lora.n > 0) {
            hipLaunchKernelGGL((skinny_kernel<ELT, NJ, GATED, XF32, true>), grid, block, 0, s, a, xf);
            return;
        }
    }
    hipLaunchKernelGGL((skinny_kernel<ELT, NJ, GATED, XF32, false>), grid, block, 0, s, a, xf);
}

template <int ELT, bool GATED, bool XF32>
void launch_nj(const DenseArgs& a, const float* xf, hipStream_t s) {
    if (a.M <= 16) launch_one<ELT, 1, GATED, XF32>(a, xf, s);
    else if (a.M <= 32) launch_one<ELT, 2, GATED, XF32>(a, xf, s);
    else launch_one<ELT, 4, GATED, XF32>(a, xf, s);
}

}  // namespace

hipError_t launch_skinny(const DenseArgs& a, int elt, int epi, const float* h_f32, hipStream_t s) {
    const bool gated = epi != kEpiOut;
    if (elt == kEltBf16) {
        if (gated) launch_nj<kEltBf16, true, false>(a, nullptr, s);
        else launch_nj<kEltBf16, false, false>(a, nullptr, s);
    } else if (gated) {
        launch_nj<kEltMx8, true, false>(a, nullptr, s);
    } else {
        launch_nj<kEltMx8, false, true>(a, h_f32, s);
    }
    return hipGetLastError();
}

}  // namespace moe
