// Dense products for few tokens (decode): C[m, n] = sum_k X[m, k] W[n, k] for
// up to 64 tokens m, bound by the stream of W from HBM.
//
// A workgroup of eight waves owns 16 rows of W (for the gated block 8 gate
// rows and their 8 up rows) and all of K: wave w takes the 128-byte K chunks
// w, w + 8, ... of every row straight into the MFMA operand registers (lane
// (i, g) holds pieces g and 4 + g of row i), with the tokens' chunks, which
// all workgroups read, coming from L2. A batch of chunks is loaded before the
// first of them is multiplied, so most of a wave's bytes are one round trip.
// The waves' sums meet in LDS, always in the same order. W is read with plain
// loads (2048 pairs over K = 3584, one token: 6.8 us, 8.0 with streaming
// ones).
//
// With more than 16 tokens the tokens' bytes count: every workgroup reads
// T x K of them next to its 16 x K of W. There the workgroup takes 64 rows
// and a part of K (or 16 rows, where W has few) and a second kernel joins the
// parts.
//
// With adapters the narrow product v = scale * A x runs in workgroups of the
// same launch (it is as short as a part of the product and does not depend on
// it), and the joining kernel adds B v.
#include "dense_epilogue.hpp"
#include "dense_tile.hpp"
#include "lora_shrink.hpp"

namespace moe {

using namespace dense;

namespace {

constexpr int kWaves = 8;

// ELT: see dense_tile.hpp. NJ: 16-token column blocks. XF32: X is fp32 and is
// quantised to MXFP8 as it is read (the second product of the MXFP8 block).
// NW: 16-row fragments of W. SPLIT: the workgroups take parts of K, into
// a.partial; those past the last part take the narrow product of the adapters
// (a token and 16 rows of its adapter each).
template <int ELT, int NJ, int NW, bool GATED, bool XF32, bool SPLIT>
__global__ __launch_bounds__(kWaves * 64) void skinny_kernel(DenseArgs a, const float* __restrict__ xf) {
    constexpr int BK = ELT == kEltBf16 ? 64 : 128;
    constexpr int ESZ = ELT == kEltBf16 ? 2 : 1;
    // Chunks in flight per wave: as many as the registers of two waves a SIMD
    // allow next to the tokens' operands.
    constexpr int kRegs = NW * 8 + NJ * (XF32 ? 32 : 8);
    constexpr int kFit = (NW * NJ > 8 ? 128 : 168) / kRegs;
    constexpr int kMost = XF32 ? 2 : ELT == kEltMx8 ? 4 : 7;
    constexpr int U = kFit < 1 ? 1 : kFit > kMost ? kMost : kFit;
    __shared__ f32x4 red[kWaves][NW * NJ][64];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    constexpr int kRows = NW * (GATED ? 8 : 16);
    int group = (int)blockIdx.x, part = 0;
    if constexpr (SPLIT) {
        const int groups = (a.N + kRows - 1) / kRows;
        part = group / groups;
        group %= groups;
        if constexpr (ELT == kEltBf16) {
            if (part >= a.splits) {
                const int e = (int)blockIdx.x - groups * a.splits, per = (a.lora.rank + 15) / 16;
                __shared__ f32x4 narrow[kShrinkWaves][4];
                shrink_token((const uint16_t*)a.x, a.ldx, a.K, a.lora, e / per, e % per * 16, narrow);
                return;
            }
        }
    }
    const int n0 = group * kRows;
    const int kb = a.K / 32;

    // Weights of at most 2^31 bytes (checked by the caller of the launcher).
    const rsrc_t rw = make_rsrc(a.w, kRecord);
    int64_t wrow[NW];
    uint32_t wo[NW];
#pragma unroll
    for (int f = 0; f < NW; ++f) {
        const int n = n0 + (GATED ? 8 * f + (i & 7) : 16 * f + i);
        wrow[f] = n < a.N ? (int64_t)(GATED && i >= 8 ? a.N + n : n) : -1;
        wo[f] = wrow[f] >= 0 ? (uint32_t)(wrow[f] * a.ldw * ESZ) + 16u * g : kOob;
    }
    const rsrc_t rx = make_rsrc(XF32 ? (const void*)xf : a.x, kRecord);
    uint32_t xo[NJ];
    int m[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        m[j] = 16 * j + i;
        xo[j] = m[j] < a.M ? (uint32_t)(m[j] * a.ldx * (XF32 ? 4 : ESZ)) + (XF32 ? 64u : 16u) * g : kOob;
    }
    f32x4 acc[NW][NJ];
#pragma unroll
    for (int f = 0; f < NW; ++f)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[f][j] = f32x4{0, 0, 0, 0};

    const int nch = (a.K + BK - 1) / BK;
    const int cbeg = SPLIT ? (int)((int64_t)nch * part / a.splits) : 0;
    const int cend = SPLIT ? (int)((int64_t)nch * (part + 1) / a.splits) : nch;
    const rsrc_t rws = make_rsrc(a.ws, kRecord), rxs = make_rsrc(a.xs, kRecord);
    u32x4 wv[U][NW][2], xv[U][NJ][XF32 ? 8 : 2];
    uint32_t ws[U][NW], xs[U][NJ];
    auto load = [&](int c0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + kWaves * u;
            const int left = c < cend ? a.K - c * BK : 0;  // <= 0 past the end: everything masked
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (4 * h + g) * (16 / ESZ);
                const bool ok = k < left;
#pragma unroll
                for (int f = 0; f < NW; ++f) wv[u][f][h] = bld16(rw, ok && wo[f] != kOob ? wo[f] + c * 128 + 64 * h : kOob);
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
#pragma unroll
                for (int f = 0; f < NW; ++f)
                    ws[u][f] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                        rws, wrow[f] >= 0 && b < kb ? (uint32_t)(wrow[f] * kb) + (uint32_t)b : kOob, 0, 0);
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
    load(cbeg + w);
    // Item (f, j, q, token): rows 4q..4q+3 of fragment f (gated: pairs, with
    // the up rows in q + 2), token 16 j + i. A thread finishes items tid,
    // tid + 512, ... (e % 16 == i for all of them).
    constexpr int Q = GATED ? 2 : 4, kItems = NW * NJ * 16 * Q;
    auto col_of = [&](int e) { return n0 + e / (NJ * 16 * Q) * (GATED ? 8 : 16) + 4 * (e / 16 % Q); };
    auto token_of = [&](int e) { return 16 * (e / (16 * Q) % NJ) + i; };
    for (int c0 = cbeg + w;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if constexpr (ELT == kEltBf16) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int f = 0; f < NW; ++f)
                            acc[f][j] = mfma16x16x32(__builtin_bit_cast(bf16x8, wv[u][f][h]),
                                                     __builtin_bit_cast(bf16x8, xv[u][j][h]), acc[f][j]);
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
#pragma unroll
                    for (int f = 0; f < NW; ++f) {
                        const u32x4 lo = wv[u][f][0], hi = wv[u][f][1];
                        const i32x8 wq = __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                        acc[f][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, acc[f][j], 0, 0, 0,
                                                                                     (int)ws[u][f], 0, (int)sx);
                    }
                }
            }
        }
        c0 += kWaves * U;
        if (c0 >= cend) break;
        load(c0);
    }
#pragma unroll
    for (int f = 0; f < NW; ++f)
#pragma unroll
        for (int j = 0; j < NJ; ++j) red[w][f * NJ + j][lane] = acc[f][j];
    __syncthreads();
#pragma unroll
    for (int e = tid; e < kItems; e += kWaves * 64) {
        const int token = token_of(e), col = col_of(e), q = e / 16 % Q, at = e / (16 * Q);
        if (token >= a.M || col >= a.N) continue;
        f32x4 v = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            v += red[k][at][16 * q + i];
            if constexpr (GATED) up += red[k][at][16 * (q + 2) + i];
        }
        if constexpr (SPLIT) {
            const int64_t cols = GATED ? 2 * (int64_t)a.N : a.N;
            float* p = a.partial + ((int64_t)part * a.M + token) * cols + col;
            *(f32x4*)p = v;
            if constexpr (GATED) *(f32x4*)(p + a.N) = up;
        } else {
            store4(a, token, col, finish4<GATED>(a, token, col, v, up));
        }
    }
}

template <int ELT, int NJ, int NW, bool GATED, bool XF32>
hipError_t launch_one(const DenseArgs& a, const float* xf, hipStream_t s) {
    constexpr int kRows = NW * (GATED ? 8 : 16);
    const unsigned groups = (unsigned)((a.N + kRows - 1) / kRows);
    const dim3 block(kWaves * 64);
    if constexpr (ELT == kEltBf16) {
        if (NW > 1 || a.splits > 1 || a.lora.n > 0) {
            const unsigned narrow = (unsigned)skinny_narrow(a);
            hipLaunchKernelGGL((skinny_kernel<ELT, NJ, NW, GATED, XF32, true>), dim3(groups * (unsigned)a.splits + narrow),
                               block, 0, s, a, xf);
            const hipError_t e = hipGetLastError();
            return e != hipSuccess ? e : launch_join(a, GATED ? kEpiGated : kEpiOut, s);
        }
    }
    if constexpr (NW == 1)
        hipLaunchKernelGGL((skinny_kernel<ELT, NJ, 1, GATED, XF32, false>), dim3(groups), block, 0, s, a, xf);
    return hipGetLastError();
}

template <int ELT, int NJ, bool GATED, bool XF32>
hipError_t launch_width(const DenseArgs& a, bool wide, const float* xf, hipStream_t s) {
    if constexpr (ELT == kEltBf16) {
        if (wide) return launch_one<ELT, NJ, 4, GATED, XF32>(a, xf, s);
    }
    return launch_one<ELT, NJ, 1, GATED, XF32>(a, xf, s);
}

// Up to 32 tokens the tokens' bytes do not pay for a second kernel, unless
// adapters need it anyway, W has few rows, or more of them than one round of
// workgroups takes and more than a batch of K (2048 pairs, K = 3584, 32
// tokens: 12.0 us, 13.5 in parts; 64 tokens: 18.9 and 16.0; 25 tokens: 4624
// rows over K = 3904 23.6 and 14.5, 6000 rows over 1024 11.6 and 11.0, over
// 512 9.1 and 10.8; 16384 rows over 3584 with 64 tokens 79 and 43).
bool one_kernel(const DenseArgs& a, bool gated) {
    const int64_t rows = gated ? 2 * (int64_t)a.N : a.N;
    return a.M <= 16 || (a.M <= 32 && a.lora.n == 0 && rows >= 2048 && (rows <= 4096 || a.K <= 512));
}

template <int ELT, bool GATED, bool XF32>
hipError_t launch_nj(const DenseArgs& a, const float* xf, hipStream_t s) {
    if (a.M <= 16) return launch_one<ELT, 1, 1, GATED, XF32>(a, xf, s);
    const bool wide = ELT == kEltBf16 && !one_kernel(a, GATED) && skinny_wide(a, GATED);
    if (a.M <= 32) return launch_width<ELT, 2, GATED, XF32>(a, wide, xf, s);
    if constexpr (ELT == kEltMx8) return hipErrorInvalidValue;  // kSkinnyMaxTokensMx
    else return launch_width<ELT, 4, GATED, XF32>(a, wide, xf, s);
}

}  // namespace

// Whether W has rows enough for 64 of them a workgroup.
bool skinny_wide(const DenseArgs& a, bool gated) { return (gated ? 2 * (int64_t)a.N : a.N) >= 2048; }

int skinny_narrow(const DenseArgs& a) { return a.lora.n > 0 ? a.M * ((a.lora.rank + 15) / 16) : 0; }

int skinny_splits(const DenseArgs& a, int elt, int epi) {
    const bool gated = epi != kEpiOut;
    const int64_t rows = gated ? 2 * (int64_t)a.N : a.N;
    if (elt != kEltBf16 || one_kernel(a, gated)) return 1;
    const int64_t groups = skinny_wide(a, gated) ? (rows + 63) / 64 : (rows + 15) / 16;
    // A part of K has a chunk for each wave; a workgroup a compute unit, those
    // of the narrow product counted.
    const int64_t most = (a.K + 63) / 64 / kWaves, room = (256 - skinny_narrow(a)) / groups;
    const int64_t s = room < most ? room : most;
    return s < 2 ? 1 : (int)s;
}

bool skinny_joins(const DenseArgs& a, int splits, int elt, int epi) {
    const bool gated = epi != kEpiOut;
    return elt == kEltBf16 && (a.lora.n > 0 || splits > 1 || (!one_kernel(a, gated) && skinny_wide(a, gated)));
}

hipError_t launch_skinny(const DenseArgs& a, int elt, int epi, const float* h_f32, hipStream_t s) {
    const bool gated = epi != kEpiOut;
    if (elt == kEltBf16)
        return gated ? launch_nj<kEltBf16, true, false>(a, nullptr, s) : launch_nj<kEltBf16, false, false>(a, nullptr, s);
    return gated ? launch_nj<kEltMx8, true, false>(a, nullptr, s) : launch_nj<kEltMx8, false, true>(a, h_f32, s);
}

}  // namespace moe
