// The narrow product of one token: v = scale * A x for 16 rows of its adapter.
#pragma once

#include "common.hpp"
#include "dense.hpp"
#include "dense_tile.hpp"

namespace moe {
namespace dense {

constexpr int kShrinkWaves = 8;

// Rows r0..r0+15 of token t's adapter, in a workgroup of kShrinkWaves waves:
// they split K, hold a batch of 128-byte K chunks in flight and meet in `red`
// in a fixed order.
__device__ __forceinline__ void shrink_token(const uint16_t* __restrict__ x, int64_t ldx, int K, const LoraArgs& l,
                                             int t, int r0, f32x4 (&red)[kShrinkWaves][4]) {
    constexpr int U = 7, kWaves = kShrinkWaves;
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int ad = l.index[t];
    if ((unsigned)ad >= (unsigned)l.n) return;
    int rank = l.ranks ? l.ranks[ad] : l.rank;
    rank = rank < l.rank ? rank : l.rank;
    const rsrc_t ra = make_rsrc(l.a + (int64_t)ad * l.rank * K, kRecord);
    const rsrc_t rx = make_rsrc(x + t * ldx, kRecord);
    const uint32_t ao = r0 + i < rank ? (uint32_t)((r0 + i) * K * 2) + 16u * g : kOob;
    const int nch = (K + 63) / 64;
    f32x4 acc = {0, 0, 0, 0};
    for (int c0 = w; c0 < nch; c0 += kWaves * U) {
        u32x4 av[U][2], xv[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + kWaves * u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool ok = (4 * h + g) * 8 < K - c * 64;
                av[u][h] = bld16(ra, ok && ao != kOob ? ao + c * 128 + 64 * h : kOob);
                // The token is the MFMA's column 0; the other columns are zeros.
                xv[u][h] = bld16(rx, ok && i == 0 ? (uint32_t)(c * 128 + 64 * h + 16 * g) : kOob);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc = mfma16x16x32(__builtin_bit_cast(bf16x8, av[u][h]), __builtin_bit_cast(bf16x8, xv[u][h]), acc);
    }
    if (i == 0) red[w][g] = acc;
    __syncthreads();
    if (tid < 4) {
        f32x4 v = red[0][tid];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v += red[k][tid];
        const float scale = l.scale ? l.scale[ad] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r0 + 4 * tid + e < rank ? v[e] * scale : 0.0f;
        *(f32x4*)(l.v + (int64_t)t * l.vld + r0 + 4 * tid) = v;
    }
}

}  // namespace dense
}  // namespace moe
