// Instances of the LDS-tiled product for the forward in bf16 (both operands
// K-major), the choice of tile and K split, and the kernel that joins a split.
#include "dense_epilogue.hpp"
#include "dense_tile.hpp"

namespace moe {

using namespace dense;

namespace {

// Sums the parts of a split K in order, adds the low-rank term and applies
// the epilogue. A thread owns four columns (gated: four pairs).
template <int EPI>
__global__ __launch_bounds__(256) void join_kernel(DenseArgs a) {  // 64 or 256 threads
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedMx;
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int per = a.N / 4;
    const int64_t m = idx / per;
    const int n = (int)(idx % per) * 4;
    const bool ok = m < a.M;  // N % 32 == 0 for MXFP8: eight threads a block, all of one row
    const int64_t cols = kGated ? 2 * (int64_t)a.N : a.N;
    f32x4 low[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (ok && a.lora.n > 0) lora_dot<kGated>(a.lora, a.N, m, n, low);
    f32x4 v = low[0], up = low[1];
    if (ok)
        for (int z = 0; z < a.splits; ++z) {
            const float* p = a.partial + ((int64_t)z * a.M + m) * cols + n;
            v += *(const f32x4*)p;
            if constexpr (kGated) up += *(const f32x4*)(p + a.N);
        }
    if constexpr (EPI == kEpiGatedBwd) {
        if (ok) backward4(a, m, n, v);
        return;
    }
    if (ok) v = finish4<kGated>(a, m, n, v, up);
    if constexpr (EPI == kEpiGatedMx) {
        float big = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) big = fmaxf(big, mx8_finite_abs(v[r]));
#pragma unroll
        for (int d = 1; d < 8; d *= 2) big = fmaxf(big, __shfl_xor(big, d));
        const uint32_t sb = mx8_scale_byte(big);
        if (!ok) return;
        *(uint32_t*)((uint8_t*)a.out + m * a.ldo + n) = mx8_pack4(v[0], v[1], v[2], v[3], mx8_inv_scale(sb));
        if ((n & 31) == 0) a.hs[m * (a.N / 32) + (n >> 5)] = (uint8_t)sb;
    } else if (ok) {
        store4(a, m, n, v);
    }
}

template <int EPI, bool LORA>
hipError_t launch_epi(const DenseArgs& a, hipStream_t s) {
    if (dense_big_tiles(a, EPI))
        return launch_tile<Tile<256, 256, 2, 4, false, false, kEltBf16, EPI, false, LORA>>(a, s);
    if (a.splits > 1) {
        const hipError_t e = launch_tile<Tile<128, 128, 2, 2, false, false, kEltBf16, EPI, true, false, 4>>(a, s);
        return e != hipSuccess ? e : launch_join(a, EPI, s);
    }
    if (dense_one_round(a, EPI)) return launch_tile<Tile<128, 128, 2, 2, false, false, kEltBf16, EPI, false, LORA, 4>>(a, s);
    return launch_tile<Tile<128, 128, 2, 2, false, false, kEltBf16, EPI, false, LORA>>(a, s);
}

}  // namespace

// 256 x 256 tiles when they come close to filling the 256 compute units, else
// 128 x 128 ones, which read twice the LDS bytes for a product.
bool dense_big_tiles(const DenseArgs& a, int epi) {
    const bool gated = epi == kEpiGated || epi == kEpiGatedMx;
    const int64_t cols = gated ? 2 * (int64_t)a.N : a.N;
    return (int64_t)((a.M + 255) / 256) * ((cols + 255) / 256) >= 160;
}

// 128 x 128 tiles with at most one workgroup a compute unit.
bool dense_one_round(const DenseArgs& a, int epi) {
    const bool gated = epi == kEpiGated || epi == kEpiGatedMx;
    const int64_t cols = gated ? 2 * (int64_t)a.N : a.N;
    return (int64_t)((a.M + 127) / 128) * ((cols + 127) / 128) <= 256;
}

int dense_splits(const DenseArgs& a, int elt, int epi) {
    if (dense_big_tiles(a, epi)) return 1;
    const bool gated = epi == kEpiGated || epi == kEpiGatedMx;
    const int64_t cols = gated ? 2 * (int64_t)a.N : a.N;
    const int64_t tiles = (int64_t)((a.M + 127) / 128) * ((cols + 127) / 128);
    if (tiles == 0) return 1;  // no tokens
    const int bk = elt == kEltBf16 ? 64 : 128;
    const int steps = (a.K + bk - 1) / bk;
    int64_t s = 256 / tiles;
    if (s > steps / 4) s = steps / 4;
    if (s > 16) s = 16;
    return s < 1 ? 1 : (int)s;
}

hipError_t launch_join(const DenseArgs& a, int epi, hipStream_t s) {
    const int64_t threads = (int64_t)a.M * (a.N / 4);
    // Small ones are latency: spread them over the compute units.
    const int size = threads < 256 * 256 ? 64 : 256;
    const dim3 grid((unsigned)((threads + size - 1) / size)), block(size);
    if (epi == kEpiOut) hipLaunchKernelGGL(join_kernel<kEpiOut>, grid, block, 0, s, a);
    else if (epi == kEpiGated) hipLaunchKernelGGL(join_kernel<kEpiGated>, grid, block, 0, s, a);
    else if (epi == kEpiGatedMx) hipLaunchKernelGGL(join_kernel<kEpiGatedMx>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(join_kernel<kEpiGatedBwd>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dense_nt(const DenseArgs& a, int epi, hipStream_t s) {
    if (epi == kEpiOut) return a.lora.n > 0 ? launch_epi<kEpiOut, true>(a, s) : launch_epi<kEpiOut, false>(a, s);
    return a.lora.n > 0 ? launch_epi<kEpiGated, true>(a, s) : launch_epi<kEpiGated, false>(a, s);
}

hipError_t launch_dense(const DenseArgs& a, int elt, int epi, hipStream_t s) {
    return elt == kEltBf16 ? launch_dense_nt(a, epi, s) : launch_dense_mx(a, epi, s);
}

}  // namespace moe
