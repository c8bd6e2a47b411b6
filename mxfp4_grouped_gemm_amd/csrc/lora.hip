// The narrow product of low-rank adapters: v[t] = scale[a] * A[a] x[t] for
// a = index[t], in fp32. The second factor, B[a] v, is added inside the
// projection's own kernels.
//
// Few tokens (decode): a workgroup a token and 16 rows of its adapter's A, so
// nothing has to be sorted or searched; rows that tokens share come from L2.
//
// Many tokens (prompts): a workgroup takes 32 tokens in their own order and
// the s-th distinct adapter among them (grid.y counts s; most of the grid of
// a batch whose tokens share adapters leaves at once), so A is read once per
// 32 tokens. Tokens of other adapters run through the products too and are
// not stored.
//
// In both, eight waves split K, hold a batch of 128-byte K chunks in flight
// and meet in LDS in a fixed order.
#include "lora_shrink.hpp"

namespace moe {

using namespace dense;

namespace {

constexpr int kWaves = kShrinkWaves;
constexpr int FR = 4;  // 16-row rank fragments a pass
// Up to this many tokens a workgroup takes one token.
constexpr int kTokenWise = 128;

__global__ __launch_bounds__(kWaves * 64) void lora_shrink_token_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                        int K, LoraArgs l) {
    __shared__ f32x4 red[kWaves][4];
    shrink_token(x, ldx, K, l, (int)blockIdx.x, (int)blockIdx.y * 16, red);
}

template <int FM>
__global__ __launch_bounds__(kWaves * 64) void lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx, int T,
                                                                  int K, LoraArgs l) {
    __shared__ f32x4 red[kWaves][FR][FM][64];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int t0 = (int)blockIdx.x * 16 * FM;
    int idx[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int t = t0 + 16 * f + i;
        const int v = t < T ? l.index[t] : -1;
        idx[f] = (unsigned)v < (unsigned)l.n ? v : 0x7fffffff;
    }
    int ad = -1;
    for (int s = 0; s <= (int)blockIdx.y; ++s) {
        int next = 0x7fffffff;
#pragma unroll
        for (int f = 0; f < FM; ++f) next = idx[f] > ad && idx[f] < next ? idx[f] : next;
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            const int o = __shfl_xor(next, d);
            next = o < next ? o : next;
        }
        next = __builtin_amdgcn_readfirstlane(next);
        if (next == 0x7fffffff) return;  // the same in every wave
        ad = next;
    }
    int rank = l.ranks ? l.ranks[ad] : l.rank;
    rank = rank < l.rank ? rank : l.rank;
    const float scale = l.scale ? l.scale[ad] : 1.0f;
    const uint16_t* ap = l.a + (int64_t)ad * l.rank * K;
    const rsrc_t ra = make_rsrc(ap, kRecord);
    const rsrc_t rx = make_rsrc(x + (int64_t)t0 * ldx, kRecord);
    uint32_t xo[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f)
        xo[f] = t0 + 16 * f + i < T ? (uint32_t)((16 * f + i) * ldx * 2) + 16u * g : kOob;
    const int nch = (K + 63) / 64;
    for (int r0 = 0; r0 < l.vld; r0 += 16 * FR) {
        f32x4 acc[FR][FM];
        uint32_t ao[FR];
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            const int row = r0 + 16 * r + i;
            ao[r] = row < rank ? (uint32_t)((int64_t)row * K * 2) + 16u * g : kOob;
#pragma unroll
            for (int f = 0; f < FM; ++f) acc[r][f] = f32x4{0, 0, 0, 0};
        }
        constexpr int U = 3;
        for (int c0 = w; c0 < nch; c0 += kWaves * U) {
            u32x4 xv[U][2][FM], av[U][2][FR];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + kWaves * u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool ok = (4 * h + g) * 8 < K - c * 64;
#pragma unroll
                    for (int f = 0; f < FM; ++f)
                        xv[u][h][f] = bld16(rx, ok && xo[f] != kOob ? xo[f] + c * 128 + 64 * h : kOob);
#pragma unroll
                    for (int r = 0; r < FR; ++r)
                        av[u][h][r] = bld16(ra, ok && ao[r] != kOob ? ao[r] + c * 128 + 64 * h : kOob);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < FR; ++r)
#pragma unroll
                        for (int f = 0; f < FM; ++f)
                            acc[r][f] = mfma16x16x32(__builtin_bit_cast(bf16x8, av[u][h][r]),
                                                     __builtin_bit_cast(bf16x8, xv[u][h][f]), acc[r][f]);
        }
        if (r0 > 0) __syncthreads();  // the previous pass has been read
#pragma unroll
        for (int r = 0; r < FR; ++r)
#pragma unroll
            for (int f = 0; f < FM; ++f) red[w][r][f][lane] = acc[r][f];
        __syncthreads();
        for (int e = tid; e < FR * FM * 64; e += kWaves * 64) {
            const int r = e / (FM * 64), f = (e / 64) % FM, ln = e % 64;
            const int t = t0 + 16 * f + (ln & 15), col = r0 + 16 * r + 4 * (ln >> 4);
            // ln & 15 == i: e % 64 == lane, since the stride is a multiple of 64.
            int mine = idx[0];
#pragma unroll
            for (int ff = 1; ff < FM; ++ff) mine = f == ff ? idx[ff] : mine;
            if (mine != ad || col >= l.vld) continue;
            f32x4 v = red[0][r][f][ln];
#pragma unroll
            for (int k = 1; k < kWaves; ++k) v += red[k][r][f][ln];
            *(f32x4*)(l.v + (int64_t)t * l.vld + col) = v * scale;
        }
    }
}

}  // namespace

hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const LoraArgs& l, hipStream_t s) {
    if (T <= kTokenWise) {
        hipLaunchKernelGGL(lora_shrink_token_kernel, dim3((unsigned)T, (unsigned)(l.vld / 16)), dim3(kWaves * 64), 0, s,
                           x, ldx, K, l);
    } else {
        const dim3 grid((unsigned)((T + 31) / 32), (unsigned)(l.n < 32 ? l.n : 32));
        hipLaunchKernelGGL(lora_shrink_kernel<2>, grid, dim3(kWaves * 64), 0, s, x, ldx, T, K, l);
    }
    return hipGetLastError();
}

}  // namespace moe
