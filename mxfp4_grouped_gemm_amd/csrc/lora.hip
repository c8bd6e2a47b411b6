// The narrow product of low-rank adapters: v[t] = scale[a] * A[a] x[t] for
// a = index[t], in fp32. The second factor, B[a] v, is added inside the
// projection's own kernels.
//
// Few tokens (decode): a workgroup a token and 16 rows of its adapter's A, so
// nothing has to be sorted or searched; rows that tokens share come from L2.
//
// Many tokens (prompts): a workgroup takes 32 tokens in their own order and
// four 16-row pieces of the A of the distinct adapters among them, in the
// order of the adapters, so A is read once per 32 tokens. Tokens of other adapters run through the products too and
// are not stored.
//
// With few groups of tokens K is split over workgroups too, and what reads v
// adds the parts. In both forms eight waves split K, hold a batch of 128-byte K chunks in flight
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

__global__ __launch_bounds__(kWaves * 64) void lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx, int T,
                                                                  int K, LoraArgs l) {
    constexpr int FM = 2;
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
        idx[f] = (unsigned)v < (unsigned)l.n ? v : kNoAdapter;
    }
    const rsrc_t rx = make_rsrc(x + (int64_t)t0 * ldx, kRecord);
    uint32_t xo[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f)
        xo[f] = t0 + 16 * f + i < T ? (uint32_t)((16 * f + i) * ldx * 2) + 16u * g : kOob;
    const int nch = (K + 63) / 64;
    const int cbeg = (int)((int64_t)nch * blockIdx.z / l.parts), cend = (int)((int64_t)nch * (blockIdx.z + 1) / l.parts);
    // Piece q is rows 16 (q % per).. of distinct adapter q / per; a workgroup's
    // groups of FR pieces are blockIdx.y, blockIdx.y + gridDim.y, ... The same
    // in every wave.
    const int per = (l.rank + 15) / 16;
    int seen = -1, last = -1;  // distinct adapters passed, the last of them
    for (int group = (int)blockIdx.y;; group += (int)gridDim.y) {
        int ad[FR], row0[FR];
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            const int q = group * FR + r;
            while (last != kNoAdapter && seen < q / per) {
                int next = kNoAdapter;
#pragma unroll
                for (int f = 0; f < FM; ++f) next = idx[f] > last && idx[f] < next ? idx[f] : next;
                last = __builtin_amdgcn_readfirstlane(min16(next));
                ++seen;
            }
            ad[r] = last;
            row0[r] = q % per * 16;
        }
        if (ad[0] == kNoAdapter) return;
        if (group >= (int)gridDim.y) __syncthreads();  // the group before has been read
        f32x4 acc[FR][FM];
        rsrc_t ra[FR];
        uint32_t ao[FR];
        float scale[FR];
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            const bool some = ad[r] != kNoAdapter;
            const int at = some ? ad[r] : 0;
            int rank = l.ranks ? l.ranks[at] : l.rank;
            rank = rank < l.rank ? rank : l.rank;
            scale[r] = l.scale ? l.scale[at] : 1.0f;
            ra[r] = make_rsrc(l.a + ((int64_t)at * l.rank + row0[r]) * K, kRecord);
            ao[r] = some && row0[r] + i < rank ? (uint32_t)(i * K * 2) + 16u * g : kOob;
#pragma unroll
            for (int f = 0; f < FM; ++f) acc[r][f] = f32x4{0, 0, 0, 0};
        }
        // One chunk is loaded while the one before it is multiplied.
        u32x4 xv[2][2][FM], av[2][2][FR];
        auto load = [&](int set, int c) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool ok = c < cend && (4 * h + g) * 8 < K - c * 64;
#pragma unroll
                for (int f = 0; f < FM; ++f) xv[set][h][f] = bld16(rx, ok && xo[f] != kOob ? xo[f] + c * 128 + 64 * h : kOob);
#pragma unroll
                for (int r = 0; r < FR; ++r) av[set][h][r] = bld16(ra[r], ok && ao[r] != kOob ? ao[r] + c * 128 + 64 * h : kOob);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto multiply = [&](int set) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < FR; ++r)
#pragma unroll
                    for (int f = 0; f < FM; ++f)
                        acc[r][f] = mfma16x16x32(__builtin_bit_cast(bf16x8, av[set][h][r]),
                                                 __builtin_bit_cast(bf16x8, xv[set][h][f]), acc[r][f]);
            __builtin_amdgcn_sched_barrier(0);
        };
        load(0, cbeg + w);
        for (int c = cbeg + w; c < cend; c += 2 * kWaves) {
            load(1, c + kWaves);
            multiply(0);
            load(0, c + 2 * kWaves);
            multiply(1);
        }
#pragma unroll
        for (int r = 0; r < FR; ++r)
#pragma unroll
            for (int f = 0; f < FM; ++f) red[w][r][f][lane] = acc[r][f];
        __syncthreads();
        // Thread (r, f, lane'): four rows of v of one token; lane' % 64 == lane.
        static_assert(FR * FM == kWaves, "a wave each");
#pragma unroll
        for (int r = 0; r < FR; ++r)
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                if (w != r * FM + f || idx[f] != ad[r] || ad[r] == kNoAdapter) continue;
                f32x4 v = red[0][r][f][lane];
#pragma unroll
                for (int k = 1; k < kWaves; ++k) v += red[k][r][f][lane];
                *(f32x4*)(l.v + blockIdx.z * l.part_stride + (int64_t)(t0 + 16 * f + i) * l.vld + row0[r] + 4 * g) = v * scale[r];
            }
    }
}

}  // namespace

// A workgroup's bytes come through its compute unit's own path to L2 (about 40
// bytes a ns), and the registers allow one workgroup a compute unit: a batch
// of few 32-token groups splits K as long as that makes one round (1024
// tokens, 8 adapters of rank 64, K = 3584: 22.4 us in one part, 9.0 in four;
// 4099 tokens: 24.3 in one, 25.7 in two, which is a second round).
int lora_parts(int T) {
    if (T <= kTokenWise) return 1;
    const int groups = (T + 31) / 32;
    return groups > 128 ? 1 : groups > 64 ? 2 : kMaxLoraParts;
}

hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const LoraArgs& l, hipStream_t s) {
    if (T <= kTokenWise) {
        hipLaunchKernelGGL(lora_shrink_token_kernel, dim3((unsigned)T, (unsigned)(l.vld / 16)), dim3(kWaves * 64), 0, s,
                           x, ldx, K, l);
    } else {
        const int64_t pieces = (int64_t)(l.n < 32 ? l.n : 32) * ((l.rank + 15) / 16);
        // Groups side by side: what one round has room for, and four in any
        // case (a workgroup without a group leaves at once, while a second
        // group in turn doubles its tokens' time: 4099 tokens in eight runs
        // 24 us, 45 with one workgroup for all groups).
        const int64_t tokens = (T + 31) / 32, groups = (pieces + FR - 1) / FR, room = 256 / (tokens * l.parts);
        const int64_t y = room < 4 ? 4 : room;
        const dim3 grid((unsigned)tokens, (unsigned)(y < groups ? y : groups), (unsigned)l.parts);
        hipLaunchKernelGGL(lora_shrink_kernel, grid, dim3(kWaves * 64), 0, s, x, ldx, T, K, l);
    }
    return hipGetLastError();
}

}  // namespace moe
