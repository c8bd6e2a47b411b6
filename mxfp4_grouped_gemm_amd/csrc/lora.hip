// The narrow product of low-rank adapters: v[t] = scale[a] * A[a] x[t] for
// a = index[t], in fp32. The second factor, B[a] v, is added inside the
// projection's own kernels.
//
// Few tokens (decode): a workgroup a token and 16 rows of its adapter's A, so
// nothing has to be sorted or searched; rows that tokens share come from L2.
//
// Many tokens: a workgroup takes 32 tokens and four 16-row pieces of the A of
// the distinct adapters among them, in the order of the adapters, so A is read
// once per 32 tokens. Tokens of other adapters run through the products too and
// are not stored. With three adapters or more the tokens are taken adapter by
// adapter, here and in the projection's tiles, after a sort: tokens that come
// mixed (a decode batch) would have each adapter among every 32.
//
// With few groups of tokens K is split over workgroups too, and what reads v
// adds the parts and then scales. In both forms eight waves split K, hold a batch of 128-byte K chunks in flight
// and meet in LDS in a fixed order.
#include "lora_shrink.hpp"

namespace moe {

using namespace dense;

namespace {

constexpr int kWaves = kShrinkWaves;
constexpr int FR = 4;  // 16-row rank fragments a pass
// Up to this many tokens a workgroup takes one token.
constexpr int kTokenWise = 128;
constexpr int kSortKeys = 1024;  // adapters of a sort, and none

__global__ __launch_bounds__(kWaves * 64) void lora_shrink_token_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                        int K, LoraArgs l) {
    __shared__ f32x4 red[kWaves][4];
    shrink_token(x, ldx, K, l, (int)blockIdx.x, (int)blockIdx.y * 16, red);
}

// Counting sort of the tokens by adapter, those without one last, in one
// workgroup: each wave counts its own run of tokens, a thread a key sums the
// waves' counts, and the tokens take their places. Their order inside an adapter
// changes no result: a token's column of a product does not see the others.
constexpr int kSortWaves = 16, kSortKeep = 8;
__global__ __launch_bounds__(kSortWaves * 64) void lora_sort_kernel(const int32_t* __restrict__ index, int T, int n,
                                                                     int32_t* __restrict__ order,
                                                                     int32_t* __restrict__ sorted) {
    __shared__ int at[kSortWaves][kSortKeys];
    __shared__ int total[kSortWaves];
    static_assert(kSortKeys == kSortWaves * 64, "a thread a key");
    const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) at[i][tid] = 0;
    const int64_t per = ((int64_t)T + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;  // tokens a wave
    const int64_t beg = w * per, end = beg + per < T ? beg + per : T;
    int key[kSortKeep];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) {
            const int64_t t = t0 + i * 64 + lane;
            const int a = t < end ? index[t] : 0;
            key[i] = (unsigned)a < (unsigned)n ? a : n;
        }
    };
    // Counts the i-th tokens and gives their places; those of one adapter (a
    // run) at once, as 64 additions to one word take their turns (4099 tokens in
    // eight runs: 11.6 us by additions alone, 7.5).
    auto take = [&](int i, int64_t t0) -> int {
        const int64_t left = end - (t0 + i * 64);
        if (left <= 0) return 0;
        const int k0 = __builtin_amdgcn_readfirstlane(key[i]);
        if (left >= 64 && __all(key[i] == k0)) {
            const int p = lane == 0 ? atomicAdd(&at[w][k0], 64) : 0;
            return __builtin_amdgcn_readfirstlane(p) + lane;
        }
        return lane < left ? atomicAdd(&at[w][key[i]], 1) : 0;
    };
    __syncthreads();
    for (int64_t t0 = beg; t0 < end; t0 += kSortKeep * 64) {
        load(t0);
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i)
            take(i, t0);
    }
    __syncthreads();
    int count = 0;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) count += at[i][tid];
    int upto = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) total[w] = upto;
    __syncthreads();
    int base = upto - count;
    for (int i = 0; i < w; ++i) base += total[i];
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
        const int c = at[i][tid];
        at[i][tid] = base;
        base += c;
    }
    __syncthreads();
    for (int64_t t0 = beg; t0 < end; t0 += kSortKeep * 64) {
        if (per > kSortKeep * 64) load(t0);
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) {
            const int64_t t = t0 + i * 64 + lane;
            const int p = take(i, t0);
            if (t >= end) continue;
            order[p] = (int32_t)t;
            sorted[p] = key[i] < n ? key[i] : -1;
        }
    }
}

__global__ __launch_bounds__(kWaves * 64) void lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx, int T,
                                                                  int K, LoraArgs l) {
    constexpr int FM = 2;
    __shared__ f32x4 red[kWaves][FR][FM][64];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int t0 = (int)blockIdx.x * 16 * FM;
    int idx[FM], row[FM];  // row: of x and v, counted from t0 or, with an order, from 0
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int t = t0 + 16 * f + i;
        const int v = t < T ? (l.order ? l.sorted : l.index)[t] : -1;
        idx[f] = (unsigned)v < (unsigned)l.n ? v : kNoAdapter;
        row[f] = l.order ? l.order[t < T ? t : 0] : 16 * f + i;
    }
    const rsrc_t rx = make_rsrc(l.order ? x : x + (int64_t)t0 * ldx, kRecord);
    uint32_t xo[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) xo[f] = t0 + 16 * f + i < T ? (uint32_t)(row[f] * ldx * 2) + 16u * g : kOob;
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
        int ranks[FR];
#pragma unroll
        for (int r = 0; r < FR; ++r) {
            const bool some = ad[r] != kNoAdapter;
            const int at = some ? ad[r] : 0;
            int rank = l.ranks ? l.ranks[at] : l.rank;
            rank = rank < l.rank ? rank : l.rank;
            scale[r] = l.scale && l.parts == 1 ? l.scale[at] : 1.0f;
            ranks[r] = rank;
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
                const int64_t to = l.order && !l.v_sorted ? row[f] : t0 + 16 * f + i;
                // Rows beyond the rank are zeros for any scale.
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = row0[r] + 4 * g + e < ranks[r] ? v[e] * scale[r] : 0.0f;
                *(f32x4*)(l.v + blockIdx.z * l.part_stride + to * l.vld + row0[r] + 4 * g) = v;
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

// The sort is 4 to 8 us (30 adapters of rank 32, K = N = 3584, 1000 tokens: mixed 105
// us in their own order, 57 by adapter; 4096 tokens, K = N = 2048, 32 of rank 64:
// mixed 243 and 69, in runs 67 and 75). Up to 256 tokens neither way is ahead
// by more than that: 205 tokens mixed 28 and 24, in runs 21 and 26.
bool lora_sorts(int T, int n) { return T > 256 && n > 2 && n < kSortKeys; }

hipError_t launch_lora_sort(const int32_t* index, int T, int n, int32_t* order, int32_t* sorted, hipStream_t s) {
    hipLaunchKernelGGL(lora_sort_kernel, dim3(1), dim3(kSortWaves * 64), 0, s, index, T, n, order, sorted);
    return hipGetLastError();
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
