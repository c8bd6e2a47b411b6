// The activation's backward of the product with bias: dz = dout act'(pre),
// rounded to bf16 (it is an operand of the two products that follow: dx and dw are
// 2.34e-3 of their 2-norm off, 1.66e-3 if their own rounding were the only one; a
// second bf16 number for what it loses would be a second pass of both products), and
// the bias gradient, the sum of its unrounded values over the rows.
//
// A workgroup takes 512 columns, eight a lane, and its four waves rows w, w + 4,
// ... of the workgroup's run of rows, four in flight each; the sums of the waves
// meet in LDS, those of the workgroups in the launch of the products. 8192 x 4096,
// GELU: 40 us, 5.2 TB/s.
#include "common.hpp"
#include "dense_epilogue.hpp"
#include "dense_tile.hpp"
#include "row_io.hpp"
#include "train.hpp"

namespace moe {

using namespace rows;

namespace {
constexpr int kAtOnce = 4;           // rows a wave has in flight
constexpr int kTurn = 4 * kAtOnce;   // rows a workgroup takes in a turn
}  // namespace

// A kernel an activation: few instructions to fetch for a call of few rows.
template <bool F32, int ACT>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearDzArgs a) {
    __shared__ f32x4 part[4][64][2];
    const int lane = (int)threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n = ((int)blockIdx.x * 64 + lane) * 8;
    const int64_t turns = ((int64_t)a.T + kTurn - 1) / kTurn;
    const int64_t beg = turns * blockIdx.y / gridDim.y * kTurn, stop = turns * (blockIdx.y + 1) / gridDim.y * kTurn;
    const int64_t end = stop < a.T ? stop : a.T;
    f32x8 sum = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n < a.N) {
        for (int64_t t0 = beg + w; t0 < end; t0 += kTurn) {
            Raw8 fd[kAtOnce], fz[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                // (A row past the end: the first one, not used.)
                const int64_t t = t0 + 4 * i < end ? t0 + 4 * i : t0;
                fd[i] = fetch8<kAligned>((const char*)a.dout + t * a.lddo * (F32 ? 4 : 2), F32, n, a.N);
                if (ACT != kActNone) fz[i] = fetch8<kAligned>(a.pre + t * a.N, false, n, a.N);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (t0 + 4 * i >= end) continue;
                f32x8 d = widen8<kAligned>(fd[i], F32, n, a.N);
                if constexpr (ACT != kActNone) {
                    const f32x8 z = widen8<kAligned>(fz[i], false, n, a.N);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] *= dense::act_slope(ACT, z[e]);
                }
                sum += d;
                if (a.dz) {
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
                    *(u32x4*)(a.dz + (t0 + 4 * i) * a.N + n) = o;
                }
            }
        }
    }
    if (!a.partial) return;
    part[w][lane][0] = __builtin_shufflevector(sum, sum, 0, 1, 2, 3);
    part[w][lane][1] = __builtin_shufflevector(sum, sum, 4, 5, 6, 7);
    __syncthreads();
    if (w >= 2 || n >= a.N) return;
    *(f32x4*)(a.partial + (int64_t)blockIdx.y * a.N + n + 4 * w) =
        (part[0][lane][w] + part[1][lane][w]) + (part[2][lane][w] + part[3][lane][w]);
}

int linear_dz_parts(int T, int N) {
    // Eight workgroups a compute unit, a turn of rows each at least.
    const int cols = (N + 511) / 512;
    const int turns = (int)(((int64_t)T + kTurn - 1) / kTurn);
    const int parts = 2048 / cols < 1 ? 1 : 2048 / cols < 256 ? 2048 / cols : 256;
    return turns < parts ? turns : parts;
}

template <int ACT>
static void launch_as(const LinearDzArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 511) / 512), (unsigned)linear_dz_parts(a.T, a.N)), block(256);
    if (a.dout_f32) hipLaunchKernelGGL((linear_dz_kernel<true, ACT>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linear_dz_kernel<false, ACT>), grid, block, 0, s, a);
}

hipError_t launch_linear_dz(const LinearDzArgs& a, hipStream_t s) {
    if (a.act == kActNone) launch_as<kActNone>(a, s);
    else if (a.act == kActRelu) launch_as<kActRelu>(a, s);
    else if (a.act == kActSilu) launch_as<kActSilu>(a, s);
    else if (a.act == kActGelu) launch_as<kActGelu>(a, s);
    else launch_as<kActGeluTanh>(a, s);
    return hipGetLastError();
}

// The products of the backward where the dense block's grid of whole sums leaves
// compute units idle.
//
// Few tokens (an expert's rows): dw is a sum of one or two steps, bound
// by what it writes, and dx a long sum of few rows. 128 x 128 tiles with two
// small buffers, so that the loads of some overlap the stores of others (three
// workgroups a compute unit), in one launch: parts of dx first, then the tiles
// of dw.
namespace {

using dense::kEltBf16;
using dense::Tile;

struct GradsArgs {
    DenseArgs dw, dx;
    int nx, nw;  // tiles of each
    ColumnJoin sums;
    int nsums;
};

// TN: tiles of dw; NN: of dx; each of them takes its product's parts first.
template <class TN, class NN>
__global__ __launch_bounds__(256, 2) void linear_grads_kernel(GradsArgs g) {
    static_assert(TN::BUF == NN::BUF && TN::NB == NN::NB && TN::THREADS == 256 && NN::THREADS == 256, "one launch");
    MOE_TILE_BUFFERS(s, NN::NB, NN::BUF);
    int id = (int)blockIdx.x - g.nsums;
    if (id < 0) {
        static_assert(NN::BUF >= column_join_lds(kFewRuns), "the sums meet in a tile's buffer");
        column_join<kFewRuns>(g.sums, (int)blockIdx.x, (float*)s[0]);
        return;
    }
    // The longer sums first.
    const int first = NN::SPLIT || !TN::SPLIT ? g.nx * g.dx.splits : g.nw * g.dw.splits;
    const bool later = id >= first;
    if (later) id -= first;
    if ((NN::SPLIT || !TN::SPLIT) != later) dense::dense_tile<NN>(g.dx, id % g.nx, id / g.nx, s);
    else dense::dense_tile<TN>(g.dw, id % g.nw, id / g.nw, s);
}

template <class TN, class NN>
hipError_t launch_grads(GradsArgs& g, hipStream_t s) {
    g.nw = g.dw.out ? (int)dense::tiles_of<TN>(g.dw) : 0;
    g.nx = g.dx.out ? (int)dense::tiles_of<NN>(g.dx) : 0;
    g.nsums = g.sums.out0 ? column_join_groups(g.sums) : 0;
    const unsigned grid = (unsigned)(g.nsums + g.nx * g.dx.splits + g.nw * g.dw.splits);
    hipLaunchKernelGGL((linear_grads_kernel<TN, NN>), dim3(grid), dim3(256), 0, s, g);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && g.nx && NN::SPLIT) e = launch_join(g.dx, kEpiOut, s);
    if (e == hipSuccess && g.nw && TN::SPLIT) e = launch_join(g.dw, kEpiOut, s);
    return e;
}

template <int EDGE, int NB, int KB, bool SPLIT>
using DwTile = Tile<EDGE, EDGE, 2, 2, true, true, kEltBf16, kEpiOut, SPLIT, false, NB, KB>;
template <int EDGE, int NB, int KB, bool SPLIT>
using DxTile = Tile<EDGE, EDGE, 2, 2, false, true, kEltBf16, kEpiOut, SPLIT, false, NB, KB>;

int64_t tiles_by(int edge, const DenseArgs& a) { return (int64_t)((a.M + edge - 1) / edge) * ((a.N + edge - 1) / edge); }

}  // namespace

// Up to 128 tokens of weights with 128 tiles and more, and up to 512 where the
// products' common grid would take dx alone and the weights are large. In us, here
// and in that grid: K = 3584, N = 4096: 1 token 21.8 and 27.4, 16 24.0 and 29.2, 64
// 26.6 and 30.6, 128 32.9 and 32.8, 300 43 and 55; K = 2048, N = 1408: 16 tokens
// 18.8 and 22.2, 256 (not here) 25.3 and 21.1; K = 1024, N = 8192: 256 tokens 33 and
// 38; K = 8192, N = 1024: 16 tokens 19.0 and 26.2, 256 (not here) 30.9 and 25.1. Large
// weights: K = 2048, N = 2816: 150 tokens 26.3 and 31.9, 256 29.0 and 32.8, 400 31.7 and
// 31.8; K = 1408, N = 4096: 256 28.8 and 26.5; K = 2560, N = 2560: 150 24.8 and 31.6;
// K = 2048, N = 2560: 256 29.1 and 31.9; smaller ones (not here): K = N = 2048: 200 26.3
// and 23.6, 256 28.3 and 24.2; K = 1024, N = 4096: 256 28.2 and 24.1, 400 29.7 and 26.9; K
// = 512, N = 9000: 150 31.2 and 28.3, but 300 33.5 and 35.9.
static bool few_tokens(const DenseArgs& dw, const DenseArgs& dx) {
    const int T = dx.M;
    if (T == 0 || T > 512 || tiles_by(128, dw) < 128) return false;
    return T <= 128 || ((int64_t)dw.M * dw.N >= 5 << 20 && dense_dx_alone(dw, DenseArgs{}, dx));
}

// Weights of few tiles and many tokens: the sum over the tokens in parts, four
// steps of 64 and more, two workgroups a compute unit. In us, here and in the grid
// of whole sums: K = N = 512: 8000 tokens 34 and 69, 4000 25 and 40, 2000 (not here)
// 22 and 17; K = N = 256: 8000 tokens 27 and 68; K = N = 768: 8000 tokens 50 and 71,
// 3000 28.5 and 35; K = 256, N = 2048: 4000 tokens 33 and 32, 3000 29 and 27; K =
// N = 896 (196 tiles, not here): 4000 tokens 41 both. Where dx's sum is as long and
// would be left whole on a few compute units, that one is in parts instead (below).
// dw in parts, dx in parts: 3000 tokens, K = 64, N = 10240 93 and 72, N = 4096 39.3 and
// 35.8; 5000, K = 8, N = 8192 94.8 and 82.1; 3500, K = 128, N = 5120 61.8 and 51.9; 4000,
// K = 128, N = 4096 44.8 and 44.0; where it is shorter: 5000, K = 64, N = 4096 52.3 and
// 54.9, 3000, K = 64, N = 2048 26.6 and 27.4 (6000, K = 64, N = 4096 66.3 and 60.8). Both
// in parts, and a launch more: 75, 38.0, 84, 55.5, 47.0.
static bool long_sums(const DenseArgs& dw, const DenseArgs& dx) {
    return dw.K >= 3000 && tiles_by(64, dw) <= 160 && (dx.K < dw.K || dense_bwd_splits(dx) < 2);
}

LinearGrads linear_grads_plan(DenseArgs& dw, DenseArgs& dx) {
    // 16 parts at most: above, the join's bytes grow with the parts. In us with 8, 16 and
    // 32: dx of 1 token, K = 1024, N = 8192 25.9, 21.1 and 22.4, 128 tokens 32.5, 28.8 and
    // 32.8, 16 tokens, N = 16384 42.9, 31.6 and 31.1, K = 512, N = 32768 73, 47 and 38; dw of
    // 30000 tokens, K = N = 128 41.5, 38.6 and 43.5, 8000 tokens, K = N = 128 20.2, 20.7 and
    // 24.9, 256 23.4, 27.4 and 31.8 (24.7 with four).
    auto parts = [](int64_t room, int64_t most) { return (int)(room < most ? (room < 16 ? room : 16) : (most < 16 ? most : 16)); };
    dw.splits = dx.splits = 1;
    if (few_tokens(dw, dx)) {
        // A workgroup a compute unit, four steps of 64 and more each.
        const int s = parts(256 / tiles_by(128, dx), dx.K / 256);
        dx.splits = s < 2 ? 1 : s;
        return kGradsFew;
    }
    if (long_sums(dw, dx)) {
        dw.splits = parts(512 / tiles_by(64, dw), dw.K / 256);
        return kGradsSmall;
    }
    // Small products whose dx would go alone, in parts: with dw in 64 x 64 tiles,
    // and in parts from 32 steps on (fewer do not pay for the join). 117 tokens, K =
    // 216, N = 1376: 17.4 us, alone 25.8; 346 tokens, K = 120, N = 2184, in parts:
    // 19.8 and 24.0; 500 tokens, K = 256, N = 4096: 19.7 and 26.0.
    const int s = dense_bwd_splits(dx);
    if (s < 2) return kGradsDense;
    dx.splits = dx.K >= 2048 ? s : 1;
    return kGradsSmall;
}

hipError_t launch_linear_grads(const DenseArgs& dw, const DenseArgs& dx, const ColumnJoin& sums, LinearGrads plan,
                               hipStream_t s) {
    GradsArgs g;
    g.dw = dw;
    g.dx = dx;
    g.sums = sums;
    if (plan == kGradsDense) return launch_dense_grads(dw, DenseArgs{}, dx, sums, s);
    if (plan == kGradsFew) {
        if (dx.splits > 1) return launch_grads<DwTile<128, 2, 64, false>, DxTile<128, 2, 64, true>>(g, s);
        return launch_grads<DwTile<128, 2, 64, false>, DxTile<128, 2, 64, false>>(g, s);
    }
    if (dw.splits > 1) return launch_grads<DwTile<64, 4, 128, true>, DxTile<64, 4, 128, false>>(g, s);
    if (dx.splits > 1) return launch_grads<DwTile<64, 4, 128, false>, DxTile<64, 4, 128, true>>(g, s);
    return launch_grads<DwTile<64, 4, 128, false>, DxTile<64, 4, 128, false>>(g, s);
}

}  // namespace moe
