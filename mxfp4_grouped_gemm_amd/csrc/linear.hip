// The activation's backward of the product with bias: dz = dout act'(pre),
// rounded to bf16 (it is an operand of the two products that follow), and the
// bias gradient, the sum of its unrounded values over the rows.
//
// A workgroup takes 512 columns, eight a lane, and its four waves rows w, w + 4,
// ... of the workgroup's run of rows, four in flight each; the sums of the waves
// meet in LDS, those of the workgroups in the launch of the products.
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

// Gradients of few tokens (an expert's rows): dw is a sum of one or two steps, bound
// by what it writes, and dx a long sum of few rows. 128 x 128 tiles with two
// small buffers, so that the loads of some overlap the stores of others (three
// workgroups a compute unit), in one launch: parts of dx first, then the tiles
// of dw.
namespace {

using dense::kEltBf16;
using dense::Tile;

struct ShortArgs {
    DenseArgs dw, dx;
    int nx, nw;  // tiles of each
    ColumnJoin sums;
    int nsums;
};

using ShortDw = Tile<128, 128, 2, 2, true, true, kEltBf16, kEpiOut, false, false, 2, 64>;
template <bool SPLIT>
using ShortDx = Tile<128, 128, 2, 2, false, true, kEltBf16, kEpiOut, SPLIT, false, 2, 64>;

template <bool SPLIT>
__global__ __launch_bounds__(256, 2) void short_grads_kernel(ShortArgs g) {
    using NN = ShortDx<SPLIT>;
    static_assert(ShortDw::BUF == NN::BUF && NN::THREADS == 256, "one launch");
    MOE_TILE_BUFFERS(s, 2, NN::BUF);
    int id = (int)blockIdx.x - g.nsums;
    if (id < 0) {
        static_assert(NN::BUF >= column_join_lds(kFewRuns), "the sums meet in a tile's buffer");
        column_join<kFewRuns>(g.sums, (int)blockIdx.x, (float*)s[0]);
        return;
    }
    const int parts = SPLIT ? g.dx.splits : 1;
    if (id < g.nx * parts) {
        dense::dense_tile<NN>(g.dx, id % g.nx, id / g.nx, s);
        return;
    }
    dense::dense_tile<ShortDw>(g.dw, id - g.nx * parts, 0, s);
}

int64_t tiles128(int M, int N) { return (int64_t)((M + 127) / 128) * ((N + 127) / 128); }

}  // namespace

// Up to 128 tokens of weights with 128 tiles and more, and up to 512 where the
// products' common grid would take dx alone and the weights are large. In us, here
// and in that grid: K = 3584, N = 4096: 1 token 21.8 and 27.4, 16 24.0 and 29.2, 64
// 26.6 and 30.6, 128 32.9 and 32.8, 300 43 and 55; K = 2048, N = 1408: 16 tokens
// 18.8 and 22.2, 256 (not here) 25.3 and 21.1; K = 1024, N = 8192: 256 tokens 33 and
// 38; K = 8192, N = 1024: 16 tokens 19.0 and 26.2, 256 (not here) 30.9 and 25.1.
bool linear_short(const DenseArgs& dw, const DenseArgs& dx) {
    const int T = dx.M;
    if (T == 0 || T > 512 || tiles128(dw.M, dw.N) < 128) return false;
    return T <= 128 || ((int64_t)dw.M * dw.N >= 1 << 22 && dense_dx_alone(dw, DenseArgs{}, dx));
}

int linear_short_splits(const DenseArgs& dx) {
    // A workgroup a compute unit, four steps of 64 and more each.
    const int64_t most = dx.K / 256, room = 256 / tiles128(dx.M, dx.N);
    const int64_t s = room < most ? room : most;
    return s < 2 ? 1 : s > 16 ? 16 : (int)s;
}

hipError_t launch_linear_short_grads(const DenseArgs& dw, const DenseArgs& dx, const ColumnJoin& sums, hipStream_t s) {
    ShortArgs g;
    g.dw = dw;
    g.dx = dx;
    g.sums = sums;
    g.nw = dw.out ? (int)tiles128(dw.M, dw.N) : 0;
    g.nx = dx.out ? (int)tiles128(dx.M, dx.N) : 0;
    g.nsums = sums.out0 ? column_join_groups(sums) : 0;
    const unsigned grid = (unsigned)(g.nsums + g.nx * dx.splits + g.nw);
    if (dx.splits > 1) hipLaunchKernelGGL(short_grads_kernel<true>, dim3(grid), dim3(256), 0, s, g);
    else hipLaunchKernelGGL(short_grads_kernel<false>, dim3(grid), dim3(256), 0, s, g);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !dx.out || dx.splits == 1 ? e : launch_join(dx, kEpiOut, s);
}

}  // namespace moe
