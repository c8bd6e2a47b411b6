// The backward of the gated block: dh = dout W2 with the activation's backward
// as its epilogue, and then dx and the two weight gradients in one launch.
// 8192 tokens, H = 3584, I = 2048: dh 118 to 130 us, the gradients 463 (1.30
// PFLOP/s; matrix cores busy 78% of the time). Called in a loop over three sets of inputs
// the backward takes 577 us, the library's four plain products 720.
#include "dense_tile.hpp"

namespace moe {

using namespace dense;

namespace {

// The three products after dh do not depend on each other, and each alone
// leaves compute units idle in its last round of tiles: their tiles form one
// grid, those with the longer sum first. (dw13 and dw2 have both operands
// transposed and sum over the tokens; dx sums over the 2 I columns.)
struct GradArgs {
    DenseArgs dw13, dw2, dx;
    int n13, n2, nx;  // tiles of each
    int dx_first;
};

// TN: tiles of the weight gradients; NN: of dx. Same buffers.
template <class TN, class NN>
__global__ __launch_bounds__(TN::THREADS, 2) void grad_kernel(GradArgs g) {
    static_assert(TN::BUF == NN::BUF && TN::NB == NN::NB && TN::THREADS == NN::THREADS, "one launch");
    MOE_TILE_BUFFERS(s, TN::NB, TN::BUF);
    int id = (int)blockIdx.x;
    if (g.dx_first) {
        id = id < g.nx ? g.n13 + g.n2 + id : id - g.nx;
    }
    if (id < g.n13 + g.n2) {
        const bool second = id >= g.n13;
        const DenseArgs a = second ? g.dw2 : g.dw13;
        dense_tile<TN>(a, second ? id - g.n13 : id, 0, s);
    } else {
        dense_tile<NN>(g.dx, id - g.n13 - g.n2, 0, s);
    }
}

template <int BM, int WM, int WN, int NB, int KB>
hipError_t launch_grad(GradArgs& g, hipStream_t s) {
    using TN = Tile<BM, BM, WM, WN, true, true, kEltBf16, kEpiOut, false, false, NB, KB>;
    using NN = Tile<BM, BM, WM, WN, false, true, kEltBf16, kEpiOut, false, false, NB, KB>;
    g.n13 = g.dw13.out ? (int)tiles_of<TN>(g.dw13) : 0;
    g.n2 = g.dw2.out ? (int)tiles_of<TN>(g.dw2) : 0;
    g.nx = g.dx.out ? (int)tiles_of<NN>(g.dx) : 0;
    g.dx_first = g.dx.K > g.dw13.K;
    const int64_t grid = (int64_t)g.n13 + g.n2 + g.nx;
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((grad_kernel<TN, NN>), dim3((unsigned)grid), dim3(TN::THREADS), 0, s, g);
    return hipGetLastError();
}

int64_t square_tiles(const DenseArgs& a, int b) {
    return a.out ? (int64_t)((a.M + b - 1) / b) * ((a.N + b - 1) / b) : 0;
}

}  // namespace

// Few tokens give dh and dx few tiles of a long sum: 64 x 64 tiles that leave
// three quarters of the compute units idle split K, eight steps a part at
// least; those that leave half idle do so for sums of 64 steps and more. (One
// token, H = 1024, I = 4096: the backward took 144 us without, 32 with.)
int dense_bwd_splits(const DenseArgs& a) {
    const int64_t tiles = (int64_t)((a.M + 63) / 64) * ((a.N + 63) / 64), steps = (a.K + 63) / 64;
    if (tiles == 0 || tiles > 128 || (tiles > 64 && steps < 64)) return 1;
    const int64_t most = steps / 8, room = 256 / tiles;
    const int64_t s = room < most ? room : most;
    return s < 2 ? 1 : s > 16 ? 16 : (int)s;
}

template <int EPI>
static hipError_t launch_split(const DenseArgs& a, hipStream_t s) {
    const hipError_t e = launch_tile<Tile<64, 64, 2, 2, false, true, kEltBf16, EPI, true, false, 8>>(a, s);
    return e != hipSuccess ? e : launch_join(a, EPI, s);
}

template <int E>
static hipError_t launch_nn(const DenseArgs& a, hipStream_t s) {
    if (a.splits > 1) return launch_split<E>(a, s);
    // (A dx of so many tiles shares a grid with the weights' gradients.)
    if constexpr (E == kEpiGatedBwd) {
        if (dense_big_tiles(a, E)) return launch_tile<Tile<256, 256, 2, 4, false, true, kEltBf16, E, false, false>>(a, s);
    }
    if (!dense_one_round(a, E)) return launch_tile<Tile<128, 128, 2, 2, false, true, kEltBf16, E, false, false>>(a, s);
    // Too few 128 x 128 tiles for half of the compute units: 64 x 64 ones.
    if (square_tiles(a, 128) < 128)
        return launch_tile<Tile<64, 64, 2, 2, false, true, kEltBf16, E, false, false, 8>>(a, s);
    return launch_tile<Tile<128, 128, 2, 2, false, true, kEltBf16, E, false, false, 4>>(a, s);
}

hipError_t launch_dense_dh(const DenseArgs& a, hipStream_t s) { return launch_nn<kEpiGatedBwd>(a, s); }

hipError_t launch_dense_grads(const DenseArgs& dw13, const DenseArgs& dw2, const DenseArgs& dx, hipStream_t s) {
    GradArgs g;
    g.dw13 = dw13;
    g.dw2 = dw2;
    g.dx = dx;
    if (dx.M == 0) g.dx.out = nullptr;  // no tokens: a grid of its own would be empty
    auto tiles = [&](int b) { return square_tiles(dw13, b) + square_tiles(dw2, b) + square_tiles(g.dx, b); };
    // 256 x 256 tiles from 192 of them on, or from 160 for long sums (H = 2048,
    // I = 1408: at 700, 1024, 1500 and 2048 tokens, 160 to 200 tiles, the whole
    // backward took 66, 83, 83 and 86 us in them, 49, 69, 85 and 112 in 128 x
    // 128 ones; H = 1024, I = 4096, 192 tiles and more: 32 and 40 us at one
    // token, 75 and 87 at 700), then 128 x 128.
    const int64_t big = tiles(256);
    const int edge = big >= 192 || (big >= 160 && dw13.K >= 1536) ? 256 : tiles(128) >= 128 ? 128 : 64;
    // dx goes alone, in tiles of its own size, where the weights' many tiles
    // would leave it few of them, each a long sum: where that sum is over 2.5
    // times the compute units' mean share of all steps. (400 tokens, H = 1024,
    // I = 4096: 8 tiles of 256 x 256 over K = 8192 took 150 us of the
    // backward's 160, now 61; H = 3584, I = 2048, where the ratio is 3.7, 2.6
    // and 1.8 at 512, 700 and 1024 tokens: 95, 108 and 120 us together, 84, 110
    // and 130 alone.)
    const int64_t share = ((square_tiles(dw13, edge) + square_tiles(dw2, edge)) * (int64_t)dw13.K +
                           square_tiles(dx, edge) * dx.K) / 256;
    if (g.dx.out && (dx.splits > 1 || (edge > 64 && 2 * (int64_t)dx.K > 5 * share))) {
        const hipError_t e = launch_nn<kEpiOut>(dx, s);
        if (e != hipSuccess) return e;
        g.dx.out = nullptr;
    }
    if (edge == 256) return launch_grad<256, 2, 4, 4, 64>(g, s);
    if (edge == 128) return launch_grad<128, 2, 2, 4, 128>(g, s);
    return launch_grad<64, 2, 2, 8, 128>(g, s);
}

}  // namespace moe
