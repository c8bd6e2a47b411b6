// The backward of the gated block: dh = dout W2 with the activation's backward
// as its epilogue, and then dx and the two weight gradients in one launch.
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
    static_assert(TN::BUF == NN::BUF && TN::NB == 4 && NN::NB == 4 && TN::THREADS == NN::THREADS, "one launch");
    __shared__ __align__(1024) uint8_t s0[TN::BUF];
    __shared__ __align__(1024) uint8_t s1[TN::BUF];
    __shared__ __align__(1024) uint8_t s2[TN::BUF];
    __shared__ __align__(1024) uint8_t s3[TN::BUF];
    int id = (int)blockIdx.x;
    if (g.dx_first) {
        id = id < g.nx ? g.n13 + g.n2 + id : id - g.nx;
    }
    if (id < g.n13 + g.n2) {
        const bool second = id >= g.n13;
        const DenseArgs a = second ? g.dw2 : g.dw13;
        dense_tile<TN>(a, second ? id - g.n13 : id, 0, s0, s1, s2, s3);
    } else {
        dense_tile<NN>(g.dx, id - g.n13 - g.n2, 0, s0, s1, s2, s3);
    }
}

template <int BM, int WM, int WN, int KB>
hipError_t launch_grad(GradArgs& g, hipStream_t s) {
    using TN = Tile<BM, BM, WM, WN, true, true, kEltBf16, kEpiOut, false, false, 4, KB>;
    using NN = Tile<BM, BM, WM, WN, false, true, kEltBf16, kEpiOut, false, false, 4, KB>;
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

hipError_t launch_dense_dh(const DenseArgs& a, hipStream_t s) {
    constexpr int E = kEpiGatedBwd;
    if (dense_big_tiles(a, E)) return launch_tile<Tile<256, 256, 2, 4, false, true, kEltBf16, E, false, false>>(a, s);
    if (!dense_one_round(a, E)) return launch_tile<Tile<128, 128, 2, 2, false, true, kEltBf16, E, false, false>>(a, s);
    // Too few 128 x 128 tiles for half of the compute units: 64 x 64 ones.
    if (square_tiles(a, 128) < 128)
        return launch_tile<Tile<64, 64, 2, 2, false, true, kEltBf16, E, false, false, 4>>(a, s);
    return launch_tile<Tile<128, 128, 2, 2, false, true, kEltBf16, E, false, false, 4>>(a, s);
}

hipError_t launch_dense_grads(const DenseArgs& dw13, const DenseArgs& dw2, const DenseArgs& dx, hipStream_t s) {
    GradArgs g;
    g.dw13 = dw13;
    g.dw2 = dw2;
    g.dx = dx;
    auto tiles = [&](int b) { return square_tiles(dw13, b) + square_tiles(dw2, b) + square_tiles(dx, b); };
    if (tiles(256) >= 160) return launch_grad<256, 2, 4, 64>(g, s);
    if (tiles(128) >= 128) return launch_grad<128, 2, 2, 128>(g, s);
    return launch_grad<64, 2, 2, 128>(g, s);
}

}  // namespace moe
