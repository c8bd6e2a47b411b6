// Instances of the LDS-tiled product for the backward of the gated block:
// dh = dout W2 with the activation's backward as its epilogue, dx, and the two
// weight gradients.
#include "dense_tile.hpp"

namespace moe {

using namespace dense;

template <bool XT, int EPI>
static hipError_t launch_epi(const DenseArgs& a, hipStream_t s) {
    if (dense_big_tiles(a, EPI)) {
        // With both operands transposed the 128-byte steps need more address
        // registers than there are; half steps in four buffers fit (4096 x
        // 3584 over 8192 tokens: 202 -> 181 us). With one they lose 3 %.
        if constexpr (XT) return launch_tile<Tile<256, 256, 2, 4, XT, true, kEltBf16, EPI, false, false, 4, 64>>(a, s);
        else return launch_tile<Tile<256, 256, 2, 4, XT, true, kEltBf16, EPI, false, false>>(a, s);
    }
    if (!dense_one_round(a, EPI)) return launch_tile<Tile<128, 128, 2, 2, XT, true, kEltBf16, EPI, false, false>>(a, s);
    // Too few 128 x 128 tiles for half of the compute units: 64 x 64 ones.
    const int64_t tiles = (int64_t)((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (tiles < 128) return launch_tile<Tile<64, 64, 2, 2, XT, true, kEltBf16, EPI, false, false, 4>>(a, s);
    return launch_tile<Tile<128, 128, 2, 2, XT, true, kEltBf16, EPI, false, false, 4>>(a, s);
}

hipError_t launch_dense_bwd(const DenseArgs& a, int order, int epi, hipStream_t s) {
    if (order == kTN) return launch_epi<true, kEpiOut>(a, s);
    return epi == kEpiOut ? launch_epi<false, kEpiOut>(a, s) : launch_epi<false, kEpiGatedBwd>(a, s);
}

}  // namespace moe
