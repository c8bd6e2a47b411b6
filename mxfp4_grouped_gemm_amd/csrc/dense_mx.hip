// Instances of the LDS-tiled product for MXFP8 operands.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes the e8m0 bytes themselves, so no
// operand is converted. It adds the eight products of a group with the
// precision of the largest of them (about 2^-14 of it is lost; sums of 128
// products of N(0, 1) codes came out 1.3e-5 off), and its results are summed
// in fp32. 4096 tokens, H = 3584, I = 2048: gated 60 us (2.0 PFLOP/s), down 42
// (1.4: 224 tiles, one round that leaves 32 compute units idle).
#include "dense_tile.hpp"

namespace moe {

using namespace dense;

template <int EPI>
static hipError_t launch_epi(const DenseArgs& a, hipStream_t s) {
    if (dense_big_tiles(a, EPI))
        return launch_tile<Tile<256, 256, 2, 4, false, false, kEltMx8, EPI, false, false>>(a, s);
    if (a.splits <= 1) return launch_tile<Tile<128, 128, 2, 2, false, false, kEltMx8, EPI, false, false>>(a, s);
    const hipError_t e = launch_tile<Tile<128, 128, 2, 2, false, false, kEltMx8, EPI, true, false>>(a, s);
    return e != hipSuccess ? e : launch_join(a, EPI, s);
}

hipError_t launch_dense_mx(const DenseArgs& a, int epi, hipStream_t s) {
    return epi == kEpiOut ? launch_epi<kEpiOut>(a, s) : launch_epi<kEpiGatedMx>(a, s);
}

}  // namespace moe
