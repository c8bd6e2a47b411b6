// The activation's backward of the product with bias: dz = dout act'(pre),
// rounded to bf16 (it is an operand of the two products that follow), and the
// bias gradient, the sum of its unrounded values over the rows.
//
// A thread goes through rows blockIdx.y, + gridDim.y, ... with eight columns,
// whose sums stay in registers; the parts are joined by a second kernel.
#include "common.hpp"
#include "dense_epilogue.hpp"
#include "row_io.hpp"
#include "train.hpp"

namespace moe {

using namespace rows;

template <bool F32>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearDzArgs a) {
    const int n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8;
    if (n >= a.N) return;
    f32x8 sum = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        f32x8 d = load8<true>((const char*)a.dout + t * a.lddo * (F32 ? 4 : 2), F32, n, a.N);
        if (a.act != kActNone) {
            const f32x8 z = load8<true>(a.pre + t * a.N, false, n, a.N);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] *= dense::act_slope(a.act, z[e]);
        }
        sum += d;
        if (a.dz) {
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
            *(u32x4*)(a.dz + t * a.N + n) = o;
        }
    }
    if (!a.partial) return;
    float* p = a.partial + (int64_t)blockIdx.y * a.N + n;
    *(f32x4*)p = __builtin_shufflevector(sum, sum, 0, 1, 2, 3);
    *(f32x4*)(p + 4) = __builtin_shufflevector(sum, sum, 4, 5, 6, 7);
}

int linear_dz_parts(int T, int N) {
    const int cols = (N + 2047) / 2048;
    int parts = 1024 / cols;
    if (parts < 1) parts = 1;
    return T < parts ? T : parts;
}

hipError_t launch_linear_dz(const LinearDzArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 2047) / 2048), (unsigned)linear_dz_parts(a.T, a.N)), block(256);
    if (a.dout_f32) hipLaunchKernelGGL(linear_dz_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(linear_dz_kernel<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
