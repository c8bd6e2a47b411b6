// Arguments and launchers of the operators of a trainable expert block: layer
// norm with its backward pass, rows sorted by expert and back, and what the
// product with bias and activation needs beside the dense tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "column_join.hpp"
#include "dense.hpp"

namespace moe {

struct LayerNormArgs {
    const uint16_t* x;
    const void* residual;
    const void* weight;
    const void* bias;
    void* residual_out;
    uint16_t* y;
    float* mean;
    float* rstd;
    int64_t ldx, ldr, ldro, ldy;
    int T, H;
    float eps;
    int res_f32, weight_f32;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);

struct LayerNormBwdArgs {
    const uint16_t* dy;
    const void* s;
    const float* mean;
    const float* rstd;
    const void* weight;
    const void* dres;  // gradient that reaches s from elsewhere, or null
    uint16_t* dx;
    void* dresidual;  // of s's type
    float* partial;   // [layer_norm_parts, 2, H rounded up to 8], where sums over the rows are asked for
    void* dweight;
    void* dbias;
    int64_t lddy, lds, lddr, lddx, lddro;
    int T, H;
    int s_f32, weight_f32;
};
hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, hipStream_t s);

// dz = dout act'(pre) and its sums over the rows. dz may be null (dz == dout).
struct LinearDzArgs {
    const void* dout;
    const uint16_t* pre;
    uint16_t* dz;
    float* partial;  // [linear_dz_parts, N] or null
    int64_t lddo;
    int T, N;
    int dout_f32, act;
};
int linear_dz_parts(int T, int N);
hipError_t launch_linear_dz(const LinearDzArgs& a, hipStream_t s);
// dw = dz^T x and dx = dz W: how they are launched, which sets the parts of their
// sums (the products' splits; one of them is in parts at most).
enum LinearGrads {
    kGradsDense,  // launch_dense_grads
    kGradsFew,    // few tokens: 128 x 128 tiles with small buffers
    kGradsSmall   // 64 x 64 tiles
};
LinearGrads linear_grads_plan(DenseArgs& dw, DenseArgs& dx);
hipError_t launch_linear_grads(const DenseArgs& dw, const DenseArgs& dx, const ColumnJoin& sums, LinearGrads plan,
                               hipStream_t s);

// Rows of elt bytes an element. `rows` [T, topk]: the sorted row of each pair,
// -1 - row for a pair of no expert.
struct PermuteArgs {
    const void* x;
    void* out;
    const int32_t* ids;
    int32_t* rows;
    int32_t* offsets;
    int32_t* counts;  // [2, chunks, E + 1] and [chunks, 16] (none for few pairs)
    int64_t ldx, ldo; // bytes
    int64_t row_bytes;
    int T, topk, E;
};
int64_t permute_workspace_bytes(int64_t pairs, int E);
// The most that so many pairs or fewer take.
int64_t permute_most_workspace_bytes(int64_t pairs, int E);
hipError_t launch_permute(const PermuteArgs& a, hipStream_t s);

struct UnpermuteArgs {
    const void* y;
    const int32_t* rows;
    const float* weights;  // or null: 1
    const void* residual;
    void* out;
    int64_t ldy, ldr, ldo;
    int64_t pairs;  // rows of y
    int T, topk, H;
    int y_f32, out_f32;
};
hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s);

struct UnpermuteBwdArgs {
    const void* dout;
    const int32_t* rows;
    const float* weights;
    const void* y;
    void* dy;        // or null
    float* dweights; // or null (needs y)
    int64_t lddo, ldy, lddy;
    int T, topk, H;
    int y_f32, out_f32;
};
hipError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, hipStream_t s);

}  // namespace moe
