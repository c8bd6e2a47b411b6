// Arguments and launchers of the dense operators around the routed experts:
// residual RMS norm, gated feed-forward block (forward and backward) and the
// projection with low-rank adapters.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "column_join.hpp"

namespace moe {

// A stack of low-rank adapters beside one projection [N, K]: token t adds
// B[a] (scale[a] * (A[a] x[t])) for a = index[t]; an index outside [0, n) adds
// nothing. v [T, vld] (fp32) receives scale * A x from the narrow product and
// is read by the projection's kernels.
constexpr int kMaxLoraParts = 4;

struct LoraArgs {
    const uint16_t* a;       // bf16 [n, rank, K]
    const uint16_t* b;       // bf16 [n, N, rank]
    const int32_t* index;    // [T]
    const int32_t* order;    // [T] tokens by adapter, or null: the tokens' own order
    const int32_t* sorted;   // [T] their adapters (-1: none), with `order`
    const int32_t* ranks;    // [n] or null (all `rank`)
    const float* scale;      // [n] or null (all 1)
    float* v;                // fp32 [parts, T, vld], vld = rank rounded up to 32
    int64_t part_stride;     // T * vld
    int n, rank, vld, parts; // v is the sum of the parts (of K), of A x without the scale if there are several
    bool v_sorted;           // row p of v is token order[p]'s, else token p's
};

// Epilogues of the dense products.
constexpr int kEpiOut = 0;      // out = acc (+ addend), bf16 or fp32
constexpr int kEpiGated = 1;    // h = silu(gate) * up, bf16; optional gate_up
constexpr int kEpiGatedMx = 2;  // the same, h in MXFP8
constexpr int kEpiGatedBwd = 3; // acc = dh: dgate_up and h from the saved gate_up
constexpr int kEpiAct = 4;      // out = act(acc + bias) (+ addend), optional pre
constexpr bool epi_gated(int epi) { return epi == kEpiGated || epi == kEpiGatedMx; }

// Activations of kEpiAct.
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

// One product C[m, n] = sum_k X[m, k] W[n, k]. Strides in elements. For the
// gated epilogues W holds 2N rows (gate rows, then up rows) and n counts pairs.
struct DenseArgs {
    const void* x;
    const void* w;
    const uint8_t* xs;  // e8m0 [M, K/32] (MXFP8)
    const uint8_t* ws;
    int64_t ldx, ldw;
    int M, N, K;
    void* out;              // kEpiOut: C; kEpiGated: h; kEpiGatedMx: h codes; kEpiGatedBwd: dgate_up
    int64_t ldo;
    int out_f32;
    const void* addend;     // [M, N], stride ldadd; bf16, or fp32 with addend_f32
    int64_t ldadd;
    int addend_f32;
    const void* bias;       // [N], bf16 or fp32, or null
    int bias_f32;
    int act;
    uint16_t* pre;          // bf16 [M, N]: acc + bias, saved (may be null)
    uint16_t* gate_up;      // kEpiGated: saved (may be null); kEpiGatedBwd: read
    uint16_t* h;            // kEpiGatedBwd: h
    uint8_t* hs;            // kEpiGatedMx: e8m0 scales of h
    float* partial;         // split K: fp32 [splits, M, N or 2N]
    int splits;             // 1: the epilogue runs in the product's kernel
    LoraArgs lora;          // lora.n == 0: none
};

// splits the launcher would take for this product, and the bytes of `partial`
// that they need.
int dense_splits(const DenseArgs& a, int elt, int epi);
// (join: the product is joined by a second kernel even if splits == 1).
inline int64_t dense_partial_bytes(const DenseArgs& a, int splits, int epi, bool join) {
    return splits <= 1 && !join ? 0 : (int64_t)splits * a.M * a.N * (epi_gated(epi) ? 2 : 1) * 4;
}
bool dense_big_tiles(const DenseArgs& a, int epi);
bool dense_one_round(const DenseArgs& a, int epi);
hipError_t launch_join(const DenseArgs& a, int epi, hipStream_t s);
// A forward product (both operands K-major).
hipError_t launch_dense(const DenseArgs& a, int elt, int epi, hipStream_t s);
hipError_t launch_dense_nt(const DenseArgs& a, int epi, hipStream_t s);
hipError_t launch_dense_mx(const DenseArgs& a, int epi, hipStream_t s);
// Backward: dh (X K-major, W with K as its row index), then the gradients of
// the weights (both operands with K as the row index) and of x (as dh). A
// gradient whose `out` is null is not computed.
// (Their a.splits: dense_bwd_splits, of dh and of dx.)
int dense_bwd_splits(const DenseArgs& a);
hipError_t launch_dense_dh(const DenseArgs& a, hipStream_t s);
// Whether launch_dense_grads takes dx in a launch of its own.
bool dense_dx_alone(const DenseArgs& dw13, const DenseArgs& dw2, const DenseArgs& dx);
// (sums: a bias gradient to be joined in the same launch, or no outputs.)
hipError_t launch_dense_grads(const DenseArgs& dw13, const DenseArgs& dw2, const DenseArgs& dx, const ColumnJoin& sums,
                              hipStream_t s);

// Up to this many tokens the products stream the weights without LDS tiles.
// (MXFP8 with H = 3584, I = 2048: 33 us at 64 tokens, 26 in tiles, where h is
// quantised once and not by every workgroup of the second product; at 32 both
// take 26.) More than 16 tokens only with fewer rows of W than give tiles of
// their own to half of the compute units with K in few parts (K = 3584, 64
// tokens: 4096 rows 15.2 us, 16.1 in tiles; 8192 rows 22.8 and 19.4; 16384
// rows 42 and 31, at 25 tokens 34 and 27); in MXFP8 with one round of
// workgroups (H = 3584, I = 8192, 32 tokens: 69 us, 38 in tiles; H = 7168, I =
// 2048: 39 and 28).
constexpr int kSkinnyMaxTokens = 64, kSkinnyMaxTokensMx = 32;
constexpr int kSkinnyManyRows = 8192, kSkinnyManyRowsMx = 4104;  // from here on 16 tokens at most
// elt 0: bf16; 1: MXFP8 activations and weights. h_f32: the fp32 h of the
// MXFP8 block between its two products (written by kEpiGated, and read and
// quantised by the second product).
// Parts of K that launch_skinny takes for this product (a.splits).
int skinny_splits(const DenseArgs& a, int elt, int epi);
bool skinny_wide(const DenseArgs& a, bool gated);
// Whether its results are joined from a.partial (even of one part).
bool skinny_joins(const DenseArgs& a, int splits, int elt, int epi);
int skinny_narrow(const DenseArgs& a);  // workgroups of the adapters' narrow product
hipError_t launch_skinny(const DenseArgs& a, int elt, int epi, const float* h_f32, hipStream_t s);

// Whether the tokens are taken adapter by adapter (l.order, l.sorted), and the
// sort for it.
bool lora_sorts(int T, int n);
hipError_t launch_lora_sort(const int32_t* index, int T, int n, int32_t* order, int32_t* sorted, hipStream_t s);
// Parts of K that launch_lora_shrink takes (l.parts).
int lora_parts(int T);
// v[t] = scale * A[index[t]] x[t].
hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const LoraArgs& l, hipStream_t s);

struct NormArgs {
    const uint16_t* x;
    const void* residual;
    const void* weight;
    void* residual_out;
    uint16_t* y;
    uint8_t* q;
    uint8_t* qs;
    int64_t ldx, ldr, ldro, ldy, ldq, ldqs;
    int T, H;
    float eps, offset;
    int res_f32, weight_f32;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);

}  // namespace moe
