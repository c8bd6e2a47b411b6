// C ABI of the row movers: tokens sorted by expert, and back.
#include "abi_checks.hpp"
#include "train.hpp"

using namespace moe::abi;

namespace {

constexpr int kMaxRowTokens = 1 << 22;
constexpr int kMaxRowTopk = 64;
constexpr int kMaxRowExperts = 1024;
constexpr int kMaxRowCols = 1 << 18;

moe_status check_rows(const char* fn, int T, int topk, int H) {
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%d < 0", fn, T);
    if (T > kMaxRowTokens) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d > %d", fn, T, kMaxRowTokens);
    if (topk < 1) return fail(MOE_ERR_INVALID_ARG, "%s: topk=%d < 1", fn, topk);
    if (topk > kMaxRowTopk) return fail(MOE_ERR_UNSUPPORTED, "%s: topk=%d > %d", fn, topk, kMaxRowTopk);
    if (H < 1) return fail(MOE_ERR_INVALID_ARG, "%s: H=%d < 1", fn, H);
    if (H > kMaxRowCols) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d > %d", fn, H, kMaxRowCols);
    return MOE_OK;
}

int size_of(moe_dtype t) { return t == MOE_DT_F32 ? 4 : t == MOE_DT_BF16 ? 2 : t == MOE_DT_U8 ? 1 : 0; }

moe_status check_float(const char* fn, moe_dtype t) {
    if (t != MOE_DT_BF16 && t != MOE_DT_F32) return fail(MOE_ERR_UNSUPPORTED, "%s: type %d unknown", fn, (int)t);
    return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_permute_workspace_size(int T, int topk, int E) {
    if (T < 0 || T > kMaxRowTokens || topk < 1 || topk > kMaxRowTopk || E < 1 || E > kMaxRowExperts) return -1;
    return moe::permute_most_workspace_bytes((int64_t)T * topk, E);
}

moe_status moe_permute(const void* x, int64_t x_stride, moe_dtype type, const int32_t* topk_ids, int T, int topk, int E,
                       int H, void* out, int64_t out_stride, int32_t* rows, int32_t* expert_offsets, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const char* fn = "moe_permute";
    CHECK(check_rows(fn, T, topk, H));
    if (E < 1) return fail(MOE_ERR_INVALID_ARG, "%s: E=%d < 1", fn, E);
    if (E > kMaxRowExperts) return fail(MOE_ERR_UNSUPPORTED, "%s: E=%d > %d", fn, E, kMaxRowExperts);
    const int size = size_of(type);
    if (!size) return fail(MOE_ERR_UNSUPPORTED, "%s: type %d unknown", fn, (int)type);
    CHECK(check_stride(fn, "x_stride", x_stride, H, 1));
    CHECK(check_stride(fn, "out_stride", out_stride, H, 1));
    if (!expert_offsets || !aligned(expert_offsets, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: null or misaligned expert_offsets", fn);
    if (T > 0) {
        if (!x || !topk_ids || !out || !rows) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
        if (!aligned(x, size) || !aligned(out, size) || !aligned(topk_ids, 4) || !aligned(rows, 4))
            return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
        CHECK(check_workspace(fn, workspace, workspace_bytes, moe::permute_workspace_bytes((int64_t)T * topk, E)));
    }
    moe::PermuteArgs a;
    a.x = x;
    a.out = out;
    a.ids = topk_ids;
    a.rows = rows;
    a.offsets = expert_offsets;
    a.counts = (int32_t*)workspace;
    a.ldx = x_stride * size;
    a.ldo = out_stride * size;
    a.row_bytes = (int64_t)H * size;
    a.T = T;
    a.topk = topk;
    a.E = E;
    return hip_status(moe::launch_permute(a, (hipStream_t)stream), fn);
}

moe_status moe_unpermute(const void* y, int64_t y_stride, moe_dtype y_type, const int32_t* rows, const float* weights,
                         const void* residual, int64_t residual_stride, int T, int topk, int H, void* out,
                         int64_t out_stride, moe_dtype out_type, void* stream) {
    const char* fn = "moe_unpermute";
    CHECK(check_rows(fn, T, topk, H));
    CHECK(check_float(fn, y_type));
    CHECK(check_float(fn, out_type));
    CHECK(check_stride(fn, "y_stride", y_stride, H, 1));
    if (residual) CHECK(check_stride(fn, "residual_stride", residual_stride, H, 1));
    CHECK(check_stride(fn, "out_stride", out_stride, H, 1));
    if (T == 0) return MOE_OK;
    if (!y || !rows || !out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(y, size_of(y_type)) || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(residual, size_of(out_type)) ||
        !aligned(out, size_of(out_type)))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    moe::UnpermuteArgs a;
    a.y = y;
    a.rows = rows;
    a.weights = weights;
    a.residual = residual;
    a.out = out;
    a.ldy = y_stride;
    a.ldr = residual_stride;
    a.ldo = out_stride;
    a.pairs = (int64_t)T * topk;
    a.T = T;
    a.topk = topk;
    a.H = H;
    a.y_f32 = y_type == MOE_DT_F32;
    a.out_f32 = out_type == MOE_DT_F32;
    return hip_status(moe::launch_unpermute(a, (hipStream_t)stream), fn);
}

moe_status moe_unpermute_backward(const void* dout, int64_t dout_stride, moe_dtype out_type, const int32_t* rows,
                                  const float* weights, const void* y, int64_t y_stride, moe_dtype y_type, int T, int topk,
                                  int H, void* dy, int64_t dy_stride, float* dweights, void* stream) {
    const char* fn = "moe_unpermute_backward";
    CHECK(check_rows(fn, T, topk, H));
    CHECK(check_float(fn, y_type));
    CHECK(check_float(fn, out_type));
    CHECK(check_stride(fn, "dout_stride", dout_stride, H, 1));
    if (dweights) CHECK(check_stride(fn, "y_stride", y_stride, H, 1));
    if (dy) CHECK(check_stride(fn, "dy_stride", dy_stride, H, 1));
    if (T == 0) return MOE_OK;
    if (!dy && !dweights) return fail(MOE_ERR_INVALID_ARG, "%s: no output", fn);
    if (!dout || !rows || (dweights && !y)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(dout, size_of(out_type)) || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(y, size_of(y_type)) ||
        !aligned(dy, size_of(y_type)) || !aligned(dweights, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    moe::UnpermuteBwdArgs a;
    a.dout = dout;
    a.rows = rows;
    a.weights = weights;
    a.y = y;
    a.dy = dy;
    a.dweights = dweights;
    a.lddo = dout_stride;
    a.ldy = y_stride;
    a.lddy = dy_stride;
    a.T = T;
    a.topk = topk;
    a.H = H;
    a.y_f32 = y_type == MOE_DT_F32;
    a.out_f32 = out_type == MOE_DT_F32;
    return hip_status(moe::launch_unpermute_bwd(a, (hipStream_t)stream), fn);
}

}  // extern "C"
