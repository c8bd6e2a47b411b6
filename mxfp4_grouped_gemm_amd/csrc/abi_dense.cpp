// C ABI of the dense operators: argument checks, workspace layout and the
// sequence of launches. As in abi.cpp, every check runs before anything is
// enqueued.
#include <cmath>
#include <cstring>

#include "abi_common.hpp"
#include "dense.hpp"

using moe::abi::align_up;
using moe::abi::aligned;
using moe::abi::fail;
using moe::abi::hip_status;

namespace {

// Tile addressing: a tile's rows (at most 256, or 64 rows of K) lie within
// 32-bit byte offsets of its first element.
constexpr int64_t kMaxCols = 1 << 18;
constexpr int64_t kMaxStride = 1 << 20;
constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxRank = 256;
constexpr int kMaxAdapters = 1 << 24;  // `ranks` has 32-bit offsets
// Weights that the few-token kernels address with 32-bit offsets.
constexpr int64_t kMaxSkinnyBytes = 0x7fff0000LL;

moe_status check_size(const char* fn, const char* name, int v, int step) {
    if (v < step || v % step != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s=%d must be a positive multiple of %d", fn, name, v, step);
    if (v > kMaxCols) return fail(MOE_ERR_UNSUPPORTED, "%s: %s=%d > %lld", fn, name, v, (long long)kMaxCols);
    return MOE_OK;
}

moe_status check_tokens(const char* fn, int T) {
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%d < 0", fn, T);
    if (T > kMaxTokens) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d > %d", fn, T, kMaxTokens);
    return MOE_OK;
}

moe_status check_stride(const char* fn, const char* name, int64_t stride, int64_t cols, int step) {
    if (stride < cols || stride % step != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s=%lld must be at least %lld and a multiple of %d", fn, name,
                    (long long)stride, (long long)cols, step);
    if (stride > kMaxStride)
        return fail(MOE_ERR_UNSUPPORTED, "%s: %s=%lld > %lld", fn, name, (long long)stride, (long long)kMaxStride);
    return MOE_OK;
}

template <int N>
moe_status check_pointers(const char* fn, const void* const (&ptrs)[N], size_t align) {
    for (const void* p : ptrs)
        if (!p) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : ptrs)
        if (!aligned(p, align)) return fail(MOE_ERR_INVALID_ARG, "%s: pointer %p not %zu-byte aligned", fn, p, align);
    return MOE_OK;
}

moe_status check_workspace(const char* fn, const void* ws, size_t have, int64_t need) {
    if (need == 0) return MOE_OK;
    if (!ws) return fail(MOE_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "%s: workspace not 256-byte aligned", fn);
    if ((int64_t)have < need)
        return fail(MOE_ERR_INVALID_ARG, "%s: workspace %zu bytes < %lld needed", fn, have, (long long)need);
    return MOE_OK;
}

// T > 0: pointers are looked at.
moe_status check_lora(const char* fn, const char* name, const moe_lora* l, int T) {
    if (!l) return MOE_OK;
    if (l->n < 1) return fail(MOE_ERR_INVALID_ARG, "%s: %s has n=%d < 1", fn, name, l->n);
    if (l->n > kMaxAdapters) return fail(MOE_ERR_UNSUPPORTED, "%s: %s has n=%d > %d", fn, name, l->n, kMaxAdapters);
    if (l->rank < 8 || l->rank % 8 != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s has rank=%d, not a positive multiple of 8", fn, name, l->rank);
    if (l->rank > kMaxRank) return fail(MOE_ERR_UNSUPPORTED, "%s: %s has rank=%d > %d", fn, name, l->rank, kMaxRank);
    if (T == 0) return MOE_OK;
    if (!l->a || !l->b || !l->index) return fail(MOE_ERR_INVALID_ARG, "%s: %s has a null pointer", fn, name);
    if (!aligned(l->a, 16) || !aligned(l->b, 16) || !aligned(l->index, 4) || !aligned(l->ranks, 4) ||
        !aligned(l->scale, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: %s has a misaligned pointer", fn, name);
    return MOE_OK;
}

#define CHECK(call)                                    \
    do {                                               \
        const moe_status st_ = (call);                 \
        if (st_ != MOE_OK) return st_;                 \
    } while (0)
#define LAUNCH(call, what)                             \
    do {                                               \
        const hipError_t e_ = (call);                  \
        if (e_ != hipSuccess) return hip_status(e_, what); \
    } while (0)

int vld_of(int rank) { return (int)align_up(rank, 32); }

// What adapters keep in the workspace: the tokens' order with its adapters (for
// any number of adapters), and v.
int64_t order_bytes(int T) { return moe::lora_sorts(T, 3) ? 2 * align_up((int64_t)T * 4, 256) : 0; }
int64_t lora_bytes(int T, int rank) {
    return rank > 0 ? order_bytes(T) + align_up((int64_t)moe::lora_parts(T) * T * vld_of(rank) * 4, 256) : 0;
}

// joined: the product's parts are joined token by token, else its tiles read v.
moe::LoraArgs lora_args(const moe_lora* l, void* ws, int T, int64_t ldx, bool joined) {
    moe::LoraArgs r;
    memset(&r, 0, sizeof r);
    if (!l) return r;
    // Rows in an order are loaded by 32-bit offsets from the first.
    if (moe::lora_sorts(T, l->n) && T * ldx * 2 < (int64_t)1 << 30) {
        r.order = (int32_t*)ws;
        r.sorted = (int32_t*)((char*)ws + order_bytes(T) / 2);
        r.v_sorted = !joined;
    }
    r.a = l->a;
    r.b = l->b;
    r.index = l->index;
    r.ranks = l->ranks;
    r.scale = l->scale;
    r.n = l->n;
    r.rank = l->rank;
    r.vld = vld_of(l->rank);
    r.v = (float*)((char*)ws + order_bytes(T));
    r.parts = moe::lora_parts(T);
    r.part_stride = (int64_t)T * r.vld;
    return r;
}

moe::DenseArgs product(const void* x, int64_t ldx, const void* w, int64_t ldw, int M, int N, int K, void* out,
                       int64_t ldo) {
    moe::DenseArgs a;
    memset(&a, 0, sizeof a);
    a.x = x;
    a.ldx = ldx;
    a.w = w;
    a.ldw = ldw;
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = out;
    a.ldo = ldo;
    a.splits = 1;
    return a;
}

bool skinny(int T, int64_t rows, int K, int elt) {
    const bool many = rows >= (elt == 0 ? moe::kSkinnyManyRows : moe::kSkinnyManyRowsMx);
    const int most = many ? 16 : elt == 0 ? moe::kSkinnyMaxTokens : moe::kSkinnyMaxTokensMx;
    return T <= most && rows * K * (elt == 0 ? 2 : 1) <= kMaxSkinnyBytes;
}

int splits_of(const moe::DenseArgs& a, int elt, int epi, bool few) {
    return few ? moe::skinny_splits(a, elt, epi) : moe::dense_splits(a, elt, epi);
}

// Bytes of split-K partials of a forward product; few: in the few-token
// kernels.
int64_t partial_bytes(int T, int N, int K, int elt, int epi, bool few, int rank) {
    moe::DenseArgs a = product(nullptr, K, nullptr, K, T, N, K, nullptr, N);
    a.lora.n = rank > 0;
    a.lora.rank = rank;
    const int splits = splits_of(a, elt, epi, few);
    return align_up(moe::dense_partial_bytes(a, splits, epi, few && moe::skinny_joins(a, splits, elt, epi)), 256);
}

// The narrow product; sorted: the order is there already (of the same index).
hipError_t run_shrink(const uint16_t* x, int64_t ldx, int T, int K, const moe::LoraArgs& l, bool sorted, hipStream_t s) {
    if (l.order && !sorted) {
        const hipError_t e = moe::launch_lora_sort(l.index, T, l.n, (int32_t*)l.order, (int32_t*)l.sorted, s);
        if (e != hipSuccess) return e;
    }
    return moe::launch_lora_shrink(x, ldx, T, K, l, s);
}

// A forward product. h_f32: see launch_skinny.
hipError_t run_product(moe::DenseArgs& a, int elt, int epi, bool few, float* partial, const float* h_f32, hipStream_t s) {
    a.splits = splits_of(a, elt, epi, few);
    a.partial = partial;
    return few ? moe::launch_skinny(a, elt, epi, h_f32, s) : moe::launch_dense(a, elt, epi, s);
}

struct FfnLayout {
    int64_t h, hs, v, partial, total;
};

FfnLayout ffn_layout(int T, int H, int I, int rank13, int rank2) {
    FfnLayout L;
    const int64_t p1 = partial_bytes(T, I, H, 0, moe::kEpiGated, skinny(T, 2 * (int64_t)I, H, 0), rank13);
    const int64_t p2 = partial_bytes(T, H, I, 0, moe::kEpiOut, skinny(T, H, I, 0), rank2);
    L.h = 0;
    L.hs = 0;
    L.v = align_up((int64_t)T * I * 2, 256);
    L.partial = L.v + lora_bytes(T, rank13 > rank2 ? rank13 : rank2);
    L.total = L.partial + (p1 > p2 ? p1 : p2);
    return L;
}

bool mx_skinny(int T, int H, int I) { return skinny(T, 2 * (int64_t)I, H, 1) && skinny(T, H, I, 1); }

FfnLayout ffn_mx_layout(int T, int H, int I) {
    FfnLayout L;
    const bool few = mx_skinny(T, H, I);
    const int64_t p1 = partial_bytes(T, I, H, 1, moe::kEpiGatedMx, few, 0), p2 = partial_bytes(T, H, I, 1, moe::kEpiOut, few, 0);
    L.h = 0;
    L.v = 0;
    // h: fp32 for the few-token kernels, else codes and scales.
    L.hs = align_up((int64_t)T * I * (few ? 4 : 1), 256);
    L.partial = L.hs + (few ? 0 : align_up((int64_t)T * (I / 32), 256));
    L.total = L.partial + (p1 > p2 ? p1 : p2);
    return L;
}

struct BwdLayout {
    int64_t h, partial, total;  // dgate_up at 0
    int splits_dh, splits_dx;
};

BwdLayout bwd_layout(int T, int H, int I) {
    BwdLayout L;
    const moe::DenseArgs dh = product(nullptr, H, nullptr, I, T, I, H, nullptr, I);
    const moe::DenseArgs dx = product(nullptr, 2 * (int64_t)I, nullptr, H, T, H, 2 * I, nullptr, H);
    L.splits_dh = moe::dense_bwd_splits(dh);
    L.splits_dx = moe::dense_bwd_splits(dx);
    const int64_t p1 = moe::dense_partial_bytes(dh, L.splits_dh, moe::kEpiGatedBwd, false);
    const int64_t p2 = moe::dense_partial_bytes(dx, L.splits_dx, moe::kEpiOut, false);
    L.h = align_up((int64_t)T * 2 * I * 2, 256);
    L.partial = L.h + align_up((int64_t)T * I * 2, 256);
    L.total = L.partial + align_up(p1 > p2 ? p1 : p2, 256);
    return L;
}

moe_status check_act(const char* fn, moe_act act) {
    if (act != MOE_ACT_SWIGLU)
        return fail(MOE_ERR_UNSUPPORTED,
                    "%s: activation %d is not implemented (only SwiGLU); refusing to compute a different activation",
                    fn, (int)act);
    return MOE_OK;
}

bool valid_sizes(int T, int a, int b, int step) {
    auto ok = [&](int v) { return v >= step && v % step == 0 && v <= kMaxCols; };
    return T >= 0 && T <= kMaxTokens && ok(a) && ok(b);
}

bool valid_rank(int r) { return r >= 0 && r % 8 == 0 && r <= kMaxRank; }

}  // namespace

extern "C" {

moe_status moe_rms_norm(const uint16_t* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        moe_dtype residual_type, const void* weight, moe_dtype weight_type, float eps,
                        float weight_offset, int T, int H, void* residual_out, int64_t residual_out_stride,
                        uint16_t* y, int64_t y_stride, uint8_t* q, int64_t q_stride, uint8_t* q_scale,
                        int64_t q_scale_stride, void* stream) {
    const char* fn = "moe_rms_norm";
    CHECK(check_tokens(fn, T));
    if (H < 1) return fail(MOE_ERR_INVALID_ARG, "%s: H=%d < 1", fn, H);
    if (H > 65536) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d > 65536", fn, H);
    if ((residual_type != MOE_DT_BF16 && residual_type != MOE_DT_F32) ||
        (weight_type != MOE_DT_BF16 && weight_type != MOE_DT_F32))
        return fail(MOE_ERR_UNSUPPORTED, "%s: type %d / %d unknown", fn, (int)residual_type, (int)weight_type);
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(MOE_ERR_INVALID_ARG, "%s: eps %g must be >= 0 and finite", fn, (double)eps);
    if ((q == nullptr) != (q_scale == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "%s: q and q_scale go together", fn);
    if (q && H % 32 != 0) return fail(MOE_ERR_INVALID_ARG, "%s: H=%d must be a multiple of 32 for the MXFP8 output", fn, H);
    CHECK(check_stride(fn, "x_stride", x_stride, H, 1));
    if (residual) CHECK(check_stride(fn, "residual_stride", residual_stride, H, 1));
    if (residual_out) CHECK(check_stride(fn, "residual_out_stride", residual_out_stride, H, 1));
    if (y) CHECK(check_stride(fn, "y_stride", y_stride, H, 1));
    if (q) {
        CHECK(check_stride(fn, "q_stride", q_stride, H, 1));
        CHECK(check_stride(fn, "q_scale_stride", q_scale_stride, H / 32, 1));
    }
    if (T == 0) return MOE_OK;
    if (!y && !q && !residual_out) return fail(MOE_ERR_INVALID_ARG, "%s: no output", fn);
    if (!x || !weight) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t ra = residual_type == MOE_DT_F32 ? 4 : 2, wa = weight_type == MOE_DT_F32 ? 4 : 2;
    if (!aligned(x, 2) || !aligned(y, 2) || !aligned(residual, ra) || !aligned(residual_out, ra) || !aligned(weight, wa))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    moe::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.residual_out = residual_out;
    a.y = y;
    a.q = q;
    a.qs = q_scale;
    a.ldx = x_stride;
    a.ldr = residual_stride;
    a.ldro = residual_out_stride;
    a.ldy = y_stride;
    a.ldq = q_stride;
    a.ldqs = q_scale_stride;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.offset = weight_offset;
    a.res_f32 = residual_type == MOE_DT_F32;
    a.weight_f32 = weight_type == MOE_DT_F32;
    return hip_status(moe::launch_rms_norm(a, (hipStream_t)stream), fn);
}

int64_t moe_lora_linear_workspace_size(int T, int K, int N, int rank) {
    if (!valid_sizes(T, K, N, 8) || !valid_rank(rank)) return -1;
    return lora_bytes(T, rank) + partial_bytes(T, N, K, 0, moe::kEpiOut, skinny(T, N, K, 0), rank);
}

moe_status moe_lora_linear(const uint16_t* x, int64_t x_stride, const uint16_t* w, const moe_lora* lora, int T, int K,
                           int N, void* out, int64_t out_stride, moe_dtype out_type, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const char* fn = "moe_lora_linear";
    CHECK(check_tokens(fn, T));
    CHECK(check_size(fn, "K", K, 8));
    CHECK(check_size(fn, "N", N, 8));
    CHECK(check_stride(fn, "x_stride", x_stride, K, 8));
    CHECK(check_stride(fn, "out_stride", out_stride, N, 8));
    if (out_type != MOE_DT_BF16 && out_type != MOE_DT_F32)
        return fail(MOE_ERR_UNSUPPORTED, "%s: out_type %d unknown", fn, (int)out_type);
    CHECK(check_lora(fn, "lora", lora, T));
    if (T == 0) return MOE_OK;
    const void* ptrs[] = {x, w, out};
    CHECK(check_pointers(fn, ptrs, 16));
    CHECK(check_workspace(fn, workspace, workspace_bytes, moe_lora_linear_workspace_size(T, K, N, lora ? lora->rank : 0)));
    hipStream_t s = (hipStream_t)stream;
    moe::DenseArgs a = product(x, x_stride, w, K, T, N, K, out, out_stride);
    a.out_f32 = out_type == MOE_DT_F32;
    const bool few = skinny(T, N, K, 0);
    a.lora = lora_args(lora, workspace, T, x_stride, splits_of(a, 0, moe::kEpiOut, few) > 1);
    float* partial = (float*)((char*)workspace + lora_bytes(T, lora ? lora->rank : 0));
    if (lora && !few) LAUNCH(run_shrink(x, x_stride, T, K, a.lora, false, s), "moe_lora_linear (shrink)");
    return hip_status(run_product(a, 0, moe::kEpiOut, few, partial, nullptr, s), fn);
}

int64_t moe_ffn_workspace_size(int T, int H, int I, int rank13, int rank2) {
    if (!valid_sizes(T, H, I, 8) || !valid_rank(rank13) || !valid_rank(rank2)) return -1;
    return ffn_layout(T, H, I, rank13, rank2).total;
}

moe_status moe_ffn_forward(const uint16_t* x, int64_t x_stride, const uint16_t* w13, const uint16_t* w2, moe_act act,
                           const uint16_t* addend, int64_t addend_stride, const moe_lora* lora13,
                           const moe_lora* lora2, int T, int H, int I, uint16_t* out, int64_t out_stride,
                           uint16_t* gate_up, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "moe_ffn_forward";
    CHECK(check_act(fn, act));
    CHECK(check_tokens(fn, T));
    CHECK(check_size(fn, "H", H, 8));
    CHECK(check_size(fn, "I", I, 8));
    CHECK(check_stride(fn, "x_stride", x_stride, H, 8));
    CHECK(check_stride(fn, "out_stride", out_stride, H, 8));
    if (addend) CHECK(check_stride(fn, "addend_stride", addend_stride, H, 8));
    CHECK(check_lora(fn, "lora13", lora13, T));
    CHECK(check_lora(fn, "lora2", lora2, T));
    if (T == 0) return MOE_OK;
    const void* ptrs[] = {x, w13, w2, out};
    CHECK(check_pointers(fn, ptrs, 16));
    if (!aligned(addend, 16) || !aligned(gate_up, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: addend and gate_up must be 16-byte aligned", fn);
    const FfnLayout L = ffn_layout(T, H, I, lora13 ? lora13->rank : 0, lora2 ? lora2->rank : 0);
    CHECK(check_workspace(fn, workspace, workspace_bytes, L.total));
    hipStream_t s = (hipStream_t)stream;
    char* ws = (char*)workspace;
    uint16_t* h = (uint16_t*)(ws + L.h);
    moe::DenseArgs a = product(x, x_stride, w13, H, T, I, H, h, I);
    a.gate_up = gate_up;
    const bool few13 = skinny(T, 2 * (int64_t)I, H, 0), few2 = skinny(T, H, I, 0);
    a.lora = lora_args(lora13, ws + L.v, T, x_stride, splits_of(a, 0, moe::kEpiGated, few13) > 1);
    if (lora13 && !few13) LAUNCH(run_shrink(x, x_stride, T, H, a.lora, false, s), "moe_ffn_forward (gate_up shrink)");
    const bool sorted = lora2 && !few13 && a.lora.order && lora2->index == lora13->index && lora2->n == lora13->n;
    LAUNCH(run_product(a, 0, moe::kEpiGated, few13, (float*)(ws + L.partial), nullptr, s), "moe_ffn_forward (gate_up)");
    a = product(h, I, w2, I, T, H, I, out, out_stride);
    a.addend = addend;
    a.ldadd = addend_stride;
    a.lora = lora_args(lora2, ws + L.v, T, I, splits_of(a, 0, moe::kEpiOut, few2) > 1);
    if (lora2 && !few2) LAUNCH(run_shrink(h, I, T, I, a.lora, sorted, s), "moe_ffn_forward (down shrink)");
    return hip_status(run_product(a, 0, moe::kEpiOut, few2, (float*)(ws + L.partial), nullptr, s), "moe_ffn_forward (down)");
}

int64_t moe_ffn_mxfp8_workspace_size(int T, int H, int I) {
    if (!valid_sizes(T, H, I, 32)) return -1;
    return ffn_mx_layout(T, H, I).total;
}

moe_status moe_ffn_forward_mxfp8(const uint8_t* x, const uint8_t* x_scale, const uint8_t* w13,
                                 const uint8_t* w13_scale, const uint8_t* w2, const uint8_t* w2_scale, moe_act act,
                                 const uint16_t* addend, int64_t addend_stride, int T, int H, int I, uint16_t* out,
                                 int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "moe_ffn_forward_mxfp8";
    CHECK(check_act(fn, act));
    CHECK(check_tokens(fn, T));
    CHECK(check_size(fn, "H", H, 32));
    CHECK(check_size(fn, "I", I, 32));
    CHECK(check_stride(fn, "out_stride", out_stride, H, 8));
    if (addend) CHECK(check_stride(fn, "addend_stride", addend_stride, H, 8));
    if (T == 0) return MOE_OK;
    const void* ptrs[] = {x, x_scale, w13, w13_scale, w2, w2_scale, out};
    CHECK(check_pointers(fn, ptrs, 16));
    if (!aligned(addend, 16)) return fail(MOE_ERR_INVALID_ARG, "%s: addend must be 16-byte aligned", fn);
    const FfnLayout L = ffn_mx_layout(T, H, I);
    CHECK(check_workspace(fn, workspace, workspace_bytes, L.total));
    hipStream_t s = (hipStream_t)stream;
    char* ws = (char*)workspace;
    moe::DenseArgs a1 = product(x, H, w13, H, T, I, H, ws + L.h, I);
    a1.xs = x_scale;
    a1.ws = w13_scale;
    moe::DenseArgs a2 = product(ws + L.h, I, w2, I, T, H, I, out, out_stride);
    a2.ws = w2_scale;
    a2.addend = addend;
    a2.ldadd = addend_stride;
    float* partial = (float*)(ws + L.partial);
    const bool few = mx_skinny(T, H, I);
    if (few) {
        a1.out_f32 = 1;
    } else {
        a1.hs = (uint8_t*)(ws + L.hs);
        a2.xs = (const uint8_t*)(ws + L.hs);
    }
    LAUNCH(run_product(a1, 1, few ? moe::kEpiGated : moe::kEpiGatedMx, few, partial, nullptr, s), "moe_ffn_forward_mxfp8 (gate_up)");
    return hip_status(run_product(a2, 1, moe::kEpiOut, few, partial, few ? (const float*)(ws + L.h) : nullptr, s),
                      "moe_ffn_forward_mxfp8 (down)");
}

int64_t moe_ffn_backward_workspace_size(int T, int H, int I) {
    if (!valid_sizes(T, H, I, 8)) return -1;
    return bwd_layout(T, H, I).total;
}

moe_status moe_ffn_backward(const uint16_t* dout, int64_t dout_stride, const uint16_t* x, int64_t x_stride,
                            const uint16_t* gate_up, const uint16_t* w13, const uint16_t* w2, moe_act act, int T,
                            int H, int I, uint16_t* dx, int64_t dx_stride, uint16_t* dw13, uint16_t* dw2,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "moe_ffn_backward";
    CHECK(check_act(fn, act));
    CHECK(check_tokens(fn, T));
    CHECK(check_size(fn, "H", H, 8));
    CHECK(check_size(fn, "I", I, 8));
    CHECK(check_stride(fn, "dout_stride", dout_stride, H, 8));
    CHECK(check_stride(fn, "x_stride", x_stride, H, 8));
    if (dx) CHECK(check_stride(fn, "dx_stride", dx_stride, H, 8));
    // (An empty dx may have no address.)
    if (!dx && !dw13 && !dw2)
        return T == 0 ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "%s: no output", fn);
    if (!aligned(dx, 16) || !aligned(dw13, 16) || !aligned(dw2, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", fn);
    hipStream_t s = (hipStream_t)stream;
    uint16_t* dgu = nullptr;
    uint16_t* h = nullptr;
    const BwdLayout L = bwd_layout(T, H, I);
    float* partial = (float*)((char*)workspace + L.partial);
    if (T > 0) {
        const void* ptrs[] = {dout, x, gate_up, w13, w2};
        CHECK(check_pointers(fn, ptrs, 16));
        CHECK(check_workspace(fn, workspace, workspace_bytes, L.total));
        dgu = (uint16_t*)workspace;
        h = (uint16_t*)((char*)workspace + L.h);
        moe::DenseArgs a = product(dout, dout_stride, w2, I, T, I, H, dgu, 2 * (int64_t)I);
        a.gate_up = const_cast<uint16_t*>(gate_up);
        a.h = dw2 ? h : nullptr;
        a.splits = L.splits_dh;
        a.partial = partial;
        LAUNCH(moe::launch_dense_dh(a, s), "moe_ffn_backward (dh)");
    }
    // With T == 0 the weights' sums are empty and write zeros.
    const moe::DenseArgs g13 = product(dgu, 2 * (int64_t)I, x, x_stride, 2 * I, H, T, dw13, H);
    const moe::DenseArgs g2 = product(dout, dout_stride, h, I, H, I, T, dw2, I);
    moe::DenseArgs gx = product(dgu, 2 * (int64_t)I, w13, H, T, H, 2 * I, dx, dx_stride);
    gx.splits = L.splits_dx;
    gx.partial = partial;
    return hip_status(moe::launch_dense_grads(g13, g2, gx, s), "moe_ffn_backward (gradients)");
}

}  // extern "C"
