// Argument checks shared by the dense operators and the row movers.
#pragma once

#include "abi_common.hpp"

namespace moe {
namespace abi {

constexpr int64_t kMaxStride = 1 << 20;
constexpr int kMaxTokens = 1 << 24;

inline moe_status check_tokens(const char* fn, int T) {
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%d < 0", fn, T);
    if (T > kMaxTokens) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d > %d", fn, T, kMaxTokens);
    return MOE_OK;
}

inline moe_status check_stride(const char* fn, const char* name, int64_t stride, int64_t cols, int step) {
    if (stride < cols || stride % step != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s=%lld must be at least %lld and a multiple of %d", fn, name,
                    (long long)stride, (long long)cols, step);
    if (stride > kMaxStride)
        return fail(MOE_ERR_UNSUPPORTED, "%s: %s=%lld > %lld", fn, name, (long long)stride, (long long)kMaxStride);
    return MOE_OK;
}

template <int N>
inline moe_status check_pointers(const char* fn, const void* const (&ptrs)[N], size_t align) {
    for (const void* p : ptrs)
        if (!p) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : ptrs)
        if (!aligned(p, align)) return fail(MOE_ERR_INVALID_ARG, "%s: pointer %p not %zu-byte aligned", fn, p, align);
    return MOE_OK;
}

inline moe_status check_workspace(const char* fn, const void* ws, size_t have, int64_t need) {
    if (need == 0) return MOE_OK;
    if (!ws) return fail(MOE_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "%s: workspace not 256-byte aligned", fn);
    if ((int64_t)have < need)
        return fail(MOE_ERR_INVALID_ARG, "%s: workspace %zu bytes < %lld needed", fn, have, (long long)need);
    return MOE_OK;
}

}  // namespace abi
}  // namespace moe

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
