// Whether the rows of two matrices share memory (host code alone).
#pragma once

#include <stdint.h>

namespace moe {
namespace abi {

// n rows of lp bytes from p, sp bytes apart (sp >= lp), and n of lq from q.
inline bool rows_overlap(int64_t p, int64_t sp, int64_t lp, int64_t q, int64_t sq, int64_t lq, int n) {
    if (n < 1 || p >= q + (n - 1) * sq + lq || q >= p + (n - 1) * sp + lp) return false;
    auto meet = [&](int64_t i, int64_t j) { return p + i * sp < q + j * sq + lq && q + j * sq < p + i * sp + lp; };
    if (sp == sq) {
        // Rows i and i + k are as far apart for every i: the two k nearest.
        const int64_t d = p - q, k = d >= 0 ? d / sp : -((-d + sp - 1) / sp);  // (rounded down)
        for (int64_t at = k; at <= k + 1; ++at)
            if (at > -n && at < n && (at >= 0 ? meet(0, at) : meet(-at, 0))) return true;
        return false;
    }
    // Both in order of address: of a pair that does not meet the lower one has no
    // later partner.
    for (int64_t i = 0, j = 0; i < n && j < n;) {
        if (meet(i, j)) return true;
        if (p + i * sp < q + j * sq) ++i;
        else ++j;
    }
    return false;
}

}  // namespace abi
}  // namespace moe
