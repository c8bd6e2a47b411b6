// Error reporting and checks shared by the files of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_a16w4.h"

namespace moe {
namespace abi {

// Records the message moe_last_error() returns on this thread; returns st.
moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status hip_status(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

}  // namespace abi
}  // namespace moe
