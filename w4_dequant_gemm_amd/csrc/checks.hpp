// Argument checks shared by the host-side sources of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4.h"
#include "status.hpp"

namespace w4 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return W4_OK;
    return fail(W4_EHIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace w4

#define W4_REQUIRE_PTR(fn, p)                                                        \
    do {                                                                             \
        if (!(p)) return w4::fail(W4_EINVAL, "%s: %s is NULL", fn, #p);                  \
        if (!w4::aligned16(p)) return w4::fail(W4_EINVAL, "%s: %s is not 16-byte aligned", fn, #p); \
    } while (0)
