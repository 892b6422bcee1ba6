// Argument checks shared by the host-side sources of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4.h"
#include "status.hpp"

namespace w4 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An array of rows x cols elements of `size` bytes (sizes that pass 64 bits: as many as there are)
struct Span {
    const void* p;
    uint64_t bytes;
    const char* name;
};
inline Span span(const void* p, int64_t rows, int64_t cols, int64_t size, const char* name) {
    int64_t n = 0;
    const bool fits = !__builtin_mul_overflow(rows, cols, &n) && !__builtin_mul_overflow(n, size, &n);
    return {p, p ? (fits ? static_cast<uint64_t>(n) : UINT64_MAX) : 0, name};
}
inline bool overlap(const Span& a, const Span& b) {
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x <= y ? y - x < a.bytes : x - y < b.bytes;
}
// Workgroups write `out` while others still read `in`: no byte of the one may be one of the other's.
inline int check_apart(const char* fn, const Span& out, const Span& in) {
    if (!overlap(out, in)) return W4_OK;
    if (out.p == in.p) return fail(W4_EINVAL, "%s: %s must not be %s", fn, out.name, in.name);
    return fail(W4_EINVAL, "%s: %s overlaps %s", fn, out.name, in.name);
}

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
