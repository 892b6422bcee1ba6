// How large a launch may be.
#pragma once

#include <cstdint>

namespace w4 {

// A dispatch counts its threads along x in 32 bits, and the runtime starts what
// is left of a larger number, without an error: such launches are refused, or go
// in pieces.
inline bool launch_fits(int64_t workgroups, int threads) { return workgroups <= 0xFFFFFFFFLL / threads; }

}  // namespace w4
