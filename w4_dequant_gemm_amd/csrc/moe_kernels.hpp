// Parameters and launchers of the mixture-of-experts kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace w4 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

struct RouteParams {
    const uint16_t* X;       // [T, H] bf16
    int64_t T;
    int H;
    const uint16_t* router;  // [E, H] bf16
    int E, k;
    bool sigmoid;            // scores: sigmoid, else softmax over the experts
    const float* bias;       // [E] or null: added to the scores to choose, not to weigh
    bool renormalize;
    float scale;
    int32_t* ids;            // [T, k]
    float* weights;          // [T, k]
    float* logits;           // [T, E] workspace
};
hipError_t launch_route(const RouteParams& p, hipStream_t stream);

struct MoeWeight {
    const uint32_t* wq;      // [E, N, K/8]: the GPU layout of each expert, one after the other
    const uint32_t* sz;      // [E, N, K/G]
};
struct MoeParams {
    const uint16_t* X;       // [T, H] bf16
    int64_t T;
    int k, E, H, I, G;
    const int32_t* ids;      // [T, k]; outside 0..E-1: no expert
    const float* weights;    // [T, k]
    MoeWeight gate, up, down;
    int act;
    const uint16_t* residual;   // [T, H] or null
    uint16_t* Y;             // [T, H]
    // workspace, see moe_workspace
    int32_t* offset;         // [E + 1] first place of each expert's rows in `order`
    int32_t* active;         // [E] experts with rows, then at [E] their number
    int32_t* order;          // [T k] slots (t k + j) by expert
    uint16_t* hi;            // [T k, I] rows of act(gate) up weight, upper and lower part
    uint16_t* lo;
    float* part;             // [T k, H] each slot's share of the result
};
// bytes of the workspace, and the pointers into it
size_t moe_workspace(MoeParams& p, void* base);
hipError_t launch_moe(const MoeParams& p, hipStream_t stream);

}  // namespace w4
