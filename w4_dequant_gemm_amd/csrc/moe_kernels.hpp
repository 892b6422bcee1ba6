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
    float* logits;           // [splits, T, E] workspace: partial logits of the K ranges
    int splits;
};
// one kernel makes the logits and chooses (no workspace)
constexpr bool route_in_one(int E, int H) { return E <= 16 && H <= 1024; }
// K ranges that the logits of these sizes are split into
int route_splits(int64_t T, int E, int H);
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
    uint16_t* hi;            // [T k, I] rows of act(gate) up weight by slot t k + j, upper and lower part
    uint16_t* lo;            // (tiled: rounded to bf16 in `hi`, in the order of `order`)
    int4* runs;              // [E] expert, first place in `order`, rows
    int32_t* order;          // [T k] slots by expert
    float* part;             // [splits, T k, H] each slot's share of the result, by ranges of the inner k
    int splits;
    // tiled products
    int4* tiles;             // expert, first place in `order`, rows
    int32_t* tile_count;
    float* x_sums;           // [T, H / G] row sums of X
    float* h_sums;           // [T k, I / G] of h, in the order of `order`
};
// bytes of the workspace, and the pointers into it
size_t moe_workspace(MoeParams& p, void* base);
hipError_t launch_moe(const MoeParams& p, hipStream_t stream);

// the tiled products (moe_tile.hip): rows of a tile, the most row sums of one
// (they lie in LDS), and the launch for at most `tiles` tiles
constexpr int kMoeTileRows = 64;
constexpr int kMoeTileSums = 16384;
hipError_t launch_moe_tile(const MoeParams& p, bool up, int64_t tiles, hipStream_t stream);

}  // namespace w4
