// C ABI of the mixture-of-experts calls: argument checks, then the launches on
// the caller's stream.  As for the products: no allocation, no state, nothing
// launched on a refused argument.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.hpp"
#include "moe_kernels.hpp"

namespace {
using w4::aligned16;
using w4::fail;
using w4::hip_status;

long long ll(int64_t v) { return static_cast<long long>(v); }

constexpr int64_t kMaxTokens = 1000000;
constexpr int64_t kMaxWidth = 65536;      // hidden and inner sizes

int check_sizes(const char* fn, int64_t T, int64_t E, int top_k) {
    if (T < 0 || T > kMaxTokens) return fail(W4_EINVAL, "%s: T = %lld outside 0..%lld", fn, ll(T), ll(kMaxTokens));
    if (E <= 0) return fail(W4_EINVAL, "%s: E = %lld must be > 0", fn, ll(E));
    if (E > w4::kMaxExperts) return fail(W4_EUNSUPPORTED, "%s: E = %lld above %d", fn, ll(E), w4::kMaxExperts);
    if (top_k <= 0) return fail(W4_EINVAL, "%s: top_k = %d must be > 0", fn, top_k);
    if (top_k > w4::kMaxTopK) return fail(W4_EUNSUPPORTED, "%s: top_k = %d above %d", fn, top_k, w4::kMaxTopK);
    return W4_OK;
}

bool widths_ok(int64_t H, int64_t I, int G) {
    return (G == 32 || G == 64 || G == 128) && H > 0 && H <= kMaxWidth && H % G == 0 && I > 0 && I <= kMaxWidth && I % G == 0;
}
}  // namespace

extern "C" {

size_t w4_route_workspace_bytes(int64_t T, int64_t H, int64_t E) {
    if (T <= 0 || T > kMaxTokens || E <= 0 || E > w4::kMaxExperts || H <= 0 || H > kMaxWidth || H % 8 != 0) return 0;
    if (w4::route_in_one(static_cast<int>(E), static_cast<int>(H))) return 0;
    return static_cast<size_t>(w4::route_splits(T, static_cast<int>(E), static_cast<int>(H))) * static_cast<size_t>(T) *
           static_cast<size_t>(E) * sizeof(float);
}

int w4_route(const uint16_t* X, int64_t T, int64_t H, const uint16_t* router, int64_t E, int top_k, int score,
             const float* bias, int renormalize, float scale, int32_t* ids, float* weights, void* workspace,
             size_t workspace_bytes, hipStream_t stream) {
    const char* fn = "w4_route";
    W4_TRY(check_sizes(fn, T, E, top_k));
    if (top_k > E) return fail(W4_EINVAL, "%s: top_k = %d of E = %lld experts", fn, top_k, ll(E));
    if (H <= 0 || H > kMaxWidth || H % 8 != 0)
        return fail(W4_EINVAL, "%s: H = %lld must be a multiple of 8 in 8..%lld", fn, ll(H), ll(kMaxWidth));
    if (score != W4_SCORE_SOFTMAX && score != W4_SCORE_SIGMOID)
        return fail(W4_EINVAL, "%s: score = %d is neither W4_SCORE_SOFTMAX nor W4_SCORE_SIGMOID", fn, score);
    if (!std::isfinite(scale)) return fail(W4_EINVAL, "%s: scale is not finite", fn);
    if (T == 0) return W4_OK;
    W4_REQUIRE_PTR(fn, X);
    W4_REQUIRE_PTR(fn, router);
    if (!ids || !weights) return fail(W4_EINVAL, "%s: ids or weights is NULL", fn);
    const size_t need = w4_route_workspace_bytes(T, H, E);
    if (need > 0) W4_REQUIRE_PTR(fn, workspace);
    if (workspace_bytes < need)
        return fail(W4_EINVAL, "%s: workspace of %zu bytes, these sizes need %zu (w4_route_workspace_bytes)", fn, workspace_bytes, need);
    // workgroups read all of these while others write: choices and weights are no
    // part of what is read, nor of each other, nor of the partial logits
    const w4::Span x = w4::span(X, T, H, 2, "X"), r = w4::span(router, E, H, 2, "router"), b = w4::span(bias, E, 1, 4, "bias"),
                   i = w4::span(ids, T, top_k, 4, "ids"), w = w4::span(weights, T, top_k, 4, "weights"),
                   ws{workspace, need, "the workspace"};
    for (const w4::Span& in : {x, r, b}) {
        W4_TRY(w4::check_apart(fn, i, in));
        W4_TRY(w4::check_apart(fn, w, in));
        W4_TRY(w4::check_apart(fn, ws, in));
    }
    W4_TRY(w4::check_apart(fn, i, w));
    W4_TRY(w4::check_apart(fn, ws, i));
    W4_TRY(w4::check_apart(fn, ws, w));
    const w4::RouteParams p{X, T, static_cast<int>(H), router, static_cast<int>(E), top_k, score == W4_SCORE_SIGMOID, bias,
                            renormalize != 0, scale, ids, weights, static_cast<float*>(workspace),
                            w4::route_splits(T, static_cast<int>(E), static_cast<int>(H))};
    return hip_status(w4::launch_route(p, stream), fn);
}

size_t w4a16_moe_workspace_bytes(int64_t T, int top_k, int64_t E, int64_t H, int64_t I, int G) {
    if (T <= 0 || T > kMaxTokens || top_k <= 0 || top_k > w4::kMaxTopK || E <= 0 || E > w4::kMaxExperts || !widths_ok(H, I, G)) return 0;
    w4::MoeParams p{};
    p.T = T;
    p.k = top_k;
    p.E = static_cast<int>(E);
    p.H = static_cast<int>(H);
    p.I = static_cast<int>(I);
    p.G = G;
    return w4::moe_workspace(p, nullptr);
}

int w4a16_moe(const uint16_t* X, int64_t T, int64_t H, const int32_t* ids, const float* weights, int top_k,
              const uint32_t* wq_gate, const uint32_t* sz_gate, const uint32_t* wq_up, const uint32_t* sz_up,
              const uint32_t* wq_down, const uint32_t* sz_down, int64_t E, int64_t I, int G, int act,
              const uint16_t* residual, uint16_t* Y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* fn = "w4a16_moe";
    W4_TRY(check_sizes(fn, T, E, top_k));
    if (G != 32 && G != 64 && G != 128)
        return fail(W4_EUNSUPPORTED, "%s: group size %d is not one of 32, 64, 128", fn, G);
    if (!widths_ok(H, I, G))
        return fail(W4_EINVAL, "%s: H = %lld and I = %lld must be multiples of the group size %d up to %lld", fn, ll(H), ll(I), G,
                    ll(kMaxWidth));
    if (act != W4_ACT_SILU && act != W4_ACT_GELU_TANH)
        return fail(W4_EINVAL, "%s: act = %d is neither W4_ACT_SILU nor W4_ACT_GELU_TANH", fn, act);
    if (T == 0) return W4_OK;
    W4_REQUIRE_PTR(fn, X);
    if (!ids || !weights) return fail(W4_EINVAL, "%s: ids or weights is NULL", fn);
    W4_REQUIRE_PTR(fn, wq_gate);
    W4_REQUIRE_PTR(fn, wq_up);
    W4_REQUIRE_PTR(fn, wq_down);
    W4_REQUIRE_PTR(fn, sz_gate);
    W4_REQUIRE_PTR(fn, sz_up);
    W4_REQUIRE_PTR(fn, sz_down);
    W4_REQUIRE_PTR(fn, Y);
    if (residual && !aligned16(residual)) return fail(W4_EINVAL, "%s: residual is not 16-byte aligned", fn);
    // (the join reads the ids again while it writes Y)
    const w4::Span y = w4::span(Y, T, H, 2, "Y"), x = w4::span(X, T, H, 2, "X"), i = w4::span(ids, T, top_k, 4, "ids"),
                   w = w4::span(weights, T, top_k, 4, "weights"), r = w4::span(residual, T, H, 2, "the residual");
    for (const w4::Span& in : {x, i, w}) W4_TRY(w4::check_apart(fn, y, in));
    if (residual != Y) W4_TRY(w4::check_apart(fn, y, r));
    W4_REQUIRE_PTR(fn, workspace);
    w4::MoeParams p{};
    p.X = X;
    p.T = T;
    p.k = top_k;
    p.E = static_cast<int>(E);
    p.H = static_cast<int>(H);
    p.I = static_cast<int>(I);
    p.G = G;
    p.ids = ids;
    p.weights = weights;
    p.gate = {wq_gate, sz_gate};
    p.up = {wq_up, sz_up};
    p.down = {wq_down, sz_down};
    p.act = act;
    p.residual = residual;
    p.Y = Y;
    const size_t need = w4::moe_workspace(p, workspace);
    if (workspace_bytes < need)
        return fail(W4_EINVAL, "%s: workspace of %zu bytes, these sizes need %zu (w4a16_moe_workspace_bytes)", fn, workspace_bytes, need);
    const w4::Span ws{workspace, need, "the workspace"};
    for (const w4::Span& in : {x, i, w, r, y}) W4_TRY(w4::check_apart(fn, ws, in));
    return hip_status(w4::launch_moe(p, stream), fn);
}

}  // extern "C"
