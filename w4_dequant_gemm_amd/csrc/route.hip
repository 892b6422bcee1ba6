// Router of a mixture-of-experts layer on gfx950: each token's experts and
// their weights.
//
//   l[t, e] = sum_h X[t, h] R[e, h]                    (fp32 sums)
//   s = softmax over e of l[t, .], or 1 / (1 + exp(-l))
// The k experts with the largest l (with a selection bias: the largest s +
// bias), ties to the lower index; their weights are s, divided by their sum if
// renormalized, times a factor.  NaN logits count as -inf.
// Where the scores chosen leave the range of fp32 (sigmoids of logits below
// -88, or experts that a bias chose far below the largest logit), their ratios
// do not: a sigmoid of l << 0 is exp(l) to exp(l) of itself, a softmax score
// exp(l) over a sum that all share, so the shares are then
//   exp(l_j - max l) / sum of the same over the choices.
//
// The logits are v_mfma_f32_16x16x32_bf16 products of 16 tokens by 16 experts,
// a wave taking every wk-th step of 32 k; the waves' sums are added through LDS
// in wave order.  One compute unit reads only some 40 bytes a nanosecond, so
// with few tokens the k are split over workgroups too, and the second kernel,
// one wave a token, adds the ranges in their order before it chooses.  (All
// experts of 16 tokens in one workgroup and one launch: 10.7 us for 64 experts
// of 2048, 23 us for 128, against 4.2 and 5.7 for the logits here and 3 for the
// choice.)  Up to 16 experts with few k one workgroup does both.
#include <type_traits>

#include "device.hpp"
#include "moe_kernels.hpp"

namespace w4 {
namespace {

constexpr int kStep = 32;
constexpr int kMaxSplits = 8;

// maximum over the wavefront: within rows of 16 lanes, then across them, with
// lane 63's value for all
__device__ __forceinline__ float wave_max_dpp(float v) {
    auto step = [&](auto ctrl, auto rows) {
        const int o = __builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value,
                                                  0xF, false);
        v = fmaxf(v, __int_as_float(o));
    };
    step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});   // row_shr:1
    step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});   // row_shr:2
    step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});   // row_shr:4
    step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});   // row_shr:8
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});   // row_bcast:15 into rows 1 and 3
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});   // row_bcast:31 into rows 2 and 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// One wave's choice for token t from its logits l; value i of a lane is expert
// 64 i + lane's.
template <int NV>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, float (&l)[NV], int lane) {
    const float ninf = -__builtin_inff();
    float rank[NV], raw[NV];
    float top = ninf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = 64 * i + lane < p.E && l[i] == l[i] ? l[i] : ninf;
        raw[i] = rank[i] = l[i];
        top = fmaxf(top, l[i]);
    }
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = 1.0f / (1.0f + expf(-l[i]));
    } else {
        top = wave_max_dpp(top);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // the largest has 1 whatever it is, unless there is none
            l[i] = l[i] == ninf ? 0.0f : (l[i] == top ? 1.0f : expf(l[i] - top));
            sum += l[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = sum > 0.0f ? l[i] / sum : 0.0f;
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            const float v = e < p.E ? l[i] + p.bias[e] : ninf;
            rank[i] = v == v ? v : ninf;
        }
    }
    uint32_t open = 0;               // bit i: value i is an expert that is not chosen yet
#pragma unroll
    for (int i = 0; i < NV; ++i) open |= 64 * i + lane < p.E ? 1u << i : 0u;
    float mine = 0.0f, all = 0.0f;   // lane j: the weight of choice j
    float my_raw = ninf, most = ninf;   // its logit, and the largest of the choices'
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
        float best = ninf;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = open >> i & 1u ? fmaxf(best, rank[i]) : best;
        best = wave_max_dpp(best);
        // the lowest expert that has it: the first value i with one, its lowest lane
        int id = 0;
        float score = 0.0f, logit = ninf;
        bool found = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint64_t has = __builtin_amdgcn_ballot_w64((open >> i & 1u) && rank[i] == best);
            if (!found && has) {
                const int at = __builtin_ctzll(has);
                found = true;
                id = 64 * i + at;
                score = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l[i]), at));
                logit = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(raw[i]), at));
                if (lane == at) open &= ~(1u << i);
            }
        }
        if (lane == j) {
            mine = score;
            my_raw = logit;
            my_id = id;
        }
        all += score;
        most = fmaxf(most, logit);
    }
    // (2^-60: what fp32 holds of a score above 2^-126 is whole, and smaller ones
    // are less than a rounding of such a sum; the largest logit has 1 whatever it is)
    if (p.renormalize && all < 0x1p-60f && most > ninf) {
        mine = lane >= p.k ? 0.0f : (my_raw == most ? 1.0f : expf(my_raw - most));
        all = wave_sum(mine);
    }
    if (lane < p.k) {
        if (p.renormalize) mine = all > 0.0f ? mine / all : 0.0f;
        p.ids[t * p.k + lane] = my_id;
        p.weights[t * p.k + lane] = mine * p.scale;
    }
}

// 16 tokens from t0 on times 16 experts from e0 on, the wave's steps; register i
// of lane (c, h): token 4 h + i, expert c
__device__ __forceinline__ float4_t logits16(const RouteParams& p, int64_t t0, int e0, int first, int steps, int wave, int wk, int lane) {
    const int c = lane & 15, h = lane >> 4;
    const int64_t t = t0 + c < p.T ? t0 + c : p.T - 1;
    const int e = e0 + c < p.E ? e0 + c : p.E - 1;
    const uint16_t* const x = p.X + t * p.H;
    const uint16_t* const r = p.router + static_cast<int64_t>(e) * p.H;
    float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    constexpr int AHEAD = 4;                        // steps in flight
    const int end = first + steps;
    for (int s0 = first + wave; s0 < end; s0 += AHEAD * wk) {
        u32x4_t a[AHEAD], b[AHEAD];
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            const int k = kStep * (s0 + d * wk) + 8 * h;
            const bool in = s0 + d * wk < end && k < p.H;   // (H is a multiple of 8)
            a[d] = *reinterpret_cast<const u32x4_t*>(x + (in ? k : 0));
            b[d] = *reinterpret_cast<const u32x4_t*>(r + (in ? k : 0));
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            // (both zero past H: an infinity there would be NaN)
            const bool in = s0 + d * wk < end && kStep * (s0 + d * wk) + 8 * h < p.H;
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, in ? a[d] : zero),
                                                          __builtin_bit_cast(bf16x8_t, in ? b[d] : zero), acc, 0, 0, 0);
        }
    }
    return acc;
}

// at most 16 experts of 16 tokens, and the choice
__global__ void __launch_bounds__(1024) route_kernel(RouteParams p, int wk) {
    __shared__ float red[16][256];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = 16 * static_cast<int64_t>(blockIdx.x);
    const float4_t acc = logits16(p, t0, 0, 0, (p.H + kStep - 1) / kStep, wave, wk, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][16 * (4 * (lane >> 4) + i) + (lane & 15)] = acc[i];
    __syncthreads();
    for (int t = wave; t < 16 && t0 + t < p.T; t += wk) {
        float l[1] = {0.0f};
        if (lane < 16)
            for (int w = 0; w < wk; ++w) l[0] += red[w][16 * t + lane];
        choose<1>(p, t0 + t, l, lane);
    }
}

__global__ void __launch_bounds__(1024) route_logits_kernel(RouteParams p, int wk) {
    __shared__ float red[16][256];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = 16 * blockIdx.x;
    const int64_t t0 = 16 * static_cast<int64_t>(blockIdx.y);
    const int steps = (p.H + kStep - 1) / kStep, z = blockIdx.z;
    const int first = z * steps / p.splits;
    const float4_t acc = logits16(p, t0, e0, first, (z + 1) * steps / p.splits - first, wave, wk, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][16 * (4 * (lane >> 4) + i) + (lane & 15)] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += blockDim.x) {
        float y = 0.0f;
        for (int w = 0; w < wk; ++w) y += red[w][o];
        const int64_t t = t0 + o / 16;
        const int e = e0 + o % 16;
        if (t < p.T && e < p.E) p.logits[(z * p.T + t) * p.E + e] = y;
    }
}

template <int NV>
__global__ void __launch_bounds__(64) route_choose_kernel(RouteParams p) {
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = 0.0f;
        if (64 * i + lane < p.E) {
            const float* const at = p.logits + t * p.E + 64 * i + lane;
            float v[kMaxSplits];
#pragma unroll
            for (int z = 0; z < kMaxSplits; ++z) v[z] = z < p.splits ? at[z * p.T * p.E] : 0.0f;
#pragma unroll
            for (int z = 0; z < kMaxSplits; ++z) l[i] += v[z];
        }
    }
    choose<NV>(p, t, l, lane);
}

}  // namespace

// About 512 k a workgroup while there are fewer workgroups than compute units.
int route_splits(int64_t T, int E, int H) {
    const int64_t tiles = ((E + 15) / 16) * ((T + 15) / 16);
    int64_t s = H / 512;
    if (s > 256 / tiles) s = 256 / tiles;
    if (s > kMaxSplits) s = kMaxSplits;
    return s < 1 ? 1 : static_cast<int>(s);
}

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
    const int steps = (p.H + kStep - 1) / kStep;
    if (route_in_one(p.E, p.H)) {
        const int wk = steps / 2 < 1 ? 1 : (steps / 2 > 16 ? 16 : steps / 2);
        hipLaunchKernelGGL(route_kernel, dim3(static_cast<unsigned>((p.T + 15) / 16)), dim3(64 * wk), 0, stream, p, wk);
        return hipGetLastError();
    }
    int wk = steps / p.splits / (p.splits > 1 ? 1 : 4);
    wk = wk < 1 ? 1 : (wk > 16 ? 16 : wk);
    hipLaunchKernelGGL(route_logits_kernel,
                       dim3(static_cast<unsigned>((p.E + 15) / 16), static_cast<unsigned>((p.T + 15) / 16),
                            static_cast<unsigned>(p.splits)),
                       dim3(64 * wk), 0, stream, p, wk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.T));
    if (p.E <= 64) hipLaunchKernelGGL((route_choose_kernel<1>), grid, dim3(64), 0, stream, p);
    else if (p.E <= 128) hipLaunchKernelGGL((route_choose_kernel<2>), grid, dim3(64), 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL((route_choose_kernel<4>), grid, dim3(64), 0, stream, p);
    else hipLaunchKernelGGL((route_choose_kernel<16>), grid, dim3(64), 0, stream, p);
    return hipGetLastError();
}

}  // namespace w4
