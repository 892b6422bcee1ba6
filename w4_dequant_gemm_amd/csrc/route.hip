// Router of a mixture-of-experts layer on gfx950: each token's experts and
// their weights.
//
//   l[t, e] = sum_h X[t, h] R[e, h]                    (fp32 sums)
//   s = softmax over e of l[t, .], or 1 / (1 + exp(-l))
// The k experts with the largest l (with a selection bias: the largest s +
// bias), ties to the lower index; their weights are s, divided by their sum if
// renormalized, times a factor.  NaN logits count as -inf.
//
// Logits: a workgroup takes 16 tokens by 16 experts on
// v_mfma_f32_16x16x32_bf16, its waves every wk-th step of 32 k; the partial
// sums are added through LDS in wave order.  Then one wave a token chooses.
#include "device.hpp"
#include "moe_kernels.hpp"

namespace w4 {
namespace {

constexpr int kStep = 32;

__global__ void __launch_bounds__(1024) route_logits_kernel(RouteParams p, int wk) {
    __shared__ float red[16][256];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int e0 = 16 * blockIdx.x;
    const int64_t t0 = 16 * static_cast<int64_t>(blockIdx.y);
    const int64_t t = t0 + c < p.T ? t0 + c : p.T - 1;
    const int e = e0 + c < p.E ? e0 + c : p.E - 1;
    const uint16_t* const x = p.X + t * p.H;
    const uint16_t* const r = p.router + static_cast<int64_t>(e) * p.H;
    const int steps = (p.H + kStep - 1) / kStep;
    float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll 4
    for (int s = wave; s < steps; s += wk) {
        const int k = kStep * s + 8 * h;
        const bool in = k < p.H;                    // (H is a multiple of 8)
        u32x4_t a = *reinterpret_cast<const u32x4_t*>(x + (in ? k : 0));
        const u32x4_t b = *reinterpret_cast<const u32x4_t*>(r + (in ? k : 0));
        u32x4_t bz = in ? b : zero;
        a = in ? a : zero;
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, bz), acc,
                                                      0, 0, 0);
    }
    // register i of lane (c, h): token 4 h + i, expert c
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][16 * (4 * h + i) + c] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += blockDim.x) {
        float y = 0.0f;
        for (int w = 0; w < wk; ++w) y += red[w][o];
        const int64_t tt = t0 + o / 16;
        const int ee = e0 + o % 16;
        if (tt < p.T && ee < p.E) p.logits[tt * p.E + ee] = y;
    }
}

// NV: logits a lane holds; expert 64 i + lane is value i
template <int NV>
__global__ void __launch_bounds__(64) route_choose_kernel(RouteParams p) {
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const float ninf = -__builtin_inff();
    float l[NV], rank[NV];
    float top = ninf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 64 * i + lane;
        const float v = e < p.E ? p.logits[t * p.E + e] : ninf;
        l[i] = v == v ? v : ninf;
        top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        rank[i] = l[i];
        if (p.sigmoid) {
            l[i] = 1.0f / (1.0f + expf(-l[i]));
        } else {
            // the largest has 1 whatever it is, unless there is none
            l[i] = l[i] == ninf ? 0.0f : (l[i] == top ? 1.0f : expf(l[i] - top));
            sum += l[i];
        }
    }
    if (!p.sigmoid) {
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
    uint32_t taken = 0;              // bit i: value i is chosen already
    float mine = 0.0f, all = 0.0f;   // lane j: the weight of choice j
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
        float best = ninf, score = 0.0f;
        int id = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            if (e < p.E && !(taken >> i & 1u) && (id == 0x7FFFFFFF || rank[i] > best)) {
                best = rank[i];
                score = l[i];
                id = e;
            }
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const float ob = __shfl_xor(best, off, kWave), os = __shfl_xor(score, off, kWave);
            const int oi = __shfl_xor(id, off, kWave);
            if (oi != 0x7FFFFFFF && (id == 0x7FFFFFFF || ob > best || (ob == best && oi < id))) {
                best = ob;
                score = os;
                id = oi;
            }
        }
        if ((id & 63) == lane) taken |= 1u << (id >> 6);
        if (lane == j) {
            mine = score;
            my_id = id;
        }
        all += score;
    }
    if (lane < p.k) {
        if (p.renormalize) mine = all > 0.0f ? mine / all : 0.0f;
        p.ids[t * p.k + lane] = my_id;
        p.weights[t * p.k + lane] = mine * p.scale;
    }
}

}  // namespace

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
    const int steps = (p.H + kStep - 1) / kStep;
    int wk = steps / 4;
    wk = wk < 1 ? 1 : (wk > 16 ? 16 : wk);
    hipLaunchKernelGGL(route_logits_kernel,
                       dim3(static_cast<unsigned>((p.E + 15) / 16), static_cast<unsigned>((p.T + 15) / 16)), dim3(64 * wk), 0,
                       stream, p, wk);
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
