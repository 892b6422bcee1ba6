// Epilogue of a product with bias, activation and residual:
//   Y[m, n] = bf16(act(y + bias[n]) + residual[m, n]),  y the fp32 sum (row
// scale applied).  Kernels take it as a template argument; without it they
// round y to bf16 as they are.
#pragma once

#include "device.hpp"
#include "kernels.hpp"

namespace w4 {

// act: 0 none, 1 SiLU, 2 GELU (tanh form), 3 ReLU, 4 GELU (erf).  With
// 1 + tanh(t) = 2 / (1 + e^-2t) the first two are x / (1 + e^-t), t = x a and
// t = x (a + b x^2): one exponential, and no cancellation where x is far below
// zero; the erf form takes erfc for the same reason.
__device__ __forceinline__ float linear_activation(int act, float x) {
    if (act == 0) return x;
    if (act == 3) return x < 0.0f ? 0.0f : x;                       // (NaN stays)
    if (act == 4) return 0.5f * x * erfcf(-0.70710678118654752f * x);
    const float a = act == 1 ? 1.0f : 1.5957691216057308f, b = act == 1 ? 0.0f : 0.071354816272600251f;
    // (x^2 kept finite: 0 times an infinity is NaN)
    return x / (1.0f + expf(-x * fmaf(b, fminf(x * x, 3.0e38f), a)));
}

// one output
template <bool EPI>
__device__ __forceinline__ uint16_t finish(const KernelParams<EPI>& p, int64_t row, int64_t col, float y) {
    if constexpr (EPI) {
        if (p.bias) y += p.bias[col];
        y = linear_activation(p.out_act, y);
        if (p.residual) y += bf16_lo(p.residual[row * p.N + col]);
    }
    return float_to_bf16_bits(y);
}

// four outputs of a row from column `col` on (a multiple of 4; those past N
// are left out), their sums in y
template <bool EPI>
__device__ __forceinline__ void finish4(const KernelParams<EPI>& p, int64_t row, int64_t col, float4 y) {
    float v[4] = {y.x, y.y, y.z, y.w};
    const int64_t at = row * p.N + col;
    const bool whole = col + 3 < p.N && p.N % 4 == 0;
    if constexpr (EPI) {
        float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.residual) {
            if (whole) {
                const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p.residual + at);
                r[0] = bf16_lo(w[0]);
                r[1] = bf16_hi(w[0]);
                r[2] = bf16_lo(w[1]);
                r[3] = bf16_hi(w[1]);
            } else {
                for (int e = 0; e < 4 && col + e < p.N; ++e) r[e] = bf16_lo(p.residual[at + e]);
            }
        }
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += p.bias[col + e < p.N ? col + e : p.N - 1];
        }
        if (p.out_act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = linear_activation(p.out_act, v[e]);
        }
        if (p.residual) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += r[e];
        }
    }
    uint16_t* const dst = p.Y + at;
    if (whole) *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
        for (int e = 0; e < 4 && col + e < p.N; ++e) dst[e] = float_to_bf16_bits(v[e]);
}

// The tiled kernels hold a wave's sums in the matrix cores' layout.  With an
// epilogue a few rows at a time go through LDS, so that bias, residual and
// output pass in 8- and 16-byte pieces of consecutive lanes, and the code of
// the activations is there once a round instead of once an output.  Column c of
// row r lies at c ^ epi_swizzle(r): the lanes of a store, 16 or 32 columns of
// rows 4 apart, then fall on different banks.
__device__ __forceinline__ int epi_swizzle(int r) { return ((r >> 2) & 1) << 5 | ((r >> 3) & 1) << 4; }

// `rows` LDS rows of BN sums: outputs (row_of(r), n0 + c)
template <int NT, int BN, bool SCALE, typename RowOf>
__device__ __forceinline__ void epilogue_rows(const MulParams& p, const float* t, int rows, int64_t n0, int tid, RowOf row_of) {
    for (int o = 4 * tid; o < rows * BN; o += 4 * NT) {
        const int r = o / BN, c = o % BN;
        const int64_t row = row_of(r), col = n0 + c;
        if (row >= p.M || col >= p.N) continue;
        float4 y = *reinterpret_cast<const float4*>(t + r * BN + (c ^ epi_swizzle(r)));
        if (SCALE && p.x_fp8) {
            const float s = p.xscale[row];
            y.x *= s; y.y *= s; y.z *= s; y.w *= s;
        }
        finish4<true>(p, row, col, y);
    }
}

}  // namespace w4
