// Mixture-of-experts layer over 4-bit experts on gfx950.
//
//   h_j = w_j act(Wg[e_j] X[t]) * (Wu[e_j] X[t])      for the experts e_j of token t
//   Y[t] = bf16(residual[t] + sum_j Wd[e_j] h_j)
//
// With few tokens an expert the layer is bound by streaming the chosen
// experts' packed weights, as the W4A16 products of few rows are.  A slot is
// a (token, choice) pair; the slots are first put in order of their expert, so
// that an expert's weights are read once for all of its rows.
//
// A workgroup owns 16 columns of one expert's gate and up weights (or 16 FJ
// columns of its down weight) and up to 16 MB of the expert's rows at a time;
// its wk waves take every wk-th 128-k step.  Lane (c, q) loads the 16 bytes of
// the 32-k tile 4 s + q of column c (1 KB contiguous in the blocked layout).
// The codes become the exact bf16 values 128 + u; with P the product with them
// and x1 the sum of the activations over a group (an MFMA against ones),
//   acc += s (P - (128 + z) x1)
// is exact in the weights.  Groups of 128: MFMA b takes from every quarter q
// the 8 k at 32 q + 8 b, as the words lie.  Groups of 32 and 64 need MFMAs
// that stay inside a group: the four words of the four quarters are
// transposed (two swaps of 32 lanes and two of 16), after which MFMA t takes
// exactly tile t, quarter q the 8 k at 32 t + 8 q.
//
// h carries the token's weight w_j already.  It is kept as two bf16 numbers,
// h = hi + lo (16 bits of mantissa), and the down product multiplies both: with
// h rounded to bf16 once the result was 1.4 times as far from the exact one
// as its own rounding to bf16 leaves it.
#include "device.hpp"
#include "moe_kernels.hpp"

namespace w4 {
namespace {

// ------------------------------------------------------------------- lists

// Slots ordered by expert, and the experts that have any.  One workgroup:
// counts in LDS, a running sum over the experts, then every slot takes a place
// behind its expert's start.  (Which place inside an expert's run is up to the
// order of the atomics; every row's result is the same at any place.)
constexpr int kListThreads = 1024;
__global__ void __launch_bounds__(kListThreads) moe_lists_kernel(MoeParams p) {
    __shared__ int count[kMaxExperts], sums[2][kListThreads];
    const int tid = threadIdx.x;
    for (int e = tid; e < p.E; e += kListThreads) count[e] = 0;
    __syncthreads();
    const int slots = static_cast<int>(p.T * p.k);
    for (int s = tid; s < slots; s += kListThreads) {
        const uint32_t e = static_cast<uint32_t>(p.ids[s]);
        if (e < static_cast<uint32_t>(p.E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    // inclusive sums over the experts (kMaxExperts threads), of the counts
    // (low 31 bits would do) and of the experts that have rows
    const int mine = tid < p.E ? count[tid] : 0;
    sums[0][tid] = mine;
    sums[1][tid] = mine > 0;
    __syncthreads();
    for (int off = 1; off < kListThreads; off <<= 1) {
        const int a = tid >= off ? sums[0][tid - off] : 0, b = tid >= off ? sums[1][tid - off] : 0;
        __syncthreads();
        sums[0][tid] += a;
        sums[1][tid] += b;
        __syncthreads();
    }
    if (tid < p.E) {
        const int start = sums[0][tid] - mine;
        p.offset[tid] = start;
        count[tid] = start;
        if (mine > 0) p.active[sums[1][tid] - 1] = tid;
        if (tid == p.E - 1) {
            p.offset[p.E] = sums[0][tid];
            p.active[p.E] = sums[1][tid];
        }
    }
    __syncthreads();
    for (int s = tid; s < slots; s += kListThreads) {
        const uint32_t e = static_cast<uint32_t>(p.ids[s]);
        if (e < static_cast<uint32_t>(p.E)) p.order[atomicAdd(&count[e], 1)] = s;
    }
}

// ------------------------------------------------------------------ products

constexpr int kStepK = 128;
constexpr int kDepth = 2;        // steps in flight a wave

// 4 x 4 transposition of words over the quarters: w[t] of quarter q becomes
// w[q] of quarter t
__device__ __forceinline__ void transpose_quarters(u32x4_t& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// UP: gate and up (FJ = 2: block 0 the gate weight, block 1 the up weight, at
// the same 16 columns), rows gathered from X; else the down product on the
// rows hi + lo.
template <int MB, int FJ, int G, bool UP>
__global__ void __launch_bounds__(512) moe_stream_kernel(MoeParams p, int wk) {
    static_assert(!UP || FJ == 2, "a block for each weight");
    constexpr int NG = kStepK / G;                 // groups in a step
    constexpr int AP = UP ? 1 : 2;                 // parts of an activation
    constexpr int COLS = UP ? 16 : 16 * FJ;
    extern __shared__ float red[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    if (static_cast<int>(blockIdx.y) >= p.active[p.E]) return;
    const int expert = p.active[blockIdx.y];
    const int first = p.offset[expert], rows = p.offset[expert + 1] - first;
    const int K = UP ? p.H : p.I, N = UP ? p.I : p.H;
    const int KS = (K + kStepK - 1) / kStepK, KQ = K / 32;
    const int n0 = COLS * blockIdx.x;
    const int64_t words = static_cast<int64_t>(N) * (K / 8), groups = static_cast<int64_t>(N) * (K / G);

    // the blocks' first words; N is a multiple of 16, so every block has 16 rows
    const uint32_t* wb[FJ];
    const uint32_t* sb[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        const MoeWeight& w = UP ? (j == 0 ? p.gate : p.up) : p.down;
        int r0 = UP ? n0 : n0 + 16 * j;
        r0 = r0 < N ? r0 : N - 16;
        wb[j] = w.wq + expert * words + static_cast<int64_t>(r0) * (K / 8) + 4 * c;
        sb[j] = w.sz + expert * groups + static_cast<int64_t>(r0) * (K / G) + c;
    }
    const uint32_t bias = opaque_vgpr(kBf16Bias128x2);
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const u32x4_t zero = {0u, 0u, 0u, 0u};

    for (int m0 = 0; m0 < rows; m0 += 16 * MB) {
        // the lane's row in each block (past the last: the last, never stored)
        const uint16_t* arow[MB][AP];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            int m = m0 + 16 * i + c;
            m = m < rows ? m : rows - 1;
            const int slot = p.order[first + m];
            if constexpr (UP) {
                arow[i][0] = p.X + static_cast<int64_t>(slot / p.k) * K;
            } else {
                arow[i][0] = p.hi + static_cast<int64_t>(slot) * K;
                arow[i][1] = p.lo + static_cast<int64_t>(slot) * K;
            }
        }
        float4_t acc[MB][FJ];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

        struct B {
            u32x4_t w[FJ];
            uint32_t s[FJ][NG];
        };
        struct A {
            u32x4_t a[MB][AP][4];
        };
        auto load_b = [&](int step, B& b) {
            int t = 4 * step + q;
            t = t < KQ ? t : KQ - 1;
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                b.w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wb[j] + 64 * t));
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    int gg = NG * step + g;
                    gg = gg < K / G ? gg : K / G - 1;
                    b.s[j][g] = sb[j][16 * gg];
                }
            }
        };
        // fragment f: the 8 k at 32 q + 8 f of the step (groups of 128), or at
        // 32 f + 8 q
        auto load_a = [&](int step, A& a) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                int t = 4 * step + (NG == 1 ? q : f);
                t = t < KQ ? t : KQ - 1;
                const int k = 32 * t + 8 * (NG == 1 ? f : q);
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int v = 0; v < AP; ++v) a.a[i][v][f] = *reinterpret_cast<const u32x4_t*>(arow[i][v] + k);
            }
        };
        auto multiply = [&](int step, B& b, const A& a) {
            if constexpr (NG > 1) {
#pragma unroll
                for (int j = 0; j < FJ; ++j) transpose_quarters(b.w[j]);
            }
            float4_t ps[MB][FJ], x1[MB];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                if (f % (4 / NG) == 0) {
#pragma unroll
                    for (int i = 0; i < MB; ++i) {
                        x1[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int j = 0; j < FJ; ++j) ps[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                }
                // K ends inside the last step of groups below 128
                const bool in = NG == 1 || 4 * step + f < KQ;
                bf16x8_t bp[FJ];
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    const uint32_t w = b.w[j][f];
                    bp[j] = __builtin_bit_cast(bf16x8_t, u32x4_t{nibble_pair_bf16(w, 0, bias), nibble_pair_bf16(w, 1, bias),
                                                                 nibble_pair_bf16(w, 2, bias), nibble_pair_bf16(w, 3, bias)});
                }
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int v = 0; v < AP; ++v) {
                        const bf16x8_t ap = __builtin_bit_cast(bf16x8_t, in ? a.a[i][v][f] : zero);
                        x1[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ap, ones, x1[i], 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < FJ; ++j)
                            ps[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ap, bp[j], ps[i][j], 0, 0, 0);
                    }
                if (f % (4 / NG) == 4 / NG - 1) {
#pragma unroll
                    for (int j = 0; j < FJ; ++j) {
                        const uint32_t sz = b.s[j][f / (4 / NG)];
                        const float sc = half_bits_to_float(sz), zc = 128.0f + half_bits_to_float(sz >> 16);
#pragma unroll
                        for (int i = 0; i < MB; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[i][j][e] = fmaf(sc, fmaf(-zc, x1[i][e], ps[i][j][e]), acc[i][j][e]);
                    }
                }
            }
        };
        // rounds of kDepth steps: their loads together, then their products;
        // the other waves on the compute unit cover the latency
        for (int step = wave; step < KS; step += kDepth * wk) {
            B b[kDepth];
            A a[kDepth];
#pragma unroll
            for (int d = 0; d < kDepth; ++d)
                if (step + d * wk < KS) {
                    load_b(step + d * wk, b[d]);
                    load_a(step + d * wk, a[d]);
                }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int d = 0; d < kDepth; ++d)
                if (step + d * wk < KS) multiply(step + d * wk, b[d], a[d]);
        }

        // the waves' sums through LDS, in wave order: register e of lane (c, q)
        // is row 4 q + e of its block, column c
        constexpr int TILE = 256 * MB * FJ;
        __syncthreads();                           // (the last rows' sums are read)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[wave * TILE + (16 * i + 4 * q + e) * (16 * FJ) + 16 * j + c] = acc[i][j][e];
        __syncthreads();
        for (int o = threadIdx.x; o < 16 * MB * COLS; o += blockDim.x) {
            const int row = o / COLS, col = o % COLS;
            if (m0 + row >= rows || n0 + col >= N) continue;
            const int slot = p.order[first + m0 + row];
            if constexpr (UP) {
                float g = 0.0f, u = 0.0f;
                for (int w = 0; w < wk; ++w) {
                    g += red[w * TILE + row * 32 + col];
                    u += red[w * TILE + row * 32 + 16 + col];
                }
                const float h = activation(p.act, g) * u * p.weights[slot];
                const uint16_t hi = float_to_bf16_bits(h);
                const float rest = h - bf16_lo(hi);
                const int64_t at = static_cast<int64_t>(slot) * N + n0 + col;
                p.hi[at] = hi;
                // (an infinite upper part has no rest)
                p.lo[at] = (hi & 0x7FFFu) == 0x7F80u ? 0 : float_to_bf16_bits(rest);
            } else {
                float y = 0.0f;
                for (int w = 0; w < wk; ++w) y += red[w * TILE + row * COLS + col];
                p.part[static_cast<int64_t>(slot) * N + n0 + col] = y;
            }
        }
    }
}

// Y = bf16(residual + the slots' shares in the order of the choices), eight
// columns a thread
__global__ void __launch_bounds__(256) moe_join_kernel(MoeParams p) {
    const int per = p.H / 8;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.T * per) return;
    const int64_t t = i / per;
    const int n = static_cast<int>(i % per) * 8;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int64_t slot = t * p.k + j;
        if (static_cast<uint32_t>(p.ids[slot]) >= static_cast<uint32_t>(p.E)) continue;
        const float4* src = reinterpret_cast<const float4*>(p.part + slot * p.H + n);
        const float4 a = src[0], b = src[1];
        y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
        y[4] += b.x; y[5] += b.y; y[6] += b.z; y[7] += b.w;
    }
    if (p.residual) {
        const u32x4_t r = *reinterpret_cast<const u32x4_t*>(p.residual + t * p.H + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] += bf16_lo(r[e]);
            y[2 * e + 1] += bf16_hi(r[e]);
        }
    }
    *reinterpret_cast<u32x4_t*>(p.Y + t * p.H + n) = u32x4_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                            pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
}

template <int MB, int FJ, int G, bool UP>
hipError_t launch_stream(const MoeParams& p, hipStream_t stream) {
    const int K = UP ? p.H : p.I, N = UP ? p.I : p.H, cols = UP ? 16 : 16 * FJ;
    const int64_t slots = p.T * p.k;
    const int experts = slots < p.E ? static_cast<int>(slots) : p.E;
    const int nb = (N + cols - 1) / cols, steps = (K + kStepK - 1) / kStepK;
    int64_t wk = 4096 / (static_cast<int64_t>(nb) * experts);
    wk = wk > 8 ? 8 : wk;
    wk = wk > steps / 2 ? steps / 2 : wk;
    wk = wk < 1 ? 1 : wk;
    hipLaunchKernelGGL((moe_stream_kernel<MB, FJ, G, UP>), dim3(static_cast<unsigned>(nb), static_cast<unsigned>(experts)),
                       dim3(static_cast<unsigned>(64 * wk)), static_cast<size_t>(wk) * 256 * MB * FJ * sizeof(float), stream, p,
                       static_cast<int>(wk));
    return hipGetLastError();
}

template <int MB, bool UP>
hipError_t launch_stream_g(const MoeParams& p, hipStream_t stream) {
    switch (p.G) {
        case 32: return launch_stream<MB, 2, 32, UP>(p, stream);
        case 64: return launch_stream<MB, 2, 64, UP>(p, stream);
        default: return launch_stream<MB, 2, 128, UP>(p, stream);
    }
}

}  // namespace

size_t moe_workspace(MoeParams& p, void* base) {
    const size_t slots = static_cast<size_t>(p.T) * p.k;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        void* q = base ? static_cast<char*>(base) + at : nullptr;
        at += (bytes + 255) & ~size_t{255};
        return q;
    };
    p.offset = static_cast<int32_t*>(take(4 * (p.E + 1)));
    p.active = static_cast<int32_t*>(take(4 * (p.E + 1)));
    p.order = static_cast<int32_t*>(take(4 * slots));
    p.hi = static_cast<uint16_t*>(take(2 * slots * p.I));
    p.lo = static_cast<uint16_t*>(take(2 * slots * p.I));
    p.part = static_cast<float*>(take(4 * slots * p.H));
    return at;
}

hipError_t launch_moe(const MoeParams& p, hipStream_t stream) {
    hipLaunchKernelGGL(moe_lists_kernel, dim3(1), dim3(kListThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_stream_g<1, true>(p, stream);
    if (e != hipSuccess) return e;
    e = launch_stream_g<1, false>(p, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_join_kernel, dim3(static_cast<unsigned>((p.T * (p.H / 8) + 255) / 256)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace w4
