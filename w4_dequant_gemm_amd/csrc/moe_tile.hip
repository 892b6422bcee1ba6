// The products of a mixture of experts with many tokens, on gfx950's matrix
// cores: tiles of 64 of one expert's rows.
//
//   up:    h = bf16(w act(Wg x) * (Wu x)) of every slot, in the order of the
//          experts' rows, and h's sums over each group
//   down:  part[slot] = Wd h, fp32
//
// A workgroup of four waves computes 64 rows by 128 columns of h (or 256
// columns of the down product); a wave owns all 64 rows of 64 weight columns,
// in two blocks of 32: the same 32 columns of the gate and of the up weight, so
// that a lane holds both sums of its outputs, or 64 columns of the down weight.
// Four 32 x 32 x 16 MFMAs then share two fragments of activations and two of
// weights: with 32 columns a wave (four 16 x 16 MFMAs to four fragments) the
// reads of the activations from LDS took as long as the matrix cores, and the
// up product of 1999 tokens by 64 experts 206 us.
//
// The activations go straight from global memory into LDS, two steps of 128 k
// ahead in three stages of 64 x 256 bytes; chunk ch (16 bytes) of row r lies at
// ch ^ (r & 15).  The weights never pass through LDS: half h of the lanes loads
// the 16 bytes of every second 32-k tile, a step ahead, and a code word becomes
// the four registers of an MFMA operand (the exact bf16 values 128 + u) right
// before its MFMAs; MFMA j of a 64-k half takes the 8 k at 32 h + 8 j.  With x1
// the row sum of the group's activations, which a kernel before has made,
//   acc += s (T - (128 + z) x1)
// per group, exact in the weights.
#include "device.hpp"
#include "moe_kernels.hpp"

namespace w4 {
namespace {

constexpr int kRows = kMoeTileRows, kThreads = 256, kStepK = 128;
constexpr int kStage = kRows * kStepK * 2;          // bytes
constexpr int kDma = kStage / (1024 * 4);           // loads to LDS a wave and step
static_assert(kRows == 64, "two row blocks of 32");

__device__ __forceinline__ u32x4_t tile_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return u32x4_t{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a))),
                   static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32))) & 0xFFFFu,
                   static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
}

// activation() with the hardware's exponential and reciprocal (a few units of
// 2^-24; what is made of it is rounded to bf16).  1 + tanh(t) = 2 / (1 + e^-2t):
// both forms are x / (1 + 2^-y), y = x (a + b x^2).  (x^2 kept finite: 0 times an
// infinity is NaN.)
__device__ __forceinline__ float quick_activation(int act, float x) {
    const float a = act == 1 ? 1.4426950408889634f : 2.3022081986685205f, b = act == 1 ? 0.0f : 0.10294324003185554f;
    const float y = x * fmaf(b, fminf(x * x, 3.0e38f), a);
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-y));
}

// Two workgroups a compute unit: 256 registers a lane.  (One, with 512: 1999
// tokens on 64 experts of 2048 x 1024, groups of 64, 370 us in place of 287;
// 1391 rows on 5 experts, groups of 32, 102 in place of 87.)  Groups of 128 fit;
// of groups of 64 3 or 4 registers and of groups of 32 17 are kept in memory: 1999
// tokens, 6 of 64 experts of 2048 x 1024, up and down product 154 and 95 us, 181 and
// 109, 238 and 140, matrix cores 48 and 38 %, 35 and 30 %, 24 and 21 % busy, and of
// groups of 32 the up product writes 53 MB for 24 of h.  (Registers kept in memory
// add loads and stores to those that the counted waits below allow, which makes
// the waits longer and never shorter.)
template <int G, bool UP>
__global__ void __launch_bounds__(kThreads, 2) moe_tile_kernel(MoeParams p) {
    constexpr int GS = kStepK / G, PER = 8 / GS;     // groups in a step, slots (MFMAs of a tile) in a group
    __shared__ __attribute__((aligned(16))) uint8_t lds_a0[kStage];
    __shared__ __attribute__((aligned(16))) uint8_t lds_a1[kStage];
    __shared__ __attribute__((aligned(16))) uint8_t lds_a2[kStage];
    __shared__ int lds_slot[kRows], lds_row[kRows];
    __shared__ float lds_weight[kRows];
    extern __shared__ __attribute__((aligned(16))) float lds_x1[];   // [step][row]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, h = lane >> 5;
    const int K = UP ? p.H : p.I, N = UP ? p.I : p.H;
    constexpr int COLS = UP ? 128 : 256;             // the workgroup's columns of the result
    const int nt = (N + COLS - 1) / COLS;
    const int zs = UP ? 1 : p.splits;                // ranges of the down product's k
    const int total = *p.tile_count * nt * zs;
    if (static_cast<int>(blockIdx.x) >= total) return;
    int job = static_cast<int>(xcd_tile(blockIdx.x, total));
    const int z = job % zs;
    job /= zs;
    // (K may end inside the last step of groups below 128: its activations are
    // zeros there)
    const int steps = (K + kStepK - 1) / kStepK, kb = z * steps / zs, KT = (z + 1) * steps / zs - kb;
    const int4 t4 = p.tiles[job / nt];
    const int expert = __builtin_amdgcn_readfirstlane(t4.x);
    const int first = __builtin_amdgcn_readfirstlane(t4.y);
    const int rows = __builtin_amdgcn_readfirstlane(t4.z);
    const int n0 = (job % nt) * COLS;
    // weights: block j's 32 columns are two 16-row blocks of the layout (N is a
    // multiple of 32); lane (c, h) reads tile 4 kt + 2 m + h of its column
    const int64_t words = static_cast<int64_t>(N) * (K / 8), groups = static_cast<int64_t>(N) * (K / G);
    const uint32_t* wb[2];
    const uint32_t* sb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const MoeWeight& w = UP ? (j == 0 ? p.gate : p.up) : p.down;
        int r0 = n0 + (UP ? 32 * wave : 64 * wave + 32 * j);
        r0 = r0 < N ? r0 : N - 32;                   // (columns past N are not stored)
        r0 += c & 16;
        wb[j] = w.wq + expert * words + static_cast<int64_t>(r0) * (K / 8) + 4 * (c & 15) + 64 * h;
        sb[j] = w.sz + expert * groups + static_cast<int64_t>(r0) * (K / G) + (c & 15);
    }
    struct Regs {
        u32x4_t q[2][2];     // [block][64-k half]
        uint32_t s[2][GS];
    };
    auto load_w = [&](int kt, Regs& r) {
        kt = kb + (kt < KT ? kt : KT - 1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                int t = 4 * kt + 2 * m;
                // (the last tile, where K ends before; its activations are zeros)
                if constexpr (GS > 1) t = t + h < K / 32 ? t : K / 32 - 1 - h;
                r.q[j][m] = *reinterpret_cast<const u32x4_t*>(wb[j] + 64 * t);
            }
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                int gg = GS * kt + g;
                if constexpr (GS > 1) gg = gg < K / G ? gg : K / G - 1;
                r.s[j][g] = sb[j][16 * gg];
            }
        }
    };
    constexpr int kWLoads = 2 * (2 + GS);
    // the first weights need no list of rows
    Regs rr[2];
    load_w(0, rr[0]);
    asm volatile("" ::: "memory");

    if (tid < kRows) {
        const int slot = p.order[first + (tid < rows ? tid : 0)];
        lds_slot[tid] = slot;
        // the row of X, or of h, which is in the order of the rows
        lds_row[tid] = UP ? slot / p.k : first + (tid < rows ? tid : 0);
        if constexpr (UP) lds_weight[tid] = p.weights[slot];
    }
    __syncthreads();

    // activations: load `it` of the wave fills stage rows 4 (4 wave + it) .. + 3,
    // lane l row 4 (4 wave + it) + l / 16 at position l % 16 (rows past the
    // tile's: its first, never stored)
    const u32x4_t a_rsrc = tile_rsrc(UP ? p.X : p.hi, static_cast<uint32_t>((UP ? p.T : p.T * p.k) * K * 2));
    uint32_t a_voff[kDma];
#pragma unroll
    for (int it = 0; it < kDma; ++it) {
        const int r = 4 * (kDma * wave + it) + (lane >> 4);
        a_voff[it] = static_cast<uint32_t>(lds_row[r]) * static_cast<uint32_t>(2 * K) + 16u * ((lane & 15) ^ (r & 15));
    }
    auto dma = [&](int kt, uint8_t* stage) {
        kt = kt < KT ? kt : KT - 1;
        const uint32_t soff = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>((kb + kt) * kStepK * 2));
        typedef __attribute__((address_space(3))) uint8_t lds_u8;
#pragma unroll
        for (int it = 0; it < kDma; ++it) {
            const uint32_t m0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)stage)) +
                                static_cast<uint32_t>((kDma * wave + it) * 1024);
            // (a load to LDS may follow a write of M0 after one wait state; it
            // has no register result, and the wait at a step's start covers it)
            uint32_t voff = a_voff[it];
            // (chunks past K: past the buffer's end, zeros)
            if constexpr (GS > 1) {
                const int r = 4 * (kDma * wave + it) + (lane >> 4);
                if ((kb + kt) * kStepK + 8 * ((lane & 15) ^ (r & 15)) >= K) voff = 0x80000000u;
            }
            asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
                         ::"v"(voff), "s"(a_rsrc), "s"(m0), "s"(soff) : "memory", "m0");
        }
    };

    dma(0, lds_a0);
    dma(1, lds_a1);
    {
        const int r = tid % kRows;
        const float* const from = (UP ? p.x_sums : p.h_sums) + static_cast<int64_t>(lds_row[r]) * (K / G) + kb * GS;
        for (int g = tid / kRows; g < KT * GS; g += kThreads / kRows)
            lds_x1[g * kRows + r] = GS == 1 || kb * GS + g < K / G ? from[g] : 0.0f;
    }

    float16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    const uint32_t bias = opaque_vgpr(kBf16Bias128x2);

    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // code word f of a step's two columns as MFMA operands.  Groups of 32: an MFMA
    // stays inside a tile, half h of the lanes taking its words 2 i + h; a swap of
    // the halves turns the words 2 i and 2 i + 1 of both halves' tiles into those
    // of the one and of the other.
    auto convert = [&](Regs& r, int f, bf16x8_t (&o)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            u32x4_t& q = r.q[j][f >> 2];
            if constexpr (G == 32) {
                if ((f & 3) < 2) {
                    const int i = f & 1;
                    const auto both = __builtin_amdgcn_permlane32_swap(q[2 * i], q[2 * i + 1], false, false);
                    q[2 * i] = both[0];
                    q[2 * i + 1] = both[1];
                }
            }
            // (the first tile's words are now 0 and 2, the second's 1 and 3)
            const uint32_t w = q[G == 32 ? 2 * (f & 1) + ((f >> 1) & 1) : f & 3];
            o[j] = __builtin_bit_cast(bf16x8_t, u32x4_t{nibble_pair_bf16(w, 0, bias), nibble_pair_bf16(w, 1, bias),
                                                        nibble_pair_bf16(w, 2, bias), nibble_pair_bf16(w, 3, bias)});
        }
    };
    // operands of slot f in b[f & 1]; slot 0 of a step is converted in slot 7 of
    // the one before
    bf16x8_t b[2][2];
    convert(rr[0], 0, b[0]);
    auto step = [&](int kt, const uint8_t* A, uint8_t* Ad, Regs& cur, Regs& next) __attribute__((always_inline)) {
        load_w(kt + 1, next);
        asm volatile("" ::: "memory");
        float16_t T[2][2];
        auto frag = [&](int i, int f) {
            const int ch = G == 32 ? 2 * f + h : 8 * (f >> 2) + 4 * h + (f & 3);
            return *reinterpret_cast<const bf16x8_t*>(A + (32 * i + c) * 256 + 16 * (ch ^ (c & 15)));
        };
        // group g's products into the sums.  Register e of lane (c, h): row 8 (e / 4)
        // + 4 h + e % 4 of its block, column c
        auto scale = [&](int g) __attribute__((always_inline)) {
            float sc[2], zc[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sc[j] = half_bits_to_float(cur.s[j][g]);
                zc[j] = 128.0f + half_bits_to_float(cur.s[j][g] >> 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4_t x1 = *reinterpret_cast<const float4_t*>(lds_x1 + (kt * GS + g) * kRows + 32 * i + 8 * r + 4 * h);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 4 * r; e < 4 * r + 4; ++e)
                            acc[i][j][e] = fmaf(sc[j], fmaf(-zc[j], x1[e % 4], T[i][j][e]), acc[i][j][e]);
                    // (with groups of 64 the scheduler would fetch all the sums at
                    // once, and 45 registers would have to go to memory)
                    if constexpr (G == 64)
                        if (r % 2 == 1) __builtin_amdgcn_sched_barrier(0);
                }
        };
        bf16x8_t a[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[0][i] = frag(i, 0);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            if (f > 0 && f % PER == 0) {
                __builtin_amdgcn_sched_barrier(0);
                scale(f / PER - 1);
            }
            // A slot: the fragments of the next one are fetched and its code words
            // converted between this one's MFMAs.
            __builtin_amdgcn_sched_barrier(0);
            if (f < 7) {
#pragma unroll
                for (int i = 0; i < 2; ++i) a[(f + 1) & 1][i] = frag(i, f + 1);
                convert(cur, f + 1, b[(f + 1) & 1]);
            } else {
                convert(next, 0, b[0]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float16_t zero = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                    T[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[f & 1][i], b[f & 1][j], f % PER == 0 ? zero : T[i][j], 0, 0, 0);
                }
            if (f < 7) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // an MFMA
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);          // VALU
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // (behind the use of the next step's first code words: the compiler's wait
        // for those, which does not know these loads, would wait for them as well)
        dma(kt + 2, Ad);
        scale(GS - 1);
        // the next step's activations are in LDS: all loads done but the last
        // step's and this one's weights and activations
        asm volatile("" ::: "memory");
        constexpr int kLeft = kWLoads + kDma;
        __builtin_amdgcn_s_waitcnt((kLeft & 15) | (7 << 4) | ((kLeft >> 4) << 14));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    int kt = 0;
    for (; kt + 6 <= KT; kt += 6) {
        step(kt, lds_a0, lds_a2, rr[0], rr[1]);
        step(kt + 1, lds_a1, lds_a0, rr[1], rr[0]);
        step(kt + 2, lds_a2, lds_a1, rr[0], rr[1]);
        step(kt + 3, lds_a0, lds_a2, rr[1], rr[0]);
        step(kt + 4, lds_a1, lds_a0, rr[0], rr[1]);
        step(kt + 5, lds_a2, lds_a1, rr[1], rr[0]);
    }
    if (kt < KT) step(kt, lds_a0, lds_a2, rr[0], rr[1]);
    if (kt + 1 < KT) step(kt + 1, lds_a1, lds_a0, rr[1], rr[0]);
    if (kt + 2 < KT) step(kt + 2, lds_a2, lds_a1, rr[0], rr[1]);
    if (kt + 3 < KT) step(kt + 3, lds_a0, lds_a2, rr[1], rr[0]);
    if (kt + 4 < KT) step(kt + 4, lds_a1, lds_a0, rr[0], rr[1]);
    __builtin_amdgcn_s_waitcnt(0);                   // nothing is on its way into LDS any more
    asm volatile("" ::: "memory");
    __syncthreads();

    if constexpr (UP) {
        // h through LDS, [row][128] bf16 (chunk ch of row r at ch ^ (r & 15)),
        // out in 16-byte pieces with the rows' sums
        uint16_t* const hl = reinterpret_cast<uint16_t*>(lds_a0);
        const int col = 32 * wave + c;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = 32 * i + 8 * (e / 4) + 4 * h + e % 4;
                const float v = quick_activation(p.act, acc[i][0][e]) * acc[i][1][e] * lds_weight[r];
                hl[r * 128 + 8 * ((col >> 3) ^ (r & 15)) + (col & 7)] = float_to_bf16_bits(v);
            }
        __syncthreads();
        const int r = tid >> 2, part = tid & 3;      // a row's quarter of 32 columns
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(hl + r * 128 + 8 * ((4 * part + b) ^ (r & 15)));
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += bf16_lo(v[e]) + bf16_hi(v[e]);
            if (r < rows && n0 + 32 * part < N) *reinterpret_cast<u32x4_t*>(p.hi + static_cast<int64_t>(first + r) * N + n0 + 32 * part + 8 * b) = v;
        }
        // sums over the groups: one, two or four quarters
        if constexpr (G >= 64) sum += __shfl_xor(sum, 1, kWave);
        if constexpr (G >= 128) sum += __shfl_xor(sum, 2, kWave);
        const int n = n0 + 32 * part;
        if (r < rows && n < N && n % G == 0) p.h_sums[static_cast<int64_t>(first + r) * (N / G) + n / G] = sum;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = 32 * i + 8 * (e / 4) + 4 * h + e % 4;
                if (r >= rows) continue;
                float* const dst = p.part + (z * p.T * p.k + lds_slot[r]) * N;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = n0 + 64 * wave + 32 * j + c;
                    if (n < N) dst[n] = acc[i][j][e];
                }
            }
    }
}

}  // namespace

namespace {
template <int G>
hipError_t launch_tile_g(const MoeParams& p, bool up, unsigned grid, size_t lds, hipStream_t stream) {
    if (up) hipLaunchKernelGGL((moe_tile_kernel<G, true>), dim3(grid), dim3(kThreads), lds, stream, p);
    else hipLaunchKernelGGL((moe_tile_kernel<G, false>), dim3(grid), dim3(kThreads), lds, stream, p);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_moe_tile(const MoeParams& p, bool up, int64_t tiles, hipStream_t stream) {
    const int K = up ? p.H : p.I, N = up ? p.I : p.H, cols = up ? 128 : 256, zs = up ? 1 : p.splits;
    const int64_t grid = tiles * ((N + cols - 1) / cols) * zs;
    const int steps = (K + kStepK - 1) / kStepK;
    const size_t lds = static_cast<size_t>((steps + zs - 1) / zs) * (kStepK / p.G) * kRows * sizeof(float);
    if (N % 32 != 0 || lds > sizeof(float) * kMoeTileSums || grid <= 0 || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    switch (p.G) {
        case 32: return launch_tile_g<32>(p, up, static_cast<unsigned>(grid), lds, stream);
        case 64: return launch_tile_g<64>(p, up, static_cast<unsigned>(grid), lds, stream);
        default: return launch_tile_g<128>(p, up, static_cast<unsigned>(grid), lds, stream);
    }
}

}  // namespace w4
