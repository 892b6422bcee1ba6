// Mixture-of-experts layer over 4-bit experts on gfx950.
//
//   h_j = w_j act(Wg[e_j] X[t]) * (Wu[e_j] X[t])      for the experts e_j of token t
//   Y[t] = bf16(residual[t] + sum_j Wd[e_j] h_j)
//
// With few tokens an expert the layer is bound by streaming the chosen
// experts' packed weights, as the W4A16 products of few rows are.  A slot is
// a (token, choice) pair; the slots are put in order of their expert, so that an
// expert's weights are read once for all of its rows.  Three forms:
//
// - one or two tokens whose rows fit 48 KB of LDS (two slots of inner sizes up to
//   5952, eight up to 1472): each slot by itself on dot products (moe_*_dot_kernel; one
//   token, 8 of 64 experts of 2048 x 1024: 8.0 and 8.6 us, of which the
//   weights' bytes are 5.5 together: launches and the chains of first reads);
// - rows streamed past (moe_stream_kernel): a wave owns 16 columns of one
//   expert's gate and up weight, or 32 of its down weight, and reads them once;
//   the workgroup's waves multiply them by the same 16 MB rows, which lie in
//   LDS.  Lane (c, q) loads the 16 bytes of the 32-k tile 4 s + q of column c
//   (1 KB contiguous in the blocked layout).  24 tokens, 2 of 8 experts of
//   4096 x 14336: 87 to 95 us for the 499 MB of gate and up (5.2 to 5.7 TB/s)
//   and 51 to 59 for the 250 MB of down;
// - from 16 rows an expert, within the widths and sizes of tile_form(), tiles on
//   the matrix cores (moe_tile.hip).
//
// The codes become the exact bf16 values 128 + u; with P the product with them
// and x1 the sum of the activations over a group (an MFMA against ones),
//   acc += s (P - (128 + z) x1)
// is exact in the weights.  Groups of 128: MFMA b takes from every quarter q
// the 8 k at 32 q + 8 b, as the words lie.  Groups of 32 and 64 need MFMAs
// that stay inside a group: the four words of the four quarters are
// transposed (two swaps of 32 lanes and two of 16), after which MFMA t takes
// exactly tile t, quarter q the 8 k at 32 t + 8 q.
//
// h carries the token's weight w_j already.  Where the weights' bytes bound the
// down product it is kept as two bf16 numbers, h = hi + lo (16 bits of
// mantissa), and the product multiplies both: with h rounded to bf16 once the
// result is 1.4 times as far from the exact one as its own rounding to bf16
// leaves it.  (The tiles, which the matrix cores bound, round it once.)
#include "device.hpp"
#include "moe_kernels.hpp"

namespace w4 {
namespace {

// ------------------------------------------------------------------- lists

// Which slots belong together: found by one workgroup, in a launch of its own
// where there are more slots than a wavefront has lanes; with fewer the gate
// and up kernel looks its rows up among the ids, and one more workgroup of it
// makes the lists that the down product needs.

// The slots ordered by expert, and the runs of equal ones: (expert, first, rows)
// of each expert that has any; runs behind the last one have no rows.  (Which place inside an
// expert's run a slot gets is up to the order of the atomics; every row's
// result is the same at any place.)
struct RunMem {
    int count[kMaxExperts];
};
// TILES: the runs cut into tiles instead, for the tiled products.
template <bool TILES>
__device__ __forceinline__ void build_runs(const MoeParams& p, RunMem& m, int tid, int threads) {
    for (int e = tid; e < p.E; e += threads) m.count[e] = 0;
    __syncthreads();
    const int slots = static_cast<int>(p.T * p.k);
    // (four ids a thread in flight)
    auto each = [&](auto take) {
        for (int s0 = tid; s0 < slots; s0 += 4 * threads) {
            uint32_t e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = s0 + i * threads < slots ? static_cast<uint32_t>(p.ids[s0 + i * threads]) : ~0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e[i] < static_cast<uint32_t>(p.E)) take(s0 + i * threads, e[i]);
        }
    };
    each([&](int, uint32_t e) { atomicAdd(&m.count[e], 1); });
    __syncthreads();
    if (tid < kWave) {
        // the first wavefront sums over the experts, 64 at a time
        int rows = 0, active = 0, tiles = 0;
        for (int e0 = 0; e0 < p.E; e0 += kWave) {
            const int e = e0 + tid;
            const int mine = e < p.E ? m.count[e] : 0;
            int upto = mine;
#pragma unroll
            for (int off = 1; off < kWave; off <<= 1) {
                const int o = __shfl_up(upto, off, kWave);
                upto += tid >= off ? o : 0;
            }
            const uint64_t some = __builtin_amdgcn_ballot_w64(mine > 0);
            const int first = rows + upto - mine;
            if (e < p.E) m.count[e] = first;
            if (!TILES && mine > 0) p.runs[active + __builtin_popcountll(some & ((uint64_t{1} << tid) - 1))] = make_int4(e, first, mine, 0);
            if constexpr (TILES) {
                constexpr int kRows = kMoeTileRows;
                const int own = (mine + kRows - 1) / kRows;
                int before = own;
#pragma unroll
                for (int off = 1; off < kWave; off <<= 1) {
                    const int o = __shfl_up(before, off, kWave);
                    before += tid >= off ? o : 0;
                }
                for (int i = 0; i < own; ++i)
                    p.tiles[tiles + before - own + i] =
                        make_int4(e, first + i * kRows, mine - i * kRows < kRows ? mine - i * kRows : kRows, 0);
                tiles += __shfl(before, kWave - 1, kWave);
            }
            rows += __shfl(upto, kWave - 1, kWave);
            active += __builtin_popcountll(some);
        }
        if (TILES && tid == 0) *p.tile_count = tiles;
        if constexpr (!TILES)
            for (int i = active + tid; i < p.E; i += kWave) p.runs[i] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    each([&](int s, uint32_t e) { p.order[atomicAdd(&m.count[e], 1)] = s; });
}

constexpr int kListThreads = 1024;
__global__ void __launch_bounds__(kListThreads) moe_lists_kernel(MoeParams p) {
    __shared__ RunMem mem;
    build_runs<false>(p, mem, threadIdx.x, kListThreads);
}

// For the tiled products: workgroup 0 makes the runs and tiles, the others the
// tokens' row sums over each group (an eighth as many lanes as it has k).
template <int G>
__global__ void __launch_bounds__(kListThreads) moe_tiles_kernel(MoeParams p) {
    constexpr int LANES = G / 8;
    __shared__ RunMem mem;
    if (blockIdx.x == 0) {
        build_runs<true>(p, mem, threadIdx.x, kListThreads);
        return;
    }
    const int64_t i = (static_cast<int64_t>(blockIdx.x - 1) * kListThreads + threadIdx.x) / LANES;
    const int64_t sums = p.T * (p.H / G);
    const u32x4_t v = reinterpret_cast<const u32x4_t*>(p.X)[(i < sums ? i : 0) * LANES + threadIdx.x % LANES];
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += bf16_lo(v[e]) + bf16_hi(v[e]);
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) s += __shfl_xor(s, off, LANES);
    if (i < sums && threadIdx.x % LANES == 0) p.x_sums[i] = s;
}

// ------------------------------------------------------------------ products

constexpr int kStepK = 128;

// 4 x 4 transposition of words over the quarters: w[t] of quarter q becomes
// w[q] of quarter t
__device__ __forceinline__ void transpose_quarters(u32x4_t& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// One 128-k step of up to 16 MB rows by 16 FJ columns; AP parts of every
// activation (hi and lo).  The weights' blocks and the rows are given by
// pointers that already include the lane's column c or row.
template <int FJ, int G>
struct StepB {
    u32x4_t w[FJ];
    uint32_t s[FJ][kStepK / G];
};
// From the blocks' first words: a step's address is uniform, the lane's offset in
// it the same for all steps.  (The step passes through an empty asm: the
// compiler would otherwise keep a pointer of its own in registers for each of the
// loads in flight.)
template <int FJ, int G>
__device__ __forceinline__ void load_b(StepB<FJ, G>& b, const uint32_t* const (&wb)[FJ], const uint32_t* const (&sb)[FJ], int step,
                                       int K, int c, int q) {
    constexpr int NG = kStepK / G;
    step = __builtin_amdgcn_readfirstlane(step);
    asm volatile("" : "+s"(step));
    uint32_t tile = q;
    if constexpr (NG > 1) {
        // K may end inside the last step of groups below 128
        const uint32_t tiles = K / 32 - 4 * step;
        tile = tile < tiles ? tile : tiles - 1;
    }
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        const uint8_t* const w = reinterpret_cast<const uint8_t*>(wb[j]) + static_cast<int64_t>(step) * 1024;
        b.w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(w + (256u * tile + 16u * c)));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            int gg = NG * step + g;
            if constexpr (NG > 1) gg = gg < K / G ? gg : K / G - 1;
            const uint8_t* const s = reinterpret_cast<const uint8_t*>(sb[j]) + static_cast<int64_t>(gg) * 64;
            b.s[j][g] = *reinterpret_cast<const uint32_t*>(s + 4u * c);
        }
    }
}
// `frag(i, v, f)`: fragment f of part v of the rows' block i: the 8 k at 32 q +
// 8 f of the step (groups of 128), or at 32 f + 8 q.  Blocks of rows from
// `blocks` on are left out.
template <int MB, int AP, int FJ, int G, typename Frag>
__device__ __forceinline__ void multiply(float4_t (&acc)[MB][FJ], const StepB<FJ, G>& b, Frag frag, int step, int K, uint32_t bias,
                                         int blocks = MB) {
    constexpr int NG = kStepK / G, PER = 4 / NG;     // groups in a step, fragments in a group
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    u32x4_t word[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        word[j] = b.w[j];
        if constexpr (NG > 1) transpose_quarters(word[j]);
    }
    float4_t ps[MB][FJ], x1[MB];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        // (the scheduler would otherwise fetch fragments ahead until the
        // registers are full, and fewer waves fit a compute unit)
        __builtin_amdgcn_sched_barrier(0);
        if (f % PER == 0) {
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                x1[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < FJ; ++j) ps[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        // K may end inside the last step of groups below 128
        const bool in = NG == 1 || 4 * step + f < K / 32;
        bf16x8_t bp[FJ];
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
            const uint32_t w = word[j][f];
            bp[j] = __builtin_bit_cast(bf16x8_t, u32x4_t{nibble_pair_bf16(w, 0, bias), nibble_pair_bf16(w, 1, bias),
                                                         nibble_pair_bf16(w, 2, bias), nibble_pair_bf16(w, 3, bias)});
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if (MB > 1 && i >= blocks) continue;
#pragma unroll
            for (int v = 0; v < AP; ++v) {
                const u32x4_t x = frag(i, v, f);
                const bf16x8_t ap = __builtin_bit_cast(bf16x8_t, in ? x : zero);
                x1[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ap, ones, x1[i], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < FJ; ++j) ps[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ap, bp[j], ps[i][j], 0, 0, 0);
            }
        }
        if (f % PER == PER - 1) {
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                const uint32_t sz = b.s[j][f / PER];
                const float sc = half_bits_to_float(sz), zc = 128.0f + half_bits_to_float(sz >> 16);
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(sc, fmaf(-zc, x1[i][e], ps[i][j][e]), acc[i][j][e]);
            }
        }
    }
}

// h as two bf16 numbers (an infinite upper part has no rest)
__device__ __forceinline__ void store_h(const MoeParams& p, int64_t at, float h) {
    const uint16_t hi = float_to_bf16_bits(h);
    p.hi[at] = hi;
    p.lo[at] = (hi & 0x7FFFu) == 0x7F80u ? 0 : float_to_bf16_bits(h - bf16_lo(hi));
}

// UP: gate and up (block 0 of the gate weight, block 1 of the up weight, at the
// same 16 columns), rows gathered from X; else the down product on the rows
// hi + lo.  SCAN (UP only, at most 64 slots): the expert's rows from the ids,
// with blockIdx.y the expert or, where there are fewer slots than experts, a
// slot, whose expert it takes if no slot before has the same; the last
// blockIdx.y makes the lists for the kernels behind.
//
// A wave streams the weights of its own columns, two 128-k steps ahead, and all
// of the workgroup's waves multiply them by the same rows, which go straight from
// global memory into LDS a piece of CS steps ahead (waves that split the k
// instead read the rows from L2 for every 32 columns anew, four times the bytes
// of the weights: 8 experts of 14336 x 4096, 24 tokens, down product 78 us).
// With blockIdx.z an expert's blocks of 16 MB rows are dealt out to `rs`
// workgroups, and the down product's k are split over others.
template <int MB, int G, bool UP, bool SCAN>
__global__ void __launch_bounds__(512, 2) moe_stream_kernel(MoeParams p, int rs) {
    static_assert(UP || !SCAN, "the lists are made by then");
    constexpr int FJ = 2, NG = kStepK / G;
    constexpr int AP = UP ? 1 : 2;                 // parts of an activation
    constexpr int RM = 16 * MB;                    // rows at a time
    // steps of weights in flight, and steps of a piece of the rows: with two of
    // each, 16 rows at a time in groups of 128 and 64 take 92 to 114 registers, so
    // that two workgroups of 8 waves share a compute unit and cover each other's
    // waits (four of each, groups of 128: 138 registers and 64 KB of LDS, one
    // workgroup, down products 5 to 10 us slower).  Groups of 32 take 140 and 148,
    // one workgroup: four words of scales a column and step, and the transposed
    // codes.  32 rows at a time have one workgroup in any case (148 to 202
    // registers), in groups of 32 with 38 to 43 of 256 in memory.  33 tokens, 8 of
    // 128 experts of 2048 x 768, up and down product: groups of 128 39 and 25 us,
    // of 64 46 and 31, of 32 64 and 43.
    constexpr int DEPTH = 2;
    constexpr int CS = 2;
    constexpr int ROW = CS * kStepK * 2;           // its bytes in a row
    constexpr int RPD = 1024 / ROW;                // rows of a load to LDS
    constexpr int LOADS = FJ * (1 + NG);           // loads of one
    constexpr int COLS = UP ? 16 : 32;             // columns of a wave
    static_assert(CS * LOADS < 64, "vmcnt range");
    __shared__ __attribute__((aligned(16))) uint8_t lds_a[2][AP * RM * ROW];
    __shared__ int row_at[RM];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    int expert, rows;
    const int* list;
    __shared__ int scanned[SCAN ? kWave : 1];
    if constexpr (SCAN) {
        const int slots = static_cast<int>(p.T * p.k);
        if (blockIdx.y == gridDim.y - 1) {
            if (blockIdx.x > 0 || blockIdx.z > 0) return;
            __shared__ RunMem mem;
            build_runs<false>(p, mem, tid, blockDim.x);
            return;
        }
        const int id = lane < slots ? p.ids[lane] : -1;
        expert = __builtin_amdgcn_readfirstlane(slots < p.E ? __builtin_amdgcn_readlane(id, blockIdx.y) : static_cast<int>(blockIdx.y));
        if (static_cast<uint32_t>(expert) >= static_cast<uint32_t>(p.E)) return;
        const uint64_t some = __builtin_amdgcn_ballot_w64(id == expert);
        rows = __builtin_popcountll(some);
        if (rows == 0 || (slots < p.E && __builtin_ctzll(some) < static_cast<int>(blockIdx.y))) return;
        // every wavefront writes the same list and reads what it wrote
        if (id == expert) scanned[__builtin_popcountll(some & ((uint64_t{1} << lane) - 1))] = lane;
        list = scanned;
    } else {
        const int4 run = p.runs[blockIdx.y];
        expert = __builtin_amdgcn_readfirstlane(run.x);
        rows = __builtin_amdgcn_readfirstlane(run.z);
        if (rows == 0) return;
        list = p.order + __builtin_amdgcn_readfirstlane(run.y);
    }
    const int K = UP ? p.H : p.I, N = UP ? p.I : p.H;
    const int KS = (K + kStepK - 1) / kStepK;
    const int z = blockIdx.z / rs, zs = gridDim.z / rs;
    const int first = z * KS / zs, n = (z + 1) * KS / zs - first;    // the workgroup's steps
    const int n0 = COLS * (blockIdx.x * waves + wave);
    const int64_t words = static_cast<int64_t>(N) * (K / 8), groups = static_cast<int64_t>(N) * (K / G);

    // the blocks' first words; N is a multiple of 32, so every block has 16
    // rows (a wave past N repeats the last columns and stores nothing)
    const uint32_t* wb[FJ];
    const uint32_t* sb[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        const MoeWeight& w = UP ? (j == 0 ? p.gate : p.up) : p.down;
        const int r0 = (n0 < N ? n0 : N - COLS) + (UP ? 0 : 16 * j);
        wb[j] = w.wq + expert * words + static_cast<int64_t>(r0) * (K / 8);
        sb[j] = w.sz + expert * groups + static_cast<int64_t>(r0) * (K / G);
    }
    const uint32_t bias = opaque_vgpr(kBf16Bias128x2);
    StepB<FJ, G> b[DEPTH];
    auto load = [&](int i, int d) { load_b<FJ, G>(b[d], wb, sb, first + i, K, c, q); };

    for (int m0 = RM * (blockIdx.z % rs); m0 < rows; m0 += RM * rs) {
        const int some = rows - m0 < RM ? rows - m0 : RM;
        // the first steps' weights need no list; the rows of m0 in LDS
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (d < n) load(d, d);
        __syncthreads();                            // (the rows before are multiplied)
        if (tid < some) {
            const int slot = list[m0 + tid];
            row_at[tid] = UP ? slot / p.k : slot;
        }
        __syncthreads();
        // piece j of the rows (its steps first + CS j ..): 16-byte chunk ch of
        // row r at ch ^ (r & 15); a lane past K reads the row's last chunk, which
        // meets zeros or nothing
        auto dma = [&](int j) {
            const int per = (some + RPD - 1) / RPD;          // loads of one part
            for (int d = wave; d < AP * per; d += waves) {
                const int v = d / per, r0 = d % per * RPD;
                int r = r0 + lane / (ROW / 16);
                const int ch = (lane % (ROW / 16)) ^ (r & 15);
                r = r < some ? r : some - 1;
                int k = (first + CS * j) * kStepK + 8 * ch;
                k = k < K ? k : K - 8;
                const uint16_t* const from = (UP ? p.X : v == 0 ? p.hi : p.lo) + static_cast<int64_t>(row_at[r]) * K + k;
                typedef __attribute__((address_space(3))) uint8_t lds_u8;
                const uint32_t m0_ = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
                    reinterpret_cast<uintptr_t>((lds_u8*)(lds_a[j & 1] + (v * RM + r0) * ROW))));
                asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(m0_) : "memory", "m0");
            }
        };
        dma(0);
        const int blocks = (some + 15) / 16;
        // where the lane's fragment f lies in a step of its row in each block (past
        // the last row: the last): f moves it among the step's 16 chunks only
        uint32_t at[MB][4];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int r = 16 * i + c < some ? 16 * i + c : some - 1;
#pragma unroll
            for (int f = 0; f < 4; ++f) at[i][f] = static_cast<uint32_t>(r * ROW + 16 * ((NG == 1 ? 4 * q + f : 4 * f + q) ^ (r & 15)));
        }
        float4_t acc[MB][FJ];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        // The piece that step i begins is in LDS for all waves, and the next one on
        // its way.  `all`: the CS steps before it were whole, each with its load of
        // weights, so exactly kBehind = CS LOADS loads of this wave came behind the
        // piece's own, and as they end in order, waiting until no more than those are
        // under way is enough.  That rests on load_b's FJ (1 + NG) loads a step: with
        // fewer the wait would be over before the piece is there (more, and what the
        // compiler adds, only make it longer).  Before the first step no load came
        // behind the piece, and in the last steps fewer than kBehind do: then all are
        // waited for.
        auto piece = [&](int i, bool all) {
            asm volatile("" ::: "memory");
            constexpr int kBehind = CS * LOADS;
            if (all) __builtin_amdgcn_s_waitcnt((kBehind & 15) | (7 << 4) | (0 << 8) | ((kBehind >> 4) << 14));
            else __builtin_amdgcn_s_waitcnt(0);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (i + CS < n) dma(i / CS + 1);
        };
        auto one = [&](int i, int s) {
            const uint8_t* const from = lds_a[(i / CS) & 1];
            multiply<MB, AP, FJ, G>(
                acc, b[s],
                [&](int rb, int v, int f) {
                    return *reinterpret_cast<const u32x4_t*>(from + at[rb][f] + (v * (RM * ROW) + 256 * (s % CS)));
                },
                first + i, K, bias, blocks);
        };
        int i = 0;
        // whole groups of DEPTH steps whose refills are all real: no branch
        // around a load, so that a step waits for its own weights only
        for (; i + 2 * DEPTH <= n; i += DEPTH) {
#pragma unroll
            for (int s = 0; s < DEPTH; ++s) {
                // (before the first group nothing was issued behind its piece)
                if (s % CS == 0) piece(i + s, i + s >= CS);
                one(i + s, s);
                load(i + DEPTH + s, s);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        for (; i < n; i += DEPTH) {
#pragma unroll
            for (int s = 0; s < DEPTH; ++s) {
                if (i + s < n) {
                    if (s % CS == 0) piece(i + s, false);
                    one(i + s, s);
                    if (i + DEPTH + s < n) load(i + DEPTH + s, s);
                }
            }
        }

        // register e of lane (c, q): row 4 q + e of its block, column c
        if (n0 >= N) continue;
#pragma unroll
        for (int rb = 0; rb < MB; ++rb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * rb + 4 * q + e;
                if (r >= some) continue;
                const int slot = UP ? list[m0 + r] : row_at[r];
                const int64_t at = static_cast<int64_t>(slot) * N + n0 + c;
                if constexpr (UP) {
                    store_h(p, at, activation(p.act, acc[rb][0][e]) * acc[rb][1][e] * p.weights[slot]);
                } else {
                    float* const dst = p.part + z * p.T * p.k * N + at;
                    dst[0] = acc[rb][0][e];
                    dst[16] = acc[rb][1][e];
                }
            }
    }
}

// One or two tokens: every slot by itself (against streaming, one token: 8 of 64
// experts of 2048 x 1024 15.7 and 25.6 us, 2 of 8 of 576 x 1536 9.7 and 15.6;
// two tokens: 30.7 and 31.0, 12.1 and 16.0).  The matrix cores would multiply 16
// rows where there is one, and each wave would load every row 16 times over;
// here the rows lie in LDS, each lane multiplies the 32 codes it loads by the 32
// activations of its tile (v_dot2_f32_bf16 on the exact 128 + u), and the
// group's scale and zero point are applied per lane, whose 32 k lie in one group
// of any size.
constexpr int kDotTokens = 2;
// bf16 pairs of a row and the sums of its tiles, in LDS words
constexpr int dot_words(int K, int parts) { return parts * (K / 2) + K / 32; }
constexpr int kDotWords = 12288;                   // most of them: 48 KB

// a tile's 32 products: the codes of one lane against `x` (16 words, 16 more of
// the second part), whose sum is xs
template <int AP>
__device__ __forceinline__ float dot_tile(const u32x4_t& w, uint32_t sz, const uint32_t* hi, const uint32_t* lo, float xs, uint32_t bias) {
    const float sc = half_bits_to_float(sz), zc = 128.0f + half_bits_to_float(sz >> 16);
    float d[2] = {-zc * xs, 0.0f};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const u32x4_t h = *reinterpret_cast<const u32x4_t*>(hi + 4 * b);
        u32x4_t l = {0u, 0u, 0u, 0u};
        if constexpr (AP == 2) l = *reinterpret_cast<const u32x4_t*>(lo + 4 * b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t pr = nibble_pair_bf16(w[b], i, bias);
            d[0] = dot2_bf16(pr, h[i], d[0]);
            if constexpr (AP == 2) d[1] = dot2_bf16(pr, l[i], d[1]);
        }
    }
    return sc * (d[0] + d[1]);
}
// tile t of a row into LDS: its 32 values as they are, and their sum
__device__ __forceinline__ float put_tile(uint32_t* to, const u32x4_t (&v)[4]) {
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        *reinterpret_cast<u32x4_t*>(to + 4 * b) = v[b];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[b] = dot2_bf16(v[b][i], 0x3F803F80u, sum[b]);
    }
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ void __launch_bounds__(512) moe_up_dot_kernel(MoeParams p, int wk) {
    constexpr int DEPTH = 4;
    extern __shared__ uint32_t x_lds[];            // the row's pairs, then its tiles' sums
    __shared__ float red[8][32];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int slot = blockIdx.y, n0 = 16 * blockIdx.x;
    const int expert = p.ids[slot];
    const float weight = p.weights[slot];
    const int K = p.H, N = p.I, KQ = K / 32, KS = (KQ + 3) / 4;
    const u32x4_t* const x = reinterpret_cast<const u32x4_t*>(p.X + static_cast<int64_t>(slot / p.k) * K);
    float* const xs = reinterpret_cast<float*>(x_lds + K / 2);
    u32x4_t xv[4];
    if (tid < KQ) {
#pragma unroll
        for (int b = 0; b < 4; ++b) xv[b] = x[4 * tid + b];
    }
    if (static_cast<uint32_t>(expert) >= static_cast<uint32_t>(p.E)) return;
    const int64_t words = static_cast<int64_t>(N) * (K / 8), groups = static_cast<int64_t>(N) * (K / p.G);
    const int per = p.G / 32;                      // tiles of a group
    const uint32_t* wb[2];
    const uint32_t* sb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const MoeWeight& w = j == 0 ? p.gate : p.up;
        wb[j] = w.wq + expert * words + static_cast<int64_t>(n0) * (K / 8) + 4 * c;
        sb[j] = w.sz + expert * groups + static_cast<int64_t>(n0) * (K / p.G) + c;
    }
    u32x4_t w[DEPTH][2];
    uint32_t sz[DEPTH][2];
    auto load = [&](int step, int d) {
        int t = 4 * step + q;
        t = t < KQ ? t : KQ - 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[d][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wb[j] + 64 * t));
            sz[d][j] = sb[j][16 * (t / per)];
        }
    };
    // the first steps' weights are on their way while the row is put into LDS
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(wave + d * wk, d);
    asm volatile("" ::: "memory");
    if (tid < KQ) xs[tid] = put_tile(x_lds + 16 * tid, xv);
    for (int t = tid + blockDim.x; t < KQ; t += blockDim.x) {
#pragma unroll
        for (int b = 0; b < 4; ++b) xv[b] = x[4 * t + b];
        xs[t] = put_tile(x_lds + 16 * t, xv);
    }
    __syncthreads();
    const uint32_t bias = opaque_vgpr(kBf16Bias128x2);
    float acc[2] = {0.0f, 0.0f};
    for (int step = wave; step < KS; step += DEPTH * wk) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int t = 4 * (step + d * wk) + q;
            if (t < KQ)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j] += dot_tile<1>(w[d][j], sz[d][j], x_lds + 16 * t, nullptr, xs[t], bias);
            load(step + (DEPTH + d) * wk, d);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        acc[j] += __shfl_xor(acc[j], 16, kWave);
        acc[j] += __shfl_xor(acc[j], 32, kWave);
        if (q == 0) red[wave][16 * j + c] = acc[j];
    }
    __syncthreads();
    if (tid < 16) {
        float g = 0.0f, u = 0.0f;
        for (int v = 0; v < wk; ++v) {
            g += red[v][tid];
            u += red[v][16 + tid];
        }
        store_h(p, static_cast<int64_t>(slot) * N + n0 + tid, activation(p.act, g) * u * weight);
    }
}

// The waves take equal runs of the (slot, step) pairs.
__global__ void __launch_bounds__(1024) moe_down_dot_kernel(MoeParams p, int wk) {
    constexpr int DEPTH = 4;
    extern __shared__ uint32_t h_lds[];            // [slot] pairs of hi, then of lo; then [slot] the tiles' sums
    __shared__ float red[16][kDotTokens][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int n0 = 16 * blockIdx.x;
    const int K = p.I, N = p.H, KQ = K / 32, KS = (KQ + 3) / 4;
    const int T = static_cast<int>(p.T), slots = T * p.k, tiles = slots * KQ;
    float* const hs = reinterpret_cast<float*>(h_lds + slots * K);
    // lane s: slot s's expert
    const int ids = lane < slots ? p.ids[lane] : -1;
    const int64_t words = static_cast<int64_t>(N) * (K / 8), groups = static_cast<int64_t>(N) * (K / p.G);
    const int per = p.G / 32;
    const int all = slots * KS, begin = all * wave / wk, end = all * (wave + 1) / wk;
    u32x4_t w[DEPTH];
    uint32_t sz[DEPTH];
    int where[DEPTH];                              // slot and step of the codes in flight, -1: none
    int slot = begin / KS, step = begin % KS;
    auto load = [&](int at, int d) {
        where[d] = -1;
        if (at >= end) return;
        const int expert = __builtin_amdgcn_readlane(ids, slot);
        if (static_cast<uint32_t>(expert) < static_cast<uint32_t>(p.E)) {
            where[d] = slot << 16 | step;
            int t = 4 * step + q;
            t = t < KQ ? t : KQ - 1;
            w[d] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(
                p.down.wq + expert * words + static_cast<int64_t>(n0) * (K / 8) + 4 * c + 64 * t));
            sz[d] = p.down.sz[expert * groups + static_cast<int64_t>(n0) * (K / p.G) + c + 16 * (t / per)];
        }
        if (++step == KS) {
            step = 0;
            ++slot;
        }
    };
    // h's first tiles, then the first steps' weights
    u32x4_t hv[2][4];
    auto take = [&](int i) {
        const int64_t at = static_cast<int64_t>(i) * 4;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            hv[0][b] = reinterpret_cast<const u32x4_t*>(p.hi)[at + b];
            hv[1][b] = reinterpret_cast<const u32x4_t*>(p.lo)[at + b];
        }
    };
    auto put = [&](int i) {
        // (rows of slots without an expert hold whatever was there; nothing reads them)
        const int s = i / KQ, t = i % KQ;
        uint32_t* const to = h_lds + s * K + 16 * t;
        hs[i] = put_tile(to, hv[0]) + put_tile(to + K / 2, hv[1]);
    };
    if (tid < tiles) take(tid);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(begin + d, d);
    float first = 0.0f;
    if (p.residual && tid < 16 * T) first = bf16_lo(p.residual[static_cast<int64_t>(tid / 16) * N + n0 + tid % 16]);
    asm volatile("" ::: "memory");
    if (tid < tiles) put(tid);
    for (int i = tid + blockDim.x; i < tiles; i += blockDim.x) {
        take(i);
        put(i);
    }
    __syncthreads();
    const uint32_t bias = opaque_vgpr(kBf16Bias128x2);
    float acc[kDotTokens] = {0.0f, 0.0f};
    for (int at = begin; at < end; at += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (where[d] >= 0) {
                const int s = where[d] >> 16, t = 4 * (where[d] & 0xFFFF) + q;
                float y = 0.0f;
                if (t < KQ) {
                    const uint32_t* const h = h_lds + s * K + 16 * t;
                    y = dot_tile<2>(w[d], sz[d], h, h + K / 2, hs[s * KQ + t], bias);
                }
                if (s < p.k) acc[0] += y;
                else acc[1] += y;
            }
            load(at + DEPTH + d, d);
        }
    }
#pragma unroll
    for (int t = 0; t < kDotTokens; ++t) {
        acc[t] += __shfl_xor(acc[t], 16, kWave);
        acc[t] += __shfl_xor(acc[t], 32, kWave);
        if (q == 0) red[wave][t][c] = acc[t];
    }
    __syncthreads();
    if (tid < 16 * T) {
        float y = 0.0f;
        for (int v = 0; v < wk; ++v) y += red[v][tid / 16][tid % 16];
        p.Y[static_cast<int64_t>(tid / 16) * N + n0 + tid % 16] = float_to_bf16_bits(y + first);
    }
}

// Y = bf16(residual + the slots' shares in the order of the choices), four
// columns a thread.  A launch has fewer than 2^32 threads (the runtime starts
// only what is left of a larger number, without an error), and a million tokens
// may have more columns than that: `turn` is which 2^30 threads these are.
constexpr int64_t kJoinThreads = int64_t{1} << 30;
__global__ void __launch_bounds__(256) moe_join_kernel(MoeParams p, int turn) {
    const int per = p.H / 4;
    const int64_t i = kJoinThreads * turn + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.T * per) return;
    const int64_t t = i / per;
    const int n = static_cast<int>(i % per) * 4;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x2_t r = {0u, 0u};
    if (p.residual) r = *reinterpret_cast<const u32x2_t*>(p.residual + t * p.H + n);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        // eight choices' shares in flight; one that is no expert has none
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int64_t slot = t * p.k + j0 + j;
            if (j0 + j < p.k && static_cast<uint32_t>(p.ids[slot]) < static_cast<uint32_t>(p.E)) {
                v[j] = *reinterpret_cast<const float4*>(p.part + slot * p.H + n);
                for (int z = 1; z < p.splits; ++z) {
                    const float4 u = *reinterpret_cast<const float4*>(p.part + (z * p.T * p.k + slot) * p.H + n);
                    v[j].x += u.x;
                    v[j].y += u.y;
                    v[j].z += u.z;
                    v[j].w += u.w;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[0] += v[j].x;
            y[1] += v[j].y;
            y[2] += v[j].z;
            y[3] += v[j].w;
        }
    }
    y[0] += bf16_lo(r[0]);
    y[1] += bf16_hi(r[0]);
    y[2] += bf16_lo(r[1]);
    y[3] += bf16_hi(r[1]);
    *reinterpret_cast<u32x2_t*>(p.Y + t * p.H + n) = u32x2_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

// Waves of a workgroup: as many columns as give two workgroups a compute unit,
// from 8 waves down to 2.
int stream_waves(int64_t columns, int per_wave, int64_t experts) {
    int w = 8;
    while (w > 2 && (columns + w * per_wave - 1) / (w * per_wave) * experts < 512) w /= 2;
    return w;
}
template <int MB, int G, bool UP>
hipError_t launch_stream(const MoeParams& p, int rs, hipStream_t stream) {
    const int N = UP ? p.I : p.H, per = UP ? 16 : 32;
    const int64_t slots = p.T * p.k, experts = slots < p.E ? slots : p.E;
    const int w = stream_waves(N, per, experts * rs * (UP ? 1 : p.splits));
    dim3 grid(static_cast<unsigned>((N + w * per - 1) / (w * per)), static_cast<unsigned>(experts),
              static_cast<unsigned>(rs * (UP ? 1 : p.splits)));
    const dim3 block(static_cast<unsigned>(64 * w));
    if constexpr (UP) {
        if (slots <= kWave) {
            grid.y += 1;
            hipLaunchKernelGGL((moe_stream_kernel<MB, G, true, true>), grid, block, 0, stream, p, rs);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((moe_stream_kernel<MB, G, UP, false>), grid, block, 0, stream, p, rs);
    return hipGetLastError();
}

// one or two tokens, their rows within LDS
bool dot_form(const MoeParams& p) {
    const int64_t slots = p.T * p.k;
    return p.T <= kDotTokens && slots <= kWave && dot_words(p.H, 1) <= kDotWords && slots * dot_words(p.I, 2) <= kDotWords;
}
hipError_t launch_dot(const MoeParams& p, hipStream_t stream) {
    const int slots = static_cast<int>(p.T * p.k);
    const int up_steps = (p.H + kStepK - 1) / kStepK;
    int wk = up_steps < 8 ? up_steps : 8;
    hipLaunchKernelGGL(moe_up_dot_kernel, dim3(static_cast<unsigned>(p.I / 16), static_cast<unsigned>(slots)),
                       dim3(static_cast<unsigned>(64 * wk)), 4 * dot_words(p.H, 1), stream, p, wk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    wk = slots * ((p.I + kStepK - 1) / kStepK);
    wk = wk > 16 ? 16 : wk;
    hipLaunchKernelGGL(moe_down_dot_kernel, dim3(static_cast<unsigned>(p.H / 16)), dim3(static_cast<unsigned>(64 * wk)),
                       4 * slots * dot_words(p.I, 2), stream, p, wk);
    return hipGetLastError();
}

// The rows of an expert in tiles on the matrix cores (moe_tile.hip), where an
// expert has enough of them, all row sums of a tile fit its LDS (widths up to 8192
// in groups of 32, 16384 of 64, 32768 of 128), and the offsets of all rows fit 31
// bits.  Beyond these limits the streamed form takes any number of rows: 2048
// tokens, 2 of 8 experts of 4096 x 14336, groups of 32, 6.1 + 4.2 ms, 38 to 43
// registers of a lane in memory, where the tiles of groups of 128 take 1.08 + 0.60
// (the whole call 10.3 and 1.64, in groups of 64 2.34); 65536 tokens, 8 of 128 of 2048 x 768, 17.5 ms.  Tiles against streaming, 64 experts of 2048 x
// 1024: 8 rows an expert 82 and 60 us, 16 rows 75 and 86, 32 rows 76 and 137;
// groups of 64, 16 rows 91 and 97; 8 experts of 4096 x 14336: 15 rows 227 and
// 227, 25 rows 215 and 270.
constexpr int64_t kTileFrom = 16;
int64_t tile_count(const MoeParams& p) {
    const int64_t slots = p.T * p.k;
    return slots / kMoeTileRows + (slots < p.E ? slots : p.E);
}
bool tile_form(const MoeParams& p) {
    // (the activations are addressed with 31-bit byte offsets)
    constexpr int64_t kMost = (int64_t{1} << 31) - 1;
    const int64_t slots = p.T * p.k, wide = p.H > p.I ? p.H : p.I;
    return slots > kWave && slots >= kTileFrom * p.E &&
           (wide + 127) / 128 * (128 / p.G) * kMoeTileRows <= kMoeTileSums && 2 * slots * wide <= kMost;
}
template <int G>
hipError_t launch_tiles(const MoeParams& p, hipStream_t stream) {
    const int64_t lanes = p.T * (p.H / 8);
    hipLaunchKernelGGL((moe_tiles_kernel<G>), dim3(static_cast<unsigned>(1 + (lanes + kListThreads - 1) / kListThreads)),
                       dim3(kListThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_moe_tile(p, true, tile_count(p), stream);
    return e != hipSuccess ? e : launch_moe_tile(p, false, tile_count(p), stream);
}

hipError_t launch_join(const MoeParams& p, hipStream_t stream) {
    int turn = 0;
    for (int64_t left = p.T * (p.H / 4); left > 0; left -= kJoinThreads) {
        const int64_t threads = left < kJoinThreads ? left : kJoinThreads;
        hipLaunchKernelGGL(moe_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, stream, p, turn++);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// K ranges of the down product, towards two workgroups of 256 columns a compute
// unit, each of at least two steps (`parts`: experts, or tiles; of at least eight,
// 14 tokens on 4 experts of 576 x 1536, groups of 32: 50 us in place of 30)
int down_splits(const MoeParams& p, int64_t parts) {
    int64_t z = 512 / ((p.H + 255) / 256 * parts);
    if (z > p.I / kStepK / 2) z = p.I / kStepK / 2;
    return z < 1 ? 1 : (z > 8 ? 8 : static_cast<int>(z));
}

template <int G>
hipError_t launch_moe_g(const MoeParams& p, hipStream_t stream) {
    const int64_t slots = p.T * p.k;
    hipError_t e;
    if (tile_form(p)) {
        e = launch_tiles<G>(p, stream);
        return e != hipSuccess ? e : launch_join(p, stream);
    }
    if (slots > kWave) {
        hipLaunchKernelGGL(moe_lists_kernel, dim3(1), dim3(kListThreads), 0, stream, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // an expert's rows, were the choices even: 16 at a time, or 32 (each read of
    // the weights then serves twice as many; 8 experts of 4096 x 14336: 10 rows an
    // expert 164 us with 16 at a time, 191 with 32, 15 rows 221 and 220, 20 rows
    // 297 and 233; 64 experts of 2048 x 1024: 12 rows 79 and 81, 16 rows 90 and 83)
    // Where gate and up have fewer waves than two a SIMD, 16 rows at a time, the
    // next ones in workgroups beside them: the time is then that of one wave's
    // steps, not of the weights' bytes (51 tokens, 3 of 12 experts of 2048 x 768,
    // groups of 32: 43 us in place of 76; 150 tokens, 2 of 24, groups of 128: 36
    // in place of 46).  One workgroup for each 8 rows of the mean, since the
    // choices are not even.
    const int64_t experts = slots < p.E ? slots : p.E;
    const bool narrow = experts * (p.I / 16) <= 2048;
    const bool few = narrow || slots <= 12 * static_cast<int64_t>(p.E);
    const int64_t rows = (slots + 8 * p.E - 1) / (8 * p.E);
    const int rs = !narrow ? 1 : (rows > 4 ? 4 : static_cast<int>(rows));
    e = few ? launch_stream<1, G, true>(p, rs, stream) : launch_stream<2, G, true>(p, rs, stream);
    if (e != hipSuccess) return e;
    e = few ? launch_stream<1, G, false>(p, rs, stream) : launch_stream<2, G, false>(p, rs, stream);
    if (e != hipSuccess) return e;
    return launch_join(p, stream);
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
    const bool dot = dot_form(p), tile = !dot && tile_form(p);
    p.hi = static_cast<uint16_t*>(take(2 * slots * p.I));
    if (!tile) p.lo = static_cast<uint16_t*>(take(2 * slots * p.I));
    if (dot) return at;
    p.order = static_cast<int32_t*>(take(4 * slots));
    const int64_t experts = static_cast<int64_t>(slots) < p.E ? slots : p.E;
    p.splits = down_splits(p, tile ? static_cast<int64_t>(slots) / kMoeTileRows + experts / 2 : experts);
    p.part = static_cast<float*>(take(4 * slots * p.H * p.splits));
    if (tile) {
        p.tiles = static_cast<int4*>(take(16 * tile_count(p)));
        p.tile_count = static_cast<int32_t*>(take(4));
        p.x_sums = static_cast<float*>(take(4 * p.T * (p.H / p.G)));
        p.h_sums = static_cast<float*>(take(4 * slots * (p.I / p.G)));
    } else {
        p.runs = static_cast<int4*>(take(16 * p.E));
    }
    return at;
}

hipError_t launch_moe(const MoeParams& p, hipStream_t stream) {
    if (dot_form(p)) return launch_dot(p, stream);
    switch (p.G) {
        case 32: return launch_moe_g<32>(p, stream);
        case 64: return launch_moe_g<64>(p, stream);
        default: return launch_moe_g<128>(p, stream);
    }
}

}  // namespace w4
