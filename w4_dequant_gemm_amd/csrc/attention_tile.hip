// Attention on many rows: a (sequence, KV head)'s nodes times its query heads.
//
// Both products on v_mfma_f32_32x32x16_bf16, transposed as in attention.hip:
//   S^T [32 tokens x 32 rows] = K Q^T,   O^T [32 dims x 32 rows] += V^T P^T,
// a row being a column of both.  A result holds row l % 32 in lane l and, in
// register r, index 8 (r / 4) + 4 h + r % 4 (h = l / 32); an operand holds 8
// values of the summed index in half h.  The tokens of K's rows are chosen so
// that half h's scores are the tokens of the V pieces it multiplies:
//   bf16: V's pieces hold 8 tokens, register r is token 16 (r / 8) + 8 h + r % 8;
//   E4M3: V's pieces hold 16 tokens, register r is token 16 h + r.
//
// A wave has 32 rows and takes 64 tokens at a time.  The tokens' pieces go from
// the cache straight to shared memory, in the order in which the operands are
// read (one linear 1 KB a piece and wavefront: no bank is asked twice), the
// next 64 tokens' while the present ones are used, one barrier a stage.  (128
// tokens a stage would halve the barriers but hold one workgroup a compute unit;
// 32 tokens: 16 trees of 60 nodes, 4000 tokens 163 us against 124.)
//
// A stage is 1100 cycles of products and 930 of VALU work a wave (32 exponentials
// of 16 cycles); two waves a SIMD keep MFMA 39 to 46 % and VALU 40 % busy, at 1.5
// to 1.6 GHz (2.0 where memory bounds).  Arranging the work otherwise changes
// nothing measurable: one unit's products interleaved with the other's
// exponentials inside a wave, long sequences first or paired with short ones, a
// higher priority in the products (all within 2 %).  Multiplying the next unit
// beside the exponentials of the present one, or 64 rows
// a wave, needs more than 256 registers and was slower (chunk of 777 tokens at the
// end of 6000: 430 to 510 us).  Measured (64 or 32 heads on 8 of 128):
//   16 trees of 40 to 60 nodes, 2000 to 4000 tokens, bf16   112 .. 124 us, 590 .. 650 TFLOP/s
//   3 chunks of 518 to 777, 3000 to 6000 tokens, bf16        212 .. 221 us, 800 .. 830 TFLOP/s
//   8 tokens after 131000, E4M3 (WK = 2, 64 splits)          65 .. 68 us with the join, 4.0 TB/s
// against 1230 TFLOP/s of a large library product.
#include <type_traits>

#include "attention.hpp"

namespace w4 {
namespace {
using namespace attn;

__device__ __forceinline__ float16_t mfma32(const uint4& a, const uint4& b, const float16_t& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ float16_t zero16() {
    float16_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.0f;
    return z;
}
__device__ __forceinline__ float max_halves(float x) {
    const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

constexpr int kTableBlocks = 1024;           // 16-token blocks looked up at a time

// WK = 2: 64 rows a workgroup, and the waves of its two halves take one unit of
// a stage each; their sums are joined at the end.
template <int D, int E, int WK>
__global__ void __launch_bounds__(256, 2) attention_tile_kernel(AttentionParams p, AttentionPlan pl) {
    constexpr int U = 2;                     // units of 32 tokens a stage
    constexpr int UW = U / WK;               // units of a stage that a wave takes
    constexpr int ROWS = 128 / WK;
    constexpr int KS = D / 16;               // operands of K, a unit
    constexpr int DB = D / 32;
    constexpr int KC = D * E / 32;           // 1 KB pieces of K, and of V, a unit
    constexpr int STAGE = 2 * U * KC;
    constexpr int MINE = STAGE / 4;          // pieces a wave loads
    static_assert(MINE == KC, "a wave loads K's pieces or V's of one unit");
    __shared__ __attribute__((aligned(16))) uint4 ring[2 * STAGE * 64];
    __shared__ int blocks[kTableBlocks];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 31, h = lane >> 5;
    const int hk = p.cache.heads, pb = p.cache.page_blocks;
    // the tiles of one (split, head, sequence) on one XCD, which then reads its tokens once
    const int xcd = blockIdx.x & 7;
    const int turn = blockIdx.x >> 3;
    const int tile = turn % pl.tiles;
    int id = (turn / pl.tiles) * 8 + xcd;
    if (id >= pl.splits * hk * p.B) return;
    // (heads before splits: the splits of a sequence differ in length, and would
    // fall on the same XCDs for every head)
    const int head = id % hk;
    id /= hk;
    const int split = id % pl.splits, b = id / pl.splits;

    Sequence s;
    sequence_rows(p, b, s.q0, s.n);
    const int rows = s.n * pl.group;
    const int tile_row = tile * ROWS;
    if (tile_row >= rows) return;
    s.len = p.kv_len[b];
    s.len = s.len < 0 ? 0 : s.len > p.max_kv ? p.max_kv : s.len;
    s.past = s.len - s.n;
    const int row_last = (tile_row + ROWS < rows ? tile_row + ROWS : rows) - 1;
    int begin, end;
    split_range(p, pl, s, b, split, tile_row / pl.group, row_last / pl.group, begin, end);

    // this wave's rows
    const int row0 = tile_row + (wave & (4 / WK - 1)) * 32;
    const int unit0 = WK == 2 ? wave >> 1 : 0;   // of a stage
    const bool works = row0 < rows;          // the last tile's waves may have none: they only load
    float scale = p.scale * 1.4426950408889634f * (E == 1 ? p.cache.k_scale[head] : 1.0f);
    const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;   // so that the largest score is the largest product
    scale = fmaxf(fabsf(scale), 1.17549435e-38f);
    uint4 Q[KS];
    float16_t O[DB];
    float ref = -INFINITY, sum = 0.0f;       // sum: of this half's p
    const bool live = row0 + m < rows;
    const int node = (live ? row0 + m : rows - 1) / pl.group;
    const int pos = p.positions ? p.positions[s.q0 + node] : s.past + node;
    const int low = p.window > 0 ? pos - p.window + 1 : 0;
    int low_most = low > 0 ? low : 0;
    {
        const int qh = head * pl.group + (live ? row0 + m : rows - 1) - node * pl.group;
        const uint16_t* q = p.q + static_cast<int64_t>(s.q0 + node) * p.q_stride + static_cast<int64_t>(qh) * D;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            // dims of operand i in half h, as K's pieces hold them
            const int d = E == 2 ? 16 * i + 8 * h : 32 * (i >> 1) + 16 * h + 8 * (i & 1);
            const uint4 v = *reinterpret_cast<const uint4*>(q + d);
            Q[i] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
        }
    }
#pragma unroll
    for (int db = 0; db < DB; ++db) O[db] = zero16();
    if (p.window > 0) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) low_most = max(low_most, __shfl_xor(low_most, off));
        low_most = __builtin_amdgcn_readfirstlane(low_most);
    }

    // this wave's pieces of a stage: K or V of one unit
    const int my_unit = wave >> 1;
    const bool values = wave & 1;
    // the token of K's row m in a unit, and the block of this lane's pieces
    const int token = E == 2 ? 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3)
                             : 16 * ((m >> 2) & 1) + 4 * (m >> 3) + (m & 3);
    const int k_offset = h * 256 + (token & 15) * 16;
    const int v_offset = (E == 2 ? h * (16 * D) : 0) + m * 16;
    const uint8_t* my_base = static_cast<const uint8_t*>(values ? p.cache.v : p.cache.k) + (values ? v_offset : k_offset);
    const int lane_block = values ? h : token >> 4;    // (bf16's V: one of each, below)
    int units = 0;                           // of the part in the table
    auto load = [&](int stage) {
        int unit = stage * U + my_unit;
        unit = unit < units ? unit : units - 1;
        // As plain instructions: the compiler would wait for all of them
        // before any read of shared memory.  Completion is the explicit
        // waits' matter; there is no register result.  The instruction's
        // offset counts in both places, so M0 makes up for the pieces' 512 B
        // in the cache against 1 KB in shared memory.  (A load to shared
        // memory may follow a write of M0 after one wait state.)
        const uint32_t to = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
            reinterpret_cast<uintptr_t>(ring + ((stage & 1) * STAGE + (my_unit * 2 + (values ? 1 : 0)) * KC) * 64)));
        auto pieces = [&](const uint8_t* from, uint32_t at, auto count) {
            constexpr int N = decltype(count)::value;
#define W4_PIECE(x)                                                                                                        \
    if constexpr (x < N)                                                                                                   \
        asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%3" ::"v"(from),          \
                     "s"(at), "n"((x) * 512), "n"((x) * 512) : "memory", "m0", "scc");
            W4_PIECE(0) W4_PIECE(1) W4_PIECE(2) W4_PIECE(3) W4_PIECE(4) W4_PIECE(5) W4_PIECE(6) W4_PIECE(7)
#undef W4_PIECE
        };
        auto block = [&](int i) {
            const int blk = blocks[2 * unit + i];
            return my_base + static_cast<int64_t>(blk < 0 ? 0 : blk) * (16 * D * E);
        };
        if (E == 2 && values) {
            pieces(block(0), to, std::integral_constant<int, DB>{});
            pieces(block(1), to + DB * 1024, std::integral_constant<int, DB>{});
        } else {
            pieces(block(lane_block), to, std::integral_constant<int, KC>{});
        }
    };
    auto mask_bits = [&](int k0) -> uint32_t {
        if (!live) return 0u;
        if (E == 2)
            return sees(p, pl, s, node, low, k0 + 8 * h, 8) | sees(p, pl, s, node, low, k0 + 16 + 8 * h, 8) << 8;
        return sees(p, pl, s, node, low, k0 + 16 * h, 16);
    };
    // tokens [plain, plain_end) are seen by all rows of the wave
    const int plain = low_most;
    // (a chain's tokens up to the first row's own node too)
    int plain_end = p.tree || p.positions ? s.past : s.past + row0 / pl.group + 1;
    plain_end = s.holes ? 0 : plain_end < s.len ? plain_end : s.len;
    auto needs_mask = [&](int k0, int tokens) { return k0 < plain || k0 + tokens > plain_end; };

    for (int from_token = begin; from_token < end; from_token += 16 * kTableBlocks) {
        // the blocks of the split (nearly always all of them), as indices of
        // the cache's; -1: outside it
        const int left = end - from_token;
        units = ((left < 16 * kTableBlocks ? left : 16 * kTableBlocks) + 31) / 32;
        if (from_token != begin) __syncthreads();
        for (int i = threadIdx.x; i < 2 * units; i += 256) {
            const int blk = min((from_token >> 4) + i, s.last_block);
            const int pg = page_of(p, pl, blk);
            const int64_t page = s.table[pg];
            blocks[i] = page < 0 || page >= p.cache.pages ? -1
                                                          : static_cast<int>((page * hk + head) * pb + (blk - pg * pb));
            // (2^31 blocks of at least 1 KB are more than the memory holds)
        }
        // every load the compiler knows of is done before the first it does not
        wait_loads<0>();
        __syncthreads();
        bool repairs = false;
        load(0);
        const int stages = (units + 1) / 2;
        for (int st = 0; st < stages; ++st) {
            // this stage is there, and all waves are done with the one before
            wait_loads<0>();
            __syncthreads();
            if (st + 1 < stages) load(st + 1);
            if (!works) continue;
            const int k0 = from_token + 64 * st + 32 * unit0;
            const uint4* at = ring + ((st & 1) * STAGE + unit0 * 2 * KC) * 64 + lane;
            float16_t acc[UW];
#pragma unroll
            for (int u = 0; u < UW; ++u) acc[u] = zero16();
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int u = 0; u < UW; ++u) {
                    const uint4 x = at[(u * 2 * KC + c) * 64];
                    if constexpr (E == 2) {
                        acc[u] = mfma32(x, Q[c], acc[u]);
                    } else {
                        uint4 lo, hi;
                        widen16(x, lo, hi);
                        acc[u] = mfma32(lo, Q[2 * c], acc[u]);
                        acc[u] = mfma32(hi, Q[2 * c + 1], acc[u]);
                    }
                }
            // the first unit's values on their way under the exponentials
            uint4 vx[KC];
#pragma unroll
            for (int c = 0; c < KC; ++c) vx[c] = at[(KC + c) * 64];
            const bool masked = needs_mask(k0, 32 * UW);
            bool odd = false;
            if (masked) {
#pragma unroll
                for (int u = 0; u < UW; ++u) {
                    const uint32_t bits = mask_bits(k0 + 32 * u);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!((bits >> i) & 1)) acc[u][i] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < KC; ++c) odd = odd || nonfinite<E>(at[((u * 2 + 1) * KC + c) * 64]);
                }
                odd = __any(odd);
                repairs = repairs || odd;
            }
            // the reference is raised where a score exceeds it by more than kRaise
            float top = acc[0][0];
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(top, acc[u][i]);
            top *= scale;
            if (__any(top > ref + kRaise)) {
                const float now = fmaxf(ref, max_halves(top));
                const float fade = now == -INFINITY ? 1.0f : exp2_fast(ref - now);
                ref = now;
                sum *= fade;
#pragma unroll
                for (int db = 0; db < DB; ++db) O[db] *= fade;
            }
            float base = ref == -INFINITY ? 0.0f : ref, by = scale;
            if (__any(fabsf(base) >= kFar)) {
#pragma unroll
                for (int u = 0; u < UW; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[u][i] = rounded_exponent(acc[u][i], scale, base);
                base = 0.0f;
                by = 1.0f;
            }
            uint4 P[UW][2];
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[i] = pack_bf16x2(exp2_fast(__builtin_fmaf(acc[u][8 * j + 2 * i], by, -base)),
                                           exp2_fast(__builtin_fmaf(acc[u][8 * j + 2 * i + 1], by, -base)));
                        sum = dot2_bf16(w[i], 0x3F803F80u, sum);   // of the rounded p
                    }
                    P[u][j] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            auto add_values = [&](auto clean) {
#pragma unroll
                for (int u = 0; u < UW; ++u) {
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        uint4 x = u == 0 ? vx[c] : at[((u * 2 + 1) * KC + c) * 64];
                        if constexpr (decltype(clean)::value) x = finite_piece<E>(x);
                        if constexpr (E == 2) {
                            O[c % DB] = mfma32(x, P[u][c / DB], O[c % DB]);
                        } else {
                            uint4 lo, hi;
                            widen16(x, lo, hi);
                            O[c] = mfma32(lo, P[u][0], O[c]);
                            O[c] = mfma32(hi, P[u][1], O[c]);
                        }
                    }
                }
            };
            // an infinity or NaN among the values of a stage that not every
            // row sees, or behind the last token (0 times it would be NaN):
            // without them here, and added after the loop where they are seen
            if (odd) add_values(std::true_type{});
            else add_values(std::false_type{});
        }
        if (repairs) {
            // for each output, how many +inf and NaN, -inf and NaN its row sees:
            // products of the rows' masks with indicators
#pragma unroll 1
            for (int u = 0; u < units; ++u) {
                const int k0 = from_token + 32 * u;
                // (the units that a wave takes of a stage were checked, and cleaned, together)
                if (!needs_mask(k0 - 32 * (u % UW), 32 * UW) || (WK == 2 && (u & 1) != unit0)) continue;
                const uint32_t bits = mask_bits(k0);
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int bj = blocks[2 * u + (E == 2 ? j : h)];
                        const uint8_t* from = static_cast<const uint8_t*>(p.cache.v) + static_cast<int64_t>(bj < 0 ? 0 : bj) * (16 * D * E) +
                                              v_offset + db * 512;
                        const uint4 c = *reinterpret_cast<const uint4*>(from);
                        uint4 x = c;
                        if constexpr (E == 1) {
                            uint4 lo, hi;
                            widen16(c, lo, hi);
                            x = j ? hi : lo;
                        }
                        uint4 plus, minus;
                        finite_part(x, plus, minus);
                        const uint4 one = ones_at(bits >> (8 * j));
                        const float16_t a = mfma32(plus, one, zero16());
#pragma unroll
                        for (int i = 0; i < 16; ++i) O[db][i] += a[i] > 0.0f ? INFINITY : 0.0f;
                        const float16_t z = mfma32(minus, one, zero16());
#pragma unroll
                        for (int i = 0; i < 16; ++i) O[db][i] += z[i] > 0.0f ? -INFINITY : 0.0f;
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
        }
    }

    if constexpr (WK == 2) {
        // the second half's sums pass through the ring to the first half's waves
        float4_t* shared = reinterpret_cast<float4_t*>(ring) + (wave & 1) * (DB * 4 * 64) + lane;
        float2_t* stats = reinterpret_cast<float2_t*>(blocks) + (wave & 1) * 64 + lane;
        __syncthreads();
        if (wave >= 2) {
            stats[0] = float2_t{ref, sum};
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    shared[(4 * db + q) * 64] = float4_t{O[db][4 * q], O[db][4 * q + 1], O[db][4 * q + 2], O[db][4 * q + 3]};
        }
        __syncthreads();
        if (wave >= 2) return;
        const float2_t other = stats[0];
        const float now = fmaxf(ref, other[0]);
        // (a half that saw nothing has sums of 0, or of NaN)
        const float mine = ref == -INFINITY ? 1.0f : exp2_fast(ref - now);
        const float theirs = other[0] == -INFINITY ? 1.0f : exp2_fast(other[0] - now);
        ref = now;
        sum = sum * mine + other[1] * theirs;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4_t x = shared[(4 * db + q) * 64];
#pragma unroll
                for (int i = 0; i < 4; ++i) O[db][4 * q + i] = O[db][4 * q + i] * mine + x[i] * theirs;
            }
    }
    if (!works) return;
    const float total = sum + __shfl_xor(sum, 32);
    if (!live) return;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            put<D, E>(p, pl, s.q0, head, split, row0 + m, 32 * db + 8 * q + 4 * h,
                      float4_t{O[db][4 * q], O[db][4 * q + 1], O[db][4 * q + 2], O[db][4 * q + 3]}, ref, total);
}

}  // namespace

hipError_t launch_attention_tiles(const AttentionParams& p, const AttentionPlan& pl, unsigned wgs, hipStream_t stream) {
    const dim3 grid(wgs), block(256);
#define W4_TILES(D, E)                                                                                              \
    do {                                                                                                            \
        if (pl.tile_rows == 64) hipLaunchKernelGGL((attention_tile_kernel<D, E, 2>), grid, block, 0, stream, p, pl); \
        else hipLaunchKernelGGL((attention_tile_kernel<D, E, 1>), grid, block, 0, stream, p, pl);                    \
    } while (0)
    if (p.cache.e4m3) {
        if (p.cache.dim == 64) W4_TILES(64, 1);
        else W4_TILES(128, 1);
    } else {
        if (p.cache.dim == 64) W4_TILES(64, 2);
        else W4_TILES(128, 2);
    }
#undef W4_TILES
    return hipGetLastError();
}

}  // namespace w4
