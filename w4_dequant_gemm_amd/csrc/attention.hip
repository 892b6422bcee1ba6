// Attention of each sequence's last tokens (one, a drafted tree, a prompt
// chunk) over the paged cache.
//
// Per KV head the rows are the nodes times the query heads of its group.  A
// wavefront takes units of S tokens (32 bf16, 64 E4M3: 16 bytes of a dim's
// tokens in each lane group) with both products on v_mfma_f32_16x16x32_bf16,
// transposed so that a row is a column of both results:
//   S^T [16 tokens x 16 rows] = K [16 x D] Q^T,   O^T [16 dims x 16 rows] += V^T [16 x S] P^T.
// A result holds row l % 16 in lane l, tokens 4 (l / 16) + 0..3; an operand
// holds 8 values of the summed index in group l / 16.  Which token is which
// index of the second sum is free as long as P and V agree, so lane group g
// takes the S/4 tokens from S/4 g on: the K rows of tile t are the tokens
// S/4 (m / 4) + 4 t + m % 4 (m = l % 16), which puts P's values where its
// operand needs them, and V's operand is one 16-byte piece of the cache as it
// lies.  Neither P nor V is transposed or passes through shared memory for it.
//
// Softmax in one pass, base 2, statistics in fp32.  The reference that is
// subtracted in the exponent need not be the maximum: it is raised (and the
// sums faded) only when a score exceeds it by more than 8, so p <= 2^8 and
// most steps neither exchange maxima between lanes nor touch the sums.  p is
// rounded to bf16, the matrix cores' operand; the sum of the same rounded p
// comes from one more product with ones, so a weight that dominates is not
// biased by its rounding.
#include "attention.hpp"
#include "launch.hpp"

namespace w4 {
namespace {
using namespace attn;

// R tiles of 16 rows of one wavefront: their queries, running sums, and the
// work of a step of one unit.
template <int D, int E, int R>
struct Core {
    static constexpr int S = 64 / E;         // tokens a unit
    static constexpr int NT = S / 16;        // K tiles a unit
    static constexpr int KP = D * E / 64;    // 16-byte pieces of a K tile in a lane
    static constexpr int KS = D / 32;        // operands of a K tile
    static constexpr int DT = D / 16;
    static constexpr int NP = S / 32;        // operands of P, and of V's piece
    static constexpr int BPU = S / 16;       // 16-token blocks a unit

    uint4 Q[R][KS];
    float4_t O[R][DT], L[R];                 // sums of p v and of p (every component)
    float ref[R], scale;
    int node[R], low[R];
    bool live[R];
    int low_most;
    bool repairs;                            // see repair()

    __device__ __forceinline__ void init(const AttentionParams& p, const AttentionPlan& pl, const Sequence& s, int head,
                                         int row0, int rows) {
        const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
        // a negative scale turns the queries' signs, so that the largest score is the largest product
        scale = p.scale * 1.4426950408889634f * (E == 1 ? p.cache.k_scale[head] : 1.0f);
        const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
        scale = fmaxf(fabsf(scale), 1.17549435e-38f);
        low_most = 0;
        repairs = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = row0 + 16 * r + m;
            live[r] = row < rows;
            const int at = live[r] ? row : rows - 1;
            node[r] = at / pl.group;
            const int h = head * pl.group + (at - node[r] * pl.group);
            const uint16_t* q = p.q + static_cast<int64_t>(s.q0 + node[r]) * p.q_stride + static_cast<int64_t>(h) * D;
            const int pos = p.positions ? p.positions[s.q0 + node[r]] : s.past + node[r];
            low[r] = p.window > 0 ? pos - p.window + 1 : 0;
            low_most = low[r] > low_most ? low[r] : low_most;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                // dims of operand i in lane group g, as K's pieces hold them
                const int d = E == 2 ? 32 * i + 8 * g : 64 * (i >> 1) + 16 * g + 8 * (i & 1);
                uint4 v = *reinterpret_cast<const uint4*>(q + d);
                Q[r][i] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
            }
            ref[r] = -INFINITY;
            L[r] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) O[r][dt] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (p.window > 0) {
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) low_most = max(low_most, __shfl_xor(low_most, off));
            low_most = __builtin_amdgcn_readfirstlane(low_most);
        }
    }

    // Tokens k0 .. k0 + S - 1: kget(i) and vget(dt) give the lane's 16-byte
    // pieces (i = tile * KP + piece); keys_done is called when the K pieces are
    // used up.  OWN: V's pieces are the wave's own registers, vown[dt].
    template <bool OWN, class KGet, class VGet, class Done>
    __device__ __forceinline__ void step(const AttentionParams& p, const AttentionPlan& pl, const Sequence& s, int k0,
                                         KGet kget, VGet vget, Done keys_done, uint4* vown) {
        const int g = (threadIdx.x & 63) >> 4;
        float4_t acc[R][NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const uint4 c = kget(t * KP + i);
                if constexpr (E == 2) {
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][t] = mfma(c, Q[r][i], acc[r][t]);
                } else {
                    uint4 a, b;
                    widen16(c, a, b);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][t] = mfma(a, Q[r][2 * i], acc[r][t]);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][t] = mfma(b, Q[r][2 * i + 1], acc[r][t]);
                }
            }
        }

        keys_done();

        const bool masked = needs_mask(s, k0);
        if (masked) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t seen = live[r] ? sees(p, pl, s, node[r], low[r], k0 + (S / 4) * g, S / 4) : 0;
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i)
                    if (!((seen >> i) & 1)) acc[r][i >> 2][i & 3] = -INFINITY;
            }
        }
        float top[R];
        bool raise = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            top[r] = -INFINITY;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; j += 2) top[r] = fmaxf(top[r], fmaxf(acc[r][t][j], acc[r][t][j + 1]));
            top[r] *= scale;
            raise = raise || top[r] > ref[r] + kRaise;
        }
        if (__any(raise)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float now = fmaxf(ref[r], max_groups(top[r]));
                const float fade = now == -INFINITY ? 1.0f : exp2_fast(ref[r] - now);
                ref[r] = now;
                L[r] *= fade;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) O[r][dt] *= fade;
            }
        }
        float base[R], by = scale;
        bool far = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            base[r] = ref[r] == -INFINITY ? 0.0f : ref[r];
            far = far || fabsf(base[r]) >= kFar;
        }
        if (__any(far)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[r][t][j] = rounded_exponent(acc[r][t][j], scale, base[r]);
                base[r] = 0.0f;
            }
            by = 1.0f;
        }
        uint4 P[R][NP];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = exp2_fast(__builtin_fmaf(acc[r][2 * q + (i >> 2)][i & 3], by, -base[r]));
                P[r][q] = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                                     pack_bf16x2(e[6], e[7]));
            }
        }
        const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < NP; ++q) L[r] = mfma(ones, P[r][q], L[r]);

        auto operands = [&](int dt, uint4 (&V)[NP]) {
            const uint4 c = vget(dt);
            if constexpr (E == 2) V[0] = c;
            else widen16(c, V[0], V[NP - 1]);
        };
        bool odd = false;
        if (masked) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) odd = odd || nonfinite<E>(vget(dt));
            odd = __any(odd);
        }
        if (odd) {
            // an infinity or NaN among the values of a step that not every row
            // sees, or behind the last token (0 times it would be NaN): without
            // them here, and repair() adds them to the rows that see them
            repairs = true;
            if constexpr (OWN) {
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) vown[dt] = finite_piece<E>(vown[dt]);
            }
        }
        if (odd && !OWN) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                uint4 V[NP];
                operands(dt, V);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    uint4 plus, minus;
                    const uint4 fine = finite_part(V[q], plus, minus);
#pragma unroll
                    for (int r = 0; r < R; ++r) O[r][dt] = mfma(fine, P[r][q], O[r][dt]);
                }
                __builtin_amdgcn_sched_barrier(0);   // registers are scarcer than time here
            }
        } else {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                uint4 V[NP];
                operands(dt, V);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int q = 0; q < NP; ++q) O[r][dt] = mfma(V[q], P[r][q], O[r][dt]);
            }
        }
    }

    // Whether a unit at k0 needs the rows' masks.
    __device__ __forceinline__ bool needs_mask(const Sequence& s, int k0) const {
        return s.holes || k0 + S > (s.past < s.len ? s.past : s.len) || k0 < low_most;
    }

    // The infinities and NaN that step() left out of the units k0, k0 + stride,
    // ... < end: for each output, how many +inf and NaN, -inf and NaN its row
    // sees (products of the rows' masks with indicators).
    __device__ __forceinline__ void repair(const AttentionParams& p, const AttentionPlan& pl, const Sequence& s, int head,
                                           int k0, int stride, int end) {
        const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll 1
        for (; k0 < end; k0 += stride) {
            if (!needs_mask(s, k0)) continue;
            const int blk = min((k0 >> 4) + (g * BPU >> 2), s.last_block);
            int64_t page = s.table[page_of(p, pl, blk)];
            page = page < 0 || page >= p.cache.pages ? 0 : page;
            const int64_t at = (page * p.cache.heads + head) * p.cache.page_blocks + (blk - page_of(p, pl, blk) * p.cache.page_blocks);
            const uint8_t* from = static_cast<const uint8_t*>(p.cache.v) + at * (16 * D * E) + (E == 2 ? (g & 1) * (16 * D) : 0) + m * 16;
            uint32_t bits[R];
#pragma unroll
            for (int r = 0; r < R; ++r) bits[r] = live[r] ? sees(p, pl, s, node[r], low[r], k0 + (S / 4) * g, S / 4) : 0;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                uint4 V[NP];
                const uint4 c = *reinterpret_cast<const uint4*>(from + dt * 256);
                if constexpr (E == 2) V[0] = c;
                else widen16(c, V[0], V[NP - 1]);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    uint4 plus, minus;
                    finite_part(V[q], plus, minus);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint4 one = ones_at(bits[r] >> (8 * q));
                        const float4_t a = mfma(plus, one, float4_t{0.0f, 0.0f, 0.0f, 0.0f});
                        const float4_t b = mfma(minus, one, float4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            O[r][dt][j] += (a[j] > 0.0f ? INFINITY : 0.0f) + (b[j] > 0.0f ? -INFINITY : 0.0f);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
    }
};

// Up to 32 rows: the time is that of reading the cache once.  The four waves
// of a workgroup hold the same rows and take steps of one unit in turn, each
// straight from memory into operand registers (no reuse to stage for; the next
// step's loads are in flight under the present one's products); their sums are
// joined through shared memory.  48 sequences of 4000 to 8000 tokens, 32 heads on
// 8 of 128, bf16: 1.19 GB in 212 us, 5.6 TB/s, what a large copy moves; one
// sequence of 517, 9 heads on 3 of 64: 8 us, of which most is the chain of a
// launch's first reads (lengths, pages, keys, values).  D = 128, E4M3 and two row
// tiles spill 12 bytes, outside the loop.
template <int D, int E, int R>
__global__ void __launch_bounds__(256, 2) attention_stream_kernel(AttentionParams p, AttentionPlan pl) {
    using C = Core<D, E, R>;
    constexpr int S = C::S, WK = 4, DT = C::DT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int hk = p.cache.heads, pb = p.cache.page_blocks;
    int id = blockIdx.x;
    const int split = id % pl.splits;
    id /= pl.splits;
    const int head = id % hk, b = id / hk;

    Sequence s;
    sequence_rows(p, b, s.q0, s.n);
    const int rows = s.n * pl.group;         // 16 R at most
    if (rows == 0) return;
    s.len = p.kv_len[b];
    s.len = s.len < 0 ? 0 : s.len > p.max_kv ? p.max_kv : s.len;
    s.past = s.len - s.n;
    int begin, end;
    split_range(p, pl, s, b, split, 0, s.n - 1, begin, end);
    C c;
    c.init(p, pl, s, head, 0, rows);

    uint4 kx[C::NT * C::KP], vx[DT];         // the pieces of the step
    auto k_block = [&](int st) { return min(st * C::BPU + (m * C::BPU >> 4), s.last_block); };
    auto v_block = [&](int st) { return min(st * C::BPU + (g * C::BPU >> 2), s.last_block); };
    auto address = [&](const void* base, int blk, int page) {
        page = page < 0 || page >= p.cache.pages ? 0 : page;
        const int64_t block = (static_cast<int64_t>(page) * hk + head) * pb + (blk - page_of(p, pl, blk) * pb);
        return static_cast<const uint8_t*>(base) + block * (16 * D * E);
    };
    auto load_k = [&](int st, int page) {
        const uint8_t* from = address(p.cache.k, k_block(st), page) + g * 256;
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
            const int token = (S / 4) * (m >> 2) + 4 * t + (m & 3);
#pragma unroll
            for (int i = 0; i < C::KP; ++i)
                kx[t * C::KP + i] = load_nt_16(reinterpret_cast<const uint32_t*>(from + (token & 15) * 16 + i * 1024));
        }
    };
    auto load_v = [&](int st, int page) {
        const uint8_t* from = address(p.cache.v, v_block(st), page) + (E == 2 ? (g & 1) * (16 * D) : 0) + m * 16;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) vx[dt] = load_nt_16(reinterpret_cast<const uint32_t*>(from + dt * 256));
    };
    auto k_page = [&](int st) { return s.table[page_of(p, pl, k_block(st))]; };
    auto v_page = [&](int st) { return s.table[page_of(p, pl, v_block(st))]; };

    // the next step's K is loaded once the present scores are done, its V once
    // the present products are; the pages are looked up a step before that
    int st = begin / S + wave;
    if (st * S < end) {
        load_k(st, k_page(st));
        load_v(st, v_page(st));
        int kp = k_page(st + WK), vp = v_page(st + WK);
        while (true) {
            const int next = st + WK;
            const bool more = next * S < end;
            const int kp2 = k_page(next + WK), vp2 = v_page(next + WK);
            c.template step<true>(p, pl, s, st * S, [&](int i) { return kx[i]; }, [&](int dt) { return vx[dt]; },
                                  [&] { if (more) load_k(next, kp); }, vx);
            if (!more) break;
            load_v(next, vp);
            kp = kp2;
            vp = vp2;
            st = next;
        }
        if (c.repairs) c.repair(p, pl, s, head, (begin / S + wave) * S, WK * S, end);
    }

    // join the waves, a quarter of the dims at a time
    constexpr int DQ = DT / 4;
    __shared__ float sm_ref[WK][16 * R], sm_sum[WK][16 * R];
    __shared__ float4_t sm_o[WK][DQ * 4][16 * R];
    if (g == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sm_ref[wave][16 * r + m] = c.ref[r];
            sm_sum[wave][16 * r + m] = c.L[r][0];
        }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float top = sm_ref[0][16 * r + m];
#pragma unroll
        for (int w = 1; w < WK; ++w) top = fmaxf(top, sm_ref[w][16 * r + m]);
        const float f = c.ref[r] == -INFINITY ? (c.L[r][0] != 0.0f ? 1.0f : 0.0f) : exp2_fast(c.ref[r] - top);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) c.O[r][dt] *= f;
    }
#pragma unroll
    for (int quarter = 0; quarter < 4; ++quarter) {
        if (quarter) __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int x = 0; x < DQ; ++x) sm_o[wave][4 * x + g][16 * r + m] = c.O[r][quarter * DQ + x];
        __syncthreads();
        for (int u = threadIdx.x; u < DQ * 4 * 16 * R; u += 256) {
            const int lr = u / (DQ * 4), d4 = u - lr * (DQ * 4);
            if (lr >= rows) continue;
            float top = sm_ref[0][lr];
#pragma unroll
            for (int w = 1; w < WK; ++w) top = fmaxf(top, sm_ref[w][lr]);
            float total = 0.0f;
            float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                // (a wave that saw nothing has sum 0; a NaN sum stays one)
                const float t = sm_ref[w][lr];
                total += sm_sum[w][lr] * (t == -INFINITY ? 1.0f : exp2_fast(t - top));
                o += sm_o[w][d4][lr];
            }
            put<D, E>(p, pl, s.q0, head, split, lr, quarter * (D / 4) + 4 * d4, o, top, total);
        }
    }
}

// Heads of 256 dims, whose pieces and sums do not fit a wave's registers in
// the other forms: each of four waves has a tile of 16 rows, and the tokens'
// pieces pass through shared memory once for the workgroup, in the order in which the
// operands are read (one linear 1 KB a piece and wavefront: no bank is asked
// twice).  Two stages of 32 KB: the loads of the next unit go straight to shared
// memory while the present one is used, one barrier a stage.  (On 32 x 32
// products as in attention_tile.hip the sums spill: 24 trees of 17 nodes, window
// 1024, E4M3: 54 us against 47, 5 of them the join.)  Bound by the work beside the
// products: widening the codes and masks at the window's and the nodes' edges
// (28 % of the cycles VALU, 19 % MFMA), at 2.3 TB/s of the cache.
template <int D, int E>
__global__ void __launch_bounds__(256, 2) attention_wide_kernel(AttentionParams p, AttentionPlan pl) {
    using C = Core<D, E, 1>;
    constexpr int S = C::S, DT = C::DT;
    constexpr int PER = D / 16;              // 1 KB pieces of K, and of V
    constexpr int STAGE = 2 * PER;
    constexpr int MINE = STAGE / 4;          // pieces a wave loads
    __shared__ __attribute__((aligned(16))) uint4 stage0[STAGE * 64];
    __shared__ __attribute__((aligned(16))) uint4 stage1[STAGE * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
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
    const int tile_row = tile * 64;
    if (tile_row >= rows) return;
    s.len = p.kv_len[b];
    s.len = s.len < 0 ? 0 : s.len > p.max_kv ? p.max_kv : s.len;
    s.past = s.len - s.n;
    const int row_last = (tile_row + 64 < rows ? tile_row + 64 : rows) - 1;
    int begin, end;
    split_range(p, pl, s, b, split, tile_row / pl.group, row_last / pl.group, begin, end);
    C c;
    c.init(p, pl, s, head, tile_row + wave * 16, rows);

    // this wave's pieces of a stage: half of K's or of V's
    const bool values = wave >> 1;
    const int part = (wave & 1) * MINE;
    auto block = [&](int k0) { return min((k0 >> 4) + (values ? g * C::BPU >> 2 : m * C::BPU >> 4), s.last_block); };
    auto page_at = [&](int k0) { return s.table[page_of(p, pl, block(k0))]; };
    auto load = [&](uint4* stage, int k0, int page) {
        page = page < 0 || page >= p.cache.pages ? 0 : page;
        const int blk = block(k0);
        const int64_t at = (static_cast<int64_t>(page) * hk + head) * pb + (blk - page_of(p, pl, blk) * pb);
        const uint8_t* src = static_cast<const uint8_t*>(values ? p.cache.v : p.cache.k) + at * (16 * D * E);
        src += values ? (E == 2 ? (g & 1) * (16 * D) : 0) + m * 16 : g * 256;
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int x = part + i;
            const int t = x / C::KP;
            const uint8_t* from = src + (values ? x * 256
                                                : (((S / 4) * (m >> 2) + 4 * t + (m & 3)) & 15) * 16 + (x - t * C::KP) * 1024);
            // As plain instructions: the compiler would wait for all of them
            // before any read of shared memory.  The wait is the explicit one
            // at the stage's end; a load the compiler does not know of only
            // makes its own waits stricter.  (A load to shared memory may
            // follow a write of M0 after one wait state.)
            const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
                reinterpret_cast<uintptr_t>(stage + ((values ? PER : 0) + x) * 64)));
            asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(m0) : "memory", "m0");
        }
    };
    auto compute = [&](const uint4* stage, int k0) {
        c.template step<false>(p, pl, s, k0, [&](int i) { return stage[i * 64 + lane]; },
                               [&](int dt) { return stage[(PER + dt) * 64 + lane]; }, [] {}, nullptr);
    };

    if (begin < end) {
        int k0 = begin;
        load(stage0, k0, page_at(k0));
        int page = page_at(k0 + S);
        while (true) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (k0 + S < end) load(stage1, k0 + S, page);
            page = page_at(k0 + 2 * S);
            compute(stage0, k0);
            k0 += S;
            if (k0 >= end) break;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (k0 + S < end) load(stage0, k0 + S, page);
            page = page_at(k0 + 2 * S);
            compute(stage1, k0);
            k0 += S;
            if (k0 >= end) break;
        }
        if (c.repairs) c.repair(p, pl, s, head, begin, S, end);
    }
    if (!c.live[0]) return;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
        put<D, E>(p, pl, s.q0, head, split, tile_row + wave * 16 + m, 16 * dt + 4 * g, c.O[0][dt], c.ref[0], c.L[0][0]);
}

// The splits of a row joined, in a fixed order: `parts` threads for each four
// dims of a row take every parts-th split, four loads in flight, and are
// joined through shared memory.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(AttentionParams p, AttentionPlan pl, int parts) {
    constexpr int L = D / 4;                 // threads a row and part
    __shared__ float4_t sm_o[256];
    __shared__ float2_t sm_ml[256];
    const int vec = threadIdx.x % L;
    const int part = (threadIdx.x / L) % parts;
    int q0, n;
    sequence_rows(p, blockIdx.y, q0, n);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / (L * parts)) + threadIdx.x / (L * parts);
    const bool live = row < static_cast<int64_t>(n) * p.hq;
    const int64_t at = static_cast<int64_t>(q0) * p.hq + (live ? row : 0);
    const int64_t all = p.T * p.hq;
    const float* ml = p.ws + static_cast<int64_t>(pl.splits) * all * D;
    float top = -INFINITY, total = 0.0f;
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](float2_t t, float4_t x) {
        if (t[1] == 0.0f) return;            // saw nothing
        const float now = fmaxf(top, t[0]);
        const float f = t[0] == -INFINITY ? 1.0f : exp2_fast(t[0] - now);
        const float g = top == -INFINITY ? 1.0f : exp2_fast(top - now);
        total = total * g + t[1] * f;
        o = o * g + x * f;
        top = now;
    };
    if (live) {
        int s = part;
        for (; s + 3 * parts < pl.splits; s += 4 * parts) {
            float2_t t[4];
            float4_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t slice = static_cast<int64_t>(s + i * parts) * all + at;
                t[i] = *reinterpret_cast<const float2_t*>(ml + 2 * slice);
                x[i] = *reinterpret_cast<const float4_t*>(p.ws + slice * D + 4 * vec);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) add(t[i], x[i]);
        }
        for (; s < pl.splits; s += parts) {
            const int64_t slice = static_cast<int64_t>(s) * all + at;
            add(*reinterpret_cast<const float2_t*>(ml + 2 * slice), *reinterpret_cast<const float4_t*>(p.ws + slice * D + 4 * vec));
        }
    }
    if (parts > 1) {
        sm_o[threadIdx.x] = o;
        sm_ml[threadIdx.x] = float2_t{top, total};
        __syncthreads();
        if (part == 0)
            for (int i = 1; i < parts; ++i) add(sm_ml[threadIdx.x + i * L], sm_o[threadIdx.x + i * L]);
    }
    if (!live || part) return;
    const float v_scale = p.cache.e4m3 ? p.cache.v_scale[(row % p.hq) / pl.group] : 1.0f;
    const float f = total != 0.0f ? v_scale / total : 0.0f;
    *reinterpret_cast<uint2*>(p.O + at * D + 4 * vec) = make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
}

// Rows a workgroup holds, by the rows a (sequence, head) has.  Up to 32: the
// streaming kernel on 16 or 32.  Above: the tile kernel on 64 up to 64 rows,
// else on 128.  256 dims: the wide kernel on 64.
int rows_per_tile(int dim, int64_t rows) {
    if (dim == 256) return 64;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

AttentionPlan make_plan(int64_t B, int hq, int hk, int dim, int64_t max_q, int64_t max_kv, int64_t window) {
    AttentionPlan pl{};
    pl.group = hq / hk;
    const int64_t rows = max_q * pl.group;
    pl.tile_rows = rows_per_tile(dim, rows);
    pl.tiles = static_cast<int>((rows + pl.tile_rows - 1) / pl.tile_rows);
    // tokens that one sequence's rows can see (a window starts at a multiple of 64)
    int64_t span = max_kv;
    if (window > 0 && window + max_q + 64 < span) span = window + max_q + 64;
    // Splits: 512 workgroups run at a time (two a compute unit).  Of the numbers
    // that just fill 1 .. 8 such rounds, and none, the one with the least
    //   rounds (tokens of a split + own cost) + cost of the join,
    // in tokens: a split writes and reads its rows' fp32 partial results (128
    // rows: as 1500 tokens), the join is a launch.  (16 trees of 60 nodes, 4000
    // tokens: one split 119 us, two 138; a chunk of 777 behind 6000: 233, 217,
    // three 231; 131000 tokens, 64 rows: 64 splits 78 us, 128 86; windows of
    // 1024: two splits' worth 51 us, five 55.)
    constexpr int64_t kSlots = 512;
    const int64_t whole = B * hk * pl.tiles;
    const int64_t own = pl.tile_rows <= 32 ? 8 * pl.tile_rows : 12 * pl.tile_rows;
    const int64_t join = pl.tile_rows <= 32 ? 400 : 200;
    const int64_t step = pl.tile_rows <= 32 ? 256 : 64;   // a multiple of what a workgroup takes at a time
    int64_t splits = 1, best = (whole + kSlots - 1) / kSlots * (span + own);
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
        int64_t s = rounds * kSlots / whole;
        const int64_t most = (span + step - 1) / step;
        if (s > most) s = most;
        if (s < 2) continue;
        const int64_t cost = (whole * s + kSlots - 1) / kSlots * ((span + s - 1) / s + own) + join;
        if (cost < best) {
            best = cost;
            splits = s;
        }
    }
    const int64_t chunk = ((span + splits - 1) / splits + step - 1) / step * step;
    pl.chunk = static_cast<int>(chunk);
    pl.splits = static_cast<int>((span + chunk - 1) / chunk);
    if (pl.splits < 1) pl.splits = 1;
    return pl;
}

template <int D, int E>
hipError_t launch_kind(const AttentionParams& p, const AttentionPlan& pl, hipStream_t stream) {
    const int64_t groups = static_cast<int64_t>(pl.splits) * p.cache.heads * p.B;
    const bool tiled = pl.tile_rows > 32;
    const int64_t wgs = tiled ? (groups + 7) / 8 * 8 * pl.tiles : groups;
    if (!launch_fits(wgs, 256)) return hipErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(wgs);
    if constexpr (D == 256) {
        // 64 KB of shared memory: two workgroups a compute unit
        hipLaunchKernelGGL((attention_wide_kernel<D, E>), dim3(grid), dim3(256), 0, stream, p, pl);
    } else if (tiled) {
        const hipError_t e = launch_attention_tiles(p, pl, grid, stream);
        if (e != hipSuccess) return e;
    } else {
        if (pl.tile_rows == 16) hipLaunchKernelGGL((attention_stream_kernel<D, E, 1>), dim3(grid), dim3(256), 0, stream, p, pl);
        else hipLaunchKernelGGL((attention_stream_kernel<D, E, 2>), dim3(grid), dim3(256), 0, stream, p, pl);
    }
    if (pl.splits > 1) {
        // threads a row and four dims: one for few splits, more while they have four each
        int parts = 1;
        while (parts * (D / 4) < 256 && parts * 4 < pl.splits) parts *= 2;
        const int rows = 256 / (D / 4 * parts);
        const dim3 jgrid(static_cast<unsigned>((static_cast<int64_t>(p.max_q) * p.hq + rows - 1) / rows), p.B);
        hipLaunchKernelGGL(attention_join_kernel<D>, jgrid, dim3(256), 0, stream, p, pl, parts);
    }
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int64_t B, int hq, int hk, int dim, bool e4m3, int64_t max_q,
                                 int64_t max_kv, int64_t window) {
    const AttentionPlan pl = make_plan(B, hq, hk, dim, max_q, max_kv, window);
    if (pl.splits == 1) return 0;
    return static_cast<size_t>(pl.splits) * T * hq * (dim + 2) * sizeof(float);
}

hipError_t launch_attention(const AttentionParams& p, hipStream_t stream) {
    AttentionPlan pl = make_plan(p.B, p.hq, p.cache.heads, p.cache.dim, p.max_q, p.max_kv > 0 ? p.max_kv : 1, p.window);
    const int pb = p.cache.page_blocks;
    pl.page_magic = pb > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + pb - 1) / pb) : 0;
    if (p.cache.e4m3)
        return p.cache.dim == 64 ? launch_kind<64, 1>(p, pl, stream)
               : p.cache.dim == 128 ? launch_kind<128, 1>(p, pl, stream) : launch_kind<256, 1>(p, pl, stream);
    return p.cache.dim == 64 ? launch_kind<64, 2>(p, pl, stream)
           : p.cache.dim == 128 ? launch_kind<128, 2>(p, pl, stream) : launch_kind<256, 2>(p, pl, stream);
}

}  // namespace w4
