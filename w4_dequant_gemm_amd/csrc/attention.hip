// Attention of each sequence's last tokens (one, a drafted tree, a prompt
// chunk) over the paged cache.
//
// Per KV head the rows are the nodes times the query heads of its group.  A
// wavefront takes steps of 64 bytes of one dim's tokens (S = 32 bf16 or 64
// E4M3 tokens) with both products on v_mfma_f32_16x16x32_bf16, transposed so
// that a row is a column of both results:
//   S^T [16 tokens x 16 rows] = K [16 x D] Q^T,   O^T [16 dims x 16 rows] += V^T [16 x S] P^T.
// A result holds row l % 16 in lane l, tokens 4 (l / 16) + 0..3; an operand
// holds 8 values of the summed index in group l / 16.  Which token is which
// index of the second sum is free as long as P and V agree, so lane group g
// takes the S/4 tokens from S/4 g on: the K rows of tile t are the tokens
// S/4 (m / 4) + 4 t + m % 4 (m = l % 16), which puts P's values where its
// operand needs them, and V's operand is one 16-byte piece of the cache as it
// lies.  Neither P nor V passes through shared memory.
//
// Softmax in one pass: running maximum and sum (fp32, base 2), the sums of O
// rescaled when the maximum rises.  p is rounded to bf16 for the second
// product (the matrix cores' operand); the sum keeps the unrounded p.
#include "device.hpp"
#include "kernels.hpp"

namespace w4 {
namespace {

// Launch plan: tokens [c * chunk, (c + 1) * chunk) of a sequence (from its
// first visible one) are split c; `tiles` row tiles a (sequence, head).
struct AttentionPlan {
    int chunk, splits, tiles;
    int group;               // query heads a KV head
    uint32_t page_magic;     // block / page_blocks as a high product (page_blocks > 1)
};

__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// 16 E4M3 codes -> two bf16 operands of 8 (exact).
__device__ __forceinline__ void widen16(const uint4& c, uint4& lo, uint4& hi) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(in[i], 1.0f, false));
        o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(in[i], 1.0f, true));
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ float4_t mfma(const uint4& a, const uint4& b, const float4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// one element of eight kept, the others zero
__device__ __forceinline__ uint4 only(const uint4& v, int e) {
    const uint32_t keep = (e & 1) ? 0xFFFF0000u : 0x0000FFFFu;
    const int w = e >> 1;
    return make_uint4(w == 0 ? v.x & keep : 0, w == 1 ? v.y & keep : 0, w == 2 ? v.z & keep : 0, w == 3 ? v.w & keep : 0);
}

// the first n of eight elements kept
__device__ __forceinline__ uint4 first_of(const uint4& v, int n) {
    auto m = [&](int i) { return n >= 2 * i + 2 ? 0xFFFFFFFFu : n == 2 * i + 1 ? 0x0000FFFFu : 0u; };
    return make_uint4(v.x & m(0), v.y & m(1), v.z & m(2), v.w & m(3));
}

// D dims, E bytes a cached element, R tiles of 16 rows a wave, WK waves along
// the tokens (the other 4 / WK along the rows).
template <int D, int E, int R, int WK>
__global__ void __launch_bounds__(256) attention_kernel(AttentionParams p, AttentionPlan pl) {
    constexpr int S = 64 / E;                // tokens a step
    constexpr int NT = S / 16;               // K tiles a step
    constexpr int KS = D / 32;               // operands of a K tile
    constexpr int DT = D / 16;
    constexpr int NP = S / 32;               // operands of P and of a V tile
    constexpr int WR = 4 / WK;
    constexpr int ROWS = 16 * R * WR;        // rows a workgroup
    constexpr int BPS = S / 16;              // 16-token blocks a step

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int hk = p.cache.heads, pb = p.cache.page_blocks;
    int id = blockIdx.x;
    const int tile = id % pl.tiles;
    id /= pl.tiles;
    const int split = id % pl.splits;
    id /= pl.splits;
    const int head = id % hk, b = id / hk;

    const int T = static_cast<int>(p.T);
    int q0 = p.q_start[b], q1 = p.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0 > T ? T : q0;
    q1 = q1 > T ? T : q1;
    q1 = q1 > q0 + p.max_q ? q0 + p.max_q : q1;
    const int n = q1 > q0 ? q1 - q0 : 0;
    const int rows = n * pl.group;
    const int tile_row = tile * ROWS;
    if (tile_row >= rows) return;
    int len = p.kv_len[b];
    len = len < 0 ? 0 : len > p.max_kv ? p.max_kv : len;
    const int past = len - n;

    // this lane's rows
    const int wk = WK > 1 ? wave : 0;
    const int row0 = tile_row + (WK > 1 ? 0 : wave * 16 * R);
    int node[R], low[R];
    bool live[R];
    const uint16_t* qp[R];
    int lo_min = 0x7FFFFFFF, lo_max = 0, node_max = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + 16 * r + m;
        live[r] = row < rows;
        const int at = live[r] ? row : rows - 1;
        node[r] = at / pl.group;
        const int h = head * pl.group + (at - node[r] * pl.group);
        qp[r] = p.q + static_cast<int64_t>(q0 + node[r]) * p.q_stride + static_cast<int64_t>(h) * D;
        const int pos = p.positions ? p.positions[q0 + node[r]] : past + node[r];
        low[r] = p.window > 0 ? pos - p.window + 1 : 0;
        lo_min = low[r] < lo_min ? low[r] : lo_min;
        lo_max = low[r] > lo_max ? low[r] : lo_max;
        node_max = node[r] > node_max ? node[r] : node_max;
    }
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
        lo_min = min(lo_min, __shfl_xor(lo_min, off));
        lo_max = max(lo_max, __shfl_xor(lo_max, off));
        node_max = max(node_max, __shfl_xor(node_max, off));
    }
    lo_min = __builtin_amdgcn_readfirstlane(lo_min);
    lo_max = __builtin_amdgcn_readfirstlane(lo_max);
    node_max = __builtin_amdgcn_readfirstlane(node_max);

    // the sequence's first visible token, where split 0 starts
    int first = 0;
    if (p.window > 0) {
        int least = past;
        if (p.positions) {
            least = 0x7FFFFFFF;
            for (int i = lane; i < n; i += 64) least = min(least, p.positions[q0 + i]);
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) least = min(least, __shfl_xor(least, off));
            least = __builtin_amdgcn_readfirstlane(least);
        }
        least = least - p.window + 1;
        first = least > past ? past : least;
        first = first < 0 ? 0 : first & ~63;
    }
    int begin = first + split * pl.chunk;
    int end = split == pl.splits - 1 ? len : begin + pl.chunk;
    // nodes beyond the last row of a chain, and tokens before every window, are seen by none
    if (!p.tree && end > past + node_max + 1) end = past + node_max + 1;
    if (end > len) end = len;
    // (with a window, nodes are seen by their positions: only context tokens are skipped by index)
    const int from = lo_min < past ? lo_min : past;
    if (begin < from) begin = from & ~63;

    uint4 Q[R][KS];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            // dims of operand s in lane group g, as K's pieces hold them
            const int d = E == 2 ? 32 * s + 8 * g : 64 * (s >> 1) + 16 * g + 8 * (s & 1);
            Q[r][s] = *reinterpret_cast<const uint4*>(qp[r] + d);
        }

    float4_t O[R][DT];
    float mx[R], sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mx[r] = -INFINITY;
        sum[r] = 0.0f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) O[r][dt] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const float scale = p.scale * 1.4426950408889634f * (E == 1 ? p.cache.k_scale[head] : 1.0f);
    const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.table_pages;
    const int last_block = len > 0 ? (len - 1) >> 4 : 0;

    // index of a block of the cache (in 16-token blocks of this head), or -1
    auto block_at = [&](int blk) -> int64_t {
        blk = blk > last_block ? last_block : blk;
        const int pg = pb > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(blk), pl.page_magic)) : blk;
        const int64_t page = table[pg];
        if (page < 0 || page >= p.cache.pages) return -1;
        return (page * hk + head) * pb + (blk - pg * pb);
    };

    for (int st = begin / S + wk; st * S < end; st += WK) {
        const int k0 = st * S;
        const int64_t kb = block_at(st * BPS + (m * BPS >> 4));
        const int64_t vb = block_at(st * BPS + (g * BPS >> 2));
        const bool absent = vb < 0;
        const uint8_t* kp = static_cast<const uint8_t*>(p.cache.k) + (kb < 0 ? 0 : kb) * (16 * D * E);
        const uint8_t* vp = static_cast<const uint8_t*>(p.cache.v) + (absent ? 0 : vb) * (16 * D * E);
        // V: the piece of this lane's dim and group of tokens (two groups share a block of bf16)
        vp += (E == 2 ? (g & 1) * (16 * D) : 0) + m * 16;

        float4_t acc[R][NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int token = (S / 4) * (m >> 2) + 4 * t + (m & 3);   // of the step
            const uint8_t* row = kp + (token & 15) * 16;
            uint4 K[KS];
            if constexpr (E == 2) {
#pragma unroll
                for (int s = 0; s < KS; ++s) K[s] = *reinterpret_cast<const uint4*>(row + (4 * s + g) * 256);
            } else {
#pragma unroll
                for (int s = 0; s < KS; s += 2) {
                    const uint4 c = *reinterpret_cast<const uint4*>(row + (2 * s + g) * 256);
                    widen16(c, K[s], K[s + 1]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                acc[r][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < KS; ++s) acc[r][t] = mfma(K[s], Q[r][s], acc[r][t]);
            }
        }

        const bool masked = k0 + S > (past < len ? past : len) || k0 < lo_max || __any(absent);
        uint32_t seen[R];                    // bit 4 t + j: this lane's row sees token (S/4) g + 4 t + j
        uint4 P[R][NP];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            seen[r] = 0xFFFFFFFFu;
            if (masked) {
                seen[r] = 0;
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) {
                    const int key = k0 + (S / 4) * g + i;
                    bool ok = live[r] && !absent && key < len;
                    if (ok && key < past) {
                        ok = key >= low[r];
                    } else if (ok) {
                        const int j = key - past;
                        ok = p.tree ? (p.tree[static_cast<int64_t>(q0 + node[r]) * p.tree_words + (j >> 6)] >> (j & 63)) & 1
                                    : j <= node[r];
                        if (p.window > 0) ok = ok && (p.positions ? p.positions[q0 + j] : key) >= low[r];
                    }
                    seen[r] |= (ok ? 1u : 0u) << i;
                }
            }
            float s[4 * NT];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4 * NT; ++i) {
                s[i] = acc[r][i >> 2][i & 3] * scale;
                if (masked) s[i] = (seen[r] >> i) & 1 ? s[i] : -INFINITY;
                top = fmaxf(top, s[i]);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(mx[r], top);
            const float ref = now == -INFINITY ? 0.0f : now;
            const float fade = exp2_fast(mx[r] - ref);
            mx[r] = now;
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * NT; ++i) {
                s[i] = exp2_fast(s[i] - ref);
                part += s[i];
            }
            sum[r] = sum[r] * fade + part;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) O[r][dt] *= fade;
#pragma unroll
            for (int q = 0; q < NP; ++q)
                P[r][q] = make_uint4(pack_bf16x2(s[8 * q], s[8 * q + 1]), pack_bf16x2(s[8 * q + 2], s[8 * q + 3]),
                                     pack_bf16x2(s[8 * q + 4], s[8 * q + 5]), pack_bf16x2(s[8 * q + 6], s[8 * q + 7]));
        }

#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            uint4 V[NP];
            const uint4 c = *reinterpret_cast<const uint4*>(vp + dt * 256);
            if constexpr (E == 2) V[0] = c;
            else widen16(c, V[0], V[NP - 1]);
            bool odd = false;
            if (masked) {
                // what lies behind the last token is not data
                const int left = len - (k0 + (S / 4) * g);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    V[q] = first_of(V[q], left - 8 * q);
                    odd = odd || nonfinite_bf16x2(V[q].x) || nonfinite_bf16x2(V[q].y) || nonfinite_bf16x2(V[q].z) ||
                          nonfinite_bf16x2(V[q].w);
                }
            }
            if (masked && __any(odd)) {
                // an infinity or NaN among the values of a step that not every
                // row sees (0 times it would be NaN): token by token, each
                // added only to the rows that see it
                for (int i = 0; i < 4 * NT; ++i)
                    for (int gg = 0; gg < 4; ++gg) {
                        const uint4 zero = make_uint4(0, 0, 0, 0);
                        const int q = i >> 3;
                        const uint4 v1 = g == gg ? only(NP > 1 && q ? V[NP - 1] : V[0], i & 7) : zero;
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const uint4 p1 = g == gg ? only(NP > 1 && q ? P[r][NP - 1] : P[r][0], i & 7) : zero;
                            const float4_t add = mfma(v1, p1, float4_t{0.0f, 0.0f, 0.0f, 0.0f});
                            const uint32_t sees = static_cast<uint32_t>(__shfl(static_cast<int>(seen[r]), 16 * gg + m));
                            if ((sees >> i) & 1) O[r][dt] += add;
                        }
                    }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int q = 0; q < NP; ++q) O[r][dt] = mfma(V[q], P[r][q], O[r][dt]);
            }
        }
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        sum[r] += __shfl_xor(sum[r], 16);
        sum[r] += __shfl_xor(sum[r], 32);
    }

    const float v_scale = E == 1 ? p.cache.v_scale[head] : 1.0f;
    const int64_t all = p.T * p.hq;
    float* part_ml = p.ws + static_cast<int64_t>(pl.splits) * all * D;
    // four dims of one row: to O, or as a partial result to the workspace
    auto put = [&](int row, int d, float4_t o, float top, float total) {
        const int nd = row / pl.group;
        const int64_t at = static_cast<int64_t>(q0 + nd) * p.hq + head * pl.group + (row - nd * pl.group);
        if (pl.splits == 1) {
            const float f = total > 0.0f || total != total ? v_scale / total : 0.0f;
            *reinterpret_cast<uint2*>(p.O + at * D + d) = make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
        } else {
            const int64_t slice = static_cast<int64_t>(split) * all + at;
            *reinterpret_cast<float4_t*>(p.ws + slice * D + d) = o;
            if (d == 0) *reinterpret_cast<float2_t*>(part_ml + 2 * slice) = float2_t{top, total};
        }
    };

    if constexpr (WK == 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!live[r]) continue;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) put(row0 + 16 * r + m, 16 * dt + 4 * g, O[r][dt], mx[r], sum[r]);
        }
    } else {
        // the waves hold the same rows over different tokens: join them, a
        // quarter of the dims at a time
        constexpr int DQ = DT / 4;
        __shared__ float sm_top[WK][16 * R], sm_sum[WK][16 * R];
        __shared__ float4_t sm_o[WK][DQ * 4][16 * R];
        if (g == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sm_top[wave][16 * r + m] = mx[r];
                sm_sum[wave][16 * r + m] = sum[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = sm_top[0][16 * r + m];
#pragma unroll
            for (int w = 1; w < WK; ++w) top = fmaxf(top, sm_top[w][16 * r + m]);
            const float f = mx[r] == -INFINITY ? 0.0f : exp2_fast(mx[r] - top);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) O[r][dt] *= f;
        }
#pragma unroll
        for (int quarter = 0; quarter < 4; ++quarter) {
            if (quarter) __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int x = 0; x < DQ; ++x) sm_o[wave][4 * x + g][16 * r + m] = O[r][quarter * DQ + x];
            __syncthreads();
            for (int u = threadIdx.x; u < DQ * 4 * 16 * R; u += 256) {
                const int lr = u / (DQ * 4), d4 = u - lr * (DQ * 4);
                if (tile_row + lr >= rows) continue;
                float top = sm_top[0][lr];
#pragma unroll
                for (int w = 1; w < WK; ++w) top = fmaxf(top, sm_top[w][lr]);
                float total = 0.0f;
                float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    // (a NaN sum stays one)
                    const float t = sm_top[w][lr];
                    total += sm_sum[w][lr] * (t == -INFINITY ? 0.0f : exp2_fast(t - top));
                    o += sm_o[w][d4][lr];
                }
                put(tile_row + lr, quarter * (D / 4) + 4 * d4, o, top, total);
            }
        }
    }
}

// The splits of a row joined in order: one wavefront a row.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(AttentionParams p, AttentionPlan pl) {
    constexpr int N = D / 64;                // dims a lane
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.y;
    const int T = static_cast<int>(p.T);
    int q0 = p.q_start[b], q1 = p.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0 > T ? T : q0;
    q1 = q1 > T ? T : q1;
    q1 = q1 > q0 + p.max_q ? q0 + p.max_q : q1;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= static_cast<int64_t>(q1 - q0) * p.hq) return;
    const int64_t at = static_cast<int64_t>(q0) * p.hq + row;
    const int64_t all = p.T * p.hq;
    const float* ml = p.ws + static_cast<int64_t>(pl.splits) * all * D;
    float top = -INFINITY;
    for (int s = lane; s < pl.splits; s += 64) top = fmaxf(top, ml[2 * (s * all + at)]);
    top = wave_max(top);
    float total = 0.0f, o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.0f;
    for (int s = 0; s < pl.splits; ++s) {
        const float2_t t = *reinterpret_cast<const float2_t*>(ml + 2 * (s * all + at));
        if (t[0] == -INFINITY && t[1] == 0.0f) continue;   // saw nothing
        const float f = t[0] == -INFINITY ? 0.0f : exp2_fast(t[0] - top);
        total += t[1] * f;
        const float* src = p.ws + (s * all + at) * D + N * lane;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] += src[i] * f;
    }
    const float v_scale = p.cache.e4m3 ? p.cache.v_scale[(row % p.hq) / pl.group] : 1.0f;
    const float f = total > 0.0f || total != total ? v_scale / total : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) p.O[at * D + N * lane + i] = float_to_bf16_bits(o[i] * f);
}

// Rows a workgroup holds, by the rows a (sequence, head) has: up to 16, 32 or
// 64 rows its four waves share them and divide the tokens; above, each wave
// has rows of its own.
int rows_per_tile(int dim, int64_t rows) {
    if (rows <= 16) return 16;
    if (rows <= 32) return 32;
    if (dim == 256) return rows <= 64 ? 32 : 128;
    return rows <= 64 ? 64 : 256;
}

AttentionPlan make_plan(int64_t B, int hq, int hk, int dim, int64_t max_q, int64_t max_kv, int64_t window) {
    AttentionPlan pl{};
    pl.group = hq / hk;
    const int64_t rows = max_q * pl.group;
    const int tile = rows_per_tile(dim, rows);
    pl.tiles = static_cast<int>((rows + tile - 1) / tile);
    // tokens that one sequence's rows can see (a window starts at a multiple of 64)
    int64_t span = max_kv;
    if (window > 0 && window + max_q + 64 < span) span = window + max_q + 64;
    const int64_t whole = B * hk * pl.tiles;
    int64_t splits = (1024 + whole - 1) / whole;
    const int64_t most = (span + 255) / 256;
    splits = splits < most ? splits : most;
    splits = splits < 1 ? 1 : splits;
    int64_t chunk = (span + splits - 1) / splits;
    chunk = (chunk + 255) / 256 * 256;
    pl.chunk = static_cast<int>(chunk);
    pl.splits = static_cast<int>((span + chunk - 1) / chunk);
    if (pl.splits < 1) pl.splits = 1;
    return pl;
}

template <int D, int E>
void launch_tiles(const AttentionParams& p, const AttentionPlan& pl, dim3 grid, hipStream_t stream) {
    switch (rows_per_tile(D, static_cast<int64_t>(p.max_q) * pl.group)) {
        case 16: hipLaunchKernelGGL((attention_kernel<D, E, 1, 4>), grid, dim3(256), 0, stream, p, pl); break;
        case 32: hipLaunchKernelGGL((attention_kernel<D, E, 2, 4>), grid, dim3(256), 0, stream, p, pl); break;
        case 64:
            if constexpr (D < 256) hipLaunchKernelGGL((attention_kernel<D, E, 4, 4>), grid, dim3(256), 0, stream, p, pl);
            break;
        default: hipLaunchKernelGGL((attention_kernel<D, E, D == 256 ? 2 : 4, 1>), grid, dim3(256), 0, stream, p, pl); break;
    }
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int64_t B, int hq, int hk, int dim, bool e4m3, int64_t max_q,
                                 int64_t max_kv, int64_t window) {
    const AttentionPlan pl = make_plan(B, hq, hk, dim, max_q, max_kv, window);
    if (pl.splits == 1) return 0;
    return static_cast<size_t>(pl.splits) * T * hq * (dim + 2) * sizeof(float);
}

hipError_t launch_attention(const AttentionParams& p, hipStream_t stream) {
    AttentionPlan pl = make_plan(p.B, p.hq, p.cache.heads, p.cache.dim, p.max_q, p.max_kv, p.window);
    const int pb = p.cache.page_blocks;
    pl.page_magic = pb > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + pb - 1) / pb) : 0;
    const int64_t groups = static_cast<int64_t>(pl.tiles) * pl.splits * p.cache.heads * p.B;
    if (groups > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(groups));
    if (p.cache.e4m3) {
        if (p.cache.dim == 64) launch_tiles<64, 1>(p, pl, grid, stream);
        else if (p.cache.dim == 128) launch_tiles<128, 1>(p, pl, grid, stream);
        else launch_tiles<256, 1>(p, pl, grid, stream);
    } else {
        if (p.cache.dim == 64) launch_tiles<64, 2>(p, pl, grid, stream);
        else if (p.cache.dim == 128) launch_tiles<128, 2>(p, pl, grid, stream);
        else launch_tiles<256, 2>(p, pl, grid, stream);
    }
    if (pl.splits > 1) {
        const dim3 jgrid(static_cast<unsigned>((static_cast<int64_t>(p.max_q) * p.hq + 3) / 4), p.B);
        if (p.cache.dim == 64) hipLaunchKernelGGL(attention_join_kernel<64>, jgrid, dim3(256), 0, stream, p, pl);
        else if (p.cache.dim == 128) hipLaunchKernelGGL(attention_join_kernel<128>, jgrid, dim3(256), 0, stream, p, pl);
        else hipLaunchKernelGGL(attention_join_kernel<256>, jgrid, dim3(256), 0, stream, p, pl);
    }
    return hipGetLastError();
}

}  // namespace w4
