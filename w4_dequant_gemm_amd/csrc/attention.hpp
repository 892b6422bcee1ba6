// Shared by the attention kernels (attention.hip, attention_tile.hip): launch
// plan, a sequence's view, masks, operand helpers.
#pragma once

#include "device.hpp"
#include "decode_kernels.hpp"

namespace w4 {
namespace attn {

// Launch plan: tokens [c * chunk, (c + 1) * chunk) of a sequence (from its
// first visible one) are split c; `tiles` row tiles a (sequence, head).
struct AttentionPlan {
    int chunk, splits, tiles;
    int group;               // query heads a KV head
    int tile_rows;           // rows a workgroup
    uint32_t page_magic;     // block / page_blocks as a high product (page_blocks > 1)
};

constexpr float kRaise = 8.0f;               // log2 of the largest p
constexpr float kFar = 0x1p28f;              // references from here on: see rounded_exponent

// whether any of a piece's values (8 bf16 or 16 E4M3) is infinite or NaN
template <int E>
__device__ __forceinline__ bool nonfinite(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // all exponent (E4M3: all) bits set: adding one to the field carries into the sign's place
        if constexpr (E == 2) any = any || (((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0;
        else any = any || (((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
    }
    return any;
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

// The exponent of p for a score far from 0.  A fused x scale - ref keeps what
// rounding the reference has lost, up to half a unit in its last place: the same
// for all scores of a row, so it cancels, but from 2^31 on it may be 128, and
// p infinite.  With the product rounded as the reference was, nothing is left.
__device__ __forceinline__ float rounded_exponent(float x, float scale, float ref) {
#pragma clang fp contract(off)
    return x * scale - ref;
}

// maximum over the four lane groups (lanes m, m + 16, m + 32, m + 48)
__device__ __forceinline__ float max_groups(float x) {
    const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Eight bf16 values with infinities and NaN replaced by 0; `plus` is 1 where
// +inf or NaN stood, `minus` where -inf or NaN did.
__device__ __forceinline__ uint4 finite_part(const uint4& v, uint4& plus, uint4& minus) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t f[4], a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t out = (((((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15)) * 0xFFFFu;
        const uint32_t nan = ((((w[i] & 0x007F007Fu) + 0x007F007Fu) & 0x00800080u) >> 7) * 0xFFFFu;
        const uint32_t neg = ((w[i] & 0x80008000u) >> 15) * 0xFFFFu;
        f[i] = w[i] & ~out;
        a[i] = out & (nan | ~neg) & 0x3F803F80u;
        b[i] = out & (nan | neg) & 0x3F803F80u;
    }
    plus = make_uint4(a[0], a[1], a[2], a[3]);
    minus = make_uint4(b[0], b[1], b[2], b[3]);
    return make_uint4(f[0], f[1], f[2], f[3]);
}

// A cached piece with its infinities and NaN replaced by 0.
template <int E>
__device__ __forceinline__ uint4 finite_piece(const uint4& v) {
    if constexpr (E == 2) {
        uint4 plus, minus;
        return finite_part(v, plus, minus);
    } else {
        auto fine = [](uint32_t w) {
            const uint32_t out = ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
            return w & ~out;
        };
        return make_uint4(fine(v.x), fine(v.y), fine(v.z), fine(v.w));
    }
}

// bf16 1 at the elements whose bit is set
__device__ __forceinline__ uint4 ones_at(uint32_t bits) {
    auto two = [&](int i) { return ((bits >> i) & 1 ? 0x3F80u : 0u) | ((bits >> i) & 2 ? 0x3F800000u : 0u); };
    return make_uint4(two(0), two(2), two(4), two(6));
}

// the low n bits (n may lie outside 0 .. 32)
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// A sequence as one workgroup sees it.
struct Sequence {
    int q0, n;               // its rows of q
    int len, past;           // cached tokens; those before its nodes
    int first;               // token that split 0 starts at
    const int32_t* table;
    int last_block;
    bool holes;              // a page of the split's range lies outside the cache
    bool spread;             // the nodes' positions differ by the window or more
};

__device__ __forceinline__ void sequence_rows(const AttentionParams& p, int b, int& q0, int& n) {
    const int T = static_cast<int>(p.T);
    int a = p.q_start[b], e = p.q_start[b + 1];
    a = a < 0 ? 0 : a > T ? T : a;
    e = e > T ? T : e;
    n = e > a ? e - a : 0;
    n = n < p.max_q ? n : p.max_q;
    q0 = a;
}

__device__ __forceinline__ int page_of(const AttentionParams& p, const AttentionPlan& pl, int blk) {
    return p.cache.page_blocks > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(blk), pl.page_magic)) : blk;
}

// The tokens [begin, end) of one split that rows up to node `node_last` can
// see (begin a multiple of 64).
__device__ __forceinline__ void split_range(const AttentionParams& p, const AttentionPlan& pl, Sequence& s, int b,
                                            int split, int node_first, int node_last, int& begin, int& end) {
    const int lane = threadIdx.x & 63;
    s.table = p.page_table + static_cast<int64_t>(b) * p.table_pages;
    s.last_block = s.len > 0 ? (s.len - 1) >> 4 : 0;
    s.first = 0;
    int lowest = 0;                          // no row of the tile sees a context token below
    s.spread = false;
    if (p.window > 0) {
        int least = s.past, most = s.past + s.n - 1;   // the lowest and highest position
        if (p.positions) {
            least = 0x7FFFFFFF;
            most = -0x7FFFFFFF;
            for (int i = lane; i < s.n; i += 64) {
                const int at = p.positions[s.q0 + i];
                least = min(least, at);
                most = max(most, at);
            }
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                least = min(least, __shfl_xor(least, off));
                most = max(most, __shfl_xor(most, off));
            }
            least = __builtin_amdgcn_readfirstlane(least);
            most = __builtin_amdgcn_readfirstlane(most);
        }
        s.spread = static_cast<int64_t>(most) - least >= p.window;
        lowest = least + (p.positions ? 0 : node_first) - p.window + 1;
        least = least - p.window + 1;
        least = least < s.past ? least : s.past;
        lowest = lowest < s.past ? lowest : s.past;
        s.first = least > 0 ? least & ~63 : 0;
        lowest = lowest > 0 ? lowest & ~63 : 0;
    }
    begin = s.first + split * pl.chunk;
    end = split == pl.splits - 1 ? s.len : begin + pl.chunk;
    if (!p.tree && end > s.past + node_last + 1) end = s.past + node_last + 1;
    if (end > s.len) end = s.len;
    if (begin < lowest) begin = lowest;
    bool bad = false;
    if (begin < end)
        for (int i = page_of(p, pl, begin >> 4) + lane; i <= page_of(p, pl, (end - 1) >> 4); i += 64) {
            const int64_t page = s.table[i];
            bad = bad || page < 0 || page >= p.cache.pages;
        }
    s.holes = __any(bad);
}

// bit i: a row (its node, its lowest visible token) sees token kf + i, for a run
// of `run` <= 16 tokens inside one 16-token block.
__device__ __forceinline__ uint32_t sees(const AttentionParams& p, const AttentionPlan& pl, const Sequence& s, int node,
                                         int low, int kf, int run) {
    const int c = s.past - kf;               // tokens of the context among them
    const int j0 = kf - s.past;              // node of the first
    uint32_t context = low_bits(c) & ~low_bits(low - kf);
    uint32_t nodes = 0;
    if (c < run && kf < s.len) {
        if (p.tree) {
            const uint64_t* words = p.tree + static_cast<int64_t>(s.q0 + node) * p.tree_words;
            if (j0 >= 0) {
                const int w = j0 >> 6, o = j0 & 63;
                uint64_t bits = w < p.tree_words ? words[w] >> o : 0;
                if (o > 64 - run && w + 1 < p.tree_words) bits |= words[w + 1] << (64 - o);
                nodes = static_cast<uint32_t>(bits);
            } else {
                nodes = static_cast<uint32_t>(words[0] << c);
            }
        } else {
            nodes = low_bits(node - j0 + 1);
        }
        if (s.spread) {
            if (p.positions) {
                for (int i = c > 0 ? c : 0; i < run && kf + i < s.len; ++i)
                    if (p.positions[s.q0 + j0 + i] < low) nodes &= ~(1u << i);
            } else {
                nodes &= ~low_bits(low - kf);
            }
        }
    }
    uint32_t bits = (context | (nodes & ~low_bits(c))) & low_bits(s.len - kf) & low_bits(run);
    if (s.holes && kf < s.len) {
        const int64_t page = s.table[page_of(p, pl, kf >> 4)];
        if (page < 0 || page >= p.cache.pages) bits = 0;
    }
    return bits;
}

// Four dims of one row: to O, or as a partial result to the workspace
// (partials [split][T hq][D], then reference and sum [split][T hq][2]).
template <int D, int E>
__device__ __forceinline__ void put(const AttentionParams& p, const AttentionPlan& pl, int q0, int head, int split, int row,
                                    int d, float4_t o, float ref, float total) {
    const int nd = row / pl.group;
    const int64_t at = static_cast<int64_t>(q0 + nd) * p.hq + head * pl.group + (row - nd * pl.group);
    if (pl.splits == 1) {
        const float f = total != 0.0f ? (E == 1 ? p.cache.v_scale[head] : 1.0f) / total : 0.0f;
        *reinterpret_cast<uint2*>(p.O + at * D + d) = make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
    } else {
        const int64_t all = p.T * p.hq;
        const int64_t slice = static_cast<int64_t>(split) * all + at;
        *reinterpret_cast<float4_t*>(p.ws + slice * D + d) = o;
        if (d == 0)
            *reinterpret_cast<float2_t*>(p.ws + static_cast<int64_t>(pl.splits) * all * D + 2 * slice) = float2_t{ref, total};
    }
}

}  // namespace attn

// launches of the tile kernel (pl.tile_rows rows a workgroup, grid of wgs)
hipError_t launch_attention_tiles(const AttentionParams& p, const attn::AttentionPlan& pl, unsigned wgs, hipStream_t stream);

}  // namespace w4
