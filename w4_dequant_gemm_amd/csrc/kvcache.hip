// The paged cache of keys and values: appending rows of a QKV product (with
// the heads' norms and the rotation on the way) and moving an accepted path.
#include <type_traits>

#include "device.hpp"
#include "decode_kernels.hpp"

namespace w4 {
namespace {

// E4M3 saturates at +-448; NaN stays one.
__device__ __forceinline__ float to_e4m3_range(float x) { return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f); }

// Eight fp32 values -> E4M3 codes of v / s.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float s) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_e4m3_range(v[i] / s);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    return make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

// The values of 16 tokens of one head, a workgroup.  A piece of V's cache holds
// C tokens of one dim, so neighbouring tokens are put together in shared memory
// and whole pieces written where their slots fill one (writes of single
// elements cost the memory a read each: 4100 tokens, E4M3: 20 us of 34).  The
// workgroup writes the pieces that begin with one of its tokens and so reads up
// to C - 1 tokens more.
template <int D, int E>
__device__ __forceinline__ void append_values(const KvAppendParams& p, int tile, int head) {
    using T = typename std::conditional<E == 1, uint8_t, uint16_t>::type;
    constexpr int C = 16 / E;                // tokens a piece
    constexpr int ROWS = 16 + C;             // one before this tile's, and C - 1 behind
    __shared__ int slots[ROWS], runs[16];
    __shared__ __attribute__((aligned(16))) uint16_t rows[ROWS - 1][D];
    const int t0 = tile * 16, tid = threadIdx.x;
    const int page_size = 16 * p.cache.page_blocks;
    const int64_t all = p.cache.pages * page_size;
    if (tid < ROWS) {
        const int t = t0 - 1 + tid;
        const int slot = t >= 0 && t < p.T ? p.slots[t] : -1;
        slots[tid] = slot < all ? slot : -1;
    }
    for (int i = tid; i < (ROWS - 1) * (D / 8); i += 256) {
        const int row = i / (D / 8), c = i % (D / 8);
        if (t0 + row < p.T)
            *reinterpret_cast<uint4*>(&rows[row][8 * c]) =
                *reinterpret_cast<const uint4*>(p.v + (t0 + row) * p.v_stride + static_cast<int64_t>(head) * D + 8 * c);
    }
    __syncthreads();
    if (tid < 16) {
        // tokens of the piece that begins here; none if it is not stored or the
        // token before lies in the same piece, just before
        const int slot = slots[tid + 1];
        int n = 0;
        if (slot >= 0 && (slot % C == 0 || slots[tid] != slot - 1)) {
            bool on = true;
#pragma unroll
            for (int i = 1; i < C; ++i) {
                on = on && slot % C + i < C && slots[tid + 1 + i] == slot + i;
                n += on;
            }
            ++n;
        }
        runs[tid] = n;
    }
    __syncthreads();
    const float scale = E == 1 ? p.cache.v_scale[head] : 1.0f;
    const int d = tid % D;
    for (int i = tid / D; i < 16; i += 256 / D) {
        const int n = runs[i];
        if (n == 0) continue;
        const int slot = slots[i + 1];
        const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(page_size);
        const int in_page = slot - static_cast<int>(page) * page_size;
        const int64_t block = (static_cast<int64_t>(page) * p.cache.heads + head) * p.cache.page_blocks + (in_page >> 4);
        T* to = static_cast<T*>(p.cache.v) + ((block * (16 / C) + (in_page & 15) / C) * D + d) * C;
        if (n == C) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (E == 2) {
                    w[j] = rows[i + 2 * j][d] | static_cast<uint32_t>(rows[i + 2 * j + 1][d]) << 16;
                } else {
                    float f[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[k] = to_e4m3_range(bf16_lo(rows[i + 4 * j + k][d]) / scale);
                    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
                    w[j] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true));
                }
            }
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int j = 0; j < n; ++j) {
                const uint16_t x = rows[i + j][d];
                if constexpr (E == 2) to[slot % C + j] = x;
                else to[slot % C + j] = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(bf16_lo(x) / scale), 0.0f, 0, false));
            }
        }
    }
}

// Bound by memory: 4100 tokens of 32 + 8 heads of 128, normed and rotated into an
// E4M3 cache, 94 MB in 23 to 25 us (3.8 to 4.1 TB/s; a copy of that size 5.4).  5
// tokens: 3.3 us, a launch.
//
// Query and key heads: D / 8 lanes (eight dims each) take four heads of one
// token, whose loads are on their way together under one lookup of the token's
// position, angles and slot (one head at a time the chain of those lookups
// bounds it: 4100 tokens, 32 us); the norm's sum and the rotation's partner
// values are exchanged inside the row's own lanes.  Neighbouring rows of lanes
// have neighbouring tokens, whose pieces of K lie side by side.  Workgroups
// from row_groups on store the values.
template <int D, int E>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendParams p, uint32_t row_groups) {
    constexpr int L = D / 8;                 // lanes a row
    constexpr int H = 4;                     // heads of a row
    const int hk = p.cache.heads;
    if (blockIdx.x >= row_groups) {
        const uint32_t id = blockIdx.x - row_groups;
        append_values<D, E>(p, static_cast<int>(id / static_cast<uint32_t>(hk)), static_cast<int>(id % static_cast<uint32_t>(hk)));
        return;
    }
    const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / L;
    const int c = threadIdx.x % L;           // dims 8c .. 8c + 7
    const uint32_t q_quads = static_cast<uint32_t>((p.hq + H - 1) / H), quads = q_quads + static_cast<uint32_t>((hk + H - 1) / H);
    const uint32_t sixteen = row >> 4, group = sixteen / quads;
    const uint32_t t = group * 16u + (row & 15u);
    if (t >= static_cast<uint32_t>(p.T)) return;   // whole rows leave together
    const uint32_t quad = sixteen - group * quads;
    const bool is_q = quad < q_quads;
    const int head0 = static_cast<int>(is_q ? quad : quad - q_quads) * H;
    const int heads = is_q ? p.hq : hk;
    const uint16_t* src = (is_q ? p.q + t * p.q_stride : p.k + t * p.k_stride) + static_cast<int64_t>(head0) * D + 8 * c;
    uint4 w[H];
#pragma unroll
    for (int i = 0; i < H; ++i) w[i] = head0 + i < heads ? *reinterpret_cast<const uint4*>(src + i * D) : make_uint4(0, 0, 0, 0);
    const float* norm = is_q ? p.q_norm : p.k_norm;
    float weight[8];
    if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) weight[i] = norm[8 * c + i];
    }
    // the angles' cosines and sines of this lane's dims (interleaved: of its four pairs)
    const int half = p.rot >> 4;             // lanes that hold the first of each pair (halves)
    const bool turns = p.rope && c < 2 * half;
    const bool first = c < half;
    bool inside = true;
    float co[8], si[8];
    if (turns) {
        const int64_t pos = p.positions[t];
        inside = pos >= 0 && pos < p.rope_rows;
        const float* cs = p.rope + (inside ? pos : 0) * p.rot + (p.interleaved ? 4 * c : 8 * (first ? c : c - half));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            co[i] = cs[i];
            si[i] = cs[(p.rot >> 1) + i];
        }
        if (!p.interleaved)
#pragma unroll
            for (int i = 4; i < 8; ++i) {
                co[i] = cs[i];
                si[i] = cs[(p.rot >> 1) + i];
            }
    }
    int64_t block = -1;
    int s = 0;
    if (!is_q) {
        const int64_t slot = p.slots[t];
        const int page_size = 16 * p.cache.page_blocks;
        if (slot >= 0 && slot < p.cache.pages * page_size) {
            const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(page_size);
            const int in_page = static_cast<int>(slot) - static_cast<int>(page) * page_size;
            s = in_page & 15;
            block = (static_cast<int64_t>(page) * hk + head0) * p.cache.page_blocks + (in_page >> 4);
        }
    }
#pragma unroll
    for (int j = 0; j < H; ++j) {
        if (head0 + j >= heads) break;       // (the same for a row's lanes)
        float x[8] = {bf16_lo(w[j].x), bf16_hi(w[j].x), bf16_lo(w[j].y), bf16_hi(w[j].y),
                      bf16_lo(w[j].z), bf16_hi(w[j].z), bf16_lo(w[j].w), bf16_hi(w[j].w)};
        if (norm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
            for (int off = L / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, L);
            const float r = 1.0f / sqrtf(sum * (1.0f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * weight[i];
        }
        if (p.rope) {
            if (p.interleaved) {
                if (turns)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = a * co[i] - b * si[i];
                        x[2 * i + 1] = b * co[i] + a * si[i];
                    }
            } else {
                const int partner = turns ? (first ? c + half : c - half) : c;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], partner, L);
                if (turns)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * co[i] - y[i] * si[i] : x[i] * co[i] + y[i] * si[i];
            }
            if (turns && !inside)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
        }
        const uint4 o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        if (is_q) {
            *reinterpret_cast<uint4*>(p.Q + (static_cast<int64_t>(t) * p.hq + head0 + j) * D + 8 * c) = o;
        } else if (block >= 0) {
            uint8_t* dst = static_cast<uint8_t*>(p.cache.k) + (block + j * p.cache.page_blocks) * (16 * D * E);
            if constexpr (E == 1) *reinterpret_cast<uint2*>(dst + (c >> 1) * 256 + s * 16 + (c & 1) * 8) = e4m3x8(x, p.cache.k_scale[head0 + j]);
            else *reinterpret_cast<uint4*>(dst + c * 256 + s * 16) = o;
        }
    }
}

// A workgroup moves 512 / D heads of one sequence and layer.  The tokens' blocks
// are looked up 64 at a time; then, as many tokens at a time as their new places
// have in one piece of V (8 or 16), all pieces are read, the loads on their way together,
// then, after a barrier, all written.  V's new pieces are read, filled in and
// written whole: writes of single elements cost the memory a read each (64 paths
// in 32 layers: 105 us against 95).  path[j] >= j and the path ascends, so no
// later token's source was written.  64 paths of up to 7 tokens, 32 layers, 8
// heads of 128: 95 to 100 us.  Of 67 MB that a move needs, 265 MB are read: a
// token's pieces of 16 bytes (K) and its elements of V's pieces each lie in a
// 64-byte sector of their own, the price of a layout whose pieces attention
// reads as operands.
template <int D, int E>
__global__ void __launch_bounds__(256) kv_move_kernel(KvMoveParams p) {
    using T = typename std::conditional<E == 1, uint8_t, uint16_t>::type;
    constexpr int C = 16 / E, PIECES = D / C;
    constexpr int KI = C * (512 / C) / 256;  // 16-byte pieces of K a thread
    constexpr int kTokens = 64;              // looked up at a time
    __shared__ int64_t from_block[kTokens];  // by new place; -1: stays
    __shared__ int from_slot[kTokens];
    __shared__ int64_t piece_block[kTokens / C];
    const int hk = p.cache.heads, pb = p.cache.page_blocks;
    const int tid = threadIdx.x, b = blockIdx.y, head0 = blockIdx.x * (512 / D);
    int n = p.count[b];
    n = n < p.path_len ? n : static_cast<int>(p.path_len);
    const int64_t base = p.base[b];
    if (base < 0) return;
    const int32_t* table = p.page_table + b * p.table_pages;
    const int32_t* path = p.path + b * p.path_len;
    const int64_t layer = static_cast<int64_t>(blockIdx.z) * p.cache.pages * hk * pb;

    // block of head 0 (head h is h pb further), or -1
    auto block_of = [&](int64_t token) -> int64_t {
        const int64_t blk = token >> 4;
        if (token < 0 || blk >= p.table_pages * pb) return -1;
        const uint32_t pg = static_cast<uint32_t>(blk) / static_cast<uint32_t>(pb);
        const int64_t page = table[pg];
        if (page < 0 || page >= p.cache.pages) return -1;
        return layer + page * hk * pb + (blk - static_cast<int64_t>(pg) * pb);
    };
    for (int64_t piece0 = base / C; piece0 * C < base + n; piece0 += kTokens / C) {
        if (tid < kTokens) {                     // the new tokens' places, and where they come from
            const int64_t to = piece0 * C + tid, j = to - base;
            const bool moves = j >= 0 && j < n && path[j] != j;
            const int64_t from = moves ? base + path[j] : 0;
            const int64_t tb = j < n ? block_of(to) : -1;
            from_block[tid] = moves && tb >= 0 ? block_of(from) : -1;
            from_slot[tid] = from & 15;
            if (tid % C == 0) piece_block[tid / C] = tb;   // (a piece lies in one block)
        }
        __syncthreads();
        for (int q = 0; q < kTokens / C && (piece0 + q) * C < base + n; ++q) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < C; ++e) any = any || from_block[q * C + e] >= 0;
            const int first_slot = static_cast<int>((piece0 + q) * C & 15);
            uint4 kx[KI], vx[2];
            auto k_item = [&](int i, int& e, int& head, int& at) {
                const int x = tid + 256 * i;
                e = x / (512 / C);
                head = head0 + x % (512 / C) / PIECES;
                at = x % PIECES;
                return head < hk && from_block[q * C + e] >= 0;
            };
            auto v_item = [&](int i, int& head, int64_t& at) {
                const int x = tid + 256 * i;
                head = head0 + x / D;
                at = ((piece_block[q] + head * pb) * (16 / C) + first_slot / C) * D + x % D;
                return any && head < hk;
            };
            int e, head, at;
            int64_t where;
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (k_item(i, e, head, at))
                    kx[i] = static_cast<const uint4*>(p.cache.k)[((from_block[q * C + e] + head * pb) * PIECES + at) * 16 + from_slot[q * C + e]];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (v_item(i, head, where)) {
                    const int d = (tid + 256 * i) % D;
                    T x[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int64_t fb = from_block[q * C + c];
                        const int fs = from_slot[q * C + c];
                        x[c] = fb < 0 ? T{0} : static_cast<const T*>(p.cache.v)[(((fb + head * pb) * (16 / C) + fs / C) * D + d) * C + fs % C];
                    }
                    const uint4 old = static_cast<const uint4*>(p.cache.v)[where];
                    uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int shift = 8 * E * (c % (4 / E));
                        const uint32_t mask = (E == 1 ? 0xFFu : 0xFFFFu) << shift;
                        if (from_block[q * C + c] >= 0) w[c * E / 4] = (w[c * E / 4] & ~mask) | static_cast<uint32_t>(x[c]) << shift;
                    }
                    vx[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (k_item(i, e, head, at))
                    static_cast<uint4*>(p.cache.k)[((piece_block[q] + head * pb) * PIECES + at) * 16 + first_slot + e] = kx[i];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (v_item(i, head, where)) static_cast<uint4*>(p.cache.v)[where] = vx[i];
        }
        __syncthreads();
    }
}

}  // namespace

// one instance for each head size and element
#define W4_BY_CACHE(LAUNCH)                                                  \
    do {                                                                     \
        const int dim = p.cache.dim;                                         \
        if (p.cache.e4m3) {                                                  \
            if (dim == 64) LAUNCH(64, 1);                                    \
            else if (dim == 128) LAUNCH(128, 1);                             \
            else LAUNCH(256, 1);                                             \
        } else {                                                             \
            if (dim == 64) LAUNCH(64, 2);                                    \
            else if (dim == 128) LAUNCH(128, 2);                             \
            else LAUNCH(256, 2);                                             \
        }                                                                    \
    } while (0)

hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t stream) {
    const int64_t sixteens = (static_cast<int64_t>(p.T) + 15) / 16;
    const int64_t rows = sixteens * 16 * ((p.hq + 3) / 4 + (p.cache.heads + 3) / 4);
    const int64_t per_wg = 256 / (p.cache.dim / 8);
    const uint32_t row_groups = static_cast<uint32_t>((rows + per_wg - 1) / per_wg);
    const dim3 grid(row_groups + static_cast<unsigned>(sixteens * p.cache.heads));
#define W4_APPEND(D, E) hipLaunchKernelGGL((kv_append_kernel<D, E>), grid, dim3(256), 0, stream, p, row_groups)
    W4_BY_CACHE(W4_APPEND);
#undef W4_APPEND
    return hipGetLastError();
}

hipError_t launch_kv_move(const KvMoveParams& p, hipStream_t stream) {
    const int heads = 512 / p.cache.dim;     // a workgroup
    const dim3 grid((p.cache.heads + heads - 1) / heads, p.B, p.cache.layers);
#define W4_MOVE(D, E) hipLaunchKernelGGL((kv_move_kernel<D, E>), grid, dim3(256), 0, stream, p)
    W4_BY_CACHE(W4_MOVE);
#undef W4_MOVE
    return hipGetLastError();
}

}  // namespace w4
