// The paged cache of keys and values: appending rows of a QKV product (with
// the heads' norms and the rotation on the way) and moving an accepted path.
#include "device.hpp"
#include "kernels.hpp"

namespace w4 {
namespace {

// Eight fp32 values -> E4M3 codes of v / s, saturating at +-448, NaN kept.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float s) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v[i] / s;
        f[i] = x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    return make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

// One head row of one token: D / 8 lanes with eight dims each.  Eight
// neighbouring heads (D = 64) share a wavefront, so the norm's sum and the
// rotation's partner values are exchanged inside the row's own lanes.
template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendParams p) {
    constexpr int L = D / 8;                 // lanes a row
    const int hk = p.cache.heads;
    const int heads = p.hq + 2 * hk;
    const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / L;
    const uint32_t t = row / static_cast<uint32_t>(heads);
    const int h = static_cast<int>(row - t * static_cast<uint32_t>(heads));
    const int c = threadIdx.x % L;           // dims 8c .. 8c + 7
    if (t >= static_cast<uint32_t>(p.T)) return;   // whole rows leave together

    const bool is_q = h < p.hq, is_v = h >= p.hq + hk;
    const int head = is_q ? h : is_v ? h - p.hq - hk : h - p.hq;
    const uint16_t* src = is_q ? p.q + t * p.q_stride : is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride;
    const uint4 w = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(head) * D + 8 * c);
    float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                  bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};

    if (!is_v) {
        const float* norm = is_q ? p.q_norm : p.k_norm;
        if (norm) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[i] * x[i];
#pragma unroll
            for (int off = L / 2; off >= 1; off >>= 1) s += __shfl_xor(s, off, L);
            const float r = 1.0f / sqrtf(s * (1.0f / D) + p.eps);
            const float4_t n0 = *reinterpret_cast<const float4_t*>(norm + 8 * c);
            const float4_t n1 = *reinterpret_cast<const float4_t*>(norm + 8 * c + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (i < 4 ? n0[i & 3] : n1[i & 3]);
        }
        if (p.rope) {
            const int half = p.rot >> 4;     // lanes that hold the first of each pair (halves)
            const int64_t pos = p.positions[t];
            const bool inside = pos >= 0 && pos < p.rope_rows;
            const float* cs = p.rope + (inside ? pos : 0) * p.rot;
            const bool turns = c < 2 * half;
            if (p.interleaved) {
                if (turns) {
                    const float4_t co = *reinterpret_cast<const float4_t*>(cs + 4 * c);
                    const float4_t si = *reinterpret_cast<const float4_t*>(cs + (p.rot >> 1) + 4 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = a * co[i] - b * si[i];
                        x[2 * i + 1] = b * co[i] + a * si[i];
                    }
                }
            } else {
                const bool first = c < half;
                const int partner = turns ? (first ? c + half : c - half) : c;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], partner, L);
                if (turns) {
                    const int j = 8 * (first ? c : c - half);
#pragma unroll
                    for (int v4 = 0; v4 < 2; ++v4) {
                        const float4_t co = *reinterpret_cast<const float4_t*>(cs + j + 4 * v4);
                        const float4_t si = *reinterpret_cast<const float4_t*>(cs + (p.rot >> 1) + j + 4 * v4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float own = x[4 * v4 + i], other = y[4 * v4 + i];
                            x[4 * v4 + i] = first ? own * co[i] - other * si[i] : own * co[i] + other * si[i];
                        }
                    }
                }
            }
            if (!inside && turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
            }
        }
        if (is_q) {
            const uint4 o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                       pack_bf16x2(x[6], x[7]));
            *reinterpret_cast<uint4*>(p.Q + (static_cast<int64_t>(t) * p.hq + head) * D + 8 * c) = o;
            return;
        }
    }

    const int64_t slot = p.slots[t];
    const int page_size = 16 * p.cache.page_blocks;
    if (slot < 0 || slot >= p.cache.pages * page_size) return;
    const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(page_size);
    const int in_page = static_cast<int>(slot) - static_cast<int>(page) * page_size;
    const int s = in_page & 15;
    const int64_t block = (static_cast<int64_t>(page) * hk + head) * p.cache.page_blocks + (in_page >> 4);
    if (p.cache.e4m3) {
        const uint2 codes = e4m3x8(x, is_v ? p.cache.v_scale[head] : p.cache.k_scale[head]);
        if (!is_v) {
            uint8_t* dst = static_cast<uint8_t*>(p.cache.k) + block * (16 * D);
            *reinterpret_cast<uint2*>(dst + (c >> 1) * 256 + s * 16 + (c & 1) * 8) = codes;
        } else {
            uint8_t* dst = static_cast<uint8_t*>(p.cache.v) + block * (16 * D) + 8 * c * 16 + s;
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i * 16] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
        }
    } else {
        const uint32_t o[4] = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                               pack_bf16x2(x[6], x[7])};
        if (!is_v) {
            uint16_t* dst = static_cast<uint16_t*>(p.cache.k) + block * (16 * D);
            *reinterpret_cast<uint4*>(dst + c * 128 + s * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            uint16_t* dst = static_cast<uint16_t*>(p.cache.v) + block * (16 * D) + (s >> 3) * (8 * D) + 64 * c + (s & 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i * 8] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// One thread owns one 16-byte column of the cache of one (layer, sequence,
// head): for K the same chunk of dims of every token (16 bytes a token), for V
// one dim (an element a token).  It walks the path in order, so no other
// thread touches what it reads or writes; path[j] >= j and the path ascends,
// so what a later step reads was not overwritten by an earlier one.
template <int E>   // bytes an element
__global__ void __launch_bounds__(256) kv_move_kernel(KvMoveParams p) {
    using T = typename std::conditional<E == 1, uint8_t, uint16_t>::type;
    constexpr int C = 16 / E;
    const int D = p.cache.dim, hk = p.cache.heads, pb = p.cache.page_blocks;
    const int per_head = D / C + D;
    const uint32_t unit = blockIdx.x * 256u + threadIdx.x;
    if (unit >= static_cast<uint32_t>(hk * per_head)) return;
    const int head = unit / per_head;
    const int u = unit - head * per_head;
    const int b = blockIdx.y;
    int n = p.count[b];
    n = n < p.path_len ? n : static_cast<int>(p.path_len);
    const int64_t base = p.base[b];
    const int32_t* table = p.page_table + b * p.table_pages;
    const int32_t* path = p.path + b * p.path_len;
    const int64_t layer = static_cast<int64_t>(blockIdx.z) * p.cache.pages * hk * pb;

    auto block_of = [&](int64_t token) -> int64_t {
        const int64_t blk = token >> 4;
        if (token < 0 || blk >= p.table_pages * pb) return -1;
        const uint32_t pg = static_cast<uint32_t>(blk) / static_cast<uint32_t>(pb);
        const int64_t page = table[pg];
        if (page < 0 || page >= p.cache.pages) return -1;
        return layer + (page * hk + head) * pb + (blk - static_cast<int64_t>(pg) * pb);
    };
    for (int j = 0; j < n; ++j) {
        const int64_t from = base + path[j], to = base + j;
        if (from == to) continue;
        const int64_t fb = block_of(from), tb = block_of(to);
        if (fb < 0 || tb < 0) continue;
        const int fs = from & 15, ts = to & 15;
        if (u < D / C) {
            uint4* k = static_cast<uint4*>(p.cache.k);
            k[(tb * (D / C) + u) * 16 + ts] = k[(fb * (D / C) + u) * 16 + fs];
        } else {
            T* v = static_cast<T*>(p.cache.v);
            const int d = u - D / C;
            v[((tb * (16 / C) + ts / C) * D + d) * C + ts % C] = v[((fb * (16 / C) + fs / C) * D + d) * C + fs % C];
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.T) * (p.hq + 2 * p.cache.heads);
    const int64_t per_wg = 256 / (p.cache.dim / 8);
    const dim3 grid(static_cast<unsigned>((rows + per_wg - 1) / per_wg));
    switch (p.cache.dim) {
        case 64: hipLaunchKernelGGL(kv_append_kernel<64>, grid, dim3(256), 0, stream, p); break;
        case 128: hipLaunchKernelGGL(kv_append_kernel<128>, grid, dim3(256), 0, stream, p); break;
        default: hipLaunchKernelGGL(kv_append_kernel<256>, grid, dim3(256), 0, stream, p); break;
    }
    return hipGetLastError();
}

hipError_t launch_kv_move(const KvMoveParams& p, hipStream_t stream) {
    const int c = p.cache.e4m3 ? 16 : 8;
    const int units = p.cache.heads * (p.cache.dim / c + p.cache.dim);
    const dim3 grid((units + 255) / 256, p.B, p.cache.layers);
    if (p.cache.e4m3) hipLaunchKernelGGL(kv_move_kernel<1>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(kv_move_kernel<2>, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace w4
