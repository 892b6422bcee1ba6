// Logits before a token is chosen: penalties for repeated tokens, biases of
// single tokens and masks, in one pass over each row.
//
// Per row, with c_all(v) how often token v is in the row's history and c(v)
// how often behind its prompt, in fp32 and in this order:
//   x = l[v];  c_all(v) > 0:  x = x > 0 ? x / repetition : x repetition
//   x = x - frequency c(v) - presence [c(v) > 0]
//   x = x + bias(v)
//   mask bit 0:  x = -inf
// and one rounding to the logits' type at the end.
//
// A workgroup owns a slice of one row's vocabulary and counts the row's
// history for that slice in LDS: counts are whole numbers, so the order in
// which the lanes add them does not matter.  Every slice reads the whole
// history (from L2 after the first); against a histogram in memory this needs
// no cleared buffer, no second launch and no workspace.  A word of LDS a token
// holds the count behind the prompt and, in bit 31, whether the token is in
// the prompt.  A second word holds one more than the highest index of a bias
// entry for the token: of several entries the last counts, whatever lane sees
// it first.  A thread has eight consecutive tokens, whose logits it loads
// before the counting starts, in 16-byte pieces at any alignment (rows of an
// odd vocabulary start anywhere).
#include "decode_kernels.hpp"
#include "device.hpp"

namespace w4 {
namespace {

constexpr int kVec = 8;                  // consecutive tokens of a thread
constexpr uint32_t kPrompt = 0x80000000u;

template <typename T>
__device__ __forceinline__ T load_any(const void* p) {
    T t;
    __builtin_memcpy(&t, p, sizeof(T));
    return t;
}

template <bool F32, int kThreads>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustParams p, int slice) {
    constexpr int SIZE = F32 ? 4 : 2;
    constexpr int kSlice = kThreads * kVec;      // most tokens of a slice: 32 or 64 KB of LDS
    __shared__ __attribute__((aligned(16))) uint32_t count[kSlice], entry[kSlice];
    const int b = blockIdx.y;
    const int v0 = blockIdx.x * slice;
    const int n = p.V - v0 < slice ? p.V - v0 : slice;
    const int tid = threadIdx.x;
    const int i = kVec * tid;                // the thread's first token in the slice
    const int left = n - i;                  // its tokens (8 or more: all)

    // where the row's lists lie and what its penalties are, then the logits: all
    // on their way at once, the latter while the history is counted
    int64_t lo = 0, hi = 0, answer = 0, blo = 0, bhi = 0;
    if (p.history) {
        lo = p.history_start[b];
        hi = p.history_start[b + 1];
        answer = p.prompt_len ? p.prompt_len[b] : 0;
    }
    if (p.bias_ids) {
        blo = p.bias_start[b];
        bhi = p.bias_start[b + 1];
    }
    const float rep = p.repetition ? p.repetition[b] : 1.0f;
    const float pres = p.presence ? p.presence[b] : 0.0f;
    const float freq = p.frequency ? p.frequency[b] : 0.0f;
    typedef uint32_t raw_t __attribute__((ext_vector_type(kVec * SIZE / 4)));
    raw_t raw = 0;
    const int64_t at = static_cast<int64_t>(v0) + i;
    const uint8_t* const src = static_cast<const uint8_t*>(p.logits) + (static_cast<int64_t>(b) * p.row_stride + at) * SIZE;
    if (left >= kVec) {
        raw = load_any<raw_t>(src);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < left) {
                if constexpr (F32) raw[e] = reinterpret_cast<const uint32_t*>(src)[e];
                else raw[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[e]) << (16 * (e & 1));
            }
    }
    uint32_t allowed = 0xFFu;
    if (p.mask && left > 0) {
        // (slices start at multiples of 32)
        const uint32_t* const mask = p.mask + b * p.mask_stride;
        allowed = mask[at >> 5] >> (at & 31) & 0xFFu;
    }

    answer += lo;
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.history_len ? p.history_len : hi;
    blo = blo < 0 ? 0 : blo;
    bhi = bhi > p.bias_len ? p.bias_len : bhi;
    const bool counts = lo < hi, biases = blo < bhi;
    if (counts || biases) {
        const u32x4_t zero = {0u, 0u, 0u, 0u};
        if (i < slice) {
            *reinterpret_cast<u32x4_t*>(count + i) = zero;
            *reinterpret_cast<u32x4_t*>(count + i + 4) = zero;
            *reinterpret_cast<u32x4_t*>(entry + i) = zero;
            *reinterpret_cast<u32x4_t*>(entry + i + 4) = zero;
        }
        __syncthreads();
        // the tokens of [from, to): four a thread and load, eight loads in flight
        auto read = [&](int64_t from, int64_t to, auto note) {
            constexpr int kAhead = 8;
            int64_t j = from + 4 * tid;
            auto four = [&](const u32x4_t& t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t v = t[e] - static_cast<uint32_t>(v0);
                    if (v < static_cast<uint32_t>(n)) note(v);
                }
            };
            for (; j + (kAhead - 1) * 4 * kThreads + 4 <= to; j += kAhead * 4 * kThreads) {
                u32x4_t t[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) t[a] = load_any<u32x4_t>(p.history + j + a * 4 * kThreads);
#pragma unroll
                for (int a = 0; a < kAhead; ++a) four(t[a]);
            }
            for (; j < to; j += 4 * kThreads) {
                u32x4_t t = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};    // (no token)
                if (j + 4 <= to) {
                    t = load_any<u32x4_t>(p.history + j);
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (j + e < to) t[e] = static_cast<uint32_t>(p.history[j + e]);
                }
                four(t);
            }
        };
        const int64_t split = answer < lo ? lo : (answer > hi ? hi : answer);
        read(lo, split, [&](uint32_t v) { atomicOr(&count[v], kPrompt); });
        read(split, hi, [&](uint32_t v) { atomicAdd(&count[v], 1u); });
        for (int64_t k = blo + tid; k < bhi; k += kThreads) {
            const uint32_t v = static_cast<uint32_t>(p.bias_ids[k]) - static_cast<uint32_t>(v0);
            if (v < static_cast<uint32_t>(n)) atomicMax(&entry[v], static_cast<uint32_t>(k - blo) + 1u);
        }
        __syncthreads();
    }
    if (left <= 0) return;
    float x[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        if constexpr (F32) x[e] = __uint_as_float(raw[e]);
        else x[e] = e & 1 ? bf16_hi(raw[e / 2]) : bf16_lo(raw[e / 2]);
    }
    if (counts || biases) {
        uint32_t c[kVec], k[kVec];
#pragma unroll
        for (int e = 0; e < kVec; e += 4) {
            *reinterpret_cast<u32x4_t*>(c + e) = *reinterpret_cast<const u32x4_t*>(count + i + e);
            *reinterpret_cast<u32x4_t*>(k + e) = *reinterpret_cast<const u32x4_t*>(entry + i + e);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            // few tokens of a vocabulary are in a history: the division and what
            // goes with it is passed over where no lane has one
            if (__builtin_amdgcn_ballot_w64((c[e] | k[e]) != 0) == 0) continue;
            const uint32_t later = c[e] & ~kPrompt;
            if (c[e]) x[e] = x[e] > 0.0f ? x[e] / rep : x[e] * rep;
            if (later) x[e] = x[e] - freq * static_cast<float>(later) - pres;
            if (k[e]) x[e] = x[e] + p.bias_values[blo + k[e] - 1];
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = allowed >> e & 1u ? x[e] : -__builtin_inff();
    uint8_t* const dst = static_cast<uint8_t*>(p.out) + (static_cast<int64_t>(b) * p.out_stride + at) * SIZE;
    if (left >= kVec) {
        raw_t o;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if constexpr (F32) o[e] = __float_as_uint(x[e]);
            else if (e & 1) o[e / 2] = pack_bf16x2(x[e - 1], x[e]);
        }
        __builtin_memcpy(dst, &o, sizeof(o));
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < left) {
                if constexpr (F32) reinterpret_cast<float*>(dst)[e] = x[e];
                else reinterpret_cast<uint16_t*>(dst)[e] = float_to_bf16_bits(x[e]);
            }
    }
}

}  // namespace

namespace {
template <int kThreads>
hipError_t launch_adjust_t(const AdjustParams& p, int slice, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.V + slice - 1) / slice), static_cast<unsigned>(p.B));
    if (p.f32) hipLaunchKernelGGL((adjust_kernel<true, kThreads>), grid, dim3(kThreads), 0, stream, p, slice);
    else hipLaunchKernelGGL((adjust_kernel<false, kThreads>), grid, dim3(kThreads), 0, stream, p, slice);
    return hipGetLastError();
}
}  // namespace

// With few rows, the smallest slices that leave at most one workgroup a compute
// unit, since each reads the whole history of its row, and as many threads as
// there can be to read it (3 rows of 131072 tokens with histories of 100000:
// 12.0 us, 14.8 with 512 threads, 20 with slices of 1024).  With more, slices of
// 4096 by 512 threads (200 rows: 37 us, 38 with 256 threads, 40 with 1024).
// (Runs of slices in one workgroup, the first tokens of the history in registers
// and the next slice's logits on their way: 39 us with two rounds of workgroups,
// 47 to 51 with one.  The many short workgroups cover each other's waits better.)
hipError_t launch_adjust(const AdjustParams& p, hipStream_t stream) {
    for (int slice = 512; slice <= 4096; slice *= 2)
        if (static_cast<int64_t>(p.B) * ((p.V + slice - 1) / slice) <= 256) return launch_adjust_t<1024>(p, slice, stream);
    return launch_adjust_t<512>(p, 4096, stream);
}

}  // namespace w4
