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

constexpr int kThreads = 512;
constexpr int kVec = 8;                  // consecutive tokens of a thread
constexpr int kSlice = kThreads * kVec;  // most tokens of a slice: 32 KB of LDS
constexpr uint32_t kPrompt = 0x80000000u;

template <typename T>
__device__ __forceinline__ T load_any(const void* p) {
    T t;
    __builtin_memcpy(&t, p, sizeof(T));
    return t;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustParams p, int slice) {
    constexpr int SIZE = F32 ? 4 : 2;
    __shared__ __attribute__((aligned(16))) uint32_t count[kSlice], entry[kSlice];
    const int b = blockIdx.y;
    const int v0 = blockIdx.x * slice;
    const int n = p.V - v0 < slice ? p.V - v0 : slice;
    const int tid = threadIdx.x;
    const int i = kVec * tid;                // the thread's first token in the slice
    const int left = n - i;                  // its tokens (8 or more: all)

    // the logits, on their way while the history is counted
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

    int64_t lo = 0, hi = 0, answer = 0;
    if (p.history) {
        lo = p.history_start[b];
        hi = p.history_start[b + 1];
        answer = lo + (p.prompt_len ? p.prompt_len[b] : 0);
        lo = lo < 0 ? 0 : lo;
        hi = hi > p.history_len ? p.history_len : hi;
    }
    int64_t blo = 0, bhi = 0;
    if (p.bias_ids) {
        blo = p.bias_start[b];
        bhi = p.bias_start[b + 1];
        blo = blo < 0 ? 0 : blo;
        bhi = bhi > p.bias_len ? p.bias_len : bhi;
    }
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
        auto note = [&](int64_t j, uint32_t token) {
            const uint32_t v = token - static_cast<uint32_t>(v0);
            if (v >= static_cast<uint32_t>(n)) return;
            if (j >= answer) atomicAdd(&count[v], 1u);
            else atomicOr(&count[v], kPrompt);
        };
        // four tokens a thread and load, four loads in flight
        constexpr int kAhead = 4;
        int64_t j = lo + 4 * tid;
        for (; j + (kAhead - 1) * 4 * kThreads + 4 <= hi; j += kAhead * 4 * kThreads) {
            u32x4_t t[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) t[a] = load_any<u32x4_t>(p.history + j + a * 4 * kThreads);
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) note(j + a * 4 * kThreads + e, t[a][e]);
        }
        for (; j < hi; j += 4 * kThreads)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < hi) note(j + e, static_cast<uint32_t>(p.history[j + e]));
        for (int64_t k = blo + tid; k < bhi; k += kThreads) {
            const uint32_t v = static_cast<uint32_t>(p.bias_ids[k]) - static_cast<uint32_t>(v0);
            if (v < static_cast<uint32_t>(n)) atomicMax(&entry[v], static_cast<uint32_t>(k - blo) + 1u);
        }
        __syncthreads();
    }
    if (left <= 0) return;
    const float rep = p.repetition ? p.repetition[b] : 1.0f;
    const float pres = p.presence ? p.presence[b] : 0.0f;
    const float freq = p.frequency ? p.frequency[b] : 0.0f;
    float x[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        if constexpr (F32) x[e] = __uint_as_float(raw[e]);
        else x[e] = e & 1 ? bf16_hi(raw[e / 2]) : bf16_lo(raw[e / 2]);
        if (counts || biases) {
            const uint32_t c = count[i + e], k = entry[i + e], later = c & ~kPrompt;
            if (c) x[e] = x[e] > 0.0f ? x[e] / rep : x[e] * rep;
            if (later) x[e] = x[e] - freq * static_cast<float>(later) - pres;
            if (k) x[e] = x[e] + p.bias_values[blo + k - 1];
        }
        if (!(allowed >> e & 1u)) x[e] = -__builtin_inff();
    }
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

// Slices of 4096 tokens, of 1024 where that leaves fewer than two workgroups a
// compute unit.
hipError_t launch_adjust(const AdjustParams& p, hipStream_t stream) {
    const int64_t most = static_cast<int64_t>(p.B) * ((p.V + kSlice - 1) / kSlice);
    const int slice = most < 512 ? 1024 : kSlice;
    const dim3 grid(static_cast<unsigned>((p.V + slice - 1) / slice), static_cast<unsigned>(p.B));
    if (p.f32) hipLaunchKernelGGL((adjust_kernel<true>), grid, dim3(kThreads), 0, stream, p, slice);
    else hipLaunchKernelGGL((adjust_kernel<false>), grid, dim3(kThreads), 0, stream, p, slice);
    return hipGetLastError();
}

}  // namespace w4
