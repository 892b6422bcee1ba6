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
// holds the count behind the prompt (bits 0..30, saturating is not needed: a
// history has fewer than 2^31 tokens) and, in bit 31, whether the token is in
// the history at all.  A second word holds one more than the highest index of
// a bias entry for the token: of several entries the last counts, whatever
// lane sees it first.
#include "decode_kernels.hpp"
#include "device.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 8192;          // tokens of a slice: 64 KB of LDS in all
constexpr uint32_t kSeen = 0x80000000u;

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int64_t v) {
    if constexpr (F32) return static_cast<const float*>(row)[v];
    else return bf16_lo(static_cast<const uint16_t*>(row)[v]);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustParams p, int slice) {
    extern __shared__ uint32_t lds[];
    uint32_t* const count = lds;
    uint32_t* const entry = lds + slice;
    const int b = blockIdx.y;
    const int v0 = blockIdx.x * slice;
    const int n = p.V - v0 < slice ? p.V - v0 : slice;
    const int tid = threadIdx.x;

    int lo = 0, hi = 0, prompt = 0;
    if (p.history) {
        lo = p.history_start[b];
        hi = p.history_start[b + 1];
        lo = lo < 0 ? 0 : lo;
        hi = hi > p.history_len ? static_cast<int>(p.history_len) : hi;
        prompt = p.prompt_len ? p.prompt_len[b] : 0;
    }
    int blo = 0, bhi = 0;
    if (p.bias_ids) {
        blo = p.bias_start[b];
        bhi = p.bias_start[b + 1];
        blo = blo < 0 ? 0 : blo;
        bhi = bhi > p.bias_len ? static_cast<int>(p.bias_len) : bhi;
    }
    const bool counts = lo < hi, biases = blo < bhi;
    if (counts || biases) {
        for (int i = tid; i < 2 * slice; i += kThreads) lds[i] = 0;
        __syncthreads();
        // (the prompt ends at lo + prompt, which may pass 32 bits)
        const int64_t answer = static_cast<int64_t>(lo) + prompt;
        for (uint32_t i = lo + tid; i < static_cast<uint32_t>(hi); i += kThreads) {
            const uint32_t v = static_cast<uint32_t>(p.history[i]) - static_cast<uint32_t>(v0);
            if (v < static_cast<uint32_t>(n)) {
                if (i >= answer) atomicAdd(&count[v], 1u);
                atomicOr(&count[v], kSeen);
            }
        }
        for (uint32_t i = blo + tid; i < static_cast<uint32_t>(bhi); i += kThreads) {
            const uint32_t v = static_cast<uint32_t>(p.bias_ids[i]) - static_cast<uint32_t>(v0);
            if (v < static_cast<uint32_t>(n)) atomicMax(&entry[v], i - static_cast<uint32_t>(blo) + 1u);
        }
        __syncthreads();
    }
    const float rep = p.repetition ? p.repetition[b] : 1.0f;
    const float pres = p.presence ? p.presence[b] : 0.0f;
    const float freq = p.frequency ? p.frequency[b] : 0.0f;
    const uint32_t* const mask = p.mask ? p.mask + b * p.mask_stride : nullptr;
    const void* const row = static_cast<const uint8_t*>(p.logits) + static_cast<int64_t>(b) * p.row_stride * (F32 ? 4 : 2);
    void* const out = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(b) * p.out_stride * (F32 ? 4 : 2);
    for (int i = tid; i < n; i += kThreads) {
        const int v = v0 + i;
        float x = logit<F32>(row, v);
        if (counts) {
            const uint32_t c = count[i];
            if (c) x = x > 0.0f ? x / rep : x * rep;
            const uint32_t later = c & ~kSeen;
            if (later) x = x - freq * static_cast<float>(later) - pres;
        }
        if (biases) {
            const uint32_t e = entry[i];
            if (e) x = x + p.bias_values[blo + static_cast<int>(e) - 1];
        }
        if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) x = -__builtin_inff();
        if constexpr (F32) static_cast<float*>(out)[v] = x;
        else static_cast<uint16_t*>(out)[v] = float_to_bf16_bits(x);
    }
}

}  // namespace

hipError_t launch_adjust(const AdjustParams& p, hipStream_t stream) {
    const int slice = 4096;
    const dim3 grid(static_cast<unsigned>((p.V + slice - 1) / slice), static_cast<unsigned>(p.B));
    if (p.f32) hipLaunchKernelGGL((adjust_kernel<true>), grid, dim3(kThreads), 8 * slice, stream, p, slice);
    else hipLaunchKernelGGL((adjust_kernel<false>), grid, dim3(kThreads), 8 * slice, stream, p, slice);
    return hipGetLastError();
}

}  // namespace w4
