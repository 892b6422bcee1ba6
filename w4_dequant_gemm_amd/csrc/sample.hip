// One token per row of logits: temperature, top-k, top-p, min-p, then the
// token at a given uniform number of the kept weights' running sum.
//
// Weights are whole numbers (units of 2^-31 of the largest), so every sum is
// exact and the same in any order.  The kept tokens are a prefix of the order
// (logit descending, index ascending): all with a key above kappa and the first
// `take` of those equal to it.  Both thresholds come from a radix selection on
// the order-preserving key, eight bits a level: by count for top-k, by weight
// for top-p.  Equal keys have equal weights, so how many of them are kept
// follows by division, without looking at indices.
#include "device.hpp"
#include "kernels.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

// fp32 -> a key in the order of the values; NaN like -inf; -0 like +0
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// rint(2^31 exp((x - top) r))
__device__ __forceinline__ uint32_t weight_of(float x, float top, float r) {
    if (x == top) return 0x80000000u;
    const float e = x == -INFINITY ? 0.0f : expf((x - top) * r);
    return static_cast<uint32_t>(rintf(e * 2147483648.0f));
}

__device__ __forceinline__ uint64_t units_of_2_24(float x, uint64_t most) {
    const float f = floorf(x * 16777216.0f);
    return f >= static_cast<float>(most) ? most : f > 0.0f ? static_cast<uint64_t>(f) : 0u;
}
// m total / 2^24 rounded down, and whether it was rounded
__device__ __forceinline__ uint64_t part_of(uint64_t m, uint64_t total, bool& more) {
    const uint64_t low = m * (total & 0xFFFFFFu);
    more = (low & 0xFFFFFFu) != 0;
    return m * (total >> 24) + (low >> 24);
}

__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(static_cast<unsigned long long>(v), off);
    return v;
}

template <bool F32>
struct Row {
    const void* base;
    int V;
    __device__ __forceinline__ float at(int i) const {
        if constexpr (F32) return static_cast<const float*>(base)[i];
        else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
    }
};

struct Shared {
    uint64_t mass[256];
    uint32_t count[256];
    uint64_t wave64[kWaves];
    uint64_t wave64b[kWaves];
    uint32_t wave32[kWaves];
    uint32_t pick;
    uint64_t above;
};

__device__ __forceinline__ uint64_t block_sum(Shared& sh, uint64_t v) {
    v = wave_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.wave64[threadIdx.x >> 6] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t += sh.wave64[w];
    return t;
}

// The key at which the running count (BY_MASS: weight) from the largest key
// down first reaches `need`, and what lies above it.  need >= 1 and at most
// the total.
template <bool F32, bool BY_MASS>
__device__ uint32_t select(Shared& sh, const Row<F32>& row, float top, float r, uint64_t need, uint64_t& above_out) {
    uint32_t prefix = 0;
    uint64_t above = 0;
    for (int shift = 24; shift >= (F32 ? 0 : 16); shift -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += kThreads) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int i = threadIdx.x; i < row.V; i += kThreads) {
            const float x = row.at(i);
            const uint32_t key = key_of(x);
            if ((key & mask) != prefix) continue;
            if constexpr (BY_MASS) {
                const uint32_t w = weight_of(value_of(key), top, r);
                if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[(key >> shift) & 255]), static_cast<unsigned long long>(w));
            } else {
                atomicAdd(&sh.count[(key >> shift) & 255], 1u);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int bin = 255;
            for (; bin > 0; --bin) {
                const uint64_t here = BY_MASS ? sh.mass[bin] : sh.count[bin];
                if (above + here >= need) break;
                above += here;
            }
            sh.pick = static_cast<uint32_t>(bin);
            sh.above = above;
        }
        __syncthreads();
        prefix |= sh.pick << shift;
        above = sh.above;
    }
    above_out = above;
    // low bits of a bf16 key are those of its complement for negative values
    if (!F32 && !(prefix >> 31)) prefix |= 0xFFFFu;
    return prefix;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
    __shared__ Shared sh;
    const int b = blockIdx.x;
    const int V = p.V;
    Row<F32> row;
    row.V = V;
    row.base = static_cast<const uint8_t*>(p.logits) + b * p.row_stride * (F32 ? 4 : 2);
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const float r = greedy ? 1.0f : 1.0f / t;

    uint32_t best = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) best = max(best, key_of(row.at(i)));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) best = max(best, static_cast<uint32_t>(__shfl_xor(static_cast<int>(best), off)));
    if ((threadIdx.x & 63) == 0) sh.wave32[threadIdx.x >> 6] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = max(best, sh.wave32[w]);
    const float top = value_of(best);
    if (top == -INFINITY) {
        if (threadIdx.x == 0) {
            p.tokens[b] = -1;
            if (p.probs) p.probs[b] = 0.0f;
        }
        return;
    }

    // kept: keys above kappa, the first `take` of those equal to it
    uint32_t kappa = 0;
    uint64_t take = static_cast<uint64_t>(V);
    int k = greedy ? 1 : p.top_k ? p.top_k[b] : 0;
    if (k > 0 && k < V) {
        uint64_t above;
        kappa = select<F32, false>(sh, row, top, r, k, above);
        take = k - above;
    }
    if (p.top_p && !greedy) {
        uint64_t mine = 0;
        for (int i = threadIdx.x; i < V; i += kThreads) {
            const uint32_t key = key_of(row.at(i));
            if (key > kappa) mine += weight_of(value_of(key), top, r);
        }
        const uint64_t w_kappa = kappa ? weight_of(value_of(kappa), top, r) : 0;
        const uint64_t total = block_sum(sh, mine) + take * w_kappa;
        bool more;
        uint64_t need = part_of(units_of_2_24(p.top_p[b], 1u << 24), total, more);
        need += more ? 1 : 0;
        if (need < 1) need = 1;
        uint64_t above;
        const uint32_t kp = select<F32, true>(sh, row, top, r, need, above);
        const uint64_t w = weight_of(value_of(kp), top, r);
        const uint64_t tp = w ? (need - above + w - 1) / w : 1;
        if (kp > kappa) {
            kappa = kp;
            take = tp;
        } else if (kp == kappa && tp < take) {
            take = tp;
        }
    }
    uint32_t least = 1;                      // smallest weight kept
    if (p.min_p && !greedy) {
        const float f = ceilf(p.min_p[b] * 2147483648.0f);
        least = f >= 4294967040.0f ? 0xFFFFFFFFu : f > 1.0f ? static_cast<uint32_t>(f) : 1u;
    }

    // weights and ties of each segment (a wavefront's share in index order)
    const int per = (V + kWaves - 1) / kWaves;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int lo = wave * per, hi = min(V, lo + per);
    const uint32_t w_kappa0 = kappa ? weight_of(value_of(kappa), top, r) : 0;
    const uint32_t w_tie = w_kappa0 >= least ? w_kappa0 : 0;
    uint64_t mass = 0, ties = 0;
    for (int i = lo + lane; i < hi; i += 64) {
        const uint32_t key = key_of(row.at(i));
        if (key > kappa) {
            const uint32_t w = weight_of(value_of(key), top, r);
            if (w >= least) mass += w;
        } else if (key == kappa) {
            ++ties;
        }
    }
    mass = wave_sum64(mass);
    ties = wave_sum64(ties);
    __syncthreads();
    if (lane == 0) {
        sh.wave64[wave] = mass;
        sh.wave64b[wave] = ties;
    }
    __syncthreads();
    uint64_t total = 0, tied = 0, before = 0, tied_before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint64_t c = tied >= take ? 0 : min(sh.wave64b[w], take - tied);
        if (w == wave) {
            before = total;
            tied_before = tied;
        }
        total += sh.wave64[w] + c * w_tie;
        tied += sh.wave64b[w];
    }
    if (total == 0) {                        // min_p above 1
        if (threadIdx.x == 0) {
            p.tokens[b] = -1;
            if (p.probs) p.probs[b] = 0.0f;
        }
        return;
    }
    bool more;
    const uint64_t target = part_of(units_of_2_24(p.u[b], (1u << 24) - 1), total, more);
    const uint64_t mine_ties = tied_before >= take ? 0 : min(ties, take - tied_before);
    if (!(target >= before && target < before + mass + mine_ties * w_tie)) return;   // a whole wavefront
    // this wavefront holds the token: 64 at a time, in order
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane;
        uint32_t key = 0;
        uint32_t w = 0;
        bool tie = false;
        if (i < hi) {
            key = key_of(row.at(i));
            tie = key == kappa;
            if (key > kappa) {
                w = weight_of(value_of(key), top, r);
                if (w < least) w = 0;
            }
        }
        const uint64_t tie_lanes = __ballot(tie);
        const uint64_t rank = tied_before + __popcll(tie_lanes & ((uint64_t{1} << lane) - 1));
        if (tie && rank < take) w = w_tie;
        uint64_t upto = w;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint64_t o = __shfl_up(static_cast<unsigned long long>(upto), off);
            if (lane >= off) upto += o;
        }
        const uint64_t hit = __ballot(before + upto > target);
        if (hit) {
            if (lane == __ffsll(static_cast<unsigned long long>(hit)) - 1) {
                p.tokens[b] = i;
                if (p.probs) p.probs[b] = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
            }
            return;
        }
        before += __shfl(static_cast<unsigned long long>(upto), 63);
        tied_before += __popcll(tie_lanes);
    }
}

}  // namespace

size_t sample_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleParams& p, hipStream_t stream) {
    if (p.f32) hipLaunchKernelGGL(sample_kernel<true>, dim3(p.B), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL(sample_kernel<false>, dim3(p.B), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace w4
