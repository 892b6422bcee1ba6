// One token per row of logits: temperature, top-k, top-p, min-p, then the
// token at a given uniform number of the kept weights' running sum.
//
// Weights are whole numbers (units of 2^-31 of the largest), so every sum is
// exact and the same in any order: atomics and any split of the work give the
// same token.  The kept tokens are a prefix of the order (logit descending,
// index ascending): all with a key above kappa, and those equal to it up to
// index iota.  Equal keys have equal weights, so how many of them are kept
// follows by division.
//
// One workgroup of 1024 threads a row, which is read from memory for the
// maximum and again from the caches for what follows:
//  - top-k: the k-th largest of the threads' own maxima bounds the k-th largest
//    logit from below, so few tokens besides the top k lie above it: they are
//    collected in shared memory and the filters and the draw work on them;
//  - top-p alone: weights of the tokens near the top are summed in bins of the
//    scaled distance to the maximum, all others together; the bin in which p of
//    the total is reached is collected and searched;
//  - neither: nothing to search.
// Searches are radix selections on the order-preserving key (or the index),
// eight bits a level: by count for top-k, by weight for top-p and the draw.
// Rows whose values crowd more tokens than shared memory holds (many equal
// logits) take the same selections over the whole row.
#include <type_traits>

#include "device.hpp"
#include "kernels.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kCandidates = 4096;            // tokens collected in shared memory
constexpr int kMine = kCandidates / kThreads;
constexpr int kBins = 2048;
constexpr float kBinsPerUnit = 64.0f;        // bins of 1/64 of the scaled distance
constexpr int kSegments = (1 << 20) / 256 + 1;

// fp32 (not NaN) -> a key in the order of the values; -0 like +0
__device__ __forceinline__ uint32_t key_of(float x) {
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
// a distance that grows as the weight falls, the same for equal values; the bin is its whole part
__device__ __forceinline__ float bin_of(float x, float top, float r) {
    return x == top ? 0.0f : fminf((top - x) * r * kBinsPerUnit, 1e9f);
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
// running sum over the lanes, this one included
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint64_t o = __shfl_up(static_cast<unsigned long long>(v), off);
        if (lane >= off) v += o;
    }
    return v;
}

struct Shared {
    union {
        struct {
            uint64_t bins[kBins];            // weights by distance
            uint32_t counts[kBins];
        };
        uint64_t segments[kSegments];
    };
    uint64_t hist[256];
    uint64_t wave64[kWaves];
    uint32_t wave32[kWaves];
    uint32_t key[kCandidates], index[kCandidates];
    uint32_t candidates;
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

// The first of n bins (ascending) at which their running sum reaches need, and
// the sum before it, by the first wavefront; n (a multiple of 64) if it is not
// reached.  Every thread gets the result.
template <class Get>
__device__ __forceinline__ int reach(Shared& sh, int n, uint64_t need, uint64_t& before, Get get) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const int per = n / 64;              // consecutive bins of a lane
        uint64_t mine = 0;
        for (int i = 0; i < per; ++i) mine += get(lane * per + i);
        const uint64_t upto = wave_scan64(mine);
        const uint64_t hit = __ballot(upto >= need);
        if (!hit) {
            if (lane == 63) {
                sh.pick = static_cast<uint32_t>(n);
                sh.above = upto;
            }
        } else if (lane == __ffsll(static_cast<unsigned long long>(hit)) - 1) {
            uint64_t sum = upto - mine;
            int i = 0;
            for (; i < per - 1; ++i) {
                const uint64_t w = get(lane * per + i);
                if (sum + w >= need) break;
                sum += w;
            }
            sh.pick = static_cast<uint32_t>(lane * per + i);
            sh.above = sum;
        }
    }
    __syncthreads();
    before = sh.above;
    const int at = static_cast<int>(sh.pick);
    __syncthreads();
    return at;
}

// The key (of `bits` bits, a multiple of 8) at which the running sum of weights
// from the largest key down reaches `need` (1 .. their total), and the sum
// above it.  each(f) calls f(key, weight) for this thread's items, weight being
// a function.
template <class Each>
__device__ __forceinline__ uint32_t select(Shared& sh, int bits, int stop, uint64_t need, uint64_t& above, Each each) {
    uint32_t prefix = 0;
    above = 0;
    for (int shift = bits - 8; shift >= stop; shift -= 8) {
        __syncthreads();
        if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t mask = shift + 8 >= 32 ? 0u : 0xFFFFFFFFu << (shift + 8);
        each([&](uint32_t key, auto weight) {
            if (((key ^ prefix) & mask) == 0) {
                const unsigned long long w = weight();
                if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.hist[(key >> shift) & 255]), w);
            }
        });
        __syncthreads();
        uint64_t before;
        const int at = reach(sh, 256, need - above, before, [&](int i) { return sh.hist[255 - i]; });
        above += before;
        prefix |= static_cast<uint32_t>(255 - at) << shift;
    }
    return prefix;
}

// V logits as 16-byte vectors; the elements of the first and last vector that
// lie outside the row count as -inf.  (They are inside the same 16 aligned
// bytes as elements of the row, so reading them touches no other page.)
template <bool F32>
struct Row {
    static constexpr int N = F32 ? 4 : 8;    // elements a vector
    const uint4* vectors;
    int shift, V, count;                     // first element's place in the first vector

    __device__ __forceinline__ Row(const void* logits, int64_t elements, int V_) : V(V_) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(logits) + elements * (F32 ? 4 : 2);
        vectors = reinterpret_cast<const uint4*>(at & ~uintptr_t{15});
        shift = static_cast<int>(at & 15) / (F32 ? 4 : 2);
        count = (V + shift + N - 1) / N;
    }
    __device__ __forceinline__ uint4 load(int v) const {
        const uint32_t none = F32 ? 0xFF800000u : 0xFF80FF80u;
        if (v >= count) return make_uint4(none, none, none, none);
        uint4 x = vectors[v];
        if (v == 0 || v == count - 1) {
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = v * N + i - shift;
                if (at < 0 || at >= V) {
                    if (F32) w[i & 3] = none;
                    else w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xFFFFu) | 0xFF800000u : (w[i >> 1] & 0xFFFF0000u) | 0xFF80u;
                }
            }
            x = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return x;
    }
    // f(value, index) for each element of vector v
    template <class F>
    __device__ __forceinline__ void elements(const uint4& x, int v, F f) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = F32 ? __uint_as_float(w[i & 3]) : (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
            f(fmaxf(y, -INFINITY), v * N + i - shift);   // (NaN like -inf)
        }
    }
    // f(vector, its number, turn) for this thread's vectors
    template <class F>
    __device__ __forceinline__ void all(F f) const {
        for (int j = 0; j * kThreads < count; j += 4) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = load(static_cast<int>(threadIdx.x) + (j + i) * kThreads);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const uint4 y = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3];
                if ((j + i) * kThreads < count) f(y, static_cast<int>(threadIdx.x) + (j + i) * kThreads, j + i);
            }
        }
    }
    template <class F>
    __device__ __forceinline__ void values(F f) const {
        all([&](const uint4& x, int v, int) { elements(x, v, f); });
    }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
    __shared__ Shared sh;
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Row<F32> row(p.logits, b * p.row_stride, p.V);
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const float r = greedy ? 1.0f : 1.0f / t;
    int k = p.top_k ? p.top_k[b] : 0;
    if (k < 0 || k >= p.V) k = 0;
    const uint64_t p_units = p.top_p ? units_of_2_24(p.top_p[b], 1u << 24) : 1u << 24;
    const bool cuts = p_units < (1u << 24);
    uint32_t least = 1;                      // smallest weight kept
    if (p.min_p) {
        const float f = ceilf(p.min_p[b] * 2147483648.0f);
        least = f >= 4294967040.0f ? 0xFFFFFFFFu : f > 1.0f ? static_cast<uint32_t>(f) : 1u;
    }
    const float uniform = p.u[b];
    auto answer = [&](int token, float prob) {
        p.tokens[b] = token;
        if (p.probs) p.probs[b] = prob;
    };

    float mine = -INFINITY;
    row.values([&](float x, int) { mine = fmaxf(mine, x); });
    float top = wave_max(mine);
    if (lane == 0) sh.wave32[wave] = __float_as_uint(top);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.bins[i] = 0;
        sh.counts[i] = 0;
    }
    if (threadIdx.x == 0) sh.candidates = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, __uint_as_float(sh.wave32[w]));
    if (top == -INFINITY) {
        if (threadIdx.x == 0) answer(-1, 0.0f);
        return;
    }
    if (greedy) {
        int first = 0x7FFFFFFF;
        row.values([&](float x, int i) { first = x == top && i < first ? i : first; });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) first = min(first, __shfl_xor(first, off));
        __syncthreads();
        if (lane == 0) sh.wave32[wave] = static_cast<uint32_t>(first);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) first = min(first, static_cast<int>(sh.wave32[w]));
        if (threadIdx.x == 0) answer(first, least <= 0x80000000u ? 1.0f : 0.0f);
        return;
    }

    uint32_t kappa = 0, iota = 0xFFFFFFFFu;  // kept: keys above kappa, and equal ones up to index iota
    uint64_t take = 0;                       // how many equal ones
    // the threads' maxima by distance: the bin in which the n-th largest lies
    auto bound = [&](int n) -> float {
        if (p.V <= kCandidates) return 1e30f;
        const float at = bin_of(mine, top, r);
        if (at < kBins) atomicAdd(&sh.counts[static_cast<int>(at)], 1u);
        __syncthreads();
        uint64_t before;
        const int bin = reach(sh, kBins, n, before, [&](int i) { return static_cast<uint64_t>(sh.counts[i]); });
        return bin < kBins ? static_cast<float>(bin + 1) : 1e30f;
    };
    auto collect = [&](float from, float below) -> int {
        row.values([&](float x, int i) {
            const float at = bin_of(x, top, r);
            if (at >= from && at < below) {
                const uint32_t n = atomicAdd(&sh.candidates, 1u);
                if (n < kCandidates) {
                    sh.key[n] = key_of(x);
                    sh.index[n] = static_cast<uint32_t>(i);
                }
            }
        });
        __syncthreads();
        return static_cast<int>(sh.candidates);
    };

    // this thread's collected tokens
    uint32_t ck[kMine], ci[kMine], cw[kMine];
    int mine_count = 0;
    auto own = [&](int n) {
        mine_count = (n - static_cast<int>(threadIdx.x) + kThreads - 1) / kThreads;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = static_cast<int>(threadIdx.x) + i * kThreads;
            ck[i] = at < n ? sh.key[at] : 0;
            ci[i] = at < n ? sh.index[at] : 0;
            cw[i] = at < n ? weight_of(value_of(ck[i]), top, r) : 0;
        }
    };
    auto collected = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (i < mine_count) f(ck[i], ci[i], cw[i]);
    };
    // ... or all tokens of the row; f(key, index, weight) with a function for the weight
    auto everything = [&](auto f) {
        row.values([&](float x, int i) {
            const uint32_t key = key_of(x);
            f(key, static_cast<uint32_t>(i), [&] { return weight_of(x, top, r); });
        });
    };
    constexpr int kStop = F32 ? 0 : 16;      // the low bits of a bf16 key follow from its sign
    auto whole_key = [&](uint32_t key) { return !F32 && !(key >> 31) ? key | 0xFFFFu : key; };
    auto weight_at = [&](uint32_t key) -> uint64_t { return weight_of(value_of(key), top, r); };

    bool few = false;                        // the kept tokens are all among the collected,
    bool listed = false;                     // or at least those equal to kappa
    if (k > 0) {
        int n = k <= kThreads || p.V <= kCandidates ? collect(0.0f, bound(k)) : kCandidates + 1;
        uint64_t above;
        if (n <= kCandidates) {
            few = listed = true;
            own(n);
            kappa = whole_key(select(sh, 32, kStop, k, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t) { f(key, [] { return 1ull; }); }); }));
        } else {
            kappa = whole_key(select(sh, 32, kStop, k, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto) { f(key, [] { return 1ull; }); }); }));
        }
        take = k - above;
        if (cuts) {
            uint64_t sum = 0;
            if (few) collected([&](uint32_t key, uint32_t, uint32_t w) { sum += key > kappa ? w : 0; });
            else everything([&](uint32_t key, uint32_t, auto w) { if (key > kappa) sum += w(); });
            const uint64_t total = block_sum(sh, sum) + take * weight_at(kappa);
            bool more;
            uint64_t need = part_of(p_units, total, more);
            need += more ? 1 : 0;
            need = need < 1 ? 1 : need;
            uint32_t at;
            if (few) at = select(sh, 32, kStop, need, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t w) { f(key, [&] { return static_cast<unsigned long long>(w); }); }); });
            else at = select(sh, 32, kStop, need, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto w) { f(key, [&] { return static_cast<unsigned long long>(w()); }); }); });
            at = whole_key(at);
            const uint64_t w = weight_at(at);
            const uint64_t n_at = w ? (need - above + w - 1) / w : 1;
            if (at > kappa) {
                kappa = at;
                take = n_at;
            } else if (n_at < take) {
                take = n_at;
            }
        }
    } else if (cuts) {
        // weights by distance, down to the 512th largest of the threads'
        // maxima; if p of the total lies further down, all
        float limit = bound(512);
        uint64_t total = 0, need = 0, before = 0;
        int bin = kBins;
        float from = 0.0f;
        while (true) {
            uint64_t rest = 0;
            row.values([&](float x, int) {
                const float at = bin_of(x, top, r);
                const uint32_t w = weight_of(x, top, r);
                if (at >= from && at < limit && at < kBins) {
                    if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[static_cast<int>(at)]), static_cast<unsigned long long>(w));
                } else if (at >= limit) {
                    rest += w;
                }
            });
            rest = block_sum(sh, rest);      // (also a barrier after the atomics)
            if (from == 0.0f) {
                uint64_t binned = 0;
                for (int i = threadIdx.x; i < kBins; i += kThreads) binned += sh.bins[i];
                total = block_sum(sh, binned) + rest;
                bool more;
                need = part_of(p_units, total, more);
                need += more ? 1 : 0;
                need = need < 1 ? 1 : need;
            }
            bin = reach(sh, kBins, need, before, [&](int i) { return sh.bins[i]; });
            if (bin < kBins || !(limit < 1e29f)) break;
            from = limit;
            limit = 1e30f;
        }
        // (2048 bins reach further than any weight of a unit or more)
        const int n = collect(static_cast<float>(bin), static_cast<float>(bin + 1));
        uint64_t above;
        if (n <= kCandidates) {
            listed = true;
            own(n);
            kappa = whole_key(select(sh, 32, kStop, need - before, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t w) { f(key, [&] { return static_cast<unsigned long long>(w); }); }); }));
            above += before;
        } else {
            kappa = whole_key(select(sh, 32, kStop, need, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto w) { f(key, [&] { return static_cast<unsigned long long>(w()); }); }); }));
        }
        const uint64_t w = weight_at(kappa);
        take = w ? (need - above + w - 1) / w : 1;
    }
    if (kappa) {
        // the take-th of the tokens equal to kappa, by index, if not all are kept
        uint64_t ties = 0, above;
        if (listed) collected([&](uint32_t key, uint32_t, uint32_t) { ties += key == kappa; });
        else everything([&](uint32_t key, uint32_t, auto) { ties += key == kappa; });
        ties = block_sum(sh, ties);
        if (take < ties) {
            uint32_t at;
            if (listed) at = select(sh, 24, 0, take, above, [&](auto f) { collected([&](uint32_t key, uint32_t i, uint32_t) { if (key == kappa) f(i ^ 0xFFFFFFu, [] { return 1ull; }); }); });
            else at = select(sh, 24, 0, take, above, [&](auto f) { everything([&](uint32_t key, uint32_t i, auto) { if (key == kappa) f(i ^ 0xFFFFFFu, [] { return 1ull; }); }); });
            iota = at ^ 0xFFFFFFu;
        }
    }
    auto keeps = [&](uint32_t key, uint32_t i) { return key > kappa || (key == kappa && i <= iota); };
    const uint64_t u_units = units_of_2_24(uniform, (1u << 24) - 1);
    bool more;

    if (few) {
        uint64_t sum = 0;
        collected([&](uint32_t key, uint32_t i, uint32_t w) { sum += keeps(key, i) && w >= least ? w : 0; });
        const uint64_t total = block_sum(sh, sum);
        if (total == 0) {                    // min_p above 1
            if (threadIdx.x == 0) answer(-1, 0.0f);
            return;
        }
        const uint64_t target = part_of(u_units, total, more);
        uint64_t above;
        const uint32_t token = select(sh, 24, 0, target + 1, above, [&](auto f) {
                                   collected([&](uint32_t key, uint32_t i, uint32_t w) {
                                       if (keeps(key, i) && w >= least) f(i ^ 0xFFFFFFu, [&] { return static_cast<unsigned long long>(w); });
                                   });
                               }) ^ 0xFFFFFFu;
        collected([&](uint32_t, uint32_t i, uint32_t w) {
            if (i == token) answer(static_cast<int>(i), static_cast<float>(static_cast<double>(w) / static_cast<double>(total)));
        });
        return;
    }

    // the kept weight of each 64 vectors (a wavefront's turn), then of the
    // vectors and elements where the target is reached
    __syncthreads();                         // (the segments lie where the bins did)
    const int segments = (row.count + 63) / 64;
    auto kept_weight = [&](float x, int i) -> uint32_t {
        const uint32_t key = key_of(x);
        if (!keeps(key, static_cast<uint32_t>(i))) return 0u;
        const uint32_t w = weight_of(x, top, r);
        return w >= least ? w : 0u;
    };
    row.all([&](const uint4& x, int v, int j) {
        uint64_t sum = 0;
        row.elements(x, v, [&](float y, int i) { sum += kept_weight(y, i); });
        sum = wave_sum64(sum);
        if (lane == 0 && j * kWaves + wave < segments) sh.segments[j * kWaves + wave] = sum;
    });
    __syncthreads();
    uint64_t total = 0;
    for (int i = threadIdx.x; i < segments; i += kThreads) total += sh.segments[i];
    total = block_sum(sh, total);
    if (total == 0) {
        if (threadIdx.x == 0) answer(-1, 0.0f);
        return;
    }
    const uint64_t target = part_of(u_units, total, more);
    uint64_t before;
    const int segment = reach(sh, (segments + 63) / 64 * 64, target + 1, before,
                              [&](int i) { return i < segments ? sh.segments[i] : uint64_t{0}; });
    if (wave != 0) return;
    const int v = segment * 64 + lane;
    const uint4 x = row.load(v);
    uint64_t sum = 0;
    row.elements(x, v, [&](float y, int i) { sum += kept_weight(y, i); });
    const uint64_t upto = before + wave_scan64(sum);
    const uint64_t hit = __ballot(upto > target);
    if (hit && lane == __ffsll(static_cast<unsigned long long>(hit)) - 1) {
        uint64_t at = upto - sum;
        bool found = false;
        row.elements(x, v, [&](float y, int i) {
            const uint32_t w = kept_weight(y, i);
            if (!found && at + w > target) {
                found = true;
                answer(i, static_cast<float>(static_cast<double>(w) / static_cast<double>(total)));
            }
            at += w;
        });
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
