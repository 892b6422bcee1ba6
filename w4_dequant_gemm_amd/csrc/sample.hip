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
// maximum, and again from the caches for what follows:
//  - top-k: the k-th largest of the threads' own maxima bounds the k-th largest
//    logit from below, so few tokens besides the top k lie above it: they are
//    collected in shared memory and the filters and the draw work on them;
//  - top-p alone, bf16: how often each value occurs is counted, which gives the
//    value at which p of the weight is reached;
//  - top-p alone, fp32: weights of the tokens near the top are summed in bins of
//    the scaled distance to the maximum, all others together; the bin in which p
//    of the total is reached is collected and searched;
//  - neither: nothing to search.
// Up to 128 collected tokens are compared each with each, which ranks them and
// sums what precedes them at once (top-k 50 of 50001 fp32 logits 17 -> 13 us; 256
// of them would take as long as the searches).  Other searches are radix
// selections on the order-preserving key (or the index), eight bits a level: by
// count for top-k, by weight for top-p and the draw.
// Where more tokens are kept than shared memory collects, the draw goes over the
// row once more; where a search's own tokens do not fit (many equal logits), it
// goes over the row for each level.
//
// Measured, 200 rows of 131072 bf16 logits (52 MB: 10 us to read once): greedy
// 15 us, top-k 50 26, top-p 0.5 44, top-p 0.95 48 (of a nearly flat row 68), no
// filter 30.  One row of 50001 fp32 logits: 10, 13, 31, 67 (126), 22, of which
// launch and binding are 9.  Bound by the row's one compute unit: each pass over
// a row from the caches is 6 us, a table entry, count or comparison for each of
// its logits 8 to 13 more.  Searches that go over the row for each level: top-k
// 1000 or 2000 144 and 135 us (one row: 96 and 92), top-k 50 of 13 different
// values 172 (99), top-p 0.9 of those 134 (142), top-k 2000 with top-p 0.9 277
// (163).
#include <type_traits>

#include "device.hpp"
#include "decode_kernels.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kCandidates = 2048;            // tokens collected in shared memory, and vectors that hold them
constexpr int kRanked = 128;                 // of those, few enough to compare each with each
constexpr int kMine = kCandidates / kThreads;
constexpr int kAhead = 8;                    // vectors a thread has on their way
constexpr int kBins = 512;
constexpr float kBinsPerUnit = 16.0f;        // bins of 1/16 of the scaled distance, down to exp(-32)
constexpr int kGroup = 4;                     // 64 vectors each a segment
constexpr int kSegments = ((1 << 20) / 4 / (64 * kGroup) / kWaves + 2) * kWaves;
constexpr int kLevels = 18;                  // of all selections of a call: 4 + 4 by key, 3 + 3 by index, and spare

// fp32 (not NaN) -> a key in the order of the values; -0 like +0
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// rint(2^31 exp((x - top) r)), without branches
__device__ __forceinline__ uint32_t weight_of(float x, float top, float r) {
    const float d = x == top ? 0.0f : (x - top) * r;   // (infinities' NaN at the top)
    const float e = fmaxf(expf(d), 0.0f);              // (NaN, of -inf at T = inf, is 0)
    return static_cast<uint32_t>(rintf(e * 2147483648.0f));
}
// a distance that grows as the weight falls, the same for equal values (NaN for
// infinities: like 0); a bin is its whole part
__device__ __forceinline__ float distance(float x, float top, float r) { return (top - x) * (r * kBinsPerUnit); }
__device__ __forceinline__ int bin_of(float d) { return static_cast<int>(fminf(fmaxf(d, 0.0f), static_cast<float>(kBins))); }

// The larger of m (no NaN) and x, NaN left out, in one instruction (fmaxf: two).
// A maximum with a signalling NaN is a quiet NaN and loses the other operand, so
// x is first put beside itself: max(max(x, x), m).
__device__ __forceinline__ float larger(float m, float x) {
    float r;
    asm("v_max3_f32 %0, %1, %1, %2" : "=v"(r) : "v"(x), "v"(m));
    return r;
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

// lane i gets lane i - n's value by a data-parallel move (0 where there is none)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xF, false);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
// running sum over the 64 lanes, this one included: shifts by 1, 2, 4, 8 within
// rows of 16 lanes, then each row's last lane to the rows after it
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
    v += moved<0x111, 0xF>(v);
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    v += moved<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) { return lane_value(wave_scan64(v), 63); }

// Weights of the bf16 values of magnitude 2^-14 .. 2^8, by sign and bits: of a
// row's many logits few are different, and reading a weight takes a fourth of
// the time of computing it (an exponential of every one of 131072 logits: 35
// us on the row's compute unit).
constexpr uint32_t kTableFrom = (127 - 14) << 7, kTableHalf = 22 << 7;

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

struct Shared {
    uint32_t table[2 * kTableHalf];          // weights of bf16 values
    uint32_t numbers[2 * kTableHalf];        // how often they occur
    uint64_t hist[kLevels][256];             // one a level: cleared at the start, used once
    uint64_t bins[kBins];                    // weights by distance
    uint64_t segments[kSegments];
    uint64_t wave64[2][kWaves];
    uint32_t counts[kBins];                  // threads' maxima by distance
    uint32_t wave32[2][kWaves];
    uint32_t key[kCandidates], index[kCandidates];
    uint32_t vectors[kCandidates];
    uint64_t outside[3];                     // weights above the table's values, between its halves, below
    uint32_t candidates, marked;
    uint32_t found;                          // and what belongs to it
    uint64_t found_above;
};

// What every wavefront of the row knows alike.
struct Turn {
    Shared& sh;
    int level = 0, sums = 0;
    // (two places in turn: one barrier a sum)
    __device__ __forceinline__ uint64_t block_sum(uint64_t v) {
        v = wave_sum64(v);
        uint64_t* at = sh.wave64[sums++ & 1];
        if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = v;
        __syncthreads();
        return wave_sum64((threadIdx.x & 63) < kWaves ? at[threadIdx.x & 63] : 0);
    }
};

// The first of 64 PER bins (ascending) at which their running sum reaches need,
// and the sum before it; 64 PER and the whole sum if it is not reached.  Every
// wavefront searches for itself, which saves the barriers of telling.
template <int PER, class Get>
__device__ __forceinline__ int reach(uint64_t need, uint64_t& before, Get get) {
    const int lane = threadIdx.x & 63;
    uint64_t w[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        w[i] = get(lane * PER + i);
        mine += w[i];
    }
    const uint64_t upto = wave_scan64(mine);
    const uint64_t hit = __ballot(upto >= need);
    if (!hit) {
        before = lane_value(upto, 63);
        return 64 * PER;
    }
    const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
    uint64_t sum = upto - mine;
    int skip = 0;
#pragma unroll
    for (int i = 0; i < PER - 1; ++i)
        if (skip == i && sum + w[i] < need) {
            sum += w[i];
            ++skip;
        }
    before = lane_value(sum, at);
    return at * PER + __builtin_amdgcn_readlane(skip, at);
}

// The key (of `bits` bits, a multiple of 8) at which the running sum of weights
// from the largest key down reaches `need` (1 .. their total), and the sum
// above it.  each(f) calls f(key, weight) for this thread's items, weight being
// a function.
template <class Each>
__device__ __forceinline__ uint32_t select(Turn& turn, int bits, int stop, uint64_t need, uint64_t& above, Each each) {
    uint32_t prefix = 0;
    above = 0;
#pragma unroll 1
    for (int shift = bits - 8; shift >= stop; shift -= 8) {
        uint64_t* hist = turn.sh.hist[turn.level++];
        const uint32_t mask = shift + 8 >= 32 ? 0u : 0xFFFFFFFFu << (shift + 8);
        each([&](uint32_t key, auto weight) {
            if (((key ^ prefix) & mask) == 0) {
                const unsigned long long w = weight();
                if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&hist[255 - ((key >> shift) & 255)]), w);
            }
        });
        __syncthreads();
        uint64_t before;
        const int at = reach<4>(need - above, before, [&](int i) { return hist[i]; });
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
        uint4 x = make_uint4(none, none, none, none);
        if (v < count) x = vectors[v];
        if ((v == 0 && shift) || v == count - 1) {
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
    // the values of vector v; that of element i has the index v N + i - shift
    static __device__ __forceinline__ void unpack(const uint4& x, float (&y)[N]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = F32 ? __uint_as_float(w[i & 3]) : (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
    // the largest of m and the values, NaN left out
    static __device__ __forceinline__ float largest(const float (&y)[N], float m = -INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i) m = larger(m, y[i]);
        return m;
    }
    // f(vector, its number, turn) for this thread's vectors, read ahead
    template <class F>
    __device__ __forceinline__ void all(F f) const {
        const int tid = static_cast<int>(threadIdx.x);
        uint4 a = load(tid), b = load(tid + kThreads), c = load(tid + 2 * kThreads), d = load(tid + 3 * kThreads);
#pragma unroll 1
        for (int j = 0; j * kThreads < count; ++j) {
            const uint4 e = load(tid + (j + 4) * kThreads);
            f(a, tid + j * kThreads, j);
            a = b;
            b = c;
            c = d;
            d = e;
        }
    }
    // f(values, number of the vector, the vector)
    template <class F>
    __device__ __forceinline__ void values(F f) const {
        all([&](const uint4& x, int v, int) {
            float y[N];
            unpack(x, y);
            f(y, v, x);
        });
    }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
    __shared__ Shared sh;
    constexpr int N = Row<F32>::N;
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Row<F32> row(p.logits, b * p.row_stride, p.V);
    // what is done to every element with few instructions: f(values, vector)
    auto light = [&](auto f) {
#pragma unroll 1
        for (int j = 0; j * kThreads < row.count; j += kAhead) {
            uint4 x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i] = row.load(static_cast<int>(threadIdx.x) + (j + i) * kThreads);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float y[N];
                row.unpack(x[i], y);
                f(y, static_cast<int>(threadIdx.x) + (j + i) * kThreads);
            }
        }
    };
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const float r = greedy ? 1.0f : 1.0f / t;
    int k = p.top_k ? p.top_k[b] : 0;
    if (k < 0 || k >= p.V) k = 0;
    const uint64_t p_units = p.top_p ? units_of_2_24(p.top_p[b], 1u << 24) : 1u << 24;
    const bool cuts = p_units < (1u << 24);
    const float min_p = p.min_p ? p.min_p[b] : 0.0f;
    uint32_t least = 1;                      // smallest weight kept
    {
        const float f = ceilf(min_p * 2147483648.0f);
        least = f >= 4294967040.0f ? 0xFFFFFFFFu : f > 1.0f ? static_cast<uint32_t>(f) : 1u;
    }
    // a weight is kept from `least` less half a unit up: the logarithm of that (2^-7 more, for the
    // exponential's and the distances' errors), in units of the scaled distance
    const float least_log = logf((static_cast<float>(least) - 0.5f) * 0x1p-31f) - 0.0078125f;
    const float uniform = p.u[b];
    auto answer = [&](int token, float prob) {
        p.tokens[b] = token;
        if (p.probs) p.probs[b] = prob;
    };
    Turn turn{sh};
    for (int i = threadIdx.x; i < kLevels * 256; i += kThreads) (&sh.hist[0][0])[i] = 0;
    if (threadIdx.x < kBins) {
        sh.bins[threadIdx.x] = 0;
        sh.counts[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) sh.candidates = sh.marked = sh.found = 0;
    if (threadIdx.x < 3) sh.outside[threadIdx.x] = 0;

    float mine = -INFINITY;
    light([&](const float (&y)[N], int) { mine = row.largest(y, mine); });
    float top = wave_max(mine);
    if (lane == 0) sh.wave32[0][wave] = __float_as_uint(top);
    __syncthreads();
    top = max16(__uint_as_float(sh.wave32[0][lane & (kWaves - 1)]));
    if (top == -INFINITY) {
        if (threadIdx.x == 0) answer(-1, 0.0f);
        return;
    }
    if (greedy) {
        int first = 0x7FFFFFFF;
        if (mine == top)
            light([&](const float (&y)[N], int v) {
#pragma unroll
                for (int i = N - 1; i >= 0; --i)
                    if (y[i] == top && v * N + i - row.shift < first) first = v * N + i - row.shift;
            });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) first = min(first, __shfl_xor(first, off));
        if (lane == 0) sh.wave32[1][wave] = static_cast<uint32_t>(first);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWaves; ++w) first = min(first, static_cast<int>(sh.wave32[1][w]));
            const bool kept_one = least <= 0x80000000u;
            answer(kept_one ? first : -1, kept_one ? 1.0f : 0.0f);
        }
        return;
    }

    uint32_t kappa = 0, iota = 0xFFFFFFFFu;  // kept: keys above kappa, and equal ones up to index iota
    uint64_t take = 0;                       // how many equal ones
    // values below have no weight, exp(-22.5) 2^31 being less than 1/2 (an infinite top: all others;
    // 22.5 / r may be infinite too)
    const float weightless = top == INFINITY ? top : top - 22.5f / r;
    bool tabled = false;
    auto entry_value = [&](uint32_t i) {
        return __uint_as_float((i < kTableHalf ? kTableFrom + i : 0x8000u + kTableFrom + i - kTableHalf) << 16);
    };
    auto fill_table = [&] {
        if (F32) return;
        for (uint32_t i = threadIdx.x; i < 2 * kTableHalf; i += kThreads) {
            const float x = entry_value(i);
            sh.table[i] = x <= top ? weight_of(x, top, r) : 0;
            sh.numbers[i] = 0;
        }
        tabled = true;
        __syncthreads();
    };
    // Entries of a vector's bf16 values, two at a time in 16 bits: magnitude
    // above the table's first, then the index.  False if some lie outside (the
    // wavefront's vectors mostly have none).
    auto entries = [&](const uint4& x, u16x2_t (&at)[4]) -> bool {
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        u16x2_t most = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u16x2_t bits = __builtin_bit_cast(u16x2_t, in[i]);
            const u16x2_t above = (bits & static_cast<uint16_t>(0x7FFF)) - static_cast<uint16_t>(kTableFrom);
            most = __builtin_elementwise_max(most, above);
            at[i] = __builtin_elementwise_min(above, u16x2_t{kTableHalf - 1, kTableHalf - 1}) +
                    (bits >> static_cast<uint16_t>(15)) * static_cast<uint16_t>(kTableHalf);
        }
        return !__any(most[0] >= kTableHalf || most[1] >= kTableHalf);
    };
    auto outside_table = [&](const uint4& x, int i) {
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        return (((i & 1) ? in[i >> 1] >> 16 : in[i >> 1]) & 0x7FFFu) - kTableFrom >= kTableHalf;
    };
    // the weights of a vector's values; whether they were computed, not read
    auto weights = [&](const uint4& x, const float (&y)[N], uint32_t (&w)[N]) -> bool {
        bool exact = F32;
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = weight_of(y[i], top, r);
        } else {
            u16x2_t at[4];
            const bool inside = entries(x, at);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = sh.table[at[i >> 1][i & 1]];
            if (!inside) {
                // masked values (-inf, the lowest) are common: without weight; others are computed
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const bool outside = outside_table(x, i);
                    exact = exact || (outside && y[i] >= weightless);
                    w[i] = outside ? 0 : w[i];
                }
                exact = __any(exact);
                if (exact) {
#pragma unroll
                    for (int i = 0; i < N; ++i) w[i] = weight_of(y[i], top, r);
                }
            }
        }
        return exact;
    };
    // a distance within which at least n of the threads' maxima lie
    auto bound = [&](int n) -> float {
        if (p.V <= kCandidates) return 1e30f;
        const int at = bin_of(distance(mine, top, r));
        if (at < kBins) atomicAdd(&sh.counts[at], 1u);
        __syncthreads();
        uint64_t before;
        const int bin = reach<kBins / 64>(n, before, [&](int i) { return static_cast<uint64_t>(sh.counts[i]); });
        return bin < kBins ? static_cast<float>(bin + 1) : 1e30f;
    };
    // The tokens of the vectors that has(values) marks, where wants(value):
    // few vectors of a row, so they are listed first and then shared among the
    // threads.  More than kCandidates: too many.
    auto gather = [&](auto has, auto wants) -> int {
        light([&](const float (&y)[N], int v) {
            if (!has(y)) return;
            const uint32_t n = atomicAdd(&sh.marked, 1u);
            if (n < kCandidates) sh.vectors[n] = static_cast<uint32_t>(v);
        });
        __syncthreads();
        const int marked = static_cast<int>(sh.marked);
        if (marked <= kCandidates)
            for (int i = threadIdx.x; i < marked; i += kThreads) {
                const int v = static_cast<int>(sh.vectors[i]);
                float y[N];
                row.unpack(row.load(v), y);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float z = fmaxf(y[e], -INFINITY);   // (NaN like -inf)
                    if (!wants(z)) continue;
                    const uint32_t n = atomicAdd(&sh.candidates, 1u);
                    if (n < kCandidates) {
                        sh.key[n] = key_of(z);
                        sh.index[n] = static_cast<uint32_t>(v * N + e - row.shift);
                    }
                }
            }
        __syncthreads();
        return marked <= kCandidates ? static_cast<int>(sh.candidates) : kCandidates + 1;
    };
    auto gather_again = [&] {
        __syncthreads();
        if (threadIdx.x == 0) sh.candidates = sh.marked = 0;
        __syncthreads();
    };
    // the tokens with from <= distance < below (infinities' NaN is 0)
    auto collect = [&](float from, float below) -> int {
        return gather([&](const float (&y)[N]) {
                          if (from == 0.0f) return !(distance(row.largest(y), top, r) >= below);
                          bool any = false;
#pragma unroll
                          for (int i = 0; i < N; ++i) {
                              const float d = distance(y[i], top, r);
                              any = any || (d >= from && d < below);
                          }
                          return any;
                      },
                      [&](float z) {
                          const float d = distance(z, top, r);
                          return !(d >= below || d < from);
                      });
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
        row.values([&](const float (&y)[N], int v, const uint4&) {
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                float x = y[0];
#pragma unroll
                for (int j = 1; j < N; ++j) x = i == j ? y[j] : x;
                x = fmaxf(x, -INFINITY);
                f(key_of(x), static_cast<uint32_t>(v * N + i - row.shift), [&] { return weight_of(x, top, r); });
            }
        });
    };
    const int index_bits = p.V <= 65536 ? 16 : 24;
    const uint32_t index_mask = (1u << index_bits) - 1u;
    constexpr int kStop = F32 ? 0 : 16;      // the low bits of a bf16 key follow from its sign
    auto whole_key = [&](uint32_t key) { return !F32 && !(key >> 31) ? key | 0xFFFFu : key; };
    auto weight_at = [&](uint32_t key) -> uint64_t { return weight_of(value_of(key), top, r); };

    // Few collected tokens: how many of them there are (0: more, or not collected)
    // and are kept at most; top-p's weight is `ranked_need`, or p of theirs (0).
    int ranked = 0;
    uint64_t ranked_first = 0, ranked_need = 0;
    bool few = false;                        // the kept tokens are all among the collected
    if (k > 0) {
        int n = k <= kThreads || p.V <= kCandidates ? collect(0.0f, bound(k)) : kCandidates + 1;
        uint64_t above = 0;
        if (n <= kRanked) {
            ranked = n;
            ranked_first = k;
        } else if (n <= kCandidates) {
            few = true;
            k = k < n ? k : n;               // (fewer than k above -inf)
            own(n);
            kappa = whole_key(select(turn, 32, kStop, k, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t) { f(key, [] { return 1ull; }); }); }));
        } else {
            kappa = whole_key(select(turn, 32, kStop, k, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto) { f(key, [] { return 1ull; }); }); }));
        }
        if (!ranked) take = k - above;
        if (!ranked && cuts) {
            uint64_t sum = 0;
            if (few) collected([&](uint32_t key, uint32_t, uint32_t w) { sum += key > kappa ? w : 0; });
            else everything([&](uint32_t key, uint32_t, auto w) { if (key > kappa) sum += w(); });
            const uint64_t total = turn.block_sum(sum) + take * weight_at(kappa);
            bool more;
            uint64_t need = part_of(p_units, total, more);
            need += more ? 1 : 0;
            need = need < 1 ? 1 : need;
            uint32_t at;
            if (few) at = select(turn, 32, kStop, need, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t w) { f(key, [&] { return static_cast<unsigned long long>(w); }); }); });
            else at = select(turn, 32, kStop, need, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto w) { f(key, [&] { return static_cast<unsigned long long>(w()); }); }); });
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
        fill_table();
        uint64_t total = 0, need = 0, before = 0, above = 0;
        auto set_need = [&] {
            bool more;
            need = part_of(p_units, total, more);
            need += more ? 1 : 0;
            need = need < 1 ? 1 : need;
        };
        bool counted = !F32;
        if constexpr (!F32) {
            // how often each value of the table occurs, and from that the value
            // at which p of the weight is reached
            row.all([&](const uint4& x, int v, int) {
                u16x2_t at[4];
                const bool inside = entries(x, at);
                if (inside) {
#pragma unroll
                    for (int i = 0; i < N; ++i) atomicAdd(&sh.numbers[at[i >> 1][i & 1]], 1u);
                } else {
                    float y[N];
                    row.unpack(x, y);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (!outside_table(x, i)) atomicAdd(&sh.numbers[at[i >> 1][i & 1]], 1u);
                        else if (y[i] >= weightless)
                            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.outside[y[i] >= 1.0f ? 0 : y[i] > -1.0f ? 1 : 2]),
                                      static_cast<unsigned long long>(weight_of(y[i], top, r)));
                    }
                }
            });
            __syncthreads();
            // from the largest value down: those above the table, its positive
            // half backwards, those between, the negative half, those below
            constexpr uint32_t kPlaces = 2 * kTableHalf + 3;
            constexpr int kShare = (kPlaces + kThreads - 1) / kThreads;
            auto entry_at = [&](uint32_t q) { return q <= kTableHalf ? kTableHalf - q : q - 2; };
            auto mass_at = [&](uint32_t q) -> uint64_t {
                if (q == 0) return sh.outside[0];
                if (q == kTableHalf + 1) return sh.outside[1];
                if (q >= kPlaces - 1) return q == kPlaces - 1 ? sh.outside[2] : 0;
                const uint32_t e = entry_at(q);
                return static_cast<uint64_t>(sh.numbers[e]) * sh.table[e];
            };
            uint64_t mass = 0;
#pragma unroll 1
            for (int i = 0; i < kShare; ++i) mass += mass_at(threadIdx.x * kShare + i);
            const uint64_t upto = wave_scan64(mass);
            uint64_t* sums = sh.wave64[turn.sums++ & 1];
            if (lane == 63) sums[wave] = upto;
            __syncthreads();
            uint64_t start = 0;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                if (i < wave) start += sums[i];
                total += sums[i];
            }
            set_need();
            uint64_t sum = start + upto - mass;
            if (sum < need && need <= start + upto) {
#pragma unroll 1
                for (int i = 0; i < kShare; ++i) {
                    const uint32_t q = threadIdx.x * kShare + i;
                    const uint64_t w = mass_at(q);
                    if (sum + w >= need) {
                        sh.found = q;
                        sh.found_above = sum;
                        break;
                    }
                    sum += w;
                }
            }
            __syncthreads();
            // (among those outside the table it would have to be searched for)
            const uint32_t q = sh.found;
            counted = q != 0 && q != kTableHalf + 1 && q != kPlaces - 1;
            if (counted) {
                const uint32_t entry = entry_at(q);
                kappa = key_of(entry_value(entry));
                above = sh.found_above;
                // the kept tokens, if they are few
                const float value = value_of(kappa);
                const uint64_t w = weight_at(kappa);
                take = (need - above + w - 1) / w;
                uint64_t kept = 0;
#pragma unroll 1
                for (int i = 0; i < kShare; ++i) {
                    const uint32_t at = threadIdx.x * kShare + i;
                    if (at < q && at != 0 && at != kTableHalf + 1) kept += sh.numbers[entry_at(at)];
                }
                if (turn.block_sum(kept) + take <= kCandidates) {
                    const int n = gather([&](const float (&y)[N]) { return row.largest(y) >= value; }, [&](float z) { return z >= value; });
                    few = n <= kCandidates;
                    if (n <= kRanked) {
                        ranked = n;
                        ranked_first = n;
                        ranked_need = need;
                    } else if (few) {
                        own(n);
                    }
                }
            }
        }
        if (!counted) {
            // the total, and the vectors with tokens nearer than the 512th
            // largest of the threads' maxima, whose weights are binned by
            // distance; if p of the total lies further down, all
            total = 0;
            const float limit = bound(512);
            auto to_bins = [&](const float (&y)[N], const uint32_t (&w)[N], float below) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float d = distance(y[i], top, r);
                    const int at = bin_of(d);
                    if (!(d >= below) && w[i] && at < kBins)
                        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[at]), static_cast<unsigned long long>(w[i]));
                }
            };
            row.values([&](const float (&y)[N], int v, const uint4& x) {
                uint32_t w[N];
                weights(x, y, w);
#pragma unroll
                for (int i = 0; i < N; ++i) total += w[i];
                if (!(distance(row.largest(y), top, r) >= limit)) {
                    const uint32_t n = atomicAdd(&sh.marked, 1u);
                    if (n < kCandidates) sh.vectors[n] = static_cast<uint32_t>(v);
                }
            });
            total = turn.block_sum(total);   // (its barrier is also that of the list)
            set_need();
            const int marked = static_cast<int>(sh.marked);
            int bin = kBins;
            auto bins = [&](int i) { return sh.bins[i]; };
            if (marked <= kCandidates) {
                for (int i = threadIdx.x; i < marked; i += kThreads) {
                    const uint4 x = row.load(static_cast<int>(sh.vectors[i]));
                    float y[N];
                    uint32_t w[N];
                    row.unpack(x, y);
#pragma unroll
                    for (int e = 0; e < N; ++e) w[e] = weight_of(y[e], top, r);
                    to_bins(y, w, limit);
                }
                __syncthreads();
                bin = reach<kBins / 64>(need, before, bins);
            }
            if (bin == kBins) {
                __syncthreads();
                if (threadIdx.x < kBins) sh.bins[threadIdx.x] = 0;
                __syncthreads();
                row.values([&](const float (&y)[N], int, const uint4& x) {
                    uint32_t w[N];
                    weights(x, y, w);
                    to_bins(y, w, 1e30f);
                });
                __syncthreads();
                bin = reach<kBins / 64>(need, before, bins);   // (a weight of a unit or more is nearer than the last bin)
            }
            // all kept tokens, or those of the bin alone, or neither fits
            gather_again();
            int n = collect(0.0f, static_cast<float>(bin + 1));
            few = n <= kCandidates;
            if (!few) {
                gather_again();
                n = collect(static_cast<float>(bin), static_cast<float>(bin + 1));
            }
            if (n <= kRanked && few) {
                ranked = n;
                ranked_first = n;
                ranked_need = need;
            } else if (n <= kCandidates) {
                own(n);
                const uint64_t skip = few ? 0 : before;
                kappa = whole_key(select(turn, 32, kStop, need - skip, above, [&](auto f) { collected([&](uint32_t key, uint32_t, uint32_t w) { f(key, [&] { return static_cast<unsigned long long>(w); }); }); }));
                above += skip;
            } else {
                kappa = whole_key(select(turn, 32, kStop, need, above, [&](auto f) { everything([&](uint32_t key, uint32_t, auto w) { f(key, [&] { return static_cast<unsigned long long>(w()); }); }); }));
            }
            const uint64_t w = weight_at(kappa);
            take = w ? (need - above + w - 1) / w : 1;
        }
    } else if (least > 1) {
        // min_p alone: what it may keep, if it fits
        const int n = collect(0.0f, -least_log * kBinsPerUnit);
        few = n <= kCandidates;
        if (few) own(n);
    }
    const uint64_t u_units = units_of_2_24(uniform, (1u << 24) - 1);
    bool more;
    if (ranked) {
        // A thread for each token and eighth of the others counts those that
        // precede it and their weight, which answers every filter, then the kept
        // weight of lower indices, which is the draw.
        typedef unsigned long long ull;
        auto& rank = sh.hist[0];             // (clear: no selection has run)
        auto& before = sh.hist[1];
        auto& lower = sh.hist[2];
        auto& weight = sh.hist[3];
        auto& kept = sh.hist[4];
        const int c = threadIdx.x % kRanked, q = threadIdx.x / kRanked;
        constexpr int kParts = kThreads / kRanked;
        const bool is = c < ranked;
        const uint32_t key = is ? sh.key[c] : 0, index = is ? sh.index[c] : 0;
        const uint64_t w = is ? weight_at(key) : 0;
        if (q == 0) weight[c] = w;
        __syncthreads();
        const uint64_t order = static_cast<uint64_t>(key) << 32 | ~index;
        uint32_t count = 0;
        uint64_t sum = 0;
#pragma unroll 8
        for (int j = q; j < ranked; j += kParts) {
            const uint64_t other = static_cast<uint64_t>(sh.key[j]) << 32 | ~sh.index[j];
            const uint64_t v = weight[j];
            count += other > order;
            sum += other > order ? v : 0;
        }
        if (is) {
            atomicAdd(reinterpret_cast<ull*>(&rank[c]), static_cast<ull>(count));
            atomicAdd(reinterpret_cast<ull*>(&before[c]), static_cast<ull>(sum));
        }
        __syncthreads();
        const bool in = is && rank[c] < ranked_first;
        uint64_t need = ranked_need;
        if (cuts && need == 0) {
            need = part_of(p_units, turn.block_sum(q == 0 && in ? w : 0), more);
            need += more ? 1 : 0;
            need = need < 1 ? 1 : need;
        }
        const bool keep = in && (!cuts || before[c] < need) && w >= least;
        if (q == 0) kept[c] = keep ? w : 0;
        const uint64_t total = turn.block_sum(q == 0 && keep ? w : 0);
        if (total == 0) {                    // min_p above 1
            if (threadIdx.x == 0) answer(-1, 0.0f);
            return;
        }
        const uint64_t target = part_of(u_units, total, more);
        sum = 0;
#pragma unroll 8
        for (int j = q; j < ranked; j += kParts) {
            const uint32_t other = sh.index[j];
            const uint64_t v = kept[j];
            sum += other < index ? v : 0;
        }
        if (is) atomicAdd(reinterpret_cast<ull*>(&lower[c]), static_cast<ull>(sum));
        __syncthreads();
        if (q == 0 && keep && lower[c] <= target && target < lower[c] + w)
            answer(static_cast<int>(index), static_cast<float>(static_cast<double>(w) / static_cast<double>(total)));
        return;
    }
    if (few && kappa) {
        // the take-th of the tokens equal to kappa, by index, if not all are kept
        uint64_t ties = 0, above;
        collected([&](uint32_t key, uint32_t, uint32_t) { ties += key == kappa; });
        ties = turn.block_sum(ties);
        if (take < ties)
            iota = select(turn, index_bits, 0, take, above, [&](auto f) { collected([&](uint32_t key, uint32_t i, uint32_t) { if (key == kappa) f(i ^ index_mask, [] { return 1ull; }); }); }) ^ index_mask;
    }
    auto keeps = [&](uint32_t key, uint32_t i) { return key > kappa || (key == kappa && i <= iota); };

    if (few) {
        uint64_t sum = 0;
        collected([&](uint32_t key, uint32_t i, uint32_t w) { sum += keeps(key, i) && w >= least ? w : 0; });
        const uint64_t total = turn.block_sum(sum);
        if (total == 0) {                    // min_p above 1
            if (threadIdx.x == 0) answer(-1, 0.0f);
            return;
        }
        const uint64_t target = part_of(u_units, total, more);
        uint64_t above;
        const uint32_t token = select(turn, index_bits, 0, target + 1, above, [&](auto f) {
                                   collected([&](uint32_t key, uint32_t i, uint32_t w) {
                                       if (keeps(key, i) && w >= least) f(i ^ index_mask, [&] { return static_cast<unsigned long long>(w); });
                                   });
                               }) ^ index_mask;
        collected([&](uint32_t, uint32_t i, uint32_t w) {
            if (i == token) answer(static_cast<int>(i), static_cast<float>(static_cast<double>(w) / static_cast<double>(total)));
        });
        return;
    }

    // Each wavefront takes a run of the row's vectors; the kept weight of its
    // segments of 4 x 64 vectors, then of the vectors and elements of the
    // segment in which the target is reached.  How many tokens of a segment equal
    // kappa is counted on the way (bits 48 and up): the first `take` are kept.
    const int turns = (row.count + 64 * kWaves - 1) / (64 * kWaves);   // of 64 vectors, a wavefront
    const int groups = (turns + kGroup - 1) / kGroup;
    const float value = value_of(kappa);
    constexpr uint64_t kSum = (uint64_t{1} << 48) - 1;
    static_assert(kGroup * 64 * N < 1 << 16, "a segment's tokens fit 16 bits, their weights 48");
    if (!tabled) fill_table();
    if (!F32 && (kappa || least > 1)) {
        // values that are not kept have no weight
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 2 * kTableHalf; i += kThreads)
            if ((kappa && entry_value(i) < value) || sh.table[i] < least) sh.table[i] = 0;
        __syncthreads();
    }
    // values below this one are not kept: kappa's, or that of min_p
    const float lowest = fmaxf(kappa ? value : -INFINITY, least > 1 ? top + least_log * t : -INFINITY);
    // the weights of a vector's tokens down to kappa, and which of them equal it
    auto kept_weights = [&](const uint4& x, uint32_t (&w)[N]) -> uint32_t {
        float y[N];
        row.unpack(x, y);
        if (F32) {                           // (an exponential each)
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = 0;
            if (row.largest(y) < lowest) return 0;
        }
        if (weights(x, y, w)) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = (kappa && !(y[i] >= value)) || w[i] < least ? 0u : w[i];
        }
        uint32_t ties = 0;
        if (kappa)
#pragma unroll
            for (int i = 0; i < N; ++i) ties |= y[i] == value ? 1u << i : 0u;
        return ties;
    };
    auto segment_sum = [&](int w, int g) {   // this lane's part
        uint64_t sum = 0;
        uint4 x[kGroup];
        const int first = (w * turns + g * kGroup) * 64 + lane;
#pragma unroll
        for (int j = 0; j < kGroup; ++j) x[j] = g * kGroup + j < turns ? row.load(first + 64 * j) : row.load(row.count);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            uint32_t kw[N];
            const uint32_t ties = kept_weights(x[j], kw);
#pragma unroll
            for (int i = 0; i < N; ++i) sum += kw[i];
            sum += static_cast<uint64_t>(__popc(ties)) << 48;
        }
        return sum;
    };
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
        const uint64_t sum = wave_sum64(segment_sum(wave, g));
        if (lane == 0) sh.segments[wave * groups + g] = sum;
    }
    __syncthreads();
    const int segments = kWaves * groups;
    if (kappa) {
        constexpr int kShare = (kSegments + kThreads - 1) / kThreads;
        uint64_t mine_ties = 0;
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const int at = static_cast<int>(threadIdx.x) * kShare + i;
            if (at < segments) mine_ties += sh.segments[at] >> 48;
        }
        const uint64_t upto = wave_scan64(mine_ties);
        uint64_t* sums = sh.wave64[turn.sums++ & 1];
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        uint64_t before = upto - mine_ties;
        for (int i = 0; i < wave; ++i) before += sums[i];
        const uint64_t one = weight_at(kappa) < least ? 0 : weight_at(kappa);
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const int at = static_cast<int>(threadIdx.x) * kShare + i;
            if (at >= segments) continue;
            const uint64_t all = sh.segments[at], ties = all >> 48;
            const uint64_t left = before < take ? take - before : 0, kept = left < ties ? left : ties;
            sh.segments[at] = (all & kSum) - (ties - kept) * one + (kept << 48);
            before += ties;
        }
        __syncthreads();
    }
    uint64_t total = 0;
    for (int i = threadIdx.x; i < segments; i += kThreads) total += sh.segments[i] & kSum;
    total = turn.block_sum(total);
    if (total == 0) {
        if (threadIdx.x == 0) answer(-1, 0.0f);
        return;
    }
    if (wave != 0) return;
    const uint64_t target = part_of(u_units, total, more);
    uint64_t before = 0, passed = 0;
    int segment = 0;
    for (;; segment += 64) {
        const int at = reach<1>(target + 1 - before, passed, [&](int i) { return segment + i < segments ? sh.segments[segment + i] & kSum : uint64_t{0}; });
        before += passed;
        if (at < 64) {
            segment += at;
            break;
        }
    }
    uint64_t left = sh.segments[segment] >> 48;
    const int first = (segment / groups * turns + segment % groups * kGroup) * 64 + lane;
#pragma unroll 1
    for (int j = 0; j < kGroup; ++j) {
        const int v = first + 64 * j;
        uint32_t w[N];
        const uint32_t ties = kept_weights(row.load(v), w);
        if (kappa) {
            const uint64_t upto = wave_scan64(static_cast<uint64_t>(__popc(ties)));
            uint64_t rank = upto - __popc(ties);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((ties >> i) & 1 && rank++ >= left) w[i] = 0;
            const uint64_t here = lane_value(upto, 63);
            left = here < left ? left - here : 0;
        }
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) sum += w[i];
        const uint64_t upto = before + wave_scan64(sum);
        const uint64_t hit = __ballot(upto > target);
        if (!hit) {
            before = lane_value(upto, 63);
            continue;
        }
        if (lane == __ffsll(static_cast<unsigned long long>(hit)) - 1) {
            uint64_t at = upto - sum;
            int i = 0;
            uint32_t here = w[0];
#pragma unroll
            for (int e = 1; e < N; ++e)
                if (i == e - 1 && at + here <= target) {
                    at += here;
                    here = w[e];
                    i = e;
                }
            answer(v * N + i - row.shift, static_cast<float>(static_cast<double>(here) / static_cast<double>(total)));
        }
        return;
    }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, hipStream_t stream) {
    const dim3 grid(p.B), block(kThreads);
    if (p.f32) hipLaunchKernelGGL(sample_kernel<true>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(sample_kernel<false>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace w4
