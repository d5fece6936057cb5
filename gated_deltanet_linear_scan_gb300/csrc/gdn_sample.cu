// gdn_sample.cu -- a token for every row of logits, from one given uniform number (sm_103a).
//
// With z_i = x_i / T the row's order is by x, largest first, the lower index first among equals.
// top-k, top-p and min-p each keep a prefix of that order, so what is kept is {x > V} and the
// first `ties` of those equal to V; the token is the first index whose running sum of e^{z_i}, over
// what is kept in index order, exceeds u times the whole sum.
//
// Whether a sum falls short of a border decides the token, so the weights are 64-bit integers in units
// of 2^-43 of the sum: integer sums do not depend on their order, and every pass over a row agrees
// with every other. Weights above 2^-20 of the sum (e^{z} in two floats) are good to a unit, smaller
// ones, of one exponential in fp32, to 2^-20 of themselves. So the edge between two tokens is off by at
// most vocab 2^-43 + 2^-20 s of the sum, s the share of the small ones. Where logits differ most of
// that cancels; it adds up where they repeat: 100,000 equal tokens beside one that is 2^20 times as
// likely are 9 % of the sum, and at 2^-22.2 of a weight and half a unit the edges among them are off by
// up to 3 10^-8, half a step of the uniform number. (With weights of 24 bits throughout, one row in some hundred
// of a vocabulary of 100,000 would come out another token.)
//
// A cluster of 1 to 8 CTAs takes a row, a warp a stretch of it. The first pass finds the largest logit;
// later ones read the row again from L2 (rows in flight fit there). Most tokens of a row are so unlikely
// that one exponential in fp32 gives their weight as well as it has to be; the others wait in a queue of the
// warp's until there are 32 of them. The border of top-k or top-p is found by two histograms of counts or
// weights, read across the cluster: bins of 1/32 in the weight's logarithm from the largest down, as
// far as they can be needed (a bound from the threads' largest logits, or from the sum of all weights), then
// 2048 parts of the bin that holds the border, whose smallest and largest logit are nearly always one
// value. What that leaves open (a part with two values, a border 64 powers of two below the largest) goes
// by the bits of the keys, 11, 11 and 10. What the first histogram takes is listed in shared memory
// where there is room, and the passes behind it read the list.
//
// Arithmetic on the logits bounds it, at 4 to 10 instructions of every lane a logit and pass. 1024 rows
// of 100003 fp32 logits, 0.41 GB (61 us at the copy rate): the largest logit alone 100 us; temperature
// 195, top-k of 50 219, top-p of 0.9 226, min-p 177, all 247 (without the lists 351, 449, 174, 592).
// Flat rows cost more, as many tokens have weights that count: top-p of 0.98 at a temperature of 1.3 1.2
// ms. One row of 128000 bf16 logits by top-p 27 us, nearly all of it barriers and latency.
#include <cstddef>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kPow = 256;            // entries of the table of powers
constexpr int kMaxVocab = 1 << 20;   // weights of 2^43 stay below 2^63 in a sum
constexpr int kAll = 0x7fffffff;
constexpr int kQueue = 32 * 5;       // a warp's room for logits that wait for company
constexpr int kListed = 416;        // of a warp's largest logits, kept in shared memory
constexpr int kSMs = 152;

typedef unsigned long long u64;
typedef unsigned __int128 u128;

// 2^{j / 256} in two floats, from the series of e^x in double (x < 0.7: 24 terms reach 2^-80).
struct PowTable {
    float hi[kPow], lo[kPow];
    constexpr PowTable() : hi(), lo() {
        for (int j = 0; j < kPow; ++j) {
            const double x = j * (0.693147180559945309417232121458 / kPow);
            double sum = 1.0, term = 1.0;
            for (int i = 1; i < 24; ++i) {
                term *= x / i;
                sum += term;
            }
            hi[j] = static_cast<float>(sum);
            lo[j] = static_cast<float>(sum - static_cast<double>(hi[j]));
        }
    }
};
__device__ const PowTable kPowers = PowTable();  // (constant memory would serve one entry at a time)

__device__ __forceinline__ float logit(float x) { return x; }
__device__ __forceinline__ float logit(__half x) { return __half2float(x); }
__device__ __forceinline__ float logit(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of logits, NaN as -infinity.
template <typename T>
struct Vec {
    static constexpr int kSize = 16 / static_cast<int>(sizeof(T));
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[kSize]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = fmaxf(__uint_as_float(w[i]), -INFINITY);
            } else {
                const float2 f = Elem<T>::unpack(w[i]);
                x[2 * i] = fmaxf(f.x, -INFINITY);
                x[2 * i + 1] = fmaxf(f.y, -INFINITY);
            }
        }
    }
};

struct SampleParams {
    const void *logits;
    const float *uniforms, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    int vocab, rows_per_set;
    long long stride;
    int32_t *err_count;
};

// What a warp found in its part of the row: the weights above the threshold, and how many equal it.
struct Part {
    u64 sum;
    int equal, pad;
};

struct __align__(16) Shared {
    float2 powers[kPow];
    unsigned lo[2][kBins], hi[2][kBins];  // histograms, two in turn
    unsigned least[kBins], most[kBins];   // keys of a part's smallest and largest logit (as ~key, key)
    Part parts[kMaxCluster * kWarps], own[kWarps];
    float queue[kWarps][kQueue];
    float list[kWarps][kListed];
    float tops[kMaxCluster];
    unsigned masses[kMaxCluster], warp_mass[kWarps];
    int firsts[kMaxCluster];
    u64 scan[kWarps];
    u64 before;      // what lies before the border's bin
    int bin;         // the bin that holds the border
    float warp_top[kWarps];
    int warp_first[kWarps];
    double log_min;  // T ln(min_p)
};
// (read 16 bytes a time; two CTAs share an SM, which keeps 1 KB of each for itself)
static_assert(offsetof(Shared, lo) % 16 == 0 && offsetof(Shared, hi) % 16 == 0 && offsetof(Shared, least) % 16 == 0 &&
              offsetof(Shared, most) % 16 == 0, "histograms are read 16 bytes a time");
static_assert(sizeof(Shared) <= 228 * 1024 / 2 - 1024, "two CTAs an SM");

// A float's place in the order of floats, as an unsigned number (-0 is +0); and back.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Weights: 2^{43 - shift} e^{(x - top) / T}, where 2^shift is no more than the sum of all over the largest
// (the sum of the largest of all quarters of threads' logits is taken for it): what is below 2^-43 of the sum does
// not count, and the flatter a row, the fewer of its tokens need a precise weight. c_hi + c_lo is
// log2(e) / T; above `likely` the weight is more than 2^-bits of the largest, bits = kLikely - shift;
// k_hi + k_lo is bits - top (c_hi + c_lo).
constexpr int kUnits = 43, kLikely = 20;
constexpr float kExpShort = 7.14e-8f;  // log2 of what the exponential falls short by, over its range (measured: 4.95e-8)
struct Weigher {
    float top, c_hi, c_lo, k_hi, k_lo, likely;
    int shift;
};

// The weight of a likely token: t = (x - top) log2(e) / T in two floats, 2^t from the table and a
// polynomial, to 2^-44.
__device__ __noinline__ u64 precise_weight(const Weigher w, float x) {
    extern __shared__ __align__(16) uint8_t dyn[];
    const float2 *powers = reinterpret_cast<const Shared *>(dyn)->powers;
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves the nearest integer
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.90465429995776e-9f;
    constexpr float kC2 = 0.2402265069591007f, kC3 = 0.05550410866482158f, kC4 = 0.009618129107628477f;
    // d + dl = x - top, exactly
    const float d = __fsub_rn(x, w.top), back = __fsub_rn(d, x);
    const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(w.top, back));
    const float t = __fmul_rn(d, w.c_hi);
    const float tl = __fmaf_rn(d, w.c_lo, __fmaf_rn(dl, w.c_hi, __fmaf_rn(d, w.c_hi, -t)));
    const float y = __fmaf_rn(t, static_cast<float>(kPow), kMagic);
    const int n = __float_as_int(y) - __float_as_int(kMagic);
    const float f = __fmaf_rn(__fsub_rn(y, kMagic), -1.0f / kPow, t);
    const float2 p = powers[n & (kPow - 1)];
    // 2^{f + tl} = 1 + q + b
    const float q = __fmul_rn(f, kLn2), g = __fadd_rn(f, tl);
    float b = __fmaf_rn(tl, kLn2, __fmaf_rn(f, kLn2Lo, __fmaf_rn(f, kLn2, -q)));
    b = __fmaf_rn(__fmul_rn(g, g), __fmaf_rn(g, __fmaf_rn(g, kC4, kC3), kC2), b);
    // (p.x + p.y) (1 + q + b) = s + r
    const float v = __fmul_rn(p.x, q);
    float r = __fadd_rn(__fmaf_rn(p.x, b, __fmaf_rn(p.x, q, -v)), __fmaf_rn(p.y, q, p.y));
    const float s = __fadd_rn(p.x, v);
    r = __fadd_rn(r, __fsub_rn(v, __fsub_rn(s, p.x)));
    // in units of 2^-44: s is a multiple of 2^-24, and r (up to 2^-18) its own 24 bits
    const unsigned big = __float2uint_rz(s * 16777216.0f);
    const int small = __float2int_rn(r * 17592186044416.0f);
    const u64 sum = (static_cast<u64>(big) << 20) + static_cast<long long>(small);
    return x == w.top ? 1ull << (kUnits - w.shift) : sum >> (1 + w.shift - (n >> 8));
}

// The weight of an unlikely one, below 2^23 and so the last bits of 2^23 more than it. Its argument
// is near 0 where the weight counts most, and all but exact there: the error is the exponential's
// (over all floats of its range at most 2^-22.7, measured) and that of kExpShort, which it has not
// everywhere: 2^-22.2 in all. Down to 2^-16 of the largest of these weights the two roundings of the
// argument make it 2^-20.
constexpr unsigned kSmallBase = 0x4B000000u;  // 2^23
__device__ __forceinline__ unsigned small_weight_bits(const Weigher &w, float x) {
    const float t = __fadd_rn(__fmaf_rn(x, w.c_hi, w.k_hi), __fmaf_rn(x, w.c_lo, w.k_lo));
    return __float_as_uint(__fmaf_rn(fast_exp2(t), static_cast<float>(1 << (kUnits - kLikely)), 8388608.0f));
}
__device__ __forceinline__ u64 weight_of(const Weigher &w, float x) {
    return x > w.likely ? precise_weight(w, x) : x > -INFINITY ? small_weight_bits(w, x) - kSmallBase : 0u;
}

__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(FULL_MASK, x, o);
    return x;
}

__device__ __forceinline__ u64 warp_scan64(u64 x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(FULL_MASK, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ int warp_scan(int x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int N>
struct Const {
    static constexpr int value = N;
};

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
}

// The address of this CTA's shared variable in CTA `rank` of the cluster.
template <typename V>
__device__ __forceinline__ V *in_cta(V *local, int rank) {
    u64 out;
    asm("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<u64>(local)), "r"(rank));
    return reinterpret_cast<V *>(out);
}

// floor(f * x) (up: ceil) for f >= 0, without rounding. f * x < 2^64.
__device__ __forceinline__ u64 times(float f, u64 x, bool up) {
    const unsigned bits = __float_as_uint(f);
    const int e = static_cast<int>(bits >> 23);
    const u64 m = e > 0 ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const u128 prod = static_cast<u128>(m) * x;
    const int down = 150 - (e > 0 ? e : 1);  // f = m 2^-down
    if (down >= 127) return up && prod != 0 ? 1 : 0;
    if (down <= 0) return static_cast<u64>(prod << -down);
    const u128 q = prod >> down;
    return static_cast<u64>(q) + (up && (q << down) != prod ? 1 : 0);
}

// Logits from .. to - 1 of a row, by a whole warp: f(x, index of the first), 16 bytes of them a lane
// between the first and the last boundary of 16 and one a lane at the ends (-infinity where there is
// none), kAhead loads ahead of this one's work. (1024 rows of 100003 fp32 logits: the largest alone 100 us with
// four ahead and 108 with two; the weights, whose registers are short, 195 with two, 206 with three, 230 with four.)
template <int kAhead = 2, typename T, typename F>
__device__ __forceinline__ void each_logit(const T *logits, int from, int to, F f) {
    constexpr int kVec = Vec<T>::kSize;
    const int lane = threadIdx.x & 31;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(logits + from) & 15u) / sizeof(T));
    const int s0 = min(to, from + (shift ? kVec - shift : 0)), n = (to - s0) / kVec, s1 = s0 + n * kVec;
    const uint4 *vecs = reinterpret_cast<const uint4 *>(logits + s0);
    const uint4 none = [] {
        const float x = -INFINITY;
        const unsigned w = sizeof(T) == 4 ? __float_as_uint(x) : __is_same(T, __half) ? 0xFC00FC00u : 0xFF80FF80u;
        return make_uint4(w, w, w, w);
    }();
    uint4 next[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) next[y] = lane + 32 * y < n ? vecs[lane + 32 * y] : none;
    auto end = [&](int first, int last) {
        const float x[1] = {first + lane < last ? fmaxf(logit(logits[first + lane]), -INFINITY) : -INFINITY};
        f(x, first + lane);
    };
    if (from < s0) end(from, s0);
#pragma unroll 1
    for (int v = lane; v < n + lane; v += 32 * kAhead) {
        uint4 raw[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            raw[y] = next[y];
            const int at = v + 32 * (kAhead + y);
            next[y] = at < n ? vecs[at] : none;
        }
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            float x[kVec];
            Vec<T>::unpack(raw[y], x);
            f(x, s0 + (v + 32 * y) * kVec);
        }
    }
    if (s1 < to) end(s1, to);
}

template <int N>
__device__ __forceinline__ float top_of(const float (&x)[N]) {
    float top = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
    return top;
}

// Those of a warp's values that are picked, 32 at a time: f(x) for one a lane (all lanes but in
// `finish`), in no particular order.
struct Queue {
    float *at;  // kQueue floats of the warp's own
    int count;
    template <int N, typename P, typename F>
    __device__ __forceinline__ void push(const float (&x)[N], P picked, F f) {
        const unsigned below = (1u << (threadIdx.x & 31)) - 1;
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {  // four values of a lane together
            #pragma unroll
            for (int e = e0; e < e0 + 4 && e < N; ++e) {
                const bool mine = picked(x[e]);
                const unsigned mask = __ballot_sync(FULL_MASK, mine);
                if (mine) at[count + __popc(mask & below)] = x[e];
                count += __popc(mask);
            }
            if (count < 32) continue;
            __syncwarp();
            do {
                count -= 32;
                f(at[count + (threadIdx.x & 31)]);
            } while (count >= 32);
            __syncwarp();
        }
    }
    template <typename F>
    __device__ __forceinline__ void finish(F f) {
        __syncwarp();
        const int lane = threadIdx.x & 31;
        if (lane < count) f(at[lane]);
        __syncwarp();
        count = 0;
    }
};

// The logits of a warp's stretch from some value on, where they have found room; more than kListed: not so.
struct List {
    float *at;
    int count;
    // `n` (of all lanes alike) values, one a lane
    __device__ __forceinline__ void add(float x, int n) {
        const int lane = threadIdx.x & 31;
        if (count + n <= kListed && lane < n) at[count + lane] = x;
        count = min(count + n, kListed + 1);
    }
    __device__ __forceinline__ bool whole() const { return count <= kListed; }
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        const int lane = threadIdx.x & 31;
        for (int i = lane; i < count + lane; i += 32) {
            const float x[1] = {i < count ? at[i] : -INFINITY};
            f(x, 0);
        }
    }
};

// A histogram's bin: 64 bits in two words.
__device__ __forceinline__ void add_weight(unsigned *lo, unsigned *hi, unsigned bin, u64 w) {
    const unsigned l = static_cast<unsigned>(w), old = atomicAdd(&lo[bin], l);
    const unsigned h = static_cast<unsigned>(w >> 32) + (old + l < old ? 1u : 0u);
    if (h != 0) atomicAdd(&hi[bin], h);
}

// Histogram 0 by weight: bins from `split` on have weights below 2^24 only, whose lower 12 bits go to one
// word and the rest to the other, which then needs no carry (2^20 of them fit).
__device__ __forceinline__ unsigned split_bin(const Weigher &w) { return 32u * (kLikely - w.shift); }
__device__ __forceinline__ void add_place(Shared &sh, const Weigher &w, unsigned bin, u64 weight) {
    if (bin < split_bin(w)) {
        add_weight(sh.lo[0], sh.hi[0], bin, weight);
    } else {
        atomicAdd(&sh.lo[0][bin], static_cast<unsigned>(weight) & 0xFFFu);
        atomicAdd(&sh.hi[0][bin], static_cast<unsigned>(weight >> 12));
    }
}

// A logit's bin of 1/32 in the logarithm of its weight, and its place in that (both roundings leave the
// order of logits as it is).
__device__ __forceinline__ float place_of(const Weigher &w, float x) {
    return x == w.top ? 0.0f : fminf((w.top - x) * (w.c_hi * 32.0f), static_cast<float>(kBins));
}

// The weights of logits from .. to - 1, by a whole warp; the likely ones listed, and in histogram 0.
template <typename T>
__device__ __noinline__ u64 whole_part(const T *logits, int from, int to, const Weigher w, float *room, List &list) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &sh = *reinterpret_cast<Shared *>(dyn);
    u64 sum = 0;
    unsigned small = 0, since = 0;
    Queue queue{room, 0};
    List mine{list.at, 0};
    auto weigh = [&](float x) {
        const u64 weight = precise_weight(w, x);
        sum += weight;
        add_place(sh, w, static_cast<unsigned>(place_of(w, x)), weight);
    };
    auto add = [&](float x) {
        weigh(x);
        mine.add(x, 32);
    };
    each_logit(logits, from, to, [&](const auto &x, int) {
        constexpr int N = static_cast<int>(sizeof(x) / sizeof(x[0]));
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const unsigned bits = small_weight_bits(w, x[e]) - kSmallBase;
            small += x[e] > -INFINITY && !(x[e] > w.likely) ? bits : 0u;
        }
        since += N;
        if (since >= 256) {
            sum += small;
            small = since = 0;
        }
        if (!__any_sync(FULL_MASK, top_of(x) > w.likely)) return;
        queue.push(x, [&](float y) { return y > w.likely; }, add);
    });
    sum += small;
    __syncwarp();
    const int left = queue.count;
    const float last = (threadIdx.x & 31) < left ? room[threadIdx.x & 31] : 0.0f;
    queue.finish(weigh);
    mine.add(last, left);
    __syncwarp();
    list.count = mine.count;
    return warp_sum64(sum);
}

// Of logits from .. to - 1, by a whole warp: the weights above the cut, and how many equal it.
__device__ __noinline__ Part part_of_list(const List list, float cut, const Weigher w) {
    Part mine{0, 0, 0};
    list.each([&](const auto &x, int) {
        if (x[0] > cut) mine.sum += weight_of(w, x[0]);
        mine.equal += x[0] == cut;
    });
    __syncwarp();
    mine.sum = warp_sum64(mine.sum);
    mine.equal = __reduce_add_sync(FULL_MASK, mine.equal);
    return mine;
}

template <typename T>
__device__ __noinline__ Part part_of(const T *logits, int from, int to, float cut, const Weigher w, float *room) {
    Part mine{0, 0, 0};
    Queue queue{room, 0};
    auto add = [&](float x) { mine.sum += precise_weight(w, x); };
    if (cut >= w.likely) {
        // few are as large
        each_logit(logits, from, to, [&](const auto &x, int) {
            if (!__any_sync(FULL_MASK, top_of(x) >= cut)) return;
#pragma unroll
            for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(x[0])); ++e) mine.equal += x[e] == cut;
            queue.push(x, [&](float y) { return y > cut; }, add);
        });
    } else {
        // (small weights are below 2^23: 2^9 of them add up to less than 2^32)
        unsigned small = 0, since = 0;
        each_logit(logits, from, to, [&](const auto &x, int) {
            constexpr int N = static_cast<int>(sizeof(x) / sizeof(x[0]));
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const unsigned bits = small_weight_bits(w, x[e]) - kSmallBase;
                small += x[e] > cut && !(x[e] > w.likely) ? bits : 0u;
                mine.equal += x[e] == cut;
            }
            since += N;
            if (since >= 256) {
                mine.sum += small;
                small = since = 0;
            }
            if (!__any_sync(FULL_MASK, top_of(x) > w.likely)) return;
            queue.push(x, [&](float y) { return y > w.likely; }, add);
        });
        mine.sum += small;
    }
    queue.finish(add);
    mine.sum = warp_sum64(mine.sum);
    mine.equal = __reduce_add_sync(FULL_MASK, mine.equal);
    return mine;
}

// The bin in which the running sum over the cluster's histograms (low words and, unless NULL, high
// ones) reaches `target`, from bin 0 up or from the last down; what lies before it goes to sh.before;
// -1 if none does. Bins from `limit` up are not needed; those from `split` up have 12 bits in their
// low word. By the whole CTA. Clears histogram `clears` (and with the second the parts' keys), which
// everybody has read before the barrier ahead of this call.
__device__ __noinline__ int find_bin(unsigned *low, unsigned *high, int clears, u64 target, bool down, int cluster,
                                     int limit = kBins, int split = kBins) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &sh = *reinterpret_cast<Shared *>(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int at = down ? kBins - 4 - 4 * tid : 4 * tid;
    u64 own[4] = {0, 0, 0, 0};
    for (int word = 0; word < (high ? 2 : 1); ++word) {
        unsigned *const hist = word ? high : low;
        const int up = word == 0 ? 0 : at < split ? 32 : 12;
        for (int r0 = 0; r0 < cluster; r0 += 4) {  // four CTAs' at a time
            uint4 x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[y] = r0 + y < cluster && at < limit ? *reinterpret_cast<const uint4 *>(in_cta(hist, r0 + y) + at) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                own[0] += static_cast<u64>(x[y].x) << up;
                own[1] += static_cast<u64>(x[y].y) << up;
                own[2] += static_cast<u64>(x[y].z) << up;
                own[3] += static_cast<u64>(x[y].w) << up;
            }
        }
    }
    const u64 sum = own[0] + own[1] + own[2] + own[3];
    u64 before = warp_scan64(sum);
    if (lane == 31) sh.scan[warp] = before;
    if (tid == 0) sh.bin = -1;
    before -= sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += sh.scan[w];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const u64 mine = down ? own[3 - y] : own[y];
        if (before < target && target <= before + mine) {
            sh.bin = down ? at + 3 - y : at + y;
            sh.before = before;
        }
        before += mine;
    }
    for (int x = tid; x < kBins; x += kThreads) {
        sh.lo[clears][x] = sh.hi[clears][x] = 0;
        if (clears == 1) sh.least[x] = sh.most[x] = 0;
    }
    __syncthreads();
    return sh.bin;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cluster) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &sh = *reinterpret_cast<Shared *>(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % cluster;
    const long long row = blockIdx.x / cluster;
    const int set = static_cast<int>(row / p.rows_per_set);

    // ---- the row's settings
    const float temperature = p.temperature ? p.temperature[set] : 1.0f;
    const float top_p = p.top_p ? p.top_p[set] : 1.0f;
    const float min_p = p.min_p ? p.min_p[set] : 0.0f;
    const int top_k = p.top_k ? p.top_k[set] : 0;
    float u = p.uniforms[row];
    u = u < 1.0f ? (u > 0.0f ? u : 0.0f) : u >= 1.0f ? 0.99999994f : 0.0f;
    // (from 2^100 on, logits further apart than the largest float could still both have weights)
    const bool valid = temperature >= 0.0f && temperature < 0x1p100f && top_p == top_p && min_p == min_p;
    if (!valid) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.err_count) atomicAdd(p.err_count, 1);
        }
        return;  // the whole cluster
    }
    if (cluster > 1) {  // (waited for ahead of the first store to another CTA, behind the first pass over the row)
        __syncwarp();
        cluster_arrive_release();
    }
    const bool greedy = temperature == 0.0f || min_p > 1.0f || top_k == 1;
    const bool by_count = top_k > 0 && top_k < p.vocab;

    // ---- this CTA's slice of the row, and this warp's stretch of that
    const T *logits = static_cast<const T *>(p.logits) + row * p.stride;
    const int per_cta = (p.vocab + cluster - 1) / cluster;
    const int per_warp = (per_cta + kThreads - 1) / kThreads * 32;
    const int cta1 = min(p.vocab, (rank + 1) * per_cta);
    const int e0 = min(cta1, rank * per_cta + warp * per_warp), e1 = min(cta1, e0 + per_warp);
    auto sync = [&] {
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    if (!greedy) {
        for (int x = tid; x < kPow; x += kThreads) sh.powers[x] = make_float2(kPowers.hi[x], kPowers.lo[x]);
        if (by_count || top_p < 1.0f)
            for (int x = tid; x < kBins; x += kThreads)
                sh.lo[0][x] = sh.hi[0][x] = sh.lo[1][x] = sh.hi[1][x] = sh.least[x] = sh.most[x] = 0;
    }

    // ---- the largest logit
    float own_tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // of four parts of the thread's logits
    each_logit<4>(logits, e0, e1, [&](const auto &x, int) {
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(x[0])); ++e) own_tops[e & 3] = fmaxf(own_tops[e & 3], x[e]);
    });
    float top = top_of(own_tops);
    __syncwarp();
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
    if (lane == 0) sh.warp_top[warp] = top;
    const float warp_top = top;
    if (tid == kThreads - 1 && min_p > 0.0f && min_p <= 1.0f)  // (64-bit arithmetic is slow: one thread's business)
        sh.log_min = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
    // log2(e) / T: the quotient, and the remainder's
    constexpr float kLog2EHi = 1.44269502162933349609f, kLog2ELo = 1.92596298909e-8f;
    const float c = kLog2EHi / temperature, c_hi = fminf(c, 3.0e38f);
    unsigned mass = 0;  // of the threads' largest logits, the largest 2^16
    auto mass_of = [&](float x, float units) { return __float2uint_rn(units * fast_exp2(x == top ? 0.0f : (x - top) * c_hi)); };
    if (!greedy) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mass += own_tops[e] == -INFINITY ? 0u : mass_of(own_tops[e], 65536.0f);
        __syncwarp();
        mass = __reduce_add_sync(FULL_MASK, mass);
        if (lane == 0) sh.warp_mass[warp] = mass;
        __syncthreads();
        mass = 0;
        for (int w = 0; w < kWarps; ++w) mass += sh.warp_mass[w];
    }
    if (cluster > 1) {
        __syncwarp();
        cluster_wait_acquire();  // every CTA of the cluster runs: until then it has no shared memory to write to
        if (tid < cluster) {
            *in_cta(&sh.tops[rank], tid) = top;
            *in_cta(&sh.masses[rank], tid) = mass;
        }
        cluster_sync();
        for (int r = 0; r < cluster; ++r) top = fmaxf(top, sh.tops[r]);
        mass = 0;
        for (int r = 0; r < cluster && !greedy; ++r)
            if (sh.tops[r] > -INFINITY) mass += mass_of(sh.tops[r], static_cast<float>(sh.masses[r]));
    }
    if (greedy || top == -INFINITY) {
        // the first index that has it: of the warps that have seen it
        int first = kAll;
        if (top > -INFINITY && warp_top == top)
            each_logit(logits, e0, e1, [&](const auto &x, int i) {
                if (top_of(x) != top) return;
#pragma unroll
                for (int e = static_cast<int>(sizeof(x) / sizeof(x[0])) - 1; e >= 0; --e)
                    if (x[e] == top) first = min(first, i + e);
            });
        __syncwarp();
        first = __reduce_min_sync(FULL_MASK, first);
        if (lane == 0) sh.warp_first[warp] = first;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) first = min(first, sh.warp_first[w]);
        if (cluster > 1) {
            if (tid == 0) *in_cta(&sh.firsts[rank], 0) = first;
            cluster_sync();
            if (rank == 0)
                for (int r = 0; r < cluster; ++r) first = min(first, sh.firsts[r]);
        }
        if (rank == 0 && tid == 0) p.tokens[row] = first == kAll ? -1 : first;
        return;
    }

    Weigher weigher;
    weigher.top = top;
    {
        weigher.shift = 31 - __clz(max(mass, 65536u) >> 16);
        const float bits = static_cast<float>(kLikely - weigher.shift);
        weigher.c_hi = c_hi;
        weigher.c_lo = c < 3.0e38f ? __fadd_rn(__fmaf_rn(-c, temperature, kLog2EHi), kLog2ELo) / temperature : 0.0f;
        // below the top itself, which is likely even where the difference rounds away
        weigher.likely = fminf(top - bits / weigher.c_hi, value_of(key_of(top) - (top == 0.0f ? 2 : 1)));
        // bits - top c, the product in two floats
        const float prod = __fmul_rn(top, weigher.c_hi), rest = __fmaf_rn(top, weigher.c_lo, __fmaf_rn(top, weigher.c_hi, -prod));
        const float k = __fsub_rn(bits, prod), back = __fsub_rn(k, bits);
        const float err = __fsub_rn(__fsub_rn(bits, __fsub_rn(k, back)), __fadd_rn(prod, back));
        weigher.k_hi = k;
        weigher.k_lo = __fadd_rn(__fsub_rn(err, rest), kExpShort);
        // An infinite top, or a product past the range: the floats next to such a top are 2^104 of z below
        // it (infinitely far, of an infinite one), so every smaller logit has a weight of 0. The
        // arguments are -infinity then, and none of their parts is NaN.
        if (!(fabsf(prod) < INFINITY)) {
            weigher.c_lo = weigher.k_lo = 0.0f;
            weigher.k_hi = -INFINITY;
        }
    }
    auto weight = [&](float x) { return weight_of(weigher, x); };
    Queue queue{sh.queue[warp], 0};
    List list{sh.list[warp], kListed + 1};

    // ---- what is kept: x > cut, and the first `ties` of those equal to it
    float cut = -INFINITY;
    int ties = 0;

    auto gather_parts = [&] {
        const Part mine = list.whole() ? part_of_list(list, cut, weigher) : part_of(logits, e0, e1, cut, weigher, queue.at);
        if (lane < cluster) *in_cta(&sh.parts[rank * kWarps + warp], lane) = mine;
        sync();
    };
    auto total_of = [&](u64 w_cut) {
        u64 sum = 0;
        int equal = 0;
        for (int x = lane; x < cluster * kWarps; x += 32) {
            sum += sh.parts[x].sum;
            equal += sh.parts[x].equal;
        }
        __syncwarp();
        sum = warp_sum64(sum);
        equal = __reduce_add_sync(FULL_MASK, equal);
        return sum + static_cast<u64>(min(equal, ties)) * w_cut;
    };

    // the logits that are still in question, or more
    auto each_left = [&](auto f) {
        if (list.whole()) list.each(f);
        else each_logit(logits, e0, e1, f);
    };
    auto add = [&](int turn, unsigned bin, u64 w) { add_weight(sh.lo[turn], sh.hi[turn], bin, w); };

    // ---- histograms
    // The cut at which `target` (a count, or a sum of weights) is reached from the top, among what is
    // kept so far: the new cut and its ties. (A count that is not reached: all are kept.) No weight
    // before `least_t` (its logarithm) is needed to reach it. counted: histogram 0 has the likely ones already.
    auto descend = [&](bool by_weight, u64 target, float least_t, bool counted) {
        const float old_cut = cut;
        // those equal to the cut so far, of which only `ties` are kept: one thread adds them
        const bool old = by_weight && ties > 0 && rank == 0 && tid == 0;
        const u64 w_old = old ? weight(old_cut) * static_cast<u64>(ties) : 0;
        auto place = [&](float x) { return place_of(weigher, x); };
        auto settle = [&](u64 rest) {
            if (by_weight) {
                const u64 w = weight(cut);
                ties = static_cast<int>((rest + w - 1) / w);
            } else {
                ties = static_cast<int>(rest);
            }
        };
        // what lies below this bin is not needed
        float end = fminf(ceilf(-least_t * 32.0f), static_cast<float>(kBins));
        if (!by_weight && target <= static_cast<u64>(4 * cluster * kThreads)) {
            // the largest of the threads' four parts, a logit each, reach it in a bin: all bins up to
            // that one hold enough
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = place(own_tops[e]);
                if (f < static_cast<float>(kBins)) atomicAdd(&sh.least[static_cast<unsigned>(f)], 1u);
            }
            sync();
            const int bin = find_bin(sh.least, nullptr, 0, target, false, cluster);
            if (bin >= 0) end = static_cast<float>(bin + 1);
        }
        if (counted && end > static_cast<float>(split_bin(weigher) - 1)) {
            // some that count are not likely
            list.count = kListed + 1;
            each_logit(logits, e0, e1, [&](const auto &x, int) {
#pragma unroll
                for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(x[0])); ++e) {
                    const float f = place(x[e]);
                    if (!(x[e] > weigher.likely) && f < end)
                        add_place(sh, weigher, static_cast<unsigned>(f), small_weight_bits(weigher, x[e]) - kSmallBase);
                }
            });
        }
        if (!counted) {
            auto note = [&](float x) {
                const unsigned bin = static_cast<unsigned>(place(x));
                if (by_weight) add_place(sh, weigher, bin, weight(x));
                else atomicAdd(&sh.lo[0][bin], 1u);
            };
            const bool lists = !list.whole() && old_cut == -INFINITY;  // (not without those that equal the cut)
            List kept{list.at, lists ? 0 : kListed + 1};
            auto note_all = [&](float x) {
                note(x);
                kept.add(x, 32);
            };
            each_left([&](const auto &x, int) {
                const float largest = top_of(x);
                if (!__any_sync(FULL_MASK, largest > old_cut && place(largest) < end)) return;
                queue.push(x, [&](float y) { return y > old_cut && place(y) < end; }, note_all);
            });
            __syncwarp();
            const int left = queue.count;
            const float last = lane < left ? queue.at[lane] : 0.0f;
            queue.finish(note);
            kept.add(last, left);
            __syncwarp();
            if (lists) list.count = kept.count;
        }
        if (old && place(old_cut) < end) add_place(sh, weigher, static_cast<unsigned>(place(old_cut)), w_old);
        sync();
        const int at = find_bin(sh.lo[0], by_weight ? sh.hi[0] : nullptr, 1, target, false, cluster, static_cast<int>(end),
                                static_cast<int>(split_bin(weigher)));
        if (at >= 0) {
            const u64 rest = target - sh.before;
            const float bin = static_cast<float>(at);
            auto note_part = [&](float x, u64 w) {
                const unsigned part = static_cast<unsigned>((place(x) - bin) * kBins), key = key_of(x);  // (exact)
                if (by_weight) add(1, part, w);
                else atomicAdd(&sh.lo[1][part], 1u);
                atomicMax(&sh.least[part], ~key);
                atomicMax(&sh.most[part], key);
            };
            auto inside = [&](float x) {
                const float f = place(x);
                return f >= bin && f < bin + 1.0f;
            };
            auto note_it = [&](float x) { note_part(x, by_weight ? weight(x) : 0ull); };
            each_left([&](const auto &x, int) {
                const float largest = top_of(x);
                if (!__any_sync(FULL_MASK, largest > old_cut && place(largest) < bin + 1.0f)) return;
                queue.push(x, [&](float y) { return y > old_cut && inside(y); }, note_it);
            });
            queue.finish(note_it);
            if (old && inside(old_cut)) note_part(old_cut, w_old);
            sync();
            const int part = max(0, find_bin(sh.lo[1], by_weight ? sh.hi[1] : nullptr, 0, rest, false, cluster));  // (one holds the border)
            unsigned least = 0, most = 0;
            for (int r = 0; r < cluster; ++r) {
                least = max(least, *(in_cta(sh.least, r) + part));
                most = max(most, *(in_cta(sh.most, r) + part));
            }
            const u64 left = rest - sh.before;
            if (~least == most) {
                cut = value_of(most);
                settle(left);
                return;
            }
        }
        // by the keys' bits (the border may lie below what is listed)
        list.count = kListed + 1;
        auto clear = [&] {
            sync();
            for (int x = tid; x < kBins; x += kThreads) sh.lo[0][x] = sh.hi[0][x] = 0;
            __syncthreads();
        };
        clear();
        unsigned prefix = 0;
        bool found = true;
#pragma unroll 1
        for (int pass = 0; pass < 3 && found; ++pass) {
            const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, turn = pass & 1;
            auto inside = [&](unsigned key) { return pass == 0 || (key >> (down + bits)) == prefix; };
            auto bin_of = [&](unsigned key) { return (key >> down) & ((1u << bits) - 1); };
            auto note_key = [&](float x) {
                if (by_weight) add(turn, bin_of(key_of(x)), weight(x));
                else atomicAdd(&sh.lo[turn][bin_of(key_of(x))], 1u);
            };
            each_logit(logits, e0, e1, [&](const auto &x, int) {
                queue.push(x, [&](float y) { return y > old_cut && inside(key_of(y)); }, note_key);
            });
            queue.finish(note_key);
            if (old && inside(key_of(old_cut))) add(turn, bin_of(key_of(old_cut)), w_old);
            sync();
            const int bin = find_bin(sh.lo[turn], by_weight ? sh.hi[turn] : nullptr, turn ^ 1, target, true, cluster);
            found = bin >= 0;
            if (found) {
                target -= sh.before;
                prefix = prefix << bits | static_cast<unsigned>(bin);
            }
        }
        if (found) {
            cut = value_of(prefix);
            settle(target);
        }
        clear();
    };

#pragma unroll 1
    for (int step = by_count ? 0 : 1; step < (top_p < 1.0f ? 2 : 1); ++step) {
        u64 target = top_k;
        float least_t = -INFINITY;
        if (step == 1) {
            if (by_count) {
                gather_parts();
            } else {
                const Part mine{whole_part(logits, e0, e1, weigher, queue.at, list), 0, 0};
                if (lane < cluster) *in_cta(&sh.parts[rank * kWarps + warp], lane) = mine;
                sync();
            }
            const u64 total = total_of(ties > 0 ? weight(cut) : 0);
            const u64 want = top_p > 0.0f ? times(top_p, total, true) : 0;
            // Where a weight times the vocabulary falls short of what may be left out, the border is behind
            // (0.02: half a bin, and fp32's errors).
            least_t = log2f(static_cast<float>(total - want) * 0x1p-43f / static_cast<float>(p.vocab)) +
                      static_cast<float>(weigher.shift) - 0.02f;
            target = want > 0 ? want : 1;
        }
        descend(step == 1, target, least_t, step == 1 && !by_count);  // (its barriers come before the parts are written again)
    }
    if (min_p > 0.0f) {
        // w >= min_p: x >= top + T ln(min_p)
        const float least = __double2float_ru(static_cast<double>(top) + sh.log_min);
        if (least > cut) {
            cut = least;
            ties = kAll;
        }
    }

    // ---- the token: the stretch in which the running sum exceeds the target, then 1 / 16 of it, then
    // 32 logits at a time
    gather_parts();
    const u64 w_cut = ties > 0 ? weight(cut) : 0;
    const u64 target = times(u, total_of(w_cut), false);
    u64 run = 0;   // weights above the cut before the stretch
    int seen = 0;  // logits equal to it
    auto upto = [&](u64 sum, int equal) { return sum + static_cast<u64>(min(equal, ties)) * w_cut; };
    // which lane's running sum exceeds the target (-1: none); run and seen move on to it, or past all
    auto advance = [&](u64 sum, int equal) {
        const u64 sums = warp_scan64(sum);
        const int equals = warp_scan(equal);
        const unsigned past = __ballot_sync(FULL_MASK, upto(run + sums, seen + equals) > target);
        const int at = past != 0 ? __ffs(past) - 1 : 31;
        run += __shfl_sync(FULL_MASK, past != 0 ? sums - sum : sums, at);
        seen += __shfl_sync(FULL_MASK, past != 0 ? equals - equal : equals, at);
        return past != 0 ? at : -1;
    };
    // which of `count` parts it is (by a whole warp): a few consecutive ones a lane, then one by one
    auto pick = [&](const Part *parts, int count) {
        const int each_lane = (count + 31) / 32, first = lane * each_lane;
        u64 sum = 0;
        int equal = 0;
        for (int x = first; x < min(count, first + each_lane); ++x) {
            sum += parts[x].sum;
            equal += parts[x].equal;
        }
        __syncwarp();
        int x = max(advance(sum, equal), 0) * each_lane;
        for (; x + 1 < count && upto(run + parts[x].sum, seen + parts[x].equal) <= target; ++x) {
            run += parts[x].sum;
            seen += parts[x].equal;
        }
        return x;
    };
    const int stretch = pick(sh.parts, cluster * kWarps);
    if (stretch / kWarps == rank) {
        const int begin = min(cta1, rank * per_cta + stretch % kWarps * per_warp), end = min(cta1, begin + per_warp);
        const int each_warp = (end - begin + kThreads - 1) / kThreads * 32;
        const int a = min(end, begin + warp * each_warp);
        const Part mine = part_of(logits, a, min(end, a + each_warp), cut, weigher, queue.at);
        if (lane == 0) sh.own[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const int from = begin + pick(sh.own, kWarps) * each_warp, to = min(end, from + each_warp);
            for (int i = from + lane; i < to + lane; i += 32) {
                const float x = i < to ? fmaxf(logit(logits[i]), -INFINITY) : -INFINITY;
                const u64 w = x > cut ? weight(x) : 0;
                __syncwarp();
                const int at = advance(w, x == cut);
                if (at < 0) continue;
                if (lane == at) p.tokens[row] = i;
                break;
            }
        }
    }
    if (cluster > 1) cluster_sync();  // no CTA leaves while another may read or write its shared memory
}

// CTAs of a row: as many as give every SM its two, of at least 2048 logits each; eight, whose barriers
// and histograms take as long as their passes, only where most of the GPU is idle anyway. (128000
// bf16 logits by top-p: one row 32 us by eight and 34 by four, 16 rows 42 and 37, 64 rows 51 by four and
// 88 by one; 1024 rows of 100003 in fp32 250 by one, 295 by two, 462 by four.)
template <typename T>
gdn_status launch(const SampleParams &p, int rows, cudaStream_t s) {
    int cluster = rows <= 8 ? kMaxCluster : 4;
    while (cluster > 1 && (static_cast<long long>(rows) * cluster > 2 * kSMs || p.vocab / cluster < 2048)) cluster /= 2;
    if (static_cast<long long>(rows) * cluster > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    auto kernel = sample_kernel<T>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, static_cast<int>(sizeof(Shared)), allowed));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, cluster) == cudaSuccess ? launch_status() : GDN_ERR_LAUNCH;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_sample(const void *logits, const float *uniforms,
                                 const float *temperature, const int32_t *top_k,
                                 const float *top_p, const float *min_p, int32_t *tokens, int rows,
                                 int vocab, int row_stride, int dtype, int rows_per_set,
                                 int32_t *err_count, gdn_stream_t stream) {
    if (!logits || !uniforms || !tokens) return GDN_ERR_NULL;
    if (rows < 0 || vocab < 1 || rows_per_set < 1 || row_stride < vocab) return GDN_ERR_SHAPE;
    if (!supported_dtype(dtype) || vocab > kMaxVocab) return GDN_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) != 0) return GDN_ERR_ALIGN;
    if (rows == 0) return GDN_OK;
    const SampleParams p{logits, uniforms, temperature, top_p, min_p, top_k, tokens, vocab,
                         rows_per_set, row_stride, err_count};
    const cudaStream_t s = as_cuda(stream);
    switch (dtype) {
        case GDN_F32: return launch<float>(p, rows, s);
        case GDN_F16: return launch<__half>(p, rows, s);
        default: return launch<__nv_bfloat16>(p, rows, s);
    }
}
