// gdn_sample.cu -- a token for every row of logits, from one given uniform number (sm_103a).
//
// With z_i = x_i / T the row's order is by x, largest first, the lower index first among equals.
// top-k, top-p and min-p each keep a prefix of that order, so what is kept is {x > V} and the
// first `ties` of those equal to V; the token is the first index whose running sum of e^{z_i}, over
// what is kept in index order, exceeds u times the whole sum.
//
// Whether a sum falls short of a border decides the token, so the weights are held to 2^-43 of the
// largest (e^{z} in two floats, then 64-bit integers): integer sums do not depend on their order,
// every pass over a row agrees with every other, and a wrong side of a border is as likely as a
// uniform number within 10^-11 of it. (With weights of 24 bits, one row in some hundred of a
// vocabulary of 100,000 would come out another token.)
//
// A cluster of 1 to 8 CTAs takes a row; each keeps its slice of the logits in shared memory as it
// was loaded, so a row is read from HBM once, and every pass after the first runs from there. A
// threshold is found by its key's bits, 11, 11 and 10 of them at a time: a histogram of counts
// (top-k) or weights (top-p) per CTA, read across the cluster.
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
__constant__ PowTable kPowers = PowTable();

template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float none() { return -INFINITY; }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};
template <typename T>
struct Logit16 {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<T>::unpack(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 none() { return __ushort_as_bfloat16(0xFF80u); }
};
template <>
struct Logit<__half> : Logit16<__half> {
    static __device__ __forceinline__ __half none() { return __ushort_as_half(0xFC00u); }
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
    Part parts[kMaxCluster * kWarps];
    float tops[kMaxCluster];
    u64 scan[kWarps];
    u64 above;       // what lies above the threshold's bin
    int bin;         // the bin that holds the threshold
    float warp_top[kWarps];
    double log_min;  // T ln(min_p)
};
static_assert(sizeof(Shared) % 16 == 0, "the logits behind it are read 16 bytes at a time");

// A float's place in the order of floats, as an unsigned number (-0 is +0); and back.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// 2^43 e^{(x - top) / T}, rounded down: t = (x - top) log2(e) / T in two floats, 2^t from the table
// and a polynomial. c_hi + c_lo is log2(e) / T.
struct Weigher {
    float top, c_hi, c_lo;
    const float2 *powers;

    __device__ __forceinline__ u64 operator()(float x) const {
        constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves the nearest integer
        constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.90465429995776e-9f;
        constexpr float kC2 = 0.2402265069591007f, kC3 = 0.05550410866482158f, kC4 = 0.009618129107628477f;
        // d + dl = x - top, exactly
        const float d = __fsub_rn(x, top), back = __fsub_rn(d, x);
        const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(top, back));
        const float t = __fmul_rn(d, c_hi);
        const float tl = __fmaf_rn(d, c_lo, __fmaf_rn(dl, c_hi, __fmaf_rn(d, c_hi, -t)));
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
        const u64 w = (static_cast<u64>(big) << 20) + static_cast<long long>(small);
        const int down = 1 - (n >> 8);
        return x == top ? 1ull << 43 : t > -44.0f && down < 64 ? w >> down : 0ull;
    }
};

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

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, int cluster) {
    constexpr int kVec = Logit<T>::kVec;
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &sh = *reinterpret_cast<Shared *>(dyn);
    uint4 *data = reinterpret_cast<uint4 *>(dyn + sizeof(Shared));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % cluster;
    const long long row = blockIdx.x / cluster;
    const int set = static_cast<int>(row / p.rows_per_set);

    // ---- the row's settings
    const float temperature = p.temperature ? p.temperature[set] : 1.0f;
    const float top_p = p.top_p ? p.top_p[set] : 1.0f;
    const float min_p = p.min_p ? p.min_p[set] : 0.0f;
    const int top_k = p.top_k ? p.top_k[set] : 0;
    float u = p.uniforms ? p.uniforms[row] : 0.0f;
    u = u < 1.0f ? (u > 0.0f ? u : 0.0f) : u >= 1.0f ? 0.99999994f : 0.0f;
    const bool valid = temperature >= 0.0f && temperature < INFINITY && top_p == top_p && min_p == min_p;
    if (!valid) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.err_count) atomicAdd(p.err_count, 1);
        }
        return;  // the whole cluster
    }

    // ---- this CTA's slice, in 16-byte parts of the row's own alignment
    const T *logits = static_cast<const T *>(p.logits) + row * p.stride;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15u) / sizeof(T));
    const uint4 *vecs = reinterpret_cast<const uint4 *>(logits - shift);
    const int n_vecs = (shift + p.vocab + kVec - 1) / kVec;
    const int per_cta = (n_vecs + cluster - 1) / cluster;
    const int per_warp = (per_cta + kThreads - 1) / kThreads * 32;
    const int cta0 = rank * per_cta, cta1 = min(n_vecs, cta0 + per_cta);
    const int v0 = cta0 + warp * per_warp, v1 = min(cta1, v0 + per_warp);  // this warp's
    for (int x = tid; x < kPow; x += kThreads) sh.powers[x] = make_float2(kPowers.hi[x], kPowers.lo[x]);
    for (int x = tid; x < kBins; x += kThreads) sh.lo[0][x] = sh.hi[0][x] = sh.lo[1][x] = sh.hi[1][x] = 0;
    float top = -INFINITY;
    {
        constexpr int kAhead = 4;
        for (int v = v0 + lane; v < v1; v += 32 * kAhead) {
            uint4 raw[kAhead];
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const int at = v + 32 * y;
                if (at >= v1) continue;
                const int first = at * kVec - shift;
                if (first >= 0 && first + kVec <= p.vocab) {
                    raw[y] = __ldcs(vecs + at);
                } else {  // the row's ends: what is not the row's counts as -infinity
                    T x[kVec];
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        x[e] = first + e >= 0 && first + e < p.vocab ? logits[first + e] : Logit<T>::none();
                    memcpy(&raw[y], x, 16);
                }
            }
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const int at = v + 32 * y;
                if (at >= v1) continue;
                data[at - cta0] = raw[y];
                float x[kVec];
                Logit<T>::unpack(raw[y], x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) top = fmaxf(top, x[e]);  // (passes over NaN)
            }
        }
    }
    // A thread only ever reads what it has stored itself: no barrier for the data.
    // f(x, index): every logit of the lane's, in index order; NaN is -infinity.
    auto each = [&](auto f) {
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[kVec];
            Logit<T>::unpack(data[v - cta0], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) f(fmaxf(x[e], -INFINITY));
        }
    };

    // ---- the largest logit
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
    if (lane == 0) sh.warp_top[warp] = top;
    if (tid == kThreads - 1 && min_p > 0.0f && min_p <= 1.0f)  // (64-bit arithmetic is slow: one thread's business)
        sh.log_min = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    __syncthreads();
    if (warp == 0) {
        top = sh.warp_top[lane % kWarps];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        if (lane < cluster) *in_cta(&sh.tops[rank], lane) = top;
    }
    cluster_sync();
    top = -INFINITY;
    for (int r = 0; r < cluster; ++r) top = fmaxf(top, sh.tops[r]);
    if (top == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) p.tokens[row] = -1;
        cluster_sync();  // (no CTA leaves while another may write to it)
        return;
    }

    Weigher weight;
    weight.top = top;
    weight.powers = sh.powers;
    {
        // log2(e) / T: the quotient, and the remainder's
        constexpr float kLog2EHi = 1.44269502162933349609f, kLog2ELo = 1.925963033500e-8f;
        const float t = temperature > 0.0f ? temperature : 1.0f, c = kLog2EHi / t;
        weight.c_hi = fminf(c, 3.0e38f);
        weight.c_lo = c < 3.0e38f ? __fadd_rn(__fmaf_rn(-c, t, kLog2EHi), kLog2ELo) / t : 0.0f;
    }

    // ---- what is kept: x > cut, and the first `ties` of those equal to it
    float cut = -INFINITY;
    int ties = 0;
    int turn = 0;  // histogram in use

    // Each warp's sum over what is kept, and its count of those equal to the cut, to every CTA.
    auto gather_parts = [&] {
        Part mine{0, 0, 0};
        each([&](float x) {
            if (x > cut) mine.sum += weight(x);
            else if (ties > 0 && x == cut) ++mine.equal;
        });
        mine.sum = warp_sum64(mine.sum);
        mine.equal = __reduce_add_sync(FULL_MASK, mine.equal);
        if (lane < cluster) *in_cta(&sh.parts[rank * kWarps + warp], lane) = mine;
        cluster_sync();
    };
    auto total_of = [&](u64 w_cut) {
        u64 sum = 0;
        int equal = 0;
        for (int x = lane; x < cluster * kWarps; x += 32) {
            sum += sh.parts[x].sum;
            equal += sh.parts[x].equal;
        }
        sum = warp_sum64(sum);
        equal = __reduce_add_sync(FULL_MASK, equal);
        return sum + static_cast<u64>(min(equal, ties)) * w_cut;
    };

    // The cut at which `target` is reached from the top (a count, or a sum of weights), among what
    // is kept so far: the new cut and its ties.
    auto descend = [&](bool by_weight, u64 target) {
        const float old_cut = cut;
        const int old_ties = ties;
        const u64 w_old = by_weight && old_ties > 0 ? weight(old_cut) : 0;
        unsigned prefix = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            unsigned *lo = sh.lo[turn], *hi = sh.hi[turn];
            auto add = [&](unsigned bin, u64 w) {
                const unsigned l = static_cast<unsigned>(w), old = atomicAdd(lo + bin, l);
                const unsigned h = static_cast<unsigned>(w >> 32) + (old + l < old ? 1u : 0u);
                if (h != 0) atomicAdd(hi + bin, h);
            };
            each([&](float x) {
                const unsigned key = key_of(x);
                if (!(x > old_cut) || (pass > 0 && (key >> (down + bits)) != prefix)) return;
                const unsigned bin = (key >> down) & ((1u << bits) - 1);
                if (by_weight) add(bin, weight(x));
                else atomicAdd(lo + bin, 1u);
            });
            if (by_weight && old_ties > 0 && rank == 0 && tid == 0) {
                // those equal to the cut so far, of which only old_ties are kept
                const unsigned key = key_of(old_cut);
                if (pass == 0 || (key >> (down + bits)) == prefix)
                    add((key >> down) & ((1u << bits) - 1), w_old * static_cast<u64>(old_ties));
            }
            cluster_sync();
            // bins from the top: a thread takes four, the highest first
            u64 own[4], sum = 0;
            {
                const int first = kBins - 4 - 4 * tid;
                uint4 l = make_uint4(0, 0, 0, 0), h = l;
                u64 a[4] = {0, 0, 0, 0};
                for (int r = 0; r < cluster; ++r) {
                    l = *reinterpret_cast<const uint4 *>(in_cta(lo, r) + first);
                    h = by_weight ? *reinterpret_cast<const uint4 *>(in_cta(hi, r) + first) : make_uint4(0, 0, 0, 0);
                    a[0] += static_cast<u64>(h.w) << 32 | l.w;
                    a[1] += static_cast<u64>(h.z) << 32 | l.z;
                    a[2] += static_cast<u64>(h.y) << 32 | l.y;
                    a[3] += static_cast<u64>(h.x) << 32 | l.x;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    own[y] = a[y];
                    sum += a[y];
                }
            }
            u64 before = warp_scan64(sum);
            if (lane == 31) sh.scan[warp] = before;
            before -= sum;
            __syncthreads();
            for (int w = 0; w < warp; ++w) before += sh.scan[w];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if (before < target && target <= before + own[y]) {
                    sh.bin = kBins - 1 - (4 * tid + y);
                    sh.above = before;
                }
                before += own[y];
            }
            // the other histogram is the next pass's: everyone has read it before this pass's barrier
            for (int x = tid; x < kBins; x += kThreads) sh.lo[turn ^ 1][x] = sh.hi[turn ^ 1][x] = 0;
            turn ^= 1;
            __syncthreads();
            target -= sh.above;
            prefix = prefix << bits | static_cast<unsigned>(sh.bin);
            __syncthreads();
        }
        cut = value_of(prefix);
        if (by_weight) {
            const u64 w = weight(cut);
            ties = static_cast<int>((target + w - 1) / w);
        } else {
            ties = static_cast<int>(min(target, static_cast<u64>(kAll)));
        }
    };

    if (temperature == 0.0f || min_p > 1.0f || top_k == 1) {
        cut = top;
        ties = 1;
    } else {
        if (top_k > 0 && top_k < p.vocab) {
            // (rows with fewer logits above -infinity keep them all)
            int there = 0;
            each([&](float x) { there += x > -INFINITY; });
            there = __reduce_add_sync(FULL_MASK, there);
            Part mine{static_cast<u64>(there), 0, 0};
            if (lane < cluster) *in_cta(&sh.parts[rank * kWarps + warp], lane) = mine;
            cluster_sync();
            const u64 all = total_of(0);
            cluster_sync();  // the parts have been read
            if (static_cast<u64>(top_k) < all) descend(false, top_k);
        }
        if (top_p < 1.0f) {
            gather_parts();
            const u64 total = total_of(ties > 0 ? weight(cut) : 0);
            cluster_sync();
            const u64 want = top_p > 0.0f ? times(top_p, total, true) : 0;
            descend(true, want > 0 ? want : 1);
        }
        if (min_p > 0.0f) {
            // w >= min_p: x >= top + T ln(min_p)
            const float least = __double2float_ru(static_cast<double>(top) + sh.log_min);
            if (least > cut) {
                cut = least;
                ties = kAll;
            }
        }
    }

    // ---- the token
    gather_parts();
    const u64 w_cut = ties > 0 ? weight(cut) : 0;
    const u64 target = times(u, total_of(w_cut), false);
    // the warp in whose part the running sum exceeds the target: every warp looks at its own
    {
        u64 before = 0;
        int equal = 0;
        for (int x = lane; x < rank * kWarps + warp; x += 32) {
            before += sh.parts[x].sum;
            equal += sh.parts[x].equal;
        }
        before = warp_sum64(before);
        equal = __reduce_add_sync(FULL_MASK, equal);
        const Part mine = sh.parts[rank * kWarps + warp];
        const u64 from = before + static_cast<u64>(min(equal, ties)) * w_cut;
        const u64 to = before + mine.sum + static_cast<u64>(min(equal + mine.equal, ties)) * w_cut;
        if (from <= target && target < to) {
            // 32 parts of 16 bytes at a time, then the lane's, then its logits
            u64 run = before;
            int seen = equal;
            for (int v = v0; v < v1; v += 32) {
                float x[kVec];
                u64 sum = 0;
                int same = 0;
                if (v + lane < v1) {
                    Logit<T>::unpack(data[v + lane - cta0], x);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        if (x[e] > cut) sum += weight(x[e]);
                        else if (ties > 0 && x[e] == cut) ++same;
                    }
                }
                const u64 sums = warp_scan64(sum);
                int sames = same;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(FULL_MASK, sames, o);
                    if (lane >= o) sames += y;
                }
                const u64 here = run + sums + static_cast<u64>(min(seen + sames, ties)) * w_cut;
                const unsigned past = __ballot_sync(FULL_MASK, here > target);
                if (past != 0) {
                    if (lane == __ffs(past) - 1) {
                        u64 s = run + sums - sum;
                        int q = seen + sames - same;
#pragma unroll 1
                        for (int e = 0; e < kVec; ++e) {
                            const float y = static_cast<float>(reinterpret_cast<const T *>(data + (v + lane - cta0))[e]);
                            if (y > cut) s += weight(y);
                            else if (ties > 0 && y == cut) ++q;
                            if (s + static_cast<u64>(min(q, ties)) * w_cut > target) {
                                p.tokens[row] = (v + lane) * kVec + e - shift;
                                break;
                            }
                        }
                    }
                    break;
                }
                run += __shfl_sync(FULL_MASK, sums, 31);
                seen += __shfl_sync(FULL_MASK, sames, 31);
            }
        }
    }
    cluster_sync();  // no CTA leaves while another may read or write its shared memory
}

template <typename T>
gdn_status launch(const SampleParams &p, int rows, cudaStream_t s) {
    constexpr int kVec = Logit<T>::kVec;
    const long long vecs = (static_cast<long long>(p.vocab) + 2 * kVec - 2) / kVec;
    auto bytes_of = [&](int cluster) { return sizeof(Shared) + static_cast<size_t>((vecs + cluster - 1) / cluster) * 16; };
    constexpr size_t kMost = 232448;
    int cluster = rows <= 64 ? 8 : 4;
    while (cluster < kMaxCluster && bytes_of(cluster) > kMost) cluster *= 2;
    while (cluster > 1 && vecs / cluster < 256) cluster /= 2;
    const size_t smem = bytes_of(cluster);
    if (smem > kMost || static_cast<long long>(rows) * cluster > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    auto kernel = sample_kernel<T>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, static_cast<int>(kMost), allowed));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
