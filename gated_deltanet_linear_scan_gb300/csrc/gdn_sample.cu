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
// A cluster of 1 to 8 CTAs takes a row, a warp a stretch of it. The first pass finds the largest logit;
// later ones read the row again from L1 and L2 (rows in flight fit there). The border of top-k or
// top-p is found by two histograms of counts or weights, read across the cluster: bins of 1/32 in the
// weight's logarithm from the largest down, then 2048 parts of the bin that holds the border, whose
// smallest and largest logit are nearly always one value. What that leaves open (a part with two
// values, a border 64 powers of two below the largest) goes by the bits of the keys, 11, 11 and 10.
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
    unsigned least[kBins], most[kBins];   // keys of a part's smallest and largest logit (as ~key, key)
    Part parts[kMaxCluster * kWarps], own[kWarps];
    float tops[kMaxCluster];
    int firsts[kMaxCluster];
    u64 scan[kWarps];
    u64 before;      // what lies before the border's bin
    int bin;         // the bin that holds the border
    float warp_top[kWarps];
    int warp_first[kWarps];
    double log_min;  // T ln(min_p)
};

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

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cluster) {
    constexpr int kVec = Logit<T>::kVec;
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
    const bool valid = temperature >= 0.0f && temperature < INFINITY && top_p == top_p && min_p == min_p;
    if (!valid) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.err_count) atomicAdd(p.err_count, 1);
        }
        return;  // the whole cluster
    }
    const bool greedy = temperature == 0.0f || min_p > 1.0f || top_k == 1;

    // ---- this CTA's slice, in 16-byte parts of the row's own alignment, and this warp's stretch of it
    const T *logits = static_cast<const T *>(p.logits) + row * p.stride;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15u) / sizeof(T));
    const uint4 *vecs = reinterpret_cast<const uint4 *>(logits - shift);
    const int n_vecs = (shift + p.vocab + kVec - 1) / kVec;
    const int per_cta = (n_vecs + cluster - 1) / cluster;
    const int per_warp = (per_cta + kThreads - 1) / kThreads * 32;
    const int cta1 = min(n_vecs, (rank + 1) * per_cta);
    const int v0 = min(cta1, rank * per_cta + warp * per_warp), v1 = min(cta1, v0 + per_warp);
    auto sync = [&] {
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    // 16 bytes of the row; at its ends, -infinity in place of what is not the row's
    auto load = [&](int v) {
        const int first = v * kVec - shift;
        if (first >= 0 && first + kVec <= p.vocab) return vecs[v];
        T x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            x[e] = first + e >= 0 && first + e < p.vocab ? logits[first + e] : Logit<T>::none();
        uint4 raw;
        memcpy(&raw, x, 16);
        return raw;
    };
    // f(logits, index of the first): the lane's logits, 16 bytes at a time, NaN as -infinity; AHEAD
    // of them are loaded together
    auto each = [&](auto ahead, int from, int to, auto f) {
        constexpr int kAhead = decltype(ahead)::value;
#pragma unroll 1
        for (int v = from + lane; v < to; v += 32 * kAhead) {
            uint4 raw[kAhead];
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                if (v + 32 * y < to) raw[y] = load(v + 32 * y);
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                if (v + 32 * y >= to) break;
                float x[kVec];
                Logit<T>::unpack(raw[y], x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[e] = fmaxf(x[e], -INFINITY);
                f(x, (v + 32 * y) * kVec - shift);
            }
        }
    };

    // ---- the largest logit, and (for a row that takes it) the first index that has it
    float top = -INFINITY;
    int first = kAll;
    if (greedy) {
        each(Const<4>(), v0, v1, [&](const float (&x)[kVec], int at) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (x[e] > top) {
                    top = x[e];
                    first = at + e;
                }
        });
    } else {
        for (int x = tid; x < kPow; x += kThreads) sh.powers[x] = make_float2(kPowers.hi[x], kPowers.lo[x]);
        for (int x = tid; x < kBins; x += kThreads)
            sh.lo[0][x] = sh.hi[0][x] = sh.lo[1][x] = sh.hi[1][x] = sh.least[x] = sh.most[x] = 0;
        each(Const<4>(), v0, v1, [&](const float (&x)[kVec], int) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) top = fmaxf(top, x[e]);
        });
    }
    auto larger = [&](float other, int other_first) {
        if (other > top || (other == top && other_first < first)) {
            top = other;
            first = other_first;
        }
    };
    __syncwarp();
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float other = __shfl_xor_sync(FULL_MASK, top, o);
        const int other_first = __shfl_xor_sync(FULL_MASK, first, o);
        larger(other, other_first);
    }
    if (lane == 0) {
        sh.warp_top[warp] = top;
        sh.warp_first[warp] = first;
    }
    if (tid == kThreads - 1 && min_p > 0.0f && min_p <= 1.0f)  // (64-bit arithmetic is slow: one thread's business)
        sh.log_min = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) larger(sh.warp_top[w], sh.warp_first[w]);
    if (cluster > 1) {
        if (tid < cluster) {
            *in_cta(&sh.tops[rank], tid) = top;
            *in_cta(&sh.firsts[rank], tid) = first;
        }
        cluster_sync();
        for (int r = 0; r < cluster; ++r) larger(sh.tops[r], sh.firsts[r]);
    }
    if (greedy || top == -INFINITY) {
        if (rank == 0 && tid == 0) p.tokens[row] = top == -INFINITY ? -1 : first;
        if (cluster > 1) cluster_sync();  // (no CTA leaves while another may write to it)
        return;
    }

    Weigher weight;
    weight.top = top;
    weight.powers = sh.powers;
    {
        // log2(e) / T: the quotient, and the remainder's
        constexpr float kLog2EHi = 1.44269502162933349609f, kLog2ELo = 1.92596298909e-8f;
        const float c = kLog2EHi / temperature;
        weight.c_hi = fminf(c, 3.0e38f);
        weight.c_lo = c < 3.0e38f ? __fadd_rn(__fmaf_rn(-c, temperature, kLog2EHi), kLog2ELo) / temperature : 0.0f;
    }

    // ---- what is kept: x > cut, and the first `ties` of those equal to it
    float cut = -INFINITY;
    int ties = 0;

    // Of vectors from .. to - 1, by a whole warp: the weights above the cut, and how many equal it.
    auto part_of = [&](int from, int to) {
        Part mine{0, 0, 0};
        each(Const<2>(), from, to, [&](const float (&x)[kVec], int) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                any |= x[e] > cut;
                mine.equal += x[e] == cut;
            }
            if (!any) return;
#pragma unroll
            for (int e = 0; e < kVec; ++e) mine.sum += x[e] > cut ? weight(x[e]) : 0ull;
        });
        __syncwarp();
        mine.sum = warp_sum64(mine.sum);
        mine.equal = __reduce_add_sync(FULL_MASK, mine.equal);
        return mine;
    };
    auto gather_parts = [&] {
        const Part mine = part_of(v0, v1);
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

    // ---- histograms
    auto add = [&](int turn, unsigned bin, u64 w) {
        const unsigned l = static_cast<unsigned>(w), old = atomicAdd(&sh.lo[turn][bin], l);
        const unsigned h = static_cast<unsigned>(w >> 32) + (old + l < old ? 1u : 0u);
        if (h != 0) atomicAdd(&sh.hi[turn][bin], h);
    };
    // The bin in which the running sum over the cluster's histograms reaches `target` (from bin 0 up,
    // or from the last down), and what lies before it; false if none does. Clears the other
    // histogram, which everybody has read before the barrier ahead of this call.
    auto find = [&](int turn, bool by_weight, u64 target, bool down) {
        const int at = down ? kBins - 4 - 4 * tid : 4 * tid;
        u64 own[4] = {0, 0, 0, 0};
        for (int r = 0; r < cluster; ++r) {
            const uint4 l = *reinterpret_cast<const uint4 *>(in_cta(sh.lo[turn], r) + at);
            uint4 h = make_uint4(0, 0, 0, 0);
            if (by_weight) h = *reinterpret_cast<const uint4 *>(in_cta(sh.hi[turn], r) + at);
            own[0] += static_cast<u64>(h.x) << 32 | l.x;
            own[1] += static_cast<u64>(h.y) << 32 | l.y;
            own[2] += static_cast<u64>(h.z) << 32 | l.z;
            own[3] += static_cast<u64>(h.w) << 32 | l.w;
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
        for (int x = tid; x < kBins; x += kThreads) sh.lo[turn ^ 1][x] = sh.hi[turn ^ 1][x] = 0;
        __syncthreads();
        return sh.bin >= 0;
    };

    // The cut at which `target` (a count, or a sum of weights) is reached from the top, among what is
    // kept so far: the new cut and its ties. (A count that is not reached: all are kept.)
    auto descend = [&](bool by_weight, u64 target) {
        const float old_cut = cut;
        // those equal to the cut so far, of which only `ties` are kept: one thread adds them
        const bool old = by_weight && ties > 0 && rank == 0 && tid == 0;
        const u64 w_old = old ? weight(old_cut) * static_cast<u64>(ties) : 0;
        const float scale = weight.c_hi * 32.0f;
        // bin and place in it (both roundings leave the order of logits as it is)
        auto place = [&](float x) { return x == top ? 0.0f : fminf((top - x) * scale, static_cast<float>(kBins)); };
        auto settle = [&](u64 rest) {
            if (by_weight) {
                const u64 w = weight(cut);
                ties = static_cast<int>((rest + w - 1) / w);
            } else {
                ties = static_cast<int>(rest);
            }
        };
        each(Const<2>(), v0, v1, [&](const float (&x)[kVec], int) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float f = place(x[e]);
                if (!(x[e] > old_cut) || f >= static_cast<float>(kBins)) continue;
                if (by_weight) add(0, static_cast<unsigned>(f), weight(x[e]));
                else atomicAdd(&sh.lo[0][static_cast<unsigned>(f)], 1u);
            }
        });
        if (old && place(old_cut) < static_cast<float>(kBins)) add(0, static_cast<unsigned>(place(old_cut)), w_old);
        sync();
        if (find(0, by_weight, target, false)) {
            const u64 rest = target - sh.before;
            const float bin = static_cast<float>(sh.bin);
            auto note = [&](float x, float f, u64 w) {
                const unsigned part = static_cast<unsigned>((f - bin) * kBins), key = key_of(x);  // (f - bin is exact)
                if (by_weight) add(1, part, w);
                else atomicAdd(&sh.lo[1][part], 1u);
                atomicMax(&sh.least[part], ~key);
                atomicMax(&sh.most[part], key);
            };
            each(Const<2>(), v0, v1, [&](const float (&x)[kVec], int) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float f = place(x[e]);
                    if (x[e] > old_cut && f >= bin && f < bin + 1.0f) note(x[e], f, by_weight ? weight(x[e]) : 0ull);
                }
            });
            if (old) {
                const float f = place(old_cut);
                if (f >= bin && f < bin + 1.0f) note(old_cut, f, w_old);
            }
            sync();
            const int part = find(1, by_weight, rest, false) ? sh.bin : 0;  // (the bin holds the border)
            unsigned least = 0, most = 0;
            for (int r = 0; r < cluster; ++r) {
                least = max(least, *(in_cta(sh.least, r) + part));
                most = max(most, *(in_cta(sh.most, r) + part));
            }
            const u64 left = rest - sh.before;
            sync();  // the parts' keys, and the second histogram, have been read
            for (int x = tid; x < kBins; x += kThreads)
                sh.lo[1][x] = sh.hi[1][x] = sh.least[x] = sh.most[x] = 0;
            __syncthreads();
            if (~least == most) {
                cut = value_of(most);
                settle(left);
                return;
            }
        } else {
            sync();
            for (int x = tid; x < kBins; x += kThreads) sh.lo[0][x] = sh.hi[0][x] = 0;
            __syncthreads();
        }
        // by the keys' bits
        unsigned prefix = 0;
        bool found = true;
#pragma unroll 1
        for (int pass = 0; pass < 3 && found; ++pass) {
            const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, turn = pass & 1;
            auto mine = [&](unsigned key) { return pass == 0 || (key >> (down + bits)) == prefix; };
            each(Const<2>(), v0, v1, [&](const float (&x)[kVec], int) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const unsigned key = key_of(x[e]);
                    if (!(x[e] > old_cut) || !mine(key)) continue;
                    const unsigned bin = (key >> down) & ((1u << bits) - 1);
                    if (by_weight) add(turn, bin, weight(x[e]));
                    else atomicAdd(&sh.lo[turn][bin], 1u);
                }
            });
            if (old && mine(key_of(old_cut))) add(turn, (key_of(old_cut) >> down) & ((1u << bits) - 1), w_old);
            sync();
            found = find(turn, by_weight, target, true);
            if (found) {
                target -= sh.before;
                prefix = prefix << bits | static_cast<unsigned>(sh.bin);
            }
        }
        if (found) {
            cut = value_of(prefix);
            settle(target);
        }
        sync();
        for (int x = tid; x < kBins; x += kThreads) sh.lo[0][x] = sh.hi[0][x] = 0;
        __syncthreads();
    };

    if (top_k > 0 && top_k < p.vocab) descend(false, top_k);
    if (top_p < 1.0f) {
        gather_parts();
        const u64 total = total_of(ties > 0 ? weight(cut) : 0);
        const u64 want = top_p > 0.0f ? times(top_p, total, true) : 0;
        descend(true, want > 0 ? want : 1);  // (its barriers come before the parts are written again)
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
    // 32 parts of 16 bytes at a time, then the lane's, then its logits
    gather_parts();
    const u64 w_cut = ties > 0 ? weight(cut) : 0;
    const u64 target = times(u, total_of(w_cut), false);
    u64 run = 0;   // weights above the cut before the stretch
    int seen = 0;  // logits equal to it
    auto upto = [&](u64 sum, int equal) { return sum + static_cast<u64>(min(equal, ties)) * w_cut; };
    // which of `count` parts it is (by a whole warp); run and seen move on to it
    auto pick = [&](const Part *parts, int count) {
        for (int x0 = 0;; x0 += 32) {
            Part mine{0, 0, 0};
            if (x0 + lane < count) mine = parts[x0 + lane];
            __syncwarp();
            const u64 sums = warp_scan64(mine.sum);
            const int equals = warp_scan(mine.equal);
            const unsigned past = __ballot_sync(FULL_MASK, upto(run + sums, seen + equals) > target);
            const int at = past != 0 ? __ffs(past) - 1 : 31;
            run += __shfl_sync(FULL_MASK, past != 0 ? sums - mine.sum : sums, at);
            seen += __shfl_sync(FULL_MASK, past != 0 ? equals - mine.equal : equals, at);
            if (past != 0 || x0 + 32 >= count) return x0 + at;
        }
    };
    const int stretch = pick(sh.parts, cluster * kWarps);
    if (stretch / kWarps == rank) {
        const int begin = min(cta1, rank * per_cta + stretch % kWarps * per_warp), end = min(cta1, begin + per_warp);
        const int each_warp = (end - begin + kThreads - 1) / kThreads * 32;
        const int a = min(end, begin + warp * each_warp);
        const Part mine = part_of(a, min(end, a + each_warp));
        if (lane == 0) sh.own[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const int from = begin + pick(sh.own, kWarps) * each_warp, to = min(end, from + each_warp);
            for (int v = from; v < to; v += 32) {
                float x[kVec];
                u64 sum = 0;
                int same = 0;
                if (v + lane < to) {
                    Logit<T>::unpack(load(v + lane), x);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        if (x[e] > cut) sum += weight(x[e]);
                        else if (x[e] == cut) ++same;
                    }
                }
                __syncwarp();
                const u64 sums = warp_scan64(sum);
                const int sames = warp_scan(same);
                const unsigned past = __ballot_sync(FULL_MASK, upto(run + sums, seen + sames) > target);
                if (past != 0) {
                    if (lane == __ffs(past) - 1) {
                        u64 s = run + sums - sum;
                        int q = seen + sames - same;
                        bool done = false;
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            if (x[e] > cut) s += weight(x[e]);
                            else if (x[e] == cut) ++q;
                            if (!done && upto(s, q) > target) {
                                p.tokens[row] = (v + lane) * kVec + e - shift;
                                done = true;
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
    if (cluster > 1) cluster_sync();  // no CTA leaves while another may read or write its shared memory
}

// CTAs of a row: as many as give every SM its two, of at least 2048 logits each.
template <typename T>
gdn_status launch(const SampleParams &p, int rows, cudaStream_t s) {
    int cluster = kMaxCluster;
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
