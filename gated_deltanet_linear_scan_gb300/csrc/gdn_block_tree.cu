// gdn_block_tree.cu -- the Gated-DeltaNet block over a tree of drafted tokens, and the states
// carried on along the accepted path (sm_103a).
//
// Every node continues its parent's state. With anc(i) the ancestors of node i, G_i the sum of
// the log-decays on its path (itself included) and S0 the sequence's state,
//   u_i = beta_i (v_i - e^{G_i} S0^T k_i - sum_{s in anc(i)} e^{G_i - G_s} (k_i . k_s) u_s)
//   y_i = scale (e^{G_i} S0^T q_i + sum_{s in anc(i) and i} e^{G_i - G_s} (q_i . k_s) u_s)
// is the recurrence unrolled: node i's state is e^{G_i} S0 + sum_{s} e^{G_i - G_s} k_s u_s^T.
// So the state is read once for all nodes and not written: a tree of N nodes moves 1 / (N + 1) of
// the bytes of a scan that keeps a snapshot per node. What an accepted path needs later are k, g
// and u of its nodes (the tape): its state is one more rank-L update, read and written once.
#include "gdn_paged.cuh"
#include "gdn_tc.cuh"
#include "gdn_tree.cuh"

namespace gdn {
namespace {

constexpr size_t kAlignFloats = 64;  // 256-byte sub-buffers

__host__ __device__ constexpr size_t round_up(size_t n) { return (n + kAlignFloats - 1) / kAlignFloats * kAlignFloats; }

// What the commit reads: k [n][N][Hk][S], g [n][N][H], u [n][N][H][S].
struct Tape {
    size_t k, g, u, floats;
    Tape(size_t rows, int hk, int h, int s) {
        k = 0;
        g = k + round_up(rows * hk * s);
        u = g + round_up(rows * h);
        floats = u + round_up(rows * h * s);
    }
};

// How the tensor-core path lays out what it prepares for a sequence and head, in bytes.
struct TcSizes {
    int pad, rows;                          // nodes, and vectors [K; Q], of an image: multiples of 8, of 16
    uint32_t image, images;                 // of one part; of a (sequence, k-head)'s three
    uint32_t weights_y, anc, beta, weights; // of a (sequence, v-head)'s: where what begins, and all
    __host__ __device__ explicit TcSizes(int n) {
        pad = (n + 7) / 8 * 8;
        rows = 2 * pad;
        image = static_cast<uint32_t>(rows) * 256u;
        images = 3u * image;
        weights_y = static_cast<uint32_t>(n * pad) * 4u;       // behind the weights in u, [n][pad]
        anc = 2u * weights_y;                                  // which nodes they are of, [n][pad]
        beta = anc + static_cast<uint32_t>(n * pad);           // [pad] each: beta, beta e^G, e^G, nodes on the path
        weights = (beta + 16u * static_cast<uint32_t>(pad) + 15u) / 16u * 16u;
    }
};

// Scratch: v [n][N][H][S] and, of states of 128, the images and weights of the tensor-core path; of others q
// [n][N][Hk][S], beta [n][N][H], the products k_i.k_s and q_i.k_s [n][Hk][N][N][2] and the nodes' paths
// [n][N] (0: not there).
struct Scratch {
    size_t v, images, weights, q, beta, gram, paths, floats;
    Scratch(size_t rows, int n_nodes, int hk, int h, int s) {
        const size_t seqs = rows / n_nodes;
        const TcSizes tc(n_nodes);
        v = images = weights = q = beta = gram = paths = 0;
        floats = round_up(rows * h * s);
        auto take = [&](size_t &at, size_t n) {
            at = floats;
            floats += round_up(n);
        };
        if (s == 128) {
            take(images, seqs * hk * (tc.images / 4));
            take(weights, seqs * h * (tc.weights / 4));
        } else {
            take(q, rows * hk * s);
            take(beta, rows * h);
            take(gram, rows * n_nodes * hk * 2);
            take(paths, rows * 2);
        }
    }
};

struct TreeParams {
    const float *qkv, *conv_w, *conv_state, *alpha, *b, *dt, *a, *z, *norm_w, *state;
    float *out;
    const int32_t *parents, *slots;
    int n_nodes, n_k_heads, n_v_heads, pool;
    float scale, l2_eps, norm_eps;
    int32_t *err_count;
    float *k, *g, *u;             // the tape
    float *v, *q, *beta, *gram;   // scratch
    uint8_t *images, *weights;
    unsigned long long *paths;
    unsigned *watchdog;
};

// ------------------------------------------------------------------ conv, norms and gates

// (Of other states than 128, whose nodes' sums have no tensor cores; the arithmetic is shared.) One
// warp per (head slice of S channels, kConvNodes nodes, sequence), lane L holding channels [E L, E L +
// E). A node's taps are its own raw input and those of its nearest ancestors, the conv history behind
// the root's; the arithmetic is the prefill block's, so a tree that is a chain has its bits. The CTAs
// behind the slices' compute the gates. A node that is not there has zeros.
constexpr int kConvWarps = 4;
constexpr int kConvNodes = 8;

// N consecutive floats, 16-byte aligned where N is a multiple of 4.
template <int N>
__device__ __forceinline__ void load_run(float (&x)[N], const float *from) {
    if constexpr (N % 4 == 0) load_vec<N>(x, from);
    else
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = from[i];
}

// SiLU of a node's convolution, channels of a lane: `own` its own raw input, x_ptr node 0's. Conditions
// are uniform over the warp.
template <int E, int K>
__device__ __forceinline__ void conv_node(const float *x_ptr, size_t conv_dim, int i, unsigned long long path,
                                          const float (&wc)[E * K], const float (&hist)[E * (K - 1)],
                                          const float (&own)[E], float (&o)[E]) {
    constexpr int TAPS = K - 1;
    const int depth = __popcll(path);
    float taps[TAPS][E];  // [t]: of the t-th oldest input before its own
    path &= ~(1ull << i);
#pragma unroll
    for (int t = TAPS - 1; t >= 0; --t)
        if (path != 0) {
            const int a = 63 - __clzll(static_cast<long long>(path));
            path &= ~(1ull << a);
            load_vec<E>(taps[t], x_ptr + static_cast<size_t>(a) * conv_dim);
        }
    // past the root: the history, newest last
#pragma unroll
    for (int d = 1; d <= TAPS; ++d)
        if (depth == d)
#pragma unroll
            for (int t = 0; t <= TAPS - d; ++t)
#pragma unroll
                for (int e = 0; e < E; ++e) taps[t][e] = hist[e * TAPS + t + d - 1];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float pre = __fmul_rn(own[e], wc[e * K + K - 1]);
#pragma unroll
        for (int t = 0; t < TAPS; ++t) pre = __fmaf_rn(taps[t][e], wc[e * K + t], pre);
        o[e] = silu(pre);
    }
}

// A vector over its length, by a whole warp.
template <int E>
__device__ __forceinline__ void normalise(float (&o)[E], float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss = __fmaf_rn(o[e], o[e], ss);
    ss = warp_allsum(ss);
    const float inv = 1.0f / fmaxf(sqrtf(ss), eps);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= inv;
}

__device__ __forceinline__ float gate_of(const TreeParams &p, size_t at, int h) {
    return p.a[h] * softplus_guarded(p.alpha[at] + p.dt[h]);
}
__device__ __forceinline__ float beta_of_node(const TreeParams &p, size_t at) { return 1.0f / (1.0f + expf(-p.b[at])); }

template <int E, int K>
__global__ void __launch_bounds__(32 * kConvWarps) tree_conv_kernel(const TreeParams p) {
    constexpr int S = 32 * E, TAPS = K - 1;
    __shared__ unsigned long long path_of[kMaxNodes];
    __shared__ int up[kMaxNodes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.z, N = p.n_nodes, Hk = p.n_k_heads, H = p.n_v_heads;
    const int slot = p.slots ? p.slots[n] : n;
    const bool skip = slot < 0 || slot >= p.pool;
    const bool counts = blockIdx.x == 0 && blockIdx.y == 0;
    if (skip) {
        if (counts && threadIdx.x == 0 && p.err_count) atomicAdd(p.err_count, 1);
        return;
    }
    const int i0 = blockIdx.y * kConvNodes, i1 = min(N, i0 + kConvNodes);
    const size_t row0 = static_cast<size_t>(n) * N;
    const int slices = 2 * Hk + H, sl = blockIdx.x * kConvWarps + warp;  // this warp's head slice
    const size_t conv_dim = static_cast<size_t>(slices) * S;
    const size_t ch0 = static_cast<size_t>(sl) * S + E * lane;
    const float *x_ptr = p.qkv + row0 * conv_dim + ch0;
    // the lane's weights [E][K] and history [E][TAPS], consecutive in memory, and the nodes' own inputs:
    // on their way while the paths are worked out (states of 256: no registers for the inputs)
    constexpr bool kEarly = E <= 4;
    float wc[E * K], hist[E * TAPS], own[kEarly ? kConvNodes : 1][E];
    if (sl < slices) {
        load_run<E * K>(wc, p.conv_w + ch0 * K);
        load_run<E * TAPS>(hist, p.conv_state + (static_cast<size_t>(slot) * conv_dim + ch0) * TAPS);
        if constexpr (kEarly)
#pragma unroll
            for (int y = 0; y < kConvNodes; ++y)
                if (i0 + y < i1) load_vec<E>(own[y], x_ptr + static_cast<size_t>(i0 + y) * conv_dim);
    }
    if (warp == 0) {
        unsigned long long paths[2];
        const bool bad = tree_paths(p.parents + static_cast<size_t>(n) * N, N, paths, path_of, up);
        if (bad && counts && lane == 0 && p.err_count) atomicAdd(p.err_count, 1);
        if (counts) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (lane + 32 * x < N) p.paths[static_cast<size_t>(n) * N + lane + 32 * x] = paths[x];
        }
    }
    __syncthreads();
    if (blockIdx.x == gridDim.x - 1) {
        // ---- the gates: g = a softplus(alpha + dt), beta = sigmoid(b)
        for (int x = threadIdx.x; x < (i1 - i0) * H; x += 32 * kConvWarps) {
            const int i = i0 + x / H, h = x % H;
            const size_t at = (row0 + i) * H + h;
            const bool here = path_of[i] != 0;
            p.g[at] = here ? gate_of(p, at, h) : 0.0f;
            p.beta[at] = here ? beta_of_node(p, at) : 0.0f;
        }
        return;
    }
    if (sl >= slices) return;
    const bool is_qk = sl < 2 * Hk;  // uniform over the warp
    float *dst = is_qk ? (sl < Hk ? p.q : p.k) + (row0 * Hk + sl % Hk) * S + E * lane
                       : p.v + (row0 * H + (sl - 2 * Hk)) * S + E * lane;
    const size_t dst_step = static_cast<size_t>(is_qk ? Hk : H) * S;
#pragma unroll
    for (int y = 0; y < kConvNodes; ++y) {
        const int i = i0 + y;
        if (i >= i1) break;  // uniform over the warp, as every condition below
        float o[E] = {};
        if (path_of[i] != 0) {
            float mine[E];
            if constexpr (kEarly) {
#pragma unroll
                for (int e = 0; e < E; ++e) mine[e] = own[y][e];
            } else {
                load_vec<E>(mine, x_ptr + static_cast<size_t>(i) * conv_dim);
            }
            conv_node<E, K>(x_ptr, conv_dim, i, path_of[i], wc, hist, mine, o);
            if (is_qk) normalise<E>(o, p.l2_eps);
        }
        store_vec<E>(dst + static_cast<size_t>(i) * dst_step, o);
    }
}

// ------------------------------------------------------------------ products of the nodes

// k_i.k_s and q_i.k_s of every node i with itself and its ancestors s: the keys in shared memory, one
// warp per node at a time, two ancestors together. Grid: (k-head, sequence).
constexpr int kGramWarps = 8;

template <int E>
__global__ void __launch_bounds__(32 * kGramWarps) tree_gram_kernel(const TreeParams p) {
    constexpr int S = 32 * E;
    extern __shared__ __align__(16) float keys[];  // [N][S]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kh = blockIdx.x, n = blockIdx.y, N = p.n_nodes, Hk = p.n_k_heads;
    const int slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.pool) return;
    const size_t base = (static_cast<size_t>(n) * N * Hk + kh) * S, step = static_cast<size_t>(Hk) * S;
    for (int x = threadIdx.x; x < N * (S / 4); x += 32 * kGramWarps)
        *reinterpret_cast<float4 *>(keys + 4 * x) =
            *reinterpret_cast<const float4 *>(p.k + base + (x / (S / 4)) * step + 4 * (x % (S / 4)));
    __syncthreads();
    const unsigned long long *path_of = p.paths + static_cast<size_t>(n) * N;
    float2 *gram = reinterpret_cast<float2 *>(p.gram) + (static_cast<size_t>(n) * Hk + kh) * N * N;
    for (int i = warp; i < N; i += kGramWarps) {
        unsigned long long path = path_of[i];
        if (path == 0) continue;
        float ki[E], qi[E];
        load_vec<E>(ki, keys + i * S + E * lane);
        load_vec<E>(qi, p.q + base + i * step + E * lane);
        while (path != 0) {
            const int s = __ffsll(static_cast<long long>(path)) - 1;
            path &= path - 1;
            const int t = path != 0 ? __ffsll(static_cast<long long>(path)) - 1 : s;
            if (path != 0) path &= path - 1;
            float ks[E], kt[E];
            load_vec<E>(ks, keys + s * S + E * lane);
            load_vec<E>(kt, keys + t * S + E * lane);
            float part[4] = {lane_dot<E>(ki, ks), lane_dot<E>(qi, ks), lane_dot<E>(ki, kt), lane_dot<E>(qi, kt)};
            const float sum = warp_sum_packed<4>(part, lane);
            // sums 0 and 1 of s, 2 and 3 of t
            const float next = __shfl_xor_sync(FULL_MASK, sum, row_home_lane<4>(1));
            if (lane == row_home_lane<4>(0)) gram[i * N + s] = make_float2(sum, next);
            if (lane == row_home_lane<4>(2)) gram[i * N + t] = make_float2(sum, next);
        }
    }
}

// ------------------------------------------------------------------ the nodes over the state

// Grid: (block of state rows, v-head, sequence), 128 threads. Rows j of the transposed state are
// value channels, and independent of one another: a CTA takes JB of them. First the products of
// its rows with all k_i and q_i (kTileRows of them at a time; a lane holds JB / 32 state rows and
// a warp 8 of the vectors), then u, node after node, and y, all of them at once.
constexpr int kStateThreads = 128;
constexpr int kTileRows = 32;

template <int E>
struct StateSmem {
    static constexpr int S = 32 * E;
    static constexpr int JB = S >= 64 ? 64 : 32;
    static constexpr int kPad = S + 4;  // lanes' 16-byte reads of their rows in different banks
    static size_t bytes(int n) {
        return sizeof(float) * (static_cast<size_t>(JB) * kPad + kTileRows * S + 2 * n * JB + 2 * n * n);
    }
};

// The sums on the nodes' paths, in two parts (hi + lo, off by 2^-40 relative): their differences
// e^{G_i - G_s} are then good to 2^-23 however long the path is. A log-decay ends at -kForgets, where its node
// forgets everything many times over: behind that node the sums' differences stay as good, however far below
// (or at -infinity) it was.
constexpr float kForgets = 16384.0f;
__device__ __forceinline__ void path_sum(unsigned long long path, const float *g, float &hi, float &lo) {
    hi = lo = 0.0f;
    while (path != 0) {
        const int s = __ffsll(static_cast<long long>(path)) - 1;
        path &= path - 1;
        const float x = g[s] < -kForgets ? -kForgets : g[s], sum = __fadd_rn(hi, x), y = __fsub_rn(sum, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, y)), __fsub_rn(x, y)));
        hi = sum;
    }
}

template <int E>
__global__ void __launch_bounds__(kStateThreads) tree_state_kernel(const TreeParams p) {
    using L = StateSmem<E>;
    constexpr int S = L::S, JB = L::JB, JL = JB / 32, kPad = L::kPad;
    extern __shared__ __align__(16) float smem[];
    __shared__ unsigned long long path_of[kMaxNodes];
    __shared__ float g_of[kMaxNodes], hi_of[kMaxNodes], lo_of[kMaxNodes], beta_of[kMaxNodes], decay[kMaxNodes];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = blockIdx.x * JB, vh = blockIdx.y, n = blockIdx.z;
    const int N = p.n_nodes, Hk = p.n_k_heads, H = p.n_v_heads, kh = vh % Hk;
    const int slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.pool) return;
    float *rows = smem;                       // [JB][kPad]
    float *tile = rows + JB * kPad;           // [kTileRows][S]
    float *d = tile + kTileRows * S;          // [2N][JB]: products with k, then u; with q
    float2 *coef = reinterpret_cast<float2 *>(d + 2 * N * JB);  // [N][N]
    const float *state = p.state + ((static_cast<size_t>(slot) * H + vh) * S + j0) * S;
    for (int x = tid; x < JB * S / 4; x += kStateThreads) {
        const int j = x / (S / 4), c = x % (S / 4);
        *reinterpret_cast<float4 *>(rows + j * kPad + 4 * c) = *reinterpret_cast<const float4 *>(state + j * S + 4 * c);
    }
    const size_t row0 = static_cast<size_t>(n) * N;
    if (tid < N) {
        path_of[tid] = p.paths[row0 + tid];
        g_of[tid] = p.g[(row0 + tid) * H + vh];
        beta_of[tid] = p.beta[(row0 + tid) * H + vh];
    }
    __syncthreads();
    if (tid < N) {
        path_sum(path_of[tid], g_of, hi_of[tid], lo_of[tid]);
        decay[tid] = expf(hi_of[tid] + lo_of[tid]);
    }
    __syncthreads();
    {
        const float2 *gram = reinterpret_cast<const float2 *>(p.gram) + (static_cast<size_t>(n) * Hk + kh) * N * N;
        for (int x = tid; x < N * N; x += kStateThreads) {
            const int i = x / N, s = x % N;
            if (!((path_of[i] >> s) & 1ull)) continue;
            const float w = expf((hi_of[i] - hi_of[s]) + (lo_of[i] - lo_of[s]));
            const float2 dot = gram[x];
            coef[x] = make_float2(beta_of[i] * w * dot.x, w * dot.y);
        }
    }
    // ---- the products with the state
    for (int t0 = 0; t0 < 2 * N; t0 += kTileRows) {
        __syncthreads();  // the tile before has been read
        const int count = min(kTileRows, 2 * N - t0);
        for (int x = tid; x < count * (S / 4); x += kStateThreads) {
            const int r = x / (S / 4), c = x % (S / 4), i = t0 + r;
            const float *src = (i < N ? p.k + ((row0 + i) * Hk + kh) * S : p.q + ((row0 + i - N) * Hk + kh) * S);
            *reinterpret_cast<float4 *>(tile + r * S + 4 * c) = *reinterpret_cast<const float4 *>(src + 4 * c);
        }
        __syncthreads();
        const float *mine = tile + warp * 8 * S;
        if (warp * 8 < count) {
            float acc[JL][8] = {};
#pragma unroll 4
            for (int c = 0; c < S; c += 4) {
                float4 x[JL];
#pragma unroll
                for (int l = 0; l < JL; ++l) x[l] = *reinterpret_cast<const float4 *>(rows + (lane + 32 * l) * kPad + c);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 y = *reinterpret_cast<const float4 *>(mine + r * S + c);
#pragma unroll
                    for (int l = 0; l < JL; ++l) {
                        acc[l][r] = fmaf(x[l].x, y.x, acc[l][r]);
                        acc[l][r] = fmaf(x[l].y, y.y, acc[l][r]);
                        acc[l][r] = fmaf(x[l].z, y.z, acc[l][r]);
                        acc[l][r] = fmaf(x[l].w, y.w, acc[l][r]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (warp * 8 + r < count)
#pragma unroll
                    for (int l = 0; l < JL; ++l) d[(t0 + warp * 8 + r) * JB + lane + 32 * l] = acc[l][r];
        }
    }
    __syncthreads();
    // ---- u, one thread a row, node after node
    if (tid < JB) {
        const float *v = p.v + (row0 * H + vh) * S + j0 + tid;
        float *u_out = p.u + (row0 * H + vh) * S + j0 + tid;
        const size_t step = static_cast<size_t>(H) * S;
        float next = v[0];
        for (int i = 0; i < N; ++i) {
            const float vi = next;
            if (i + 1 < N) next = v[(i + 1) * step];
            unsigned long long path = path_of[i] & ~(1ull << i);
            float u = beta_of[i] * (vi - decay[i] * d[i * JB + tid]);
            while (path != 0) {
                const int s = __ffsll(static_cast<long long>(path)) - 1;
                path &= path - 1;
                u = fmaf(-coef[i * N + s].x, d[s * JB + tid], u);
            }
            if (path_of[i] == 0) u = 0.0f;
            d[i * JB + tid] = u;
            u_out[i * step] = u;
        }
    }
    __syncthreads();
    // ---- y
    for (int x = tid; x < N * JB; x += kStateThreads) {
        const int i = x / JB, j = x % JB;
        unsigned long long path = path_of[i];
        float y = 0.0f;
        if (path != 0) {
            y = decay[i] * d[(N + i) * JB + j];
            while (path != 0) {
                const int s = __ffsll(static_cast<long long>(path)) - 1;
                path &= path - 1;
                y = fmaf(coef[i * N + s].y, d[s * JB + j], y);
            }
        }
        p.out[((row0 + i) * H + vh) * S + j0 + j] = p.scale * y;
    }
}

// ------------------------------------------------------------------ the same on the tensor cores

// State size 128: all products of a head's state with its nodes' k and q are one tcgen05 product
// D = S [K; Q]^T, and the nodes' sums and the gated norm follow in the same CTA, so a state is read
// once and y never leaves the SM. 256 threads take (sequence, v-head) after (sequence, v-head); two CTAs
// share an SM as long as 16 nodes fill half of tensor memory.
//
// The products keep fp32's precision: each operand is split into three bf16 parts, x = x1 + x2 + x3
// (8 bits each, the rest below 2^-27 of x), and the six products of parts whose sizes multiply to
// 2^-18 or more are summed in fp32; what is left out is below 2^-25 of |S| |k|. (Two parts would leave
// 2^-16, a hundred times the error of fp32 arithmetic.) The state's parts lie in tensor memory (lane =
// value channel j), the nodes' in shared memory: three images of [K; Q], K-major core matrices.
// S1 and S2 multiply the first two images at once, into two column groups that are added up later.
//
// A kernel ahead of it convolves the values, and per (sequence, k-head) convolves q and k, writes the
// images, and for every v-head of the k-head solves the nodes' triangular system: with A[i][s] =
// beta_i e^{G_i - G_s} k_i.k_s (s above i) and T = (I + A)^-1,
//   R_s = beta_s (v_s - e^{G_s} S0^T k_s),   u_i = sum_{s on the path to i} T[i][s] R_s,
//   y_i = scale (e^{G_i} S0^T q_i + sum_s W[i][s] R_s),   W = B T, B[i][s] = e^{G_i - G_s} q_i.k_s,
// so that over the state all nodes are independent of one another. T and W are lists along the paths.
//
// 64 sequences of 16 nodes, 16 k- and 32 v-heads: 102 us, of which the kernel ahead takes 44 (issue
// and latency; with a kernel of its own for the convolution 28 and 29) and this one 56 (it reads 198
// MB and writes 19 in that time: 3.9 TB/s; between barriers its 16 warps an SM issue in 4 cycles of
// 10). One sequence of 48 nodes: 36 us, 13 of them here. (Node after node over the state instead of T:
// 122 and 45.)
constexpr int kTcThreads = 256;
constexpr uint32_t kColA = 0, kColD = 192;  // tensor memory: the state's parts, 64 columns each; D, two groups

// Shared memory of the state's kernel: the state, the images, the weights, D. Up to about 40 nodes D and
// a second head's weights have places of their own, and what the next head needs is on its way as
// soon as this one's products are under way; with more, D lies over the state.
struct TcSmem {
    static constexpr uint32_t kMost = 225u * 1024u;
    uint32_t images, weights, turn, d, bytes;  // turn: from a head's weights to the next one's
    bool apart;
    __host__ __device__ TcSmem(const TcSizes &z, int n) {
        images = 65536;
        weights = images + z.images;
        const uint32_t two = weights + 2 * z.weights, all = two + 1024u * static_cast<uint32_t>(n);
        apart = all <= kMost;
        turn = apart ? z.weights : 0;
        d = apart ? two : 0;
        bytes = apart ? all : weights + z.weights;
    }
};
__host__ __device__ inline uint32_t tmem_cols(const TcSizes &z) {
    return kColD + 2u * static_cast<uint32_t>(z.rows) <= 256u ? 256u : 512u;
}

// Convolution, images and weights. CTAs of (k-head, part of its v-heads, sequence): 4 warps, 8 or 16
// where that leaves SMs idle, and then with few sequences a part for every v-head. q and k, a warp a
// node; the nodes' products, a warp a node; then, for a few v-heads at a time, A and B as lists along
// the paths, one thread an entry, and T and W, all rows of one depth together. The CTAs behind them
// convolve the values, a warp a v-head of up to kConvNodes nodes.
constexpr int kPrepThreads = 512;
constexpr int kPrepHeads = 4;

struct PrepSmem {
    static constexpr int kLd = 128 + 4;       // floats of a vector: rows' 16-byte pieces in different banks
    int heads;                                // at a time
    uint32_t b, t, head, gram, anc, bytes;    // of a v-head: A, B and T, [N][pad]
    __host__ __device__ explicit PrepSmem(int n) {
        const uint32_t lists = TcSizes(n).weights_y;
        b = lists;
        t = 2 * lists;
        head = 3 * lists;
        heads = static_cast<int>(131072u / head);
        heads = heads < 1 ? 1 : heads > kPrepHeads ? kPrepHeads : heads;
        const uint32_t vectors = static_cast<uint32_t>(2 * n * kLd) * 4u, work = static_cast<uint32_t>(heads) * head;
        gram = vectors > work ? vectors : work;  // behind the vectors, whose place A, B and T take
        anc = gram + static_cast<uint32_t>(n * n) * 8u;
        bytes = anc + lists / 4;
    }
};

constexpr int kPrepSmem = 196608;  // no number of nodes needs more

template <int K>
__global__ void __launch_bounds__(kPrepThreads, K <= 4 ? 2 : 1) tree_prepare_kernel(const TreeParams p, int prepares, int parts) {
    constexpr int S = 128, kLd = PrepSmem::kLd;
    extern __shared__ __align__(16) uint8_t dyn[];
    constexpr int E = 4, TAPS = K - 1;
    __shared__ unsigned long long path_of[kMaxNodes];
    __shared__ int up[kMaxNodes];
    __shared__ int level[kMaxNodes + 1];      // [d]: where the nodes of depth d + 1 begin in by_depth
    __shared__ uint8_t by_depth[kMaxNodes];
    __shared__ float g_of[kPrepHeads][kMaxNodes], beta_of[kPrepHeads][kMaxNodes];
    __shared__ float hi_of[kPrepHeads][kMaxNodes], lo_of[kPrepHeads][kMaxNodes];  // the sums of g on the paths
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x, warps = threads / 32;
    const int N = p.n_nodes, Hk = p.n_k_heads, H = p.n_v_heads;
    const bool prepare = static_cast<int>(blockIdx.x) < prepares;
    // the others: v-heads of a block of nodes of a sequence, one a warp
    const int groups_v = (H + warps - 1) / warps, node_blocks = (N + kConvNodes - 1) / kConvNodes;
    const int other = static_cast<int>(blockIdx.x) - prepares;
    const int n = prepare ? blockIdx.x / (Hk * parts) : other / (groups_v * node_blocks), kh = prepare ? blockIdx.x % Hk : 0;
    const int part = prepare ? blockIdx.x / Hk % parts : 0;  // of the v-heads; the first writes what all share
    const int slot = p.slots ? p.slots[n] : n;
    const bool counts = prepare && kh == 0 && part == 0;
    if (slot < 0 || slot >= p.pool) {
        if (counts && tid == 0 && p.err_count) atomicAdd(p.err_count, 1);
        return;
    }
    const size_t row0 = static_cast<size_t>(n) * N, conv_dim = static_cast<size_t>(2 * Hk + H) * S;
    // this warp's head slice: of q (even warps) or k (odd ones), or of v; its weights [E][K] and history [E][TAPS]
    const int vh_mine = other % groups_v * warps + warp;
    const int slice = prepare ? (warp & 1) * Hk + kh : 2 * Hk + vh_mine;
    const bool has_slice = prepare || vh_mine < H;
    const size_t ch0 = static_cast<size_t>(slice) * S + E * lane;
    const float *x_ptr = p.qkv + row0 * conv_dim + ch0;
    float wc[E * K], hist[E * TAPS];
    if (has_slice) {
        load_run<E * K>(wc, p.conv_w + ch0 * K);
        load_run<E * TAPS>(hist, p.conv_state + (static_cast<size_t>(slot) * conv_dim + ch0) * TAPS);
    }
    if (warp == 0) {
        unsigned long long paths[2];
        const bool bad = tree_paths(p.parents + row0, N, paths, path_of, up);
        if (bad && counts && lane == 0 && p.err_count) atomicAdd(p.err_count, 1);
    }
    __syncthreads();
    if (!prepare) {
        if (!has_slice) return;
        const int i0 = other / groups_v % node_blocks * kConvNodes, i1 = min(N, i0 + kConvNodes);
#pragma unroll 2
        for (int i = i0; i < i1; ++i) {
            float o[E] = {};
            if (path_of[i] != 0) {
                float mine[E];
                load_vec<E>(mine, x_ptr + static_cast<size_t>(i) * conv_dim);
                conv_node<E, K>(x_ptr, conv_dim, i, path_of[i], wc, hist, mine, o);
            }
            store_vec<E>(p.v + ((row0 + i) * H + vh_mine) * S + E * lane, o);
        }
        return;
    }
    const TcSizes z(N);
    const PrepSmem L(N);
    float *rows = reinterpret_cast<float *>(dyn);  // k of all nodes, then q
    float2 *gram = reinterpret_cast<float2 *>(dyn + L.gram);
    uint8_t *anc = dyn + L.anc;  // [N][pad]: the path's nodes in order, then its first again
    // ---- k and q
#pragma unroll 2
    for (int i = warp >> 1; i < N; i += warps / 2) {
        float o[E] = {};
        if (path_of[i] != 0) {
            float mine[E];
            load_vec<E>(mine, x_ptr + static_cast<size_t>(i) * conv_dim);
            conv_node<E, K>(x_ptr, conv_dim, i, path_of[i], wc, hist, mine, o);
            normalise<E>(o, p.l2_eps);
        }
        store_vec<E>(rows + ((warp & 1) ? i : N + i) * kLd + E * lane, o);
        if ((warp & 1) && part == 0) store_vec<E>(p.k + ((row0 + i) * Hk + kh) * S + E * lane, o);
    }
    __syncthreads();
    // ---- as images (rows past the nodes zero)
    uint8_t *images = p.images + (static_cast<size_t>(n) * Hk + kh) * z.images;
    for (int x = part == 0 ? tid : z.rows * (S / 8); x < z.rows * (S / 8); x += threads) {
        const int r = x / S * 8 + x % 8, c = x / 8 % (S / 8), i = r < z.pad ? r : r - z.pad;
        float v[8] = {};
        if (i < N) load_vec<8>(v, rows + (r < z.pad ? i : N + i) * kLd + 8 * c);
        uint32_t w[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) tc::split3(v[2 * e], v[2 * e + 1], w[0][e], w[1][e], w[2][e]);
        uint8_t *to = images + tc::kmajor_offset16(r, 8 * c, 128, S / 8 * 128);
#pragma unroll
        for (int y = 0; y < 3; ++y)
            *reinterpret_cast<uint4 *>(to + y * z.image) = make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
    }
    // ---- the paths as lists; the nodes by how deep they stand
    for (int i = warp; i < N; i += threads / 32) {
        const unsigned long long path = path_of[i];
        for (int k = lane; k < z.pad; k += 32) {
            if ((path >> k) & 1ull) anc[i * z.pad + __popcll(path & ((1ull << k) - 1))] = static_cast<uint8_t>(k);
            if (k >= __popcll(path)) anc[i * z.pad + k] = path != 0 ? static_cast<uint8_t>(__ffsll(static_cast<long long>(path)) - 1) : 0;
        }
    }
    if (tid < N) {
        const int depth = __popcll(path_of[tid]);
        int before = 0, upto = 0;  // nodes in front of this one; nodes that stand no deeper than tid + 1
        for (int i = 0; i < N; ++i) {
            const int other = __popcll(path_of[i]);
            before += other < depth || (other == depth && i < tid);
            upto += other <= tid;
        }
        by_depth[before] = static_cast<uint8_t>(tid);
        level[tid] = upto;
        if (tid == N - 1) level[N] = N;
    }
    __syncthreads();
    for (int i = warp; i < N; i += threads / 32) {
        const int count = __popcll(path_of[i]);
        if (count == 0) continue;
        float ki[4], qi[4];
        load_vec<4>(ki, rows + i * kLd + 4 * lane);
        load_vec<4>(qi, rows + (N + i) * kLd + 4 * lane);
        for (int k = 0; k < count; k += 4) {
            const uint32_t which = *reinterpret_cast<const uint32_t *>(anc + i * z.pad + k);
            float part[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float ks[4];
                load_vec<4>(ks, rows + ((which >> (8 * m)) & 255u) * kLd + 4 * lane);
                part[2 * m] = lane_dot<4>(ki, ks);
                part[2 * m + 1] = lane_dot<4>(qi, ks);
            }
            const float sum = warp_sum_packed<8>(part, lane);
            const float next = __shfl_xor_sync(FULL_MASK, sum, row_home_lane<8>(1));
#pragma unroll
            for (int m = 0; m < 4; ++m)
                if (lane == row_home_lane<8>(2 * m) && k + m < count)
                    gram[i * N + ((which >> (8 * m)) & 255u)] = make_float2(sum, next);
        }
    }
    const int groups = H / Hk;  // v-heads of this k-head: kh, kh + Hk, ..
    const int at_once = parts > 1 ? 1 : min(L.heads, threads / kMaxNodes);
    for (int h0 = part * at_once; h0 < groups; h0 += parts * at_once) {
        const int heads = min(at_once, groups - h0);
        __syncthreads();  // the products, or the v-heads before, are done with
        auto out_of = [&](int h) { return p.weights + (static_cast<size_t>(n) * H + kh + (h0 + h) * Hk) * z.weights; };
        // (a thread a node and v-head)
        const int hx = tid / kMaxNodes, ix = tid % kMaxNodes;
        if (hx < heads && ix < N) {
            const size_t at = (row0 + ix) * H + kh + (h0 + hx) * Hk;
            const bool here = path_of[ix] != 0;
            g_of[hx][ix] = p.g[at] = here ? gate_of(p, at, kh + (h0 + hx) * Hk) : 0.0f;
            beta_of[hx][ix] = here ? beta_of_node(p, at) : 0.0f;
        }
        __syncthreads();
        if (hx < heads && ix < z.pad) {
            float hi = 0.0f, lo = 0.0f, beta = 0.0f;
            if (ix < N) {
                path_sum(path_of[ix], g_of[hx], hi, lo);
                beta = beta_of[hx][ix];
                hi_of[hx][ix] = hi;
                lo_of[hx][ix] = lo;
            }
            const float decay = expf(hi + lo);
            float *out = reinterpret_cast<float *>(out_of(hx) + z.beta);
            out[ix] = beta;
            out[z.pad + ix] = beta * decay;
            out[2 * z.pad + ix] = decay;
            reinterpret_cast<int *>(out)[3 * z.pad + ix] = ix < N ? __popcll(path_of[ix]) : 0;
        }
        __syncthreads();
        for (int i = warp; i < N; i += threads / 32) {
            const int count = __popcll(path_of[i]);
            for (int k = lane; k < z.pad; k += 32) {
                const int at = i * z.pad + k, s = anc[at];
                const bool on = k < count - 1;  // (the node itself is taken apart)
                const float2 dot = on ? gram[i * N + s] : make_float2(0.0f, 0.0f);
                for (int h = 0; h < heads; ++h) {
                    const float e = on ? expf((hi_of[h][i] - hi_of[h][s]) + (lo_of[h][i] - lo_of[h][s])) : 0.0f;
                    float *list = reinterpret_cast<float *>(dyn + h * L.head);
                    list[at] = on ? -beta_of[h][i] * e * dot.x : 0.0f;
                    list[L.b / 4 + at] = on ? e * dot.y : k == count - 1 ? gram[i * N + i].y : 0.0f;
                    list[L.t / 4 + at] = 0.0f;
                    uint8_t *out = out_of(h);
                    if (k % 4 == 0) *reinterpret_cast<uint32_t *>(out + z.anc + at) = *reinterpret_cast<const uint32_t *>(anc + at);
                }
            }
        }
        __syncthreads();
        // T, kept like A: entry k of row i is the column of the path's k-th node, which is the k-th of
        // the path of every node between the two as well. Rows of one depth need only those above: a
        // lane an entry, 32 / width rows to a warp.
        const int h = warp % heads, part = warp / heads, per = threads / 32 / heads;
        const float *list = reinterpret_cast<const float *>(dyn + h * L.head);
        float *t_of = reinterpret_cast<float *>(dyn + h * L.head + L.t);
        for (int d = 1; d <= N && level[d - 1] < N; ++d) {
            const int bits = d <= 8 ? 3 : d <= 16 ? 4 : 5, k = lane & ((1 << bits) - 1);
            const int end = part < per ? level[d] : 0;
            for (int r = level[d - 1] + (part << (5 - bits)) + (lane >> bits); r < end; r += per << (5 - bits)) {
                const int at = by_depth[r] * z.pad;
                float t[2] = {k == d - 1 ? 1.0f : 0.0f, k + 32 == d - 1 ? 1.0f : 0.0f};
                for (int m0 = 0; m0 < d - 1; m0 += 4) {
                    const uint32_t which = *reinterpret_cast<const uint32_t *>(anc + at + m0);
                    float a[4];
                    load_vec<4>(a, list + at + m0);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float *y = t_of + ((which >> (8 * m)) & 255u) * z.pad + k;
                        t[0] = fmaf(a[m], y[0], t[0]);
                        if (d > 32 && k + 32 < d) t[1] = fmaf(a[m], y[32], t[1]);
                    }
                }
                if (k < d) t_of[at + k] = t[0];
                if (k + 32 < d) t_of[at + k + 32] = t[1];
            }
            __syncthreads();
        }
        // W = B T, and both to their places
        for (int i = warp; i < N; i += threads / 32) {
            const int count = __popcll(path_of[i]), at = i * z.pad;
            if (count == 0) continue;
            for (int k = lane; k < z.pad; k += 32) {
                for (int h = 0; h < heads; ++h) {
                    const float *b_list = reinterpret_cast<const float *>(dyn + h * L.head + L.b);
                    const float *t_list = reinterpret_cast<const float *>(dyn + h * L.head + L.t);
                    float w = 0.0f;
                    for (int m0 = 0; m0 < count; m0 += 4) {
                        const uint32_t which = *reinterpret_cast<const uint32_t *>(anc + at + m0);
                        float b[4];
                        load_vec<4>(b, b_list + at + m0);
#pragma unroll
                        for (int m = 0; m < 4; ++m) w = fmaf(b[m], t_list[((which >> (8 * m)) & 255u) * z.pad + k], w);
                    }
                    reinterpret_cast<float *>(out_of(h))[at + k] = t_list[at + k];
                    reinterpret_cast<float *>(out_of(h) + z.weights_y)[at + k] = w;
                }
            }
        }
    }
}

__global__ void __launch_bounds__(kTcThreads, 2) tree_state_tc_kernel(const __grid_constant__ CUtensorMap state_map,
                                                                      const TreeParams p, int items) {
    constexpr int S = 128;
    extern __shared__ uint8_t dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t state_full, images_full, d_full;
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.n_nodes, Hk = p.n_k_heads, H = p.n_v_heads;
    const TcSizes z(N);
    const TcSmem L(z, N);
    // the next head from `item` on whose sequence has a slot, or `items`
    auto from = [&](int item) {
        for (; item < items; item += gridDim.x) {
            const int slot = p.slots ? p.slots[item / H] : item / H;
            if (slot >= 0 && slot < p.pool) break;
        }
        return min(item, items);
    };
    auto load_state = [&](int item) {
        const int slot = p.slots ? p.slots[item / H] : item / H;
        mbar_arrive_expect_tx(&state_full, S * S * 4);
        tma_load_3d(smem, &state_map, 0, (slot * H + item % H) * S, 0, &state_full);
    };
    auto load_images = [&](int item, int turn) {
        const size_t image = static_cast<size_t>(item / H) * Hk + item % H % Hk;
        mbar_arrive_expect_tx(&images_full, z.images + z.weights);
        bulk_g2s(smem + L.images, p.images + image * z.images, z.images, &images_full);
        bulk_g2s(smem + L.weights + turn * L.turn, p.weights + static_cast<size_t>(item) * z.weights, z.weights, &images_full);
    };
    int item = from(blockIdx.x);
    if (item == items) return;
    if (tid == 0) {
        mbar_init(&state_full, 1);
        mbar_init(&images_full, 1);
        mbar_init(&d_full, 1);
        fence_mbar_init();
        load_state(item);
        load_images(item, 0);
    }
    if (warp == 1) {
        tc::tmem_alloc(&tmem_base, tmem_cols(z));
        tc::tmem_relinquish();  // (another CTA's turn)
    }
    float norm_w[4];
    load_vec<4>(norm_w, p.norm_w + 4 * lane);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int half = warp >> 2, j = (warp & 3) * 32 + lane;  // state row of this thread, which half of its cells
    const int v_count = N * (S / 4);
    const size_t step = static_cast<size_t>(H) * S;
    float *d = reinterpret_cast<float *>(smem + L.d);  // [2N][128]
    bool ok = true;
    for (int turn = 0, phase = 0; item < items && ok; turn ^= 1, phase ^= 1) {
        const int after = from(item + gridDim.x);
        const size_t at0 = (static_cast<size_t>(item / H) * N * H + item % H) * S;
        // the nodes' values, 16 bytes a time, and gates of the warp's first node
        float4 v_part[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int x = tid + y * kTcThreads;
            if (x < v_count) v_part[y] = *reinterpret_cast<const float4 *>(p.v + at0 + x / (S / 4) * step + 4 * (x % (S / 4)));
        }
        float gate[4] = {};
        if (warp < N) load_vec<4>(gate, p.z + at0 + warp * step + 4 * lane);
        // ---- the state's parts
        ok = mbar_wait(&state_full, phase);
        if (ok) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // 32 cells: a 128-byte column
                const int col = 2 * half + b;
                uint32_t w1[16], w2[16], w3[16];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 x = *reinterpret_cast<const float4 *>(smem + col * 16384 + j * 128 + ((c ^ (j & 7)) << 4));
                    tc::split3(x.x, x.y, w1[2 * c], w2[2 * c], w3[2 * c]);
                    tc::split3(x.z, x.w, w1[2 * c + 1], w2[2 * c + 1], w3[2 * c + 1]);
                }
                tc::tmem_st16(lanes + kColA + 16 * col, w1);
                tc::tmem_st16(lanes + kColA + 64 + 16 * col, w2);
                tc::tmem_st16(lanes + kColA + 128 + 16 * col, w3);
            }
            tc::tmem_st_wait();
        }
        ok = mbar_wait(&images_full, phase) && ok;
        tc::fence_before_sync();
        ok = __syncthreads_and(ok);
        tc::fence_after_sync();
        if (ok && warp == 0) {
            if (elect_one()) {
                const uint64_t image = tc::smem_desc(smem + L.images, 128, S / 8 * 128);
                const uint32_t part = z.image >> 4;  // from an image to the next, in 16 bytes
                const uint32_t wide = tc::idesc_bf16(128, 2 * z.rows), one = tc::idesc_bf16(128, z.rows);
#pragma unroll
                for (int x = 0; x < 8; ++x) {  // 16 cells at a time
                    const uint32_t a = tmem + kColA + 8 * x;
                    const uint64_t b = image + 16 * x;
                    tc::mma_bf16_ts(tmem + kColD, a, b, wide, x > 0);
                    tc::mma_bf16_ts(tmem + kColD, a + 64, b, wide, true);
                    tc::mma_bf16_ts(tmem + kColD, a, b + 2 * part, one, true);
                    tc::mma_bf16_ts(tmem + kColD, a + 128, b, one, true);
                }
                tc::mma_commit(&d_full);
                if (L.apart && after < items) load_state(after);
            }
            __syncwarp();
        }
        ok = ok && mbar_wait(&d_full, phase);
        tc::fence_after_sync();
        if (ok) {
            // (the weights' other place was last read before the barrier above)
            if (L.apart && tid == 0 && after < items) load_images(after, turn ^ 1);
            for (int c = 16 * half; c < z.rows; c += 32) {
                uint32_t x[16], y[16];
                tc::tmem_ld16_nowait(lanes + kColD + c, x);
                tc::tmem_ld16_nowait(lanes + kColD + z.rows + c, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = c + e, i = r < z.pad ? r : r - z.pad;
                    if (i < N) d[(r < z.pad ? i : N + i) * S + j] = __uint_as_float(x[e]) + __uint_as_float(y[e]);
                }
            }
        }
        tc::fence_before_sync();
        ok = __syncthreads_and(ok);
        tc::fence_after_sync();
        if (!ok) break;  // (nothing of this head is written)
        // ---- R over the products with k
        const uint8_t *w = smem + L.weights + turn * L.turn;
        const float *weights_u = reinterpret_cast<const float *>(w), *weights_y = reinterpret_cast<const float *>(w + z.weights_y);
        const float *beta = reinterpret_cast<const float *>(w + z.beta);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int x = tid + y * kTcThreads, i = x / (S / 4);
            if (x >= v_count) break;
            float4 r = *reinterpret_cast<const float4 *>(d + 4 * x);
            const float b = beta[i], bd = -beta[z.pad + i];
            r = make_float4(fmaf(bd, r.x, b * v_part[y].x), fmaf(bd, r.y, b * v_part[y].y),
                            fmaf(bd, r.z, b * v_part[y].z), fmaf(bd, r.w, b * v_part[y].w));
            *reinterpret_cast<float4 *>(d + 4 * x) = r;
        }
        __syncthreads();
        // ---- u, y and the gated norm, a warp a node: the lane's four channels
        for (int i = warp; i < N; i += kTcThreads / 32) {
            const float *wu = weights_u + i * z.pad, *wy = weights_y + i * z.pad;
            const uint32_t *which = reinterpret_cast<const uint32_t *>(w + z.anc + i * z.pad);
            const int count = reinterpret_cast<const int *>(beta)[3 * z.pad + i];  // (0: no node)
            float u[4] = {}, y[4] = {}, next_gate[4] = {};
            if (i + kTcThreads / 32 < N) load_vec<4>(next_gate, p.z + at0 + (i + kTcThreads / 32) * step + 4 * lane);
            if (count > 0) {
                load_vec<4>(y, d + (N + i) * S + 4 * lane);
                const float decay = beta[2 * z.pad + i];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= decay;
                for (int k = 0; k < count; k += 4) {
                    const uint32_t a = which[k / 4];
                    float us[4], ys[4];
                    load_vec<4>(us, wu + k);
                    load_vec<4>(ys, wy + k);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        float r[4];
                        load_vec<4>(r, d + ((a >> (8 * m)) & 255u) * S + 4 * lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u[e] = fmaf(us[m], r[e], u[e]);
                            y[e] = fmaf(ys[m], r[e], y[e]);
                        }
                    }
                }
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] *= p.scale;
                    ss = __fmaf_rn(y[e], y[e], ss);
                }
                ss = warp_allsum(ss);
                const float inv_rms = 1.0f / sqrtf(ss / static_cast<float>(S) + p.norm_eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = y[e] * inv_rms * norm_w[e] * silu(gate[e]);
            }
            store_vec<4>(p.u + at0 + i * step + 4 * lane, u);
            store_vec<4>(p.out + at0 + i * step + 4 * lane, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) gate[e] = next_gate[e];
        }
        if (!L.apart) {  // D's and the weights' places are the next head's
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0 && after < items) {
                load_state(after);
                load_images(after, 0);
            }
        }
        item = after;
    }
    if (!ok) {
        // (no copy may still be on its way into a CTA that has ended)
        mbar_wait(&d_full, 0);
        mbar_wait(&d_full, 1);
        mbar_wait(&state_full, 0);
        mbar_wait(&state_full, 1);
        mbar_wait(&images_full, 0);
        mbar_wait(&images_full, 1);
        if (tid == 0) atomicOr(p.watchdog, WD_STATE_COPY);
    }
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, tmem_cols(z));
    }
}

// ------------------------------------------------------------------ the gated norm

// One warp per head row, as gdn_gated_norm; rows of nodes that are not there are zeros.
constexpr int kNormThreads = 256;

template <int E>
__global__ void __launch_bounds__(kNormThreads) tree_norm_kernel(const TreeParams p, long long rows) {
    constexpr int D = 32 * E;
    const long long row = blockIdx.x * static_cast<long long>(kNormThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    float yv[E], zv[E], wv[E];
    load_vec<E>(yv, p.out + row * D + lane * E);
    load_vec<E>(zv, p.z + row * D + lane * E);
    load_vec<E>(wv, p.norm_w + lane * E);
    const long long node = row / p.n_v_heads;
    if (p.slots) {
        const int slot = p.slots[node / p.n_nodes];
        if (slot < 0 || slot >= p.pool) return;
    }
    if (p.paths[node] == 0) return;  // (y is zeros)
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss = __fmaf_rn(yv[e], yv[e], ss);
    ss = warp_allsum(ss);
    const float inv_rms = 1.0f / sqrtf(ss / static_cast<float>(D) + p.norm_eps);
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = yv[e] * inv_rms * wv[e] * silu(zv[e]);
    store_vec<E>(p.out + row * D + lane * E, o);
}

// ------------------------------------------------------------------ the commit

struct CommitParams {
    const float *qkv;
    float *conv_state, *state;
    const int32_t *parents, *accepted, *slots;
    int n_seqs, n_nodes, n_k_heads, n_v_heads, conv_dim, taps, pool;
    int32_t *err_count;
    const float *k, *g, *u;
    unsigned *watchdog;
};

// S <- e^{G_l} S0 + sum_{s on the path to l} e^{G_l - G_s} k_s u_s^T: the state in and out once bounds
// it. Work is dealt out in blocks of 16 KB of state rows, a contiguous range to each of the first
// `state_ctas` CTAs; a block's rows are fetched by a bulk copy, and its path's k, u and g into
// registers, while the block before is worked on. 64 sequences, 32 heads of 128: 60 us, 0.71 of the
// copy rate (a CTA per 64 rows, each with its lookups, path and loads behind one another: 65). The
// other CTAs roll the conv history, a share of a sequence's channels each.
constexpr int kCommitThreads = 256;
constexpr int kCommitNodes = 16;
constexpr int kCommitChannels = kCommitThreads * 4;
constexpr int kCommitCtas = 4;  // an SM (three, with room for those of the conv history: 65 us)

template <int E>
struct CommitSmem {
    static constexpr int S = 32 * E;
    static constexpr int kRows = S == 64 ? 64 : 32;  // of a block
    static constexpr int kBlock = kRows * S;
    static constexpr int kBytes = (2 * kBlock + kCommitNodes * (S + 2 * kRows)) * 4;  // rows, k, u of two blocks
};

template <int E>
__global__ void __launch_bounds__(kCommitThreads, E == 8 ? 2 : 4) tree_commit_kernel(const CommitParams p, int state_ctas) {
    using L = CommitSmem<E>;
    constexpr int S = L::S, kRows = L::kRows, R = kRows / 8;  // R rows a warp
    constexpr int kPerHead = S / kRows;
    constexpr int kLoadsK = (kCommitNodes * S / 4 + kCommitThreads - 1) / kCommitThreads;
    constexpr int kLoadsU = (kCommitNodes * kRows / 4 + kCommitThreads - 1) / kCommitThreads;
    extern __shared__ __align__(128) float dyn_floats[];
    float *const ks = dyn_floats + 2 * L::kBlock, *const us_of = ks + kCommitNodes * S;
    __shared__ __align__(8) uint64_t full[2];
    __shared__ unsigned long long path_of[kMaxNodes];
    __shared__ int up[kMaxNodes], walk[kMaxNodes];
    __shared__ float g_of[kMaxNodes], weight[kMaxNodes + 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.n_nodes, Hk = p.n_k_heads, H = p.n_v_heads;
    // The path to the accepted node of sequence n as `walk`, by the whole CTA; its length, 0 if nothing is
    // accepted or the node is not there.
    auto walk_of = [&](int n, bool counts) {
        const int slot = p.slots ? p.slots[n] : n, m = p.accepted[n];
        const bool range = slot >= 0 && slot < p.pool && m >= 0 && m <= N;
        if (range && m == 0) return 0;
        __syncthreads();  // (of the sequence before)
        if (warp == 0 && range) {
            unsigned long long paths[2];
            tree_paths(p.parents + static_cast<size_t>(n) * N, N, paths, path_of, up);
        }
        __syncthreads();
        const unsigned long long path = range ? path_of[m - 1] : 0;
        if (path == 0 && counts && tid == 0 && p.err_count) atomicAdd(p.err_count, 1);
        if (tid < kMaxNodes && ((path >> tid) & 1ull)) walk[__popcll(path & ((1ull << tid) - 1))] = tid;
        __syncthreads();
        return __popcll(path);
    };
    if (static_cast<int>(blockIdx.x) >= state_ctas) {
        // ---- the conv history
        const int shares = (p.conv_dim + kCommitChannels - 1) / kCommitChannels;
        const int n = (blockIdx.x - state_ctas) / shares, share = (blockIdx.x - state_ctas) % shares;
        const int len = walk_of(n, share == 0);
        if (len == 0) return;
        const int slot = p.slots ? p.slots[n] : n;
        for (int c = share * kCommitChannels + tid; c < min(p.conv_dim, (share + 1) * kCommitChannels); c += kCommitThreads) {
            float *hs = p.conv_state + (static_cast<size_t>(slot) * p.conv_dim + c) * p.taps;
            // entry t is the path's input len - taps + t, or the old entry len + t before those:
            // entries move down only
            for (int t = 0; t < p.taps; ++t) {
                const int at = len - p.taps + t;
                hs[t] = at >= 0 ? p.qkv[(static_cast<size_t>(n) * N + walk[at]) * p.conv_dim + c] : hs[len + t];
            }
        }
        return;
    }
    // ---- the states
    const int blocks = H * kPerHead;  // of a sequence
    const long long all = static_cast<long long>(p.n_seqs) * blocks;
    const long long first = all * blockIdx.x / state_ctas, last = all * (blockIdx.x + 1) / state_ctas;
    // a sequence's place, and block of it; sequences without a state to change (as far as that shows
    // without their paths) are passed over
    struct Place {
        int n, r, left;  // left: blocks of the range from here on
        float *rows;
    };
    auto settle = [&](Place &at) {
        while (at.left > 0) {
            if (at.r == blocks) {
                at.r = 0;
                ++at.n;
            }
            const int slot = p.slots ? p.slots[at.n] : at.n, m = p.accepted[at.n];
            if (slot >= 0 && slot < p.pool && m >= 1 && m <= N) {
                at.rows = p.state + (static_cast<size_t>(slot) * blocks + at.r) * L::kBlock;
                return;
            }
            at.left -= blocks - at.r;
            at.r = blocks;
        }
    };
    auto behind = [&](Place at) {
        ++at.r;
        --at.left;
        if (at.left > 0 && at.r < blocks) at.rows += L::kBlock;
        else settle(at);
        return at;
    };
    Place b{static_cast<int>(first / blocks), static_cast<int>(first % blocks), static_cast<int>(last - first), nullptr};
    settle(b);
    if (b.left <= 0) return;
    if (tid == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        fence_mbar_init();
    }
    auto fetch = [&](const Place &block, int turn) {
        mbar_arrive_expect_tx(&full[turn], L::kBlock * 4);
        bulk_g2s(dyn_floats + turn * L::kBlock, block.rows, L::kBlock * 4, &full[turn]);
    };
    if (tid == 0) fetch(b, 0);
    int n = -1, len = 0, head = -1;  // head: whose k, weights and decay lie in shared memory
    float g_next = 0.0f;
    float4 k_next[kLoadsK], u_next[kLoadsU];
    // the first nodes' u of a block of this sequence and, of another head, k and g
    auto prefetch = [&](const Place &block) {
        const size_t row0 = static_cast<size_t>(block.n) * N;
        const int vh = block.r / kPerHead, j0 = block.r % kPerHead * kRows;
        const int count = min(len, kCommitNodes);
#pragma unroll
        for (int y = 0; y < kLoadsU; ++y) {
            const int x = tid + y * kCommitThreads;
            if (x < count * (kRows / 4))
                u_next[y] = *reinterpret_cast<const float4 *>(p.u + ((row0 + walk[x / (kRows / 4)]) * H + vh) * S + j0 + 4 * (x % (kRows / 4)));
        }
        if (vh == head) return;
        if (tid < N) g_next = p.g[(row0 + tid) * H + vh];
#pragma unroll
        for (int y = 0; y < kLoadsK; ++y) {
            const int x = tid + y * kCommitThreads;
            if (x < count * (S / 4))
                k_next[y] = *reinterpret_cast<const float4 *>(p.k + ((row0 + walk[x / (S / 4)]) * Hk + vh % Hk) * S + 4 * (x % (S / 4)));
        }
    };
    bool ok = true;
    uint32_t phase = 0;  // bit t: of full[t]
    for (int turn = 0; b.left > 0; turn ^= 1) {
        if (b.n != n) {
            n = b.n;
            head = -1;
            len = walk_of(n, false);  // (counted with the conv history)
            if (len > 0) prefetch(b);
        }
        const Place after = behind(b);
        float *const us = us_of + turn * kCommitNodes * kRows;
        if (len > 0) {
#pragma unroll
            for (int y = 0; y < kLoadsU; ++y) {
                const int x = tid + y * kCommitThreads;
                if (x < min(len, kCommitNodes) * (kRows / 4)) *reinterpret_cast<float4 *>(us + 4 * x) = u_next[y];
            }
            if (b.r / kPerHead != head) {
                head = len <= kCommitNodes ? b.r / kPerHead : -1;  // (a longer path's k pass through)
                __syncthreads();  // the head before is done with
                if (tid < N) g_of[tid] = g_next;
#pragma unroll
                for (int y = 0; y < kLoadsK; ++y) {
                    const int x = tid + y * kCommitThreads;
                    if (x < min(len, kCommitNodes) * (S / 4)) *reinterpret_cast<float4 *>(ks + 4 * x) = k_next[y];
                }
                __syncthreads();
                // weight[i]: the decay behind node walk[i]; weight[len]: of the whole path
                if (tid <= len) {
                    float sum = 0.0f;
                    for (int i = len - 1; i > (tid == len ? -1 : tid); --i) sum += g_of[walk[i]];
                    weight[tid] = expf(sum);
                }
            }
            if (after.left > 0 && after.n == n) prefetch(after);
        }
        ok = mbar_wait(&full[turn], (phase >> turn) & 1u);
        phase ^= 1u << turn;
        ok = __syncthreads_and(ok);
        if (!ok) break;  // (this block keeps its state)
        if (tid == 0 && after.left > 0) fetch(after, turn ^ 1);  // (its place has been read by all)
        if (len > 0) {
            const float *mine = dyn_floats + turn * L::kBlock + warp * R * S + E * lane;
            const float decay = weight[len];
            float x[R][E];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_vec<E>(x[r], mine + r * S);
#pragma unroll
                for (int e = 0; e < E; ++e) x[r][e] *= decay;
            }
            const size_t row0 = static_cast<size_t>(n) * N;
            const int vh = b.r / kPerHead, j0 = b.r % kPerHead * kRows;
            for (int a = 0; a < len; a += kCommitNodes) {
                const int count = min(kCommitNodes, len - a);
                if (a > 0) {
                    __syncthreads();
                    for (int y = tid; y < count * (S / 4); y += kCommitThreads)
                        *reinterpret_cast<float4 *>(ks + 4 * y) =
                            *reinterpret_cast<const float4 *>(p.k + ((row0 + walk[a + y / (S / 4)]) * Hk + vh % Hk) * S + 4 * (y % (S / 4)));
                    for (int y = tid; y < count * (kRows / 4); y += kCommitThreads)
                        *reinterpret_cast<float4 *>(us + 4 * y) =
                            *reinterpret_cast<const float4 *>(p.u + ((row0 + walk[a + y / (kRows / 4)]) * H + vh) * S + j0 + 4 * (y % (kRows / 4)));
                    __syncthreads();
                }
                for (int y = 0; y < count; ++y) {
                    float kc[E], uc[R];
                    load_vec<E>(kc, ks + y * S + E * lane);
                    load_vec<R>(uc, us + y * kRows + warp * R);
                    const float w = weight[a + y];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float uw = uc[r] * w;
#pragma unroll
                        for (int e = 0; e < E; ++e) x[r][e] = fmaf(kc[e], uw, x[r][e]);
                    }
                }
            }
            float *to = b.rows + warp * R * S + E * lane;
#pragma unroll
            for (int r = 0; r < R; ++r) store_vec<E>(to + r * S, x[r]);
        }
        b = after;
    }
    if (!ok) {
        // (no copy may still be on its way into a CTA that has ended)
        mbar_wait(&full[0], 0);
        mbar_wait(&full[0], 1);
        mbar_wait(&full[1], 0);
        mbar_wait(&full[1], 1);
        if (tid == 0) atomicOr(p.watchdog, WD_STATE_COPY);
    }
}

// ------------------------------------------------------------------ host side

template <int E, int K>
gdn_status launch_conv(const TreeParams &p, int n_seqs, cudaStream_t s) {
    const int slices = 2 * p.n_k_heads + p.n_v_heads;
    const dim3 grid((slices + kConvWarps - 1) / kConvWarps + 1, (p.n_nodes + kConvNodes - 1) / kConvNodes, n_seqs);
    tree_conv_kernel<E, K><<<grid, 32 * kConvWarps, 0, s>>>(p);
    return launch_status();
}

// States of 128, on the tensor cores.
template <int K>
gdn_status launch_tc(const TreeParams &p, int n_seqs, cudaStream_t s) {
    CUtensorMap map;
    GDN_TRY(encode_blocks_map(&map, p.state, GDN_F32, 128, static_cast<uint64_t>(p.pool) * p.n_v_heads * 128, 512, 128, 4));
    static std::atomic<unsigned long long> allowed{0}, prepare_allowed{0};
    GDN_TRY(allow_smem(tree_prepare_kernel<K>, kPrepSmem, prepare_allowed));
    GDN_TRY(allow_smem(tree_state_tc_kernel, TcSmem::kMost + 1024, allowed));
    // all CTAs that prepare at once, and as many warps as that leaves
    const int groups = p.n_v_heads / p.n_k_heads;
    const int parts = static_cast<long long>(n_seqs) * p.n_v_heads <= 152 ? groups : 1;  // (few trees: a CTA a v-head)
    const long long prepares = static_cast<long long>(n_seqs) * p.n_k_heads * parts;
    const int threads = prepares <= 152 ? kPrepThreads : prepares <= 4 * 152 ? kPrepThreads / 2 : kPrepThreads / 4, warps = threads / 32;
    const int head_groups = (p.n_v_heads + warps - 1) / warps, node_blocks = (p.n_nodes + kConvNodes - 1) / kConvNodes;
    const long long others = static_cast<long long>(n_seqs) * head_groups * node_blocks;
    if (prepares + others > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    tree_prepare_kernel<K><<<static_cast<unsigned>(prepares + others), threads, PrepSmem(p.n_nodes).bytes, s>>>(
        p, static_cast<int>(prepares), parts);
    GDN_TRY(launch_status());
    const TcSizes z(p.n_nodes);
    const uint32_t smem = TcSmem(z, p.n_nodes).bytes + 1024;
    const int items = n_seqs * p.n_v_heads, wide = 152 * (tmem_cols(z) <= 256 && smem <= 113 * 1024 ? 2 : 1);
    tree_state_tc_kernel<<<items < wide ? items : wide, kTcThreads, smem, s>>>(map, p, items);
    return launch_status();
}

// Other states, on the FP32 pipes.
template <int E, int K>
gdn_status launch_fp32(const TreeParams &p, int n_seqs, cudaStream_t s) {
    GDN_TRY((launch_conv<E, K>(p, n_seqs, s)));
    const size_t keys = static_cast<size_t>(p.n_nodes) * 32 * E * sizeof(float);
    static std::atomic<unsigned long long> gram_allowed{0};
    GDN_TRY(allow_smem(tree_gram_kernel<E>, kMaxNodes * 32 * E * static_cast<int>(sizeof(float)), gram_allowed));
    tree_gram_kernel<E><<<dim3(p.n_k_heads, n_seqs), 32 * kGramWarps, keys, s>>>(p);
    GDN_TRY(launch_status());
    using L = StateSmem<E>;
    // (the most that any tree takes: a limit of this call's own would be under another thread's larger one)
    static std::atomic<unsigned long long> state_allowed{0};
    GDN_TRY(allow_smem(tree_state_kernel<E>, static_cast<int>(L::bytes(kMaxNodes)), state_allowed));
    tree_state_kernel<E><<<dim3(L::S / L::JB, p.n_v_heads, n_seqs), kStateThreads, L::bytes(p.n_nodes), s>>>(p);
    GDN_TRY(launch_status());
    const long long rows = static_cast<long long>(n_seqs) * p.n_nodes * p.n_v_heads;
    tree_norm_kernel<E><<<static_cast<unsigned>((rows + kNormThreads / 32 - 1) / (kNormThreads / 32)),
                          kNormThreads, 0, s>>>(p, rows);
    return launch_status();
}

template <int E, int K>
gdn_status launch_block_of(const TreeParams &p, int n_seqs, cudaStream_t s) {
    if constexpr (E == 4) return launch_tc<K>(p, n_seqs, s);
    else return launch_fp32<E, K>(p, n_seqs, s);
}

template <int E>
gdn_status launch_block(const TreeParams &p, int n_seqs, int conv_kernel, cudaStream_t s) {
    switch (conv_kernel) {
        case 2: return launch_block_of<E, 2>(p, n_seqs, s);
        case 3: return launch_block_of<E, 3>(p, n_seqs, s);
        case 4: return launch_block_of<E, 4>(p, n_seqs, s);
        case 5: return launch_block_of<E, 5>(p, n_seqs, s);
        case 6: return launch_block_of<E, 6>(p, n_seqs, s);
        case 7: return launch_block_of<E, 7>(p, n_seqs, s);
        default: return launch_block_of<E, 8>(p, n_seqs, s);
    }
}

template <int E>
gdn_status launch_commit(const CommitParams &p, cudaStream_t s) {
    using L = CommitSmem<E>;
    const long long blocks = static_cast<long long>(p.n_seqs) * p.n_v_heads * (L::S / L::kRows);
    const long long conv = static_cast<long long>(p.n_seqs) * ((p.conv_dim + kCommitChannels - 1) / kCommitChannels);
    if (blocks > 0x7fffffffLL || conv > 0x7fff0000LL) return GDN_ERR_UNSUPPORTED;
    constexpr int kCtas = 152 * (E == 8 ? 2 : kCommitCtas);
    const int state_ctas = static_cast<int>(blocks < kCtas ? blocks : kCtas);
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(tree_commit_kernel<E>, L::kBytes, allowed));
    tree_commit_kernel<E><<<static_cast<unsigned>(state_ctas + conv), kCommitThreads, L::kBytes, s>>>(p, state_ctas);
    return launch_status();
}

// Sizes that both calls share. (The grids' y and z are 16-bit, rows of heads 32-bit.)
gdn_status check_sizes(int n_seqs, int n_nodes, int n_k_heads, int n_v_heads, int state_size, int conv_kernel) {
    if (conv_kernel < 2 || conv_kernel > 8) return GDN_ERR_SHAPE;
    GDN_TRY(check_heads(n_k_heads, n_v_heads, state_size));
    if (n_seqs > 65535 || n_v_heads > 65535 ||
        static_cast<long long>(n_seqs) * n_nodes * n_v_heads > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

bool valid_sizes(int n_seqs, int n_nodes, int n_k_heads, int n_v_heads, int state_size) {
    return n_seqs >= 0 && n_nodes >= 1 && n_nodes <= kMaxNodes &&
           check_heads(n_k_heads, n_v_heads, state_size) == GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_block_tree_tape_size(int n_seqs, int n_nodes, int n_k_heads, int n_v_heads, int state_size) {
    if (!valid_sizes(n_seqs, n_nodes, n_k_heads, n_v_heads, state_size)) return 0;
    return Tape(static_cast<size_t>(n_seqs) * n_nodes, n_k_heads, n_v_heads, state_size).floats * sizeof(float);
}

size_t gdn_block_tree_workspace_size(int n_seqs, int n_nodes, int n_k_heads, int n_v_heads, int state_size) {
    if (!valid_sizes(n_seqs, n_nodes, n_k_heads, n_v_heads, state_size)) return 0;
    return Scratch(static_cast<size_t>(n_seqs) * n_nodes, n_nodes, n_k_heads, n_v_heads, state_size).floats * sizeof(float);
}

gdn_status gdn_block_tree(const float *qkv, const float *conv_w, const float *conv_state,
                          const float *alpha, const float *b, const float *dt, const float *a,
                          const float *z, const float *norm_w, const float *state, float *out,
                          const int32_t *parents, int n_seqs, int n_nodes, int n_k_heads,
                          int n_v_heads, int state_size, int conv_kernel, float scale, float l2_eps,
                          float norm_eps, const int32_t *slots, int pool, int32_t *err_count,
                          void *tape, size_t tape_bytes, void *workspace, size_t workspace_bytes,
                          gdn_stream_t stream) {
    if (!qkv || !conv_w || !conv_state || !alpha || !b || !dt || !a || !z || !norm_w || !state || !out)
        return GDN_ERR_NULL;
    GDN_TRY(check_tree(parents, n_seqs, n_nodes));
    GDN_TRY(check_sizes(n_seqs, n_nodes, n_k_heads, n_v_heads, state_size, conv_kernel));
    GDN_TRY(check_pool(n_seqs, slots, pool));
    // (rows of a tensor map are counted in 32 bits; so many are a terabyte)
    if (state_size == 128 && static_cast<long long>(pool) * n_v_heads * 128 > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    if (!aligned16(qkv) || !aligned16(conv_w) || !aligned16(conv_state) || !aligned16(state) ||
        !aligned16(z) || !aligned16(out) || !aligned16(norm_w))
        return GDN_ERR_ALIGN;
    if (n_seqs == 0) return GDN_OK;
    if (!tape || !workspace) return GDN_ERR_NULL;
    if (!aligned16(tape) || !aligned16(workspace)) return GDN_ERR_ALIGN;
    const size_t rows = static_cast<size_t>(n_seqs) * n_nodes;
    const Tape T(rows, n_k_heads, n_v_heads, state_size);
    const Scratch W(rows, n_nodes, n_k_heads, n_v_heads, state_size);
    if (tape_bytes < T.floats * sizeof(float) || workspace_bytes < W.floats * sizeof(float))
        return GDN_ERR_SHAPE;
    float *t = static_cast<float *>(tape), *w = static_cast<float *>(workspace);
    const TreeParams p{qkv, conv_w, conv_state, alpha, b, dt, a, z, norm_w, state, out, parents,
                       slots, n_nodes, n_k_heads, n_v_heads, pool, scale, l2_eps, norm_eps,
                       err_count, t + T.k, t + T.g, t + T.u, w + W.v, w + W.q, w + W.beta, w + W.gram,
                       reinterpret_cast<uint8_t *>(w + W.images), reinterpret_cast<uint8_t *>(w + W.weights),
                       reinterpret_cast<unsigned long long *>(w + W.paths), watchdog_block()};
    if (p.watchdog == nullptr) return GDN_ERR_LAUNCH;
    const cudaStream_t s = as_cuda(stream);
    switch (state_size) {
        case 32: return launch_block<1>(p, n_seqs, conv_kernel, s);
        case 64: return launch_block<2>(p, n_seqs, conv_kernel, s);
        case 128: return launch_block<4>(p, n_seqs, conv_kernel, s);
        default: return launch_block<8>(p, n_seqs, conv_kernel, s);
    }
}

gdn_status gdn_block_tree_commit(const float *qkv, float *conv_state, float *state,
                                 const int32_t *parents, const int32_t *accepted, int n_seqs,
                                 int n_nodes, int n_k_heads, int n_v_heads, int state_size,
                                 int conv_kernel, const int32_t *slots, int pool, int32_t *err_count,
                                 const void *tape, size_t tape_bytes, gdn_stream_t stream) {
    if (!qkv || !conv_state || !state || !accepted) return GDN_ERR_NULL;
    GDN_TRY(check_tree(parents, n_seqs, n_nodes));
    GDN_TRY(check_sizes(n_seqs, n_nodes, n_k_heads, n_v_heads, state_size, conv_kernel));
    GDN_TRY(check_pool(n_seqs, slots, pool));
    if (!aligned16(state)) return GDN_ERR_ALIGN;
    if (n_seqs == 0) return GDN_OK;
    if (!tape) return GDN_ERR_NULL;
    if (!aligned16(tape)) return GDN_ERR_ALIGN;
    const Tape T(static_cast<size_t>(n_seqs) * n_nodes, n_k_heads, n_v_heads, state_size);
    if (tape_bytes < T.floats * sizeof(float)) return GDN_ERR_SHAPE;
    const float *t = static_cast<const float *>(tape);
    const CommitParams p{qkv, conv_state, state, parents, accepted, slots, n_seqs, n_nodes, n_k_heads,
                         n_v_heads, (2 * n_k_heads + n_v_heads) * state_size, conv_kernel - 1, pool,
                         err_count, t + T.k, t + T.g, t + T.u, watchdog_block()};
    if (p.watchdog == nullptr) return GDN_ERR_LAUNCH;
    const cudaStream_t s = as_cuda(stream);
    switch (state_size) {
        case 32: return launch_commit<1>(p, s);
        case 64: return launch_commit<2>(p, s);
        case 128: return launch_commit<4>(p, s);
        default: return launch_commit<8>(p, s);
    }
}

}  // extern "C"
