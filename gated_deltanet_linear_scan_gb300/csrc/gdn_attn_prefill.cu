// gdn_attn_prefill.cu -- attention of a ragged batch of prompts, or chunks of prompts, over
// the paged key/value cache (sm_103a).
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = e^{scale q_i.k_j - m_i} over the keys i sees
//
// All query heads of a key head share its keys, so a tile of rows is (tokens x heads of one
// key head): the keys are read once for all of them, and a tile spans few positions, which
// keeps the work wasted at the causal diagonal and at the window's edge small.
#include "gdn_paged.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

__device__ unsigned g_watchdog_attn_prefill;

struct PrefillParams {
    PagedCache cache;
    AttnMask mask;
    SeqMap seqs;
    const void *q, *k_pages, *v_pages;
    void *out;
    int n_seqs, n_q_heads, group, q_stride;
    int heads_per_tile, tokens_per_tile, head_groups;
    float scale_log2;
    int32_t *err_count;
};

// The rows of one CTA: tokens token0 .. of sequence n, heads head0 .. .
struct RowTile {
    int slot, len;        // of the sequence, in the cache
    int new_tokens;       // of the sequence in this call
    size_t row0;          // packed row of the sequence's first new token
    int token0, tokens;   // of this tile
    int kvh, head0, heads;
    int p_first, p_last;  // positions of the tile's first and last token
};

// Finds the tile of this CTA (blockIdx.x: a tile slot, blockIdx.y: key head and head group);
// false when it has none. Called by whole warps. Also counts the skipped sequences once.
__device__ __forceinline__ bool find_tile(const PrefillParams &p, RowTile &t) {
    const int x = blockIdx.x;
    if (blockIdx.y == 0 && x < p.n_seqs && threadIdx.x == 0 && p.err_count) {
        size_t r0;
        int m, slot, len;
        if (!p.seqs.range(x, r0, m) || !p.cache.lookup(x, slot, len)) atomicAdd(p.err_count, 1);
    }
    const int n = warp_seq_of_slot(p.seqs.cu, p.n_seqs, p.tokens_per_tile, x);
    if (n < 0 || !p.seqs.range(n, t.row0, t.new_tokens) || !p.cache.lookup(n, t.slot, t.len))
        return false;
    const int block = x - (static_cast<int>(t.row0) / p.tokens_per_tile + n);
    t.token0 = block * p.tokens_per_tile;
    if (t.token0 >= t.new_tokens) return false;
    t.tokens = min(p.tokens_per_tile, t.new_tokens - t.token0);
    t.kvh = blockIdx.y / p.head_groups;
    const int hg = blockIdx.y % p.head_groups;
    t.head0 = t.kvh * p.group + hg * p.heads_per_tile;
    t.heads = min(p.heads_per_tile, p.group - hg * p.heads_per_tile);
    t.p_first = t.len - t.new_tokens + t.token0;
    t.p_last = t.p_first + t.tokens - 1;
    return true;
}

// ------------------------------------------------------------------ on the FP32 pipes

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = Elem<__half>::unpack(v.x), b = Elem<__half>::unpack(v.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = Elem<__nv_bfloat16>::unpack(v.x), b = Elem<__nv_bfloat16>::unpack(v.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
}

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 32;

template <int D>
constexpr int simt_smem() {
    return ((kSimtRows + 2 * kSimtKeys) * (D + 4) + kSimtRows * (kSimtKeys + 4)) * 4;
}

// 64 rows by 32 keys a step, everything in fp32: a thread holds 4 rows x 4 keys of S (8
// lanes span the keys) and 4 rows x D/8 columns of O. Rows of shared memory are padded by 16
// bytes, so the 8 lanes of a quarter-warp read different banks.
template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads)
attn_prefill_simt_kernel(const PrefillParams p) {
    constexpr int P = D + 4, PP = kSimtKeys + 4;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + kSimtRows * P, *sv = sk + kSimtKeys * P, *sp = sv + kSimtKeys * P;
    RowTile t;
    if (!find_tile(p, t)) return;
    const int tid = threadIdx.x, tx = tid & 7, ty = tid >> 3;
    const T *q = static_cast<const T *>(p.q);
    const T *k_pages = static_cast<const T *>(p.k_pages), *v_pages = static_cast<const T *>(p.v_pages);
    const int ps = 1 << p.cache.log2_ps;

    for (int x = tid; x < kSimtRows * (D / 4); x += kSimtThreads) {
        const int r = x / (D / 4), c = (x % (D / 4)) * 4;
        const int tok = r / p.heads_per_tile, h = r % p.heads_per_tile;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tok < t.tokens && h < t.heads)
            v = load4(q + (t.row0 + t.token0 + tok) * p.q_stride + static_cast<size_t>(t.head0 + h) * D + c);
        *reinterpret_cast<float4 *>(sq + r * P + c) = v;
    }
    float o[4][D / 8], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) o[i][c] = 0.0f;
    }
    const TileWalk walk = walk_tiles<kSimtKeys>(p.mask, t.p_first, t.p_last);
    for (int w = 0; w < walk.count; ++w) {
        const int key0 = walk.tile(w) * kSimtKeys;
        __syncthreads();  // the previous tile has been read
        for (int x = tid; x < kSimtKeys * (D / 4); x += kSimtThreads) {
            const int i = x / (D / 4), c = (x % (D / 4)) * 4, key = key0 + i;
            float4 kv = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vv = kv;
            // keys no row of the tile sees are not looked up: their pages may be gone, and
            // whatever a page holds past the length must not reach the sums
            if (key <= t.p_last && (t.p_first - key < p.mask.window || key < p.mask.sinks)) {
                const int page = p.cache.page_of(t.slot, key);
                if (p.cache.page_ok(page)) {
                    const size_t at =
                        ((static_cast<size_t>(page) * p.cache.n_kv_heads + t.kvh) * ps + (key & (ps - 1))) * D + c;
                    kv = load4(k_pages + at);
                    vv = load4(v_pages + at);
                } else if (c == 0 && blockIdx.y == 0 && p.err_count && (key & (ps - 1)) == 0) {
                    atomicAdd(p.err_count, 1);
                }
            }
            *reinterpret_cast<float4 *>(sk + i * P + c) = kv;
            *reinterpret_cast<float4 *>(sv + i * P + c) = vv;
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + i) * P + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(sk + (tx + 8 * j) * P + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                    s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                    s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                    s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pos = t.p_first + (ty * 4 + i) / p.heads_per_tile;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = key0 + tx + 8 * j;
                bool ok = p.mask.sees(pos, key) && key <= t.p_last;
                if (ok) ok = p.cache.page_ok(p.cache.page_of(t.slot, key));
                s[i][j] = ok ? s[i][j] * p.scale_log2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, d));
            const float old = m[i];
            m[i] = fmaxf(m[i], top);
            const float base = m[i] == -INFINITY ? 0.0f : m[i];
            const float corr = fast_exp2(old - base);
            l[i] *= corr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w_ = fast_exp2(s[i][j] - base);
                l[i] += w_;
                sp[(ty * 4 + i) * PP + tx + 8 * j] = w_;
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c) o[i][c] *= corr;
        }
        __syncwarp();  // P's rows are read by the warp that wrote them
#pragma unroll 2
        for (int j = 0; j < kSimtKeys; j += 4) {
            float4 w4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w4[i] = *reinterpret_cast<const float4 *>(sp + (ty * 4 + i) * PP + j);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(sv + (j + jj) * P + tx * 4 + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float wi = jj == 0 ? w4[i].x : jj == 1 ? w4[i].y : jj == 2 ? w4[i].z : w4[i].w;
                        o[i][4 * c] = fmaf(wi, v.x, o[i][4 * c]);
                        o[i][4 * c + 1] = fmaf(wi, v.y, o[i][4 * c + 1]);
                        o[i][4 * c + 2] = fmaf(wi, v.z, o[i][4 * c + 2]);
                        o[i][4 * c + 3] = fmaf(wi, v.w, o[i][4 * c + 3]);
                    }
                }
            }
        }
    }
    T *out = static_cast<T *>(p.out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i, tok = r / p.heads_per_tile, h = r % p.heads_per_tile;
        float sum = l[i];
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
        if (tok >= t.tokens || h >= t.heads) continue;
        const float inv = 1.0f / sum;
        T *row = out + ((t.row0 + t.token0 + tok) * p.n_q_heads + t.head0 + h) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sum != 0.0f)
                v = make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
                                o[i][4 * c + 3] * inv);
            store4(row + tx * 4 + 32 * c, v);
        }
    }
}

template <typename T, int D>
gdn_status launch_simt(PrefillParams p, cudaStream_t s) {
    p.heads_per_tile = p.group < kSimtRows ? p.group : kSimtRows;
    p.head_groups = (p.group + p.heads_per_tile - 1) / p.heads_per_tile;
    p.tokens_per_tile = kSimtRows / p.heads_per_tile;
    const long long tiles = p.seqs.total / p.tokens_per_tile + p.n_seqs;
    const long long ys = static_cast<long long>(p.cache.n_kv_heads) * p.head_groups;
    if (tiles > 0x7fffffffLL || ys > 65535) return GDN_ERR_UNSUPPORTED;
    auto kernel = attn_prefill_simt_kernel<T, D>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, simt_smem<D>()) !=
        cudaSuccess)
        return GDN_ERR_LAUNCH;
    kernel<<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(ys)), kSimtThreads,
             simt_smem<D>(), s>>>(p);
    return launch_status();
}

template <typename T>
gdn_status launch_simt_dim(int d, const PrefillParams &p, cudaStream_t s) {
    switch (d) {
        case 64: return launch_simt<T, 64>(p, s);
        case 128: return launch_simt<T, 128>(p, s);
        default: return launch_simt<T, 256>(p, s);
    }
}

// ------------------------------------------------------------------ on the tensor cores

// 16-bit types. A CTA takes kTiles tiles of 128 rows and walks the keys in tiles of 128:
//   S = Q K^T      tcgen05, Q and K from shared memory, S in tensor memory
//   P = 2^(scale log2(e) S - m)   four warps per row tile, one thread per row: the row's
//                  maximum and sum need no exchange; P goes back to tensor memory over S,
//                  in the cache's type (half a unit of the type per weight, which averages
//                  out below the output's own rounding)
//   O += P V       tcgen05, P from tensor memory, V from shared memory as it lies there
//                  (rows are keys: the MN-major operand form, no transposition)
// O stays in tensor memory. It is rescaled only when a row's maximum has grown by more than
// 2^8 since the reference the weights use (they stay below 2^8, far inside both types).
//
// Two row tiles (head_dim 64, 128) share every key tile and alternate: one tile's softmax
// runs while the tensor pipe works for the other. With head_dim 256 O fills half the tensor
// memory, so there is one row tile and two S buffers: S of the next key tile is computed
// during the softmax of this one.
//
// K and V stream through two rings of slots, each fed by a warp of its own (one warp's copies,
// barriers and page lookups would take longer than the products: a copy costs its warp about
// 60 cycles, a barrier 30 to 60). Pages are loaded one by one; a V slot keeps their rows apart
// ([page][128-byte column][row]), so that one copy brings all of a page's columns, and the
// MMA's descriptor strides say where they lie.
constexpr int kTcKeys = 128;
constexpr int kTcRows = 128;
constexpr int kDescs = 8;
constexpr float kLazy = 8.0f;  // log2 of the growth of a maximum that makes O rescale

template <int D>
struct Tc {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kBufs = D == 256 ? 2 : 1;              // S buffers of a row tile
    static constexpr int kSubs = D == 256 ? 2 : 1;              // slots of a K (or V) tile
    static constexpr int kSlots = D == 64 ? 4 : 2;              // of each ring
    static constexpr int kSlotBytes = kTcKeys * D * 2 / kSubs;
    static constexpr int kCols = D / 64 / kSubs;                // 128-byte columns of a K slot
    static constexpr int kVKeys = kTcKeys / kSubs;              // keys of a V slot
    static constexpr int kLog2VKeys = kSubs == 2 ? 6 : 7;
    static constexpr int kQBytes = kTcRows * D * 2;             // of a row tile
    static constexpr int kSmem = kTiles * kQBytes + 2 * kSlots * kSlotBytes + 1024;
    static constexpr int kThreads = kTiles * 128 + 128;         // softmax; MMA, K, V, an idle warp
    static constexpr int kS = 0, kO = 256;                      // tensor-memory columns
};

// Bounded wait; once one gave up, the CTA's later waits return at once and none of its rows
// are written.
__device__ __forceinline__ void wait_or_flag(uint64_t *bar, uint32_t parity, volatile int *dead) {
    if (mbar_test(bar, parity) || *dead) return;
    if (!mbar_wait(bar, parity)) {
        *dead = 1;
        atomicOr(&g_watchdog_attn_prefill, WD_STAGE_COPY);
    }
}

// Bits lo .. hi - 1 of a 32-bit word (any of them outside the word).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t skip = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below & ~skip;
}

template <typename T, int D>
__global__ void __launch_bounds__(Tc<D>::kThreads, 1)
attn_prefill_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const PrefillParams p) {
    using C = Tc<D>;
    constexpr bool kBf16 = !__is_same(T, __half);
    constexpr uint32_t kIdescS = tc::idesc_16bit(kBf16, kTcRows, kTcKeys, false);
    constexpr uint32_t kIdescO = tc::idesc_16bit(kBf16, kTcRows, D, true);
    extern __shared__ uint8_t dyn[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *k_ring = smem + C::kTiles * C::kQBytes;
    uint8_t *v_ring = k_ring + C::kSlots * C::kSlotBytes;
    __shared__ __align__(8) uint64_t k_full[C::kSlots], k_empty[C::kSlots];
    __shared__ __align__(8) uint64_t v_full[C::kSlots], v_empty[C::kSlots];
    __shared__ __align__(8) uint64_t q_full, s_full[2], p_ready[2], o_done[2], desc_full[kDescs];
    __shared__ int2 descs[kDescs];  // first key and loaded 8-key blocks of a key tile
    __shared__ uint32_t tmem_base;
    __shared__ int sh_dead;

    RowTile t;
    if (!find_tile(p, t)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = p.tokens_per_tile / C::kTiles;  // tokens of one 128-row tile
    const int tiles = t.tokens > per ? 2 : 1;
    const TileWalk walk = walk_tiles<kTcKeys>(p.mask, t.p_first, t.p_last);
    const int n = walk.count;
    // key tiles of row tile 0: a last one past its positions is left out
    int n0 = n;
    if (tiles == 2 && n > 0 && walk.tile(n - 1) * kTcKeys > t.p_first + per - 1) --n0;
    const int log2_bv = min(p.cache.log2_ps, C::kLog2VKeys);  // keys of a V load
    const int bv = 1 << log2_bv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kDescs; ++i) mbar_init(&desc_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(&q_full, 1);
        fence_mbar_init();
        sh_dead = 0;
    }
    if (warp == C::kTiles * 4) tc::tmem_alloc(&tmem_base, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base;

    // Two row tiles: 384 threads of 168 registers; the softmax threads take 224 each, the
    // third warp group keeps 56 (2 * 224 + 56 = 3 * 168).
    if (warp >= C::kTiles * 4) {
        if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // The loading and the MMA warp run converged, with one elected lane issuing: the
        // operands of a copy or an MMA are then the same in every lane, as the hardware
        // wants them.
        const bool leader = elect_one();
        const int ps = 1 << p.cache.log2_ps;
        const int log2_bk = min(p.cache.log2_ps, 7);  // keys of a page's part of a key tile
        const int bk = 1 << log2_bk, n_bk = kTcKeys >> log2_bk;
        // The page of lane i's part of key tile j, or -1 for a part that nobody sees (its id
        // is not read: pages before the window may be gone).
        auto page_at = [&](int j) -> int {
            if (lane >= n_bk) return -1;
            const int key = walk.tile(j) * kTcKeys + lane * bk;
            if (key > t.p_last) return -1;
            if (!(t.p_first - (key + bk - 1) < p.mask.window || key < p.mask.sinks)) return -1;
            return p.cache.page_of(t.slot, key);
        };
        if (warp == C::kTiles * 4 + 1 && n > 0) {
            // ------------------------------------------------------ the K warp
            if (leader) {
                tma_prefetch_map(&k_map);
                mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(tiles * p.heads_per_tile * per) * D * 2u);
                for (int i = 0; i < tiles; ++i)
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_3d(smem + i * C::kQBytes + cb * kTcRows * 128, &q_map, cb * 64,
                                    t.head0, static_cast<int>(t.row0) + t.token0 + i * per, &q_full);
            }
            __syncwarp();
            int page = page_at(0), slot = 0, round = 0;
            for (int j = 0; j < n; ++j) {
                const int next_page = j + 1 < n ? page_at(j + 1) : -1;
                const int key0 = walk.tile(j) * kTcKeys;
                const bool ok = p.cache.page_ok(page);
                const unsigned have = __ballot_sync(FULL_MASK, ok);
                if (!ok && blockIdx.y == 0 && p.err_count) {
                    // a part that somebody sees, without a page
                    const int key = key0 + lane * bk;
                    if (lane < n_bk && key <= t.p_last &&
                        (t.p_first - (key + bk - 1) < p.mask.window || key < p.mask.sinks))
                        atomicAdd(p.err_count, 1);
                }
                const int row = (page * p.cache.n_kv_heads + t.kvh) * ps + (key0 & (ps - 1));
                if (leader) {
                    unsigned blocks = 0;
                    for (int i = 0; i < kTcKeys / 8; ++i)
                        if ((have >> ((i * 8) >> log2_bk)) & 1u) blocks |= 1u << i;
                    descs[j % kDescs] = make_int2(key0, static_cast<int>(blocks));
                    mbar_arrive(&desc_full[j % kDescs]);
                }
                __syncwarp();
                for (int s = 0; s < C::kSubs; ++s) {
                    if (round > 0) wait_or_flag(&k_empty[slot], (round - 1) & 1, &sh_dead);
                    uint8_t *to = k_ring + slot * C::kSlotBytes;
                    if (leader)
                        mbar_arrive_expect_tx(&k_full[slot], (static_cast<uint32_t>(__popc(have)) << (log2_bk + 7)) * C::kCols);
                    if (n_bk == 1) {  // one page: its columns in one copy
                        const int r = __shfl_sync(FULL_MASK, row, 0);
                        if (leader && have) tma_load_3d(to, &k_map, 0, r, s * C::kCols, &k_full[slot]);
                    } else {
                        for (int i = 0; i < n_bk; ++i) {
                            const int r = __shfl_sync(FULL_MASK, row, i);
                            if (leader && ((have >> i) & 1u)) {
#pragma unroll
                                for (int c = 0; c < C::kCols; ++c)
                                    tma_load_3d(to + c * kTcKeys * 128 + (i << (log2_bk + 7)), &k_map, 0, r,
                                                s * C::kCols + c, &k_full[slot]);
                            }
                        }
                    }
                    __syncwarp();
                    if (++slot == C::kSlots) {
                        slot = 0;
                        ++round;
                    }
                }
                page = next_page;
            }
        } else if (warp == C::kTiles * 4 + 2 && n > 0) {
            // ------------------------------------------------------ the V warp
            if (leader) tma_prefetch_map(&v_map);
            int page = page_at(0), slot = 0, round = 0;
            for (int j = 0; j < n; ++j) {
                const int next_page = j + 1 < n ? page_at(j + 1) : -1;
                const int key0 = walk.tile(j) * kTcKeys;
                const unsigned have = __ballot_sync(FULL_MASK, p.cache.page_ok(page));
                const int row = (page * p.cache.n_kv_heads + t.kvh) * ps + (key0 & (ps - 1));
                for (int s = 0; s < C::kSubs; ++s) {
                    if (round > 0) wait_or_flag(&v_empty[slot], (round - 1) & 1, &sh_dead);
                    uint8_t *to = v_ring + slot * C::kSlotBytes;
                    // this slot's copies of bv keys, from the parts they lie in
                    const int i0 = s << (C::kLog2VKeys - log2_bv), i1 = (s + 1) << (C::kLog2VKeys - log2_bv);
                    const bool here = lane >= i0 && lane < i1 && ((have >> ((lane << log2_bv) >> log2_bk)) & 1u);
                    const unsigned loads = __popc(__ballot_sync(FULL_MASK, here));
                    if (leader) mbar_arrive_expect_tx(&v_full[slot], loads * static_cast<uint32_t>(bv) * D * 2u);
                    for (int i = i0; i < i1; ++i) {
                        const int part = (i << log2_bv) >> log2_bk;
                        const int r = __shfl_sync(FULL_MASK, row, part) + ((i << log2_bv) & (bk - 1));
                        if (leader && ((have >> part) & 1u))
                            tma_load_3d(to + (i - i0) * (bv * D * 2), &v_map, 0, r, 0, &v_full[slot]);
                    }
                    __syncwarp();
                    if (++slot == C::kSlots) {
                        slot = 0;
                        ++round;
                    }
                }
                page = next_page;
            }
        } else if (warp == C::kTiles * 4 && n > 0) {
            // ------------------------------------------------------ the MMA warp
            wait_or_flag(&q_full, 0, &sh_dead);
            const uint64_t q_desc = tc::smem_desc_sw128(smem_addr(smem));
            const uint64_t k_desc = tc::smem_desc_sw128(smem_addr(k_ring));
            // V lies page by page, every page's 128-byte columns one behind the other: 16 keys
            // are two groups of 8 rows, in one page (bv >= 16) or in two
            const uint64_t v_desc = tc::smem_desc_sw128_mn(smem_addr(v_ring), bv * 128, bv >= 16 ? 1024 : D * 16);
            uint32_t v_step[C::kVKeys / 16];
#pragma unroll
            for (int x = 0; x < C::kVKeys / 16; ++x)
                v_step[x] = (((x * 16) >> log2_bv) * (bv * D * 2) + ((x * 16) & (bv - 1)) * 128) >> 4;
            // S of row tile i over key tile j
            auto issue_s = [&](int i, int j, bool release) {
                const int buf = C::kBufs == 2 ? j & 1 : i;
                const uint32_t to = tmem + C::kS + buf * kTcKeys;
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int g = j * C::kSubs + s, slot = g % C::kSlots;
                    wait_or_flag(&k_full[slot], (g / C::kSlots) & 1, &sh_dead);
                    tc::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int c = 0; c < C::kCols; ++c)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                tc::mma_bf16(to,
                                             q_desc + ((i * C::kQBytes + (s * C::kCols + c) * kTcRows * 128 + x * 32) >> 4),
                                             k_desc + ((slot * C::kSlotBytes + c * kTcKeys * 128 + x * 32) >> 4),
                                             kIdescS, s + c + x > 0);
                        if (release) tc::mma_commit(&k_empty[slot]);
                        if (s == C::kSubs - 1) tc::mma_commit(&s_full[buf]);
                    }
                    __syncwarp();
                }
            };
            // O of row tile i += P V over key tile j
            auto issue_o = [&](int i, int j, bool release) {
                const int buf = C::kBufs == 2 ? j & 1 : i;
                wait_or_flag(&p_ready[buf], (C::kBufs == 2 ? j >> 1 : j) & 1, &sh_dead);
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int g = j * C::kSubs + s, slot = g % C::kSlots;
                    wait_or_flag(&v_full[slot], (g / C::kSlots) & 1, &sh_dead);
                    tc::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int x = 0; x < C::kVKeys / 16; ++x)
                            tc::mma_bf16_ts(tmem + C::kO + i * D,
                                            tmem + C::kS + buf * kTcKeys + (s * C::kVKeys + x * 16) / 2,
                                            v_desc + ((slot * C::kSlotBytes) >> 4) + v_step[x], kIdescO,
                                            j > 0 || s + x > 0);
                        if (release) tc::mma_commit(&v_empty[slot]);
                        if (s == C::kSubs - 1) tc::mma_commit(&o_done[i]);
                    }
                    __syncwarp();
                }
            };
            if constexpr (C::kTiles == 2) {
                if (n0 > 0) issue_s(0, 0, tiles == 1);
                if (tiles == 2) issue_s(1, 0, true);
                for (int j = 0; j < n; ++j) {
                    if (j < n0) {
                        issue_o(0, j, tiles == 1);
                        if (j + 1 < n0) issue_s(0, j + 1, tiles == 1);
                    }
                    if (tiles == 2) {
                        issue_o(1, j, true);
                        if (j + 1 < n) issue_s(1, j + 1, true);
                    }
                }
            } else {
                issue_s(0, 0, true);
                for (int j = 0; j < n; ++j) {
                    if (j + 1 < n) issue_s(0, j + 1, true);
                    issue_o(0, j, true);
                }
            }
        }
    } else {
        if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        if (warp / 4 < tiles) {
            // ------------------------------------------------------ softmax, one row a thread
            const int i = warp / 4, row = threadIdx.x & 127;
            const int my_n = i == 0 ? n0 : n;
            const int token = i * per + row / p.heads_per_tile;
            const int head = row % p.heads_per_tile;
            const int pos = t.p_first + token;
            const int p_first = t.p_first + i * per;  // of the row tile
            const int p_last = min(p_first + per - 1, t.p_last);
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t o_addr = tmem + lanes + C::kO + i * D;
            const bool positive = p.scale_log2 > 0.0f;
            const float mult = positive ? p.scale_log2 : 1.0f;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < my_n; ++j) {
                const int buf = C::kBufs == 2 ? j & 1 : i;
                const uint32_t s_addr = tmem + lanes + C::kS + buf * kTcKeys;
                wait_or_flag(&desc_full[j % kDescs], (j / kDescs) & 1, &sh_dead);
                const int2 desc = descs[j % kDescs];
                const int key0 = desc.x;
                const unsigned blocks = static_cast<unsigned>(desc.y);
                // every row of the CTA, and of this row tile, sees every key of the tile
                const bool alive = blocks == 0xFFFFu && key0 + kTcKeys - 1 <= t.p_last &&
                                   (t.p_first - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                const bool clean = blocks == 0xFFFFu && key0 + kTcKeys - 1 <= p_first &&
                                   (p_last - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                wait_or_flag(&s_full[buf], (C::kBufs == 2 ? j >> 1 : j) & 1, &sh_dead);
                tc::fence_after_sync();
                float s[128];
                {
                    uint32_t raw[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_ld32_nowait(s_addr + c * 32, raw[c]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(raw[c >> 5][c & 31]);
                }
                if (!alive && (i == 0 || j >= n0)) {
                    // V rows that no row of the CTA sees are cleared, so that whatever the page
                    // holds there (an infinity, a NaN) cannot reach O through a weight of 0.
                    // (Two S buffers: once the O product before this tile's is complete, the
                    // ring slots of V are at most one phase from the one waited for.)
                    if (C::kBufs == 2 && j > 0) wait_or_flag(&o_done[0], (j - 1) & 1, &sh_dead);
                    const int key = key0 + row;
                    const bool dead = !((blocks >> (row >> 3)) & 1u) || key > t.p_last ||
                                      !(t.p_first - key < p.mask.window || key < p.mask.sinks);
                    for (int y = 0; y < C::kSubs; ++y) {
                        const int g = j * C::kSubs + y, slot = g % C::kSlots;
                        wait_or_flag(&v_full[slot], (g / C::kSlots) & 1, &sh_dead);
                        if (dead && (row >> C::kLog2VKeys) == y) {
                            const int r = row & (C::kVKeys - 1);
                            uint8_t *at = v_ring + slot * C::kSlotBytes + (r >> log2_bv) * (bv * D * 2) + (r & (bv - 1)) * 128;
                            for (int x = 0; x < D / 8; ++x)
                                *reinterpret_cast<uint4 *>(at + (x >> 3) * bv * 128 + (x & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (!positive) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) s[c] *= p.scale_log2;
                }
                if (!clean) {
                    // the keys this row sees: from its window's first to itself, and the sinks
                    const int hi = pos - key0 + 1;
                    const int lo = pos - key0 < p.mask.window ? 0 : pos - p.mask.window + 1 - key0;
                    const int sink = min(p.mask.sinks - key0, hi);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t see = bits_between(lo - 32 * w, hi - 32 * w) | bits_between(0, sink - 32 * w);
                        uint32_t there = 0;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if ((blocks >> (4 * w + x)) & 1u) there |= 0xFFu << (8 * x);
                        see &= there;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(see & (1u << c))) s[32 * w + c] = -INFINITY;
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x) top[x] = fmaxf(fmaxf(top[x], s[c + 2 * x]), s[c + 2 * x + 1]);
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                if (j == 0) {
                    m = mx;
                } else {
                    const bool grow = (mx - m) * mult > kLazy;
                    if (__any_sync(FULL_MASK, grow)) {
                        // O is complete up to the tile before: S of this tile was issued after
                        // it (two S buffers: after the one before that)
                        if (C::kBufs == 2) {
                            wait_or_flag(&o_done[0], (j - 1) & 1, &sh_dead);
                            tc::fence_after_sync();
                        }
                        const float f = grow ? fast_exp2((m - mx) * mult) : 1.0f;
                        if (grow) m = mx;
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32_nowait(o_addr + c, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tc::tmem_st32(o_addr + c, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m * mult;
                const float2 mul2 = make_float2(mult, mult), sub2 = make_float2(-base, -base);
                float2 sum[4] = {};
#pragma unroll
                for (int c = 0; c < 128; c += 64) {
                    uint32_t w[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        float2 a = __ffma2_rn(make_float2(s[c + 2 * x], s[c + 2 * x + 1]), mul2, sub2);
                        a.x = fast_exp2(a.x);
                        a.y = fast_exp2(a.y);
                        sum[x & 3] = __fadd2_rn(sum[x & 3], a);
                        w[x] = Elem<T>::pack(a.x, a.y);
                    }
                    tc::tmem_st32(s_addr + c / 2, w);
                }
                sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += sum[0].x + sum[0].y;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                // keeps this thread at most one phase behind o_done
                if (C::kBufs == 2 && j > 0) wait_or_flag(&o_done[0], (j - 1) & 1, &sh_dead);
                if (lane == 0) mbar_arrive(&p_ready[buf]);
            }
            // ------------------------------------------------------ O out
            T *out = static_cast<T *>(p.out) +
                     ((t.row0 + t.token0 + token) * p.n_q_heads + t.head0 + head) * D;
            const bool mine = token < t.tokens && row / p.heads_per_tile < per && head < t.heads;
            if (my_n > 0) {
                wait_or_flag(&o_done[i], (my_n - 1) & 1, &sh_dead);
                tc::fence_after_sync();
            }
            const float inv = 1.0f / l;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc::tmem_ld32_nowait(o_addr + c, o);
                tc::tmem_ld_wait();
                if (mine && !sh_dead) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = l == 0.0f ? 0u
                                             : Elem<T>::pack(__uint_as_float(o[x + 2 * y]) * inv,
                                                             __uint_as_float(o[x + 2 * y + 1]) * inv);
                        *reinterpret_cast<uint4 *>(out + c + x) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc::fence_before_sync();
        }
    }
    __syncthreads();
    if (warp == C::kTiles * 4) {
        tc::fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D>
gdn_status launch_tc(PrefillParams p, int dtype, cudaStream_t s) {
    using C = Tc<D>;
    const int ps = 1 << p.cache.log2_ps;
    p.heads_per_tile = p.group < kTcRows ? p.group : kTcRows;
    p.head_groups = (p.group + p.heads_per_tile - 1) / p.heads_per_tile;
    const int per = kTcRows / p.heads_per_tile;
    p.tokens_per_tile = per * C::kTiles;
    const long long tiles = p.seqs.total / p.tokens_per_tile + p.n_seqs;
    const long long ys = static_cast<long long>(p.cache.n_kv_heads) * p.head_groups;
    if (tiles > 0x7fffffffLL || ys > 65535) return GDN_ERR_UNSUPPORTED;
    CUtensorMap q_map, k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(p.cache.n_pages) * p.cache.n_kv_heads * ps;
    GDN_TRY(encode_heads_map(&q_map, p.q, dtype, D, p.n_q_heads, static_cast<uint64_t>(p.seqs.total),
                             static_cast<uint64_t>(p.q_stride) * 2, p.heads_per_tile, per));
    GDN_TRY(encode_blocks_map(&k_map, p.k_pages, dtype, D, rows, D * 2, ps < kTcKeys ? ps : kTcKeys,
                              ps < kTcKeys ? 1 : C::kCols));
    GDN_TRY(encode_blocks_map(&v_map, p.v_pages, dtype, D, rows, D * 2, ps < C::kVKeys ? ps : C::kVKeys,
                              D / 64));
    auto kernel = attn_prefill_tc_kernel<T, D>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    kernel<<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(ys)), C::kThreads, C::kSmem, s>>>(
        q_map, k_map, v_map, p);
    return launch_status();
}

template <typename T>
gdn_status launch_tc_dim(int d, const PrefillParams &p, int dtype, cudaStream_t s) {
    switch (d) {
        case 64: return launch_tc<T, 64>(p, dtype, s);
        case 128: return launch_tc<T, 128>(p, dtype, s);
        default: return launch_tc<T, 256>(p, dtype, s);
    }
}

}  // namespace

unsigned read_and_clear_watchdog_attn_prefill(cudaStream_t s) {
    unsigned flags = 0;
    const unsigned zero = 0;
    cudaMemcpyFromSymbolAsync(&flags, g_watchdog_attn_prefill, sizeof(flags), 0,
                              cudaMemcpyDeviceToHost, s);
    cudaMemcpyToSymbolAsync(g_watchdog_attn_prefill, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
    cudaStreamSynchronize(s);
    return flags;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_attn_prefill_workspace_size(int n_seqs, int total_tokens, int n_q_heads, int n_kv_heads,
                                       int head_dim) {
    if (n_seqs < 0 || total_tokens < 0 || n_kv_heads < 1 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads != 0 || !supported_head_dim(head_dim))
        return 0;
    return 0;
}

gdn_status gdn_attn_prefill(const void *q, const void *k_pages, const void *v_pages,
                            const int32_t *page_table, const int32_t *kv_lens, void *out,
                            const int32_t *cu_seqlens, int n_seqs, int total_tokens,
                            int max_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                            int page_size, int n_pages, int max_pages, int window, int n_sinks,
                            float scale, int q_stride, int dtype, const int32_t *slots, int pool,
                            int32_t *err_count, void *workspace, size_t workspace_bytes,
                            gdn_stream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !out) return GDN_ERR_NULL;
    GDN_TRY(check_varlen(cu_seqlens, n_seqs, total_tokens, max_tokens));
    if (n_q_heads < 1 || window < 0 || n_sinks < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_cache(n_kv_heads, head_dim, page_size, n_pages, max_pages, dtype));
    if (n_q_heads % n_kv_heads != 0) return GDN_ERR_SHAPE;
    if (static_cast<long long>(n_q_heads) * head_dim > q_stride) return GDN_ERR_SHAPE;
    GDN_TRY(check_pool(n_seqs, slots, pool));
    const long long es = dtype_bytes(dtype);
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
        q_stride * es % 16 != 0)
        return GDN_ERR_ALIGN;
    if (n_seqs == 0 || total_tokens == 0) return GDN_OK;
    PrefillParams p{};
    p.cache = PagedCache{page_table, kv_lens, slots, pool, max_pages, n_pages, n_kv_heads,
                         log2_of(page_size)};
    p.mask = make_mask(window, n_sinks);
    p.seqs = SeqMap{cu_seqlens, max_tokens, total_tokens};
    p.q = q;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.out = out;
    p.n_seqs = n_seqs;
    p.n_q_heads = n_q_heads;
    p.group = n_q_heads / n_kv_heads;
    p.q_stride = q_stride;
    p.scale_log2 = scale * kLog2E;
    p.err_count = err_count;
    const cudaStream_t s = as_cuda(stream);
    switch (dtype) {
        case GDN_F32: return launch_simt_dim<float>(head_dim, p, s);
        case GDN_F16: return launch_tc_dim<__half>(head_dim, p, dtype, s);
        default: return launch_tc_dim<__nv_bfloat16>(head_dim, p, dtype, s);
    }
}

}  // extern "C"
