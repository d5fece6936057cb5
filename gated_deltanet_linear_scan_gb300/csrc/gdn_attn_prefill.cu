// gdn_attn_prefill.cu -- attention of a ragged batch of prompts, or chunks of prompts, over
// the paged key/value cache (sm_103a).
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = e^{scale q_i.k_j - m_i} over the keys i sees
//
// All query heads of a key head share its keys, so a tile of rows is (tokens x heads of one
// key head): the keys are read once for all of them, and a tile spans few positions, which
// keeps the work wasted at the causal diagonal and at the window's edge small.
#include "gdn_attn_prefill.cuh"

namespace gdn {
namespace {

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

__device__ __forceinline__ float4 load_float4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 32;

template <int D>
constexpr int simt_smem() {
    return ((kSimtRows + 4 * kSimtKeys) * (D + 4) + kSimtRows * (kSimtKeys + 4)) * 4;
}

// 64 rows by 32 keys a step, everything in fp32: a thread holds 4 rows x 4 keys of S (8
// lanes span the keys) and 4 rows x D/8 columns of O. Rows of shared memory are padded by 16
// bytes, so the 8 lanes of a quarter-warp read different banks.
//
// The tensor cores have no fp32 product, so the FP32 pipes bound it (78 TFLOP/s), and before
// them the reads of shared memory that feed them: 8 reads of 16 bytes for 64 multiply-adds of
// S, 5 for 64 of O, at 4 cycles of the SM's one port a read. 16384 ragged prompt tokens: 5.47
// ms at head_dim 128 with 32 heads (31.7 TFLOP/s), 1.51 ms at 64 with 16 (28.7), 9.25 ms at
// 256 with 24 (28.1; 12.9 ms before K and V were loaded a tile ahead).
template <int D>
__global__ void __launch_bounds__(kSimtThreads)
attn_prefill_f32_kernel(const PrefillParams p) {
    constexpr int P = D + 4, PP = kSimtKeys + 4;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *skv = sq + kSimtRows * P, *sp = skv + 4 * kSimtKeys * P;  // K, V, twice
    RowTile t;
    if (!find_tile(p, t)) return;
    const int tid = threadIdx.x, lane = tid & 31, tx = tid & 7, ty = tid >> 3;
    const float *q = static_cast<const float *>(p.q);
    const float *k_pages = static_cast<const float *>(p.k_pages);
    const float *v_pages = static_cast<const float *>(p.v_pages);
    const int ps = 1 << p.cache.log2_ps;

    for (int x = tid; x < kSimtRows * (D / 4); x += kSimtThreads) {
        const int r = x / (D / 4), c = (x % (D / 4)) * 4;
        const int tok = r / p.heads_per_tile, h = r % p.heads_per_tile;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tok < t.tokens && h < t.heads)
            v = load_float4(q + (t.row0 + t.token0 + tok) * p.q_stride + static_cast<size_t>(t.head0 + h) * D + c);
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
    // The page of this lane's key of tile w, -1 for keys that no row of the tile sees: they are
    // not looked up, their pages may be gone, and whatever a page holds past the length must
    // not reach the sums.
    auto page_at = [&](int w) {
        if (w >= walk.count) return -1;
        const int key = walk.tile(w) * kSimtKeys + lane;
        const bool seen = key <= t.p_last && (t.p_first - key < p.mask.window || key < p.mask.sinks);
        const int page = seen ? p.cache.page_of(t.slot, key) : -1;
        const bool ok = p.cache.page_ok(page);
        if (__any_sync(FULL_MASK, seen && !ok) && tid == 0 && blockIdx.y == 0 && p.err_count)
            atomicAdd(p.err_count, 1);
        return ok ? page : -1;
    };
    // Asks for tile w's rows (keys that nobody sees are zeros); returns which keys are there.
    auto load = [&](int w, int page) {
        const unsigned there = __ballot_sync(FULL_MASK, page >= 0);
        float *sk = skv + (w & 1) * 2 * kSimtKeys * P, *sv = sk + kSimtKeys * P;
        const int in_page = (walk.tile(w) * kSimtKeys + lane) & (ps - 1);
        const int row = ((page * p.cache.n_kv_heads) + t.kvh) * ps + in_page;  // (fits: the cache's rows do)
#pragma unroll 4
        for (int x = tid; x < kSimtKeys * (D / 4); x += kSimtThreads) {
            const int i = x / (D / 4), c = (x % (D / 4)) * 4;
            const size_t at = static_cast<size_t>(__shfl_sync(FULL_MASK, row, i)) * D + c;
            if ((there >> i) & 1u) {
                cp_async16(sk + i * P + c, k_pages + at);
                cp_async16(sv + i * P + c, v_pages + at);
            } else {
                *reinterpret_cast<float4 *>(sk + i * P + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                *reinterpret_cast<float4 *>(sv + i * P + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
        return there;
    };
    // tile w + 1 is on its way while tile w is computed, and the pages of tile w + 2 are looked up
    unsigned next_there = walk.count > 0 ? load(0, page_at(0)) : 0;
    int next_page = page_at(1);
    for (int w = 0; w < walk.count; ++w) {
        const int key0 = walk.tile(w) * kSimtKeys;
        const unsigned there = next_there;
        const float *sk = skv + (w & 1) * 2 * kSimtKeys * P, *sv = sk + kSimtKeys * P;
        cp_async_wait_all();
        __syncthreads();  // this tile is there, and the one before has been read
        if (w + 1 < walk.count) {
            next_there = load(w + 1, next_page);
            next_page = page_at(w + 2);
        }
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
                const int k = tx + 8 * j;
                const bool ok = ((there >> k) & 1u) && p.mask.sees(pos, key0 + k);
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
    float *out = static_cast<float *>(p.out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i, tok = r / p.heads_per_tile, h = r % p.heads_per_tile;
        float sum = l[i];
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
        if (tok >= t.tokens || h >= t.heads) continue;
        const float inv = 1.0f / sum;
        float *row = out + ((t.row0 + t.token0 + tok) * p.n_q_heads + t.head0 + h) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sum != 0.0f)
                v = make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
                                o[i][4 * c + 3] * inv);
            *reinterpret_cast<float4 *>(row + tx * 4 + 32 * c) = v;
        }
    }
}

template <int D>
gdn_status launch_f32(PrefillParams p, cudaStream_t s) {
    p.heads_per_tile = p.group < kSimtRows ? p.group : kSimtRows;
    p.head_groups = (p.group + p.heads_per_tile - 1) / p.heads_per_tile;
    p.tokens_per_tile = kSimtRows / p.heads_per_tile;
    const long long tiles = p.seqs.total / p.tokens_per_tile + p.n_seqs;
    const long long ys = static_cast<long long>(p.cache.n_kv_heads) * p.head_groups;
    if (tiles > 0x7fffffffLL || ys > 65535) return GDN_ERR_UNSUPPORTED;
    auto kernel = attn_prefill_f32_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, simt_smem<D>(), allowed));
    kernel<<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(ys)), kSimtThreads,
             simt_smem<D>(), s>>>(p);
    return launch_status();
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

// The kernels need none now; the argument keeps room for one that does.
size_t gdn_attn_prefill_workspace_size(int, int, int, int, int) { return 0; }

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
    if (dtype != GDN_F32) return launch_attn_prefill_tc(p, dtype, head_dim, s);
    switch (head_dim) {
        case 64: return launch_f32<64>(p, s);
        case 128: return launch_f32<128>(p, s);
        default: return launch_f32<256>(p, s);
    }
}

}  // extern "C"
