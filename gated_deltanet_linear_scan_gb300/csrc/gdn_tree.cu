// gdn_tree.cu -- acceptance of a tree of drafts: the path along which the sampled tokens agree
// with the drafted ones, and its keys and values moved together in the paged cache.
//
// A walk is at most 64 steps of a warp over nodes that lie in its registers, one vote a step. The
// rows to move are few (a path's), so the call is latency: every CTA of a sequence walks for
// itself, and moves its share of (plane, head, 16 bytes of a row). 64 trees of 16 with 16 planes of 8
// heads' rows of 256 bytes: 5.4 us (the rows' bytes alone 1.1); one of 64: 6.9, a walk and a move behind
// a launch.
#include "gdn_paged.cuh"
#include "gdn_tree.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // rows in flight a thread

struct AcceptParams {
    const int32_t *parents, *tokens, *sampled;
    int32_t *accepted, *n_kept, *new_lens, *next_tokens, *path;
    uint4 *pages;
    PagedCache cache;
    int n_nodes, row_vecs, n_planes;  // row_vecs: 16-byte parts of a row
    size_t page_vecs;
    int32_t *err_count;
};

// Grid: (sequence, share of its (plane, head, part of a row)).
__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const AcceptParams p) {
    __shared__ int walk[kMaxNodes], kept_sh, up[kMaxNodes];
    __shared__ unsigned long long path_of[kMaxNodes];
    __shared__ long long from[kMaxNodes], to[kMaxNodes];  // rows, in 16-byte parts of a plane's head 0
    const int n = blockIdx.x, N = p.n_nodes, tid = threadIdx.x, lane = tid & 31;
    const bool first = blockIdx.y == 0;
    int slot = p.cache.slots ? p.cache.slots[n] : n, len = 0;
    bool ok = slot >= 0 && slot < p.cache.pool;
    if (p.cache.kv_lens) {
        ok = ok && p.cache.lookup(n, slot, len);
        ok = ok && len >= N;
    }
    if (tid < 32) {
        const int32_t *parents = p.parents + static_cast<size_t>(n) * N;
        const int32_t *tokens = p.tokens + static_cast<size_t>(n) * N;
        const int32_t *sampled = p.sampled + static_cast<size_t>(n) * N;
        const int last = N - 1, a = min(lane, last), b = min(lane + 32, last);
        // (a node past the tree is nobody's child)
        const int parent0 = lane < N ? parents[a] : GDN_NO_NODE, token0 = tokens[a], pick0 = sampled[a];
        const int parent1 = lane + 32 < N ? parents[b] : GDN_NO_NODE, token1 = tokens[b], pick1 = sampled[b];
        if (first) {
            unsigned long long paths[2];
            const bool bad = tree_paths(parents, N, paths, path_of, up);
            if ((!ok || bad) && lane == 0 && p.err_count) atomicAdd(p.err_count, 1);
        }
        int at = 0, kept = 0, pick = -1;
        if (ok && __shfl_sync(FULL_MASK, parent0, 0) == -1) {
            for (;;) {
                if (lane == 0) walk[kept] = at;
                ++kept;
                pick = __shfl_sync(FULL_MASK, at < 32 ? pick0 : pick1, at & 31);
                // a child lies behind its parent: the walk ends
                const unsigned lo = __ballot_sync(FULL_MASK, parent0 == at && lane > at && token0 == pick);
                const unsigned hi = __ballot_sync(FULL_MASK, parent1 == at && lane + 32 > at && token1 == pick);
                if (lo == 0 && hi == 0) break;
                at = lo != 0 ? __ffs(lo) - 1 : 31 + __ffs(hi);
            }
        }
        if (lane == 0) kept_sh = kept;
        if (first) {
            __syncwarp();
            if (lane == 0) {
                p.accepted[n] = kept > 0 ? at + 1 : 0;
                p.n_kept[n] = kept;
                if (p.new_lens) p.new_lens[n] = ok ? len - N + kept : max(len, 0);
                p.next_tokens[n] = pick;
            }
            for (int i = lane; i < N && p.path; i += 32) p.path[static_cast<size_t>(n) * N + i] = i < kept ? walk[i] : -1;
        }
    }
    __syncthreads();
    const int kept = kept_sh;
    if (p.n_planes == 0 || kept < 2) return;
    if (tid < kept) {
        const int base = len - N, ps_mask = (1 << p.cache.log2_ps) - 1;
        long long src = -1, dst = -1;
        if (walk[tid] != tid) {
            const int sp = p.cache.page_of(slot, base + walk[tid]), dp = p.cache.page_of(slot, base + tid);
            if (p.cache.page_ok(sp) && p.cache.page_ok(dp)) {
                src = static_cast<long long>(sp * p.page_vecs) +
                      static_cast<long long>((base + walk[tid]) & ps_mask) * p.row_vecs;
                dst = static_cast<long long>(dp * p.page_vecs) +
                      static_cast<long long>((base + tid) & ps_mask) * p.row_vecs;
            } else if (first && p.err_count) {
                atomicAdd(p.err_count, 1);
            }
        }
        from[tid] = src;
        to[tid] = dst;
    }
    __syncthreads();
    const int per_plane = p.cache.n_kv_heads * p.row_vecs;
    const long long items = static_cast<long long>(per_plane) * p.n_planes;
    for (long long x = blockIdx.y * static_cast<long long>(kThreads) + tid; x < items;
         x += static_cast<long long>(gridDim.y) * kThreads) {
        const int plane = static_cast<int>(x / per_plane), rest = static_cast<int>(x - static_cast<long long>(plane) * per_plane);
        const int head = rest / p.row_vecs, vec = rest - head * p.row_vecs;
        uint4 *at = p.pages + plane * (p.page_vecs * p.cache.n_pages) +
                    (static_cast<size_t>(head) << p.cache.log2_ps) * p.row_vecs + vec;
        // Node walk[i] goes to row i <= walk[i]: no row is written before it has been read, and
        // those read ahead are rows of later nodes, behind every row written so far.
        for (int i = 1; i < kept; i += kAhead) {
            uint4 row[kAhead];
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                if (i + y < kept && from[i + y] >= 0) row[y] = at[from[i + y]];
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                if (i + y < kept && from[i + y] >= 0) at[to[i + y]] = row[y];
        }
    }
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_tree_accept(const int32_t *parents, const int32_t *tokens,
                                      const int32_t *sampled, int32_t *accepted, int32_t *n_kept,
                                      int32_t *new_lens, int32_t *next_tokens, int32_t *path,
                                      int n_seqs, int n_nodes, void *pages,
                                      const int32_t *page_table, const int32_t *kv_lens,
                                      int n_kv_heads, int page_size, int n_planes, int n_pages,
                                      size_t page_bytes, int max_pages, const int32_t *slots,
                                      int pool, int32_t *err_count, gdn_stream_t stream) {
    GDN_TRY(check_tree(parents, n_seqs, n_nodes));
    if (!tokens || !sampled || !accepted || !n_kept || !next_tokens) return GDN_ERR_NULL;
    GDN_TRY(check_pool(n_seqs, slots, pool));
    if (n_planes < 0) return GDN_ERR_SHAPE;
    AcceptParams p{};
    if (n_planes > 0 || kv_lens || new_lens) {
        if (!kv_lens || !new_lens) return GDN_ERR_NULL;
        if (page_size < 1 || max_pages < 1) return GDN_ERR_SHAPE;
        if (!supported_page_size(page_size) ||
            static_cast<long long>(max_pages) * page_size > 0x7fffffffLL)
            return GDN_ERR_UNSUPPORTED;
    }
    if (n_planes > 0) {
        if (!pages || !page_table) return GDN_ERR_NULL;
        if (n_kv_heads < 1 || n_pages < 1 || page_bytes == 0 ||
            page_bytes % (static_cast<size_t>(n_kv_heads) * page_size * 16) != 0)
            return GDN_ERR_SHAPE;
        if (!aligned16(pages)) return GDN_ERR_ALIGN;
        const size_t row_vecs = page_bytes / 16 / page_size / n_kv_heads;
        if (row_vecs * n_kv_heads > 0x7fffffffu) return GDN_ERR_UNSUPPORTED;
        p.row_vecs = static_cast<int>(row_vecs);
    }
    if (n_seqs == 0) return GDN_OK;
    p.parents = parents;
    p.tokens = tokens;
    p.sampled = sampled;
    p.accepted = accepted;
    p.n_kept = n_kept;
    p.new_lens = new_lens;
    p.next_tokens = next_tokens;
    p.path = path;
    p.pages = static_cast<uint4 *>(pages);
    p.cache = PagedCache{page_table, kv_lens, slots, pool, max_pages, n_pages, n_kv_heads,
                         kv_lens ? log2_of(page_size) : 0};
    p.n_nodes = n_nodes;
    p.n_planes = n_planes;
    p.page_vecs = page_bytes / 16;
    p.err_count = err_count;
    const long long items = static_cast<long long>(n_planes) * n_kv_heads * p.row_vecs;
    const long long shares = (items + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(n_seqs),
                    static_cast<unsigned>(shares < 1 ? 1 : shares > 65535 ? 65535 : shares));
    tree_accept_kernel<<<grid, kThreads, 0, as_cuda(stream)>>>(p);
    return launch_status();
}
