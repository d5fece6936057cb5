// gdn_pages.cu -- the paged cache's bookkeeping: new rows appended to the pages, pages
// reserved, forked, truncated (freed), compacted and copied.
//
// All of it is bound by the bytes moved (pages, appended rows) or, for the books alone, by
// launch latency. Pages are handed out in one order, lowest free page first and in call
// order, so the results are the same bits every time; the plan (who gets which page) is
// made by one CTA, the pages are then copied by the whole GPU.
#include "gdn_paged.cuh"

namespace gdn {
namespace {

constexpr int kPlan = 1024;  // threads of a planning CTA
constexpr int kSMs = 152;

// ------------------------------------------------------------------ append

struct AppendParams {
    PagedCache cache;
    SeqMap seqs;
    const uint4 *k, *v;
    uint4 *k_pages, *v_pages;
    size_t k_row, v_row;  // 16-byte units between tokens
    int n_seqs, head_vec;  // 16-byte units of a head's row
    int log2_parts;        // warps sharing a token
    int32_t *err_count;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendEach = 4;  // 16-byte units of a plane a lane holds at a time

// A few warps per new position: four while the batch is small and latency counts, one when
// there are enough tokens to fill the GPU (16 a SM). 64 tokens of 16 bf16 heads of 128: 2.7 us
// with four, 3.2 with one; 16384 tokens of 8 f16 heads of 128: 20.7 us with one (0.95 of the
// copy rate, with most of what it writes left in L2; 24 to 28 us from a cold L2), 28.3 with
// four. The rows are loaded first and find their place -- sequence, slot, length, page: four
// dependent loads -- while they are under way. Also, the warp of number n checks sequence n,
// last, and counts it when it is skipped.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    const int lane = threadIdx.x & 31;
    const long long warp = static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int part = static_cast<int>(warp & ((1 << p.log2_parts) - 1));
    const long long w = warp >> p.log2_parts;
    // start and position of sequence n's first new row; false when it is skipped
    auto find = [&](int n, size_t &t0, int &m, int &slot, int &len) {
        return p.seqs.range(n, t0, m) && p.cache.lookup(n, slot, len) && m <= len;
    };
    if (w < p.seqs.total) {
        const uint4 *k = p.k + w * p.k_row, *v = p.v + w * p.v_row;
        const int vecs = p.cache.n_kv_heads * p.head_vec, step = 32 << p.log2_parts;
        const int first = part * 32 + lane;
        uint4 kx[kAppendEach], vx[kAppendEach];
        auto load = [&](int i0) {
#pragma unroll
            for (int x = 0; x < kAppendEach; ++x) {
                const int i = i0 + x * step;
                if (i < vecs) {
                    kx[x] = k[i];
                    vx[x] = v[i];
                }
            }
        };
        load(first);
        const int n = p.seqs.cu ? warp_seq_of_position(p.seqs.cu, p.n_seqs, w)
                                : static_cast<int>(w / p.seqs.n_tokens);
        size_t t0;
        int m, slot, len;
        if (n >= 0 && find(n, t0, m, slot, len) && w < static_cast<long long>(t0) + m) {
            const int pos = len - m + static_cast<int>(w - static_cast<long long>(t0));
            const int page = p.cache.page_of(slot, pos);
            if (p.cache.page_ok(page)) {
                const int ps = 1 << p.cache.log2_ps;
                const size_t base =
                    (static_cast<size_t>(page) * p.cache.n_kv_heads * ps + (pos & (ps - 1))) * p.head_vec;
                for (int i0 = first; i0 < vecs; i0 += kAppendEach * step) {
                    if (i0 != first) load(i0);
#pragma unroll
                    for (int x = 0; x < kAppendEach; ++x) {
                        const int i = i0 + x * step;
                        if (i >= vecs) break;
                        const int h = i / p.head_vec;
                        const size_t to = base + static_cast<size_t>(h) * ps * p.head_vec + (i - h * p.head_vec);
                        p.k_pages[to] = kx[x];
                        p.v_pages[to] = vx[x];
                    }
                }
            } else if (part == 0 && lane == 0 && p.err_count) {
                atomicAdd(p.err_count, 1);
            }
        }
    }
    if (w < p.n_seqs && part == 0 && lane == 0 && p.err_count) {
        size_t t0;
        int m, slot, len;
        if (!find(static_cast<int>(w), t0, m, slot, len)) atomicAdd(p.err_count, 1);
    }
}

// ------------------------------------------------------------------ plans

// A call's scratch in its workspace.
struct Scratch {
    int32_t *head;   // [0] pages to copy, [1] live pages
    int32_t *free;   // free pages, ascending (compaction: the holes)
    int32_t *src, *dst;
    int32_t *remap;  // compaction: new place of page p, for p at or above the live count
    int32_t *state;  // per sequence or fork: the parent's length, -1 when skipped
};

__host__ __device__ inline Scratch scratch_of(void *ws, int n_pages) {
    int32_t *p = static_cast<int32_t *>(ws);
    const size_t n = static_cast<size_t>(n_pages);
    return Scratch{p, p + 16, p + 16 + n, p + 16 + 2 * n, p + 16 + 3 * n, p + 16 + 4 * n};
}

// Exclusive prefix of x over the CTA's threads, and the total. `part` holds 33 values.
__device__ __forceinline__ long long block_prefix(long long x, long long *part, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(FULL_MASK, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();  // earlier readers of part are done
    if (lane == 31) part[warp] = y;
    __syncthreads();
    if (warp == 0) {
        const long long own = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0;
        long long z = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(FULL_MASK, z, o);
            if (lane >= o) z += t;
        }
        part[lane] = z - own;
        if (lane == 31) part[32] = z;
    }
    __syncthreads();
    total = part[32];
    return part[warp] + y - x;
}

// Lists the first `want` free pages in ascending order; returns how many there are (at most
// `want`). Stops reading once it has them.
__device__ int list_free(const int32_t *refs, int n_pages, long long want, int32_t *out,
                         long long *part) {
    constexpr int kEach = 8;
    long long found = 0;
    for (long long base = 0; base < n_pages && found < want; base += kPlan * kEach) {
        const long long p0 = base + threadIdx.x * kEach;
        unsigned free = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (p0 + i < n_pages && refs[p0 + i] == 0) free |= 1u << i;
        long long total;
        long long rank = found + block_prefix(__popc(free), part, total);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if ((free >> i) & 1u) {
                if (rank < want) out[rank] = static_cast<int32_t>(p0 + i);
                ++rank;
            }
        found += total;
    }
    __syncthreads();
    return static_cast<int>(found < want ? found : want);
}

struct Books {
    int32_t *table, *kv_lens, *refs;
    const int32_t *slots;
    int pool, max_pages, n_pages, log2_ps;
    int32_t *err_count;

    __device__ __forceinline__ bool lookup(int slot, int &len) const {
        if (slot < 0 || slot >= pool) return false;
        len = kv_lens[slot];
        return len >= 0 && len <= (static_cast<long long>(max_pages) << log2_ps);
    }
    __device__ __forceinline__ int32_t *row(int slot) const {
        return table + static_cast<size_t>(slot) * max_pages;
    }
    __device__ __forceinline__ int pages(int len) const {
        return static_cast<int>((static_cast<long long>(len) + (1 << log2_ps) - 1) >> log2_ps);
    }
    __device__ __forceinline__ bool page_ok(int p) const { return p >= 0 && p < n_pages; }
    __device__ __forceinline__ void count_error() const {
        if (err_count) atomicAdd(err_count, 1);
    }
};

__global__ void __launch_bounds__(kPlan) reserve_plan_kernel(const Books b, const int32_t *n_new,
                                                             int n_seqs, Scratch ws) {
    __shared__ long long part[33];
    __shared__ int moves;
    if (threadIdx.x == 0) moves = 0;
    const int per = (n_seqs + kPlan - 1) / kPlan;
    const int i0 = min(static_cast<int>(threadIdx.x) * per, n_seqs), i1 = min(i0 + per, n_seqs);
    // pages sequence i asks for; -1 when it is skipped. `cow`: its last page is partly full
    // and shared, so it gets a copy of its own before it is written.
    auto need_of = [&](int i, int &slot, int &len, bool &cow) -> int {
        slot = b.slots ? b.slots[i] : i;
        const int add = n_new[i];
        if (!b.lookup(slot, len) || add < 0 ||
            static_cast<long long>(len) + add > (static_cast<long long>(b.max_pages) << b.log2_ps))
            return -1;
        cow = false;
        if (add > 0 && (len & ((1 << b.log2_ps) - 1)) != 0) {
            const int page = b.row(slot)[len >> b.log2_ps];
            cow = b.page_ok(page) && b.refs[page] > 1;
        }
        return b.pages(len + add) - b.pages(len) + (cow ? 1 : 0);
    };
    long long sum = 0;
    for (int i = i0; i < i1; ++i) {
        int slot, len;
        bool cow;
        const int need = need_of(i, slot, len, cow);
        ws.state[i] = need < 0 ? -1 : 2 * need + (cow ? 1 : 0);
        sum += max(need, 0);
    }
    long long total;
    long long rank = block_prefix(sum, part, total);
    const int n_free = list_free(b.refs, b.n_pages, min(total, static_cast<long long>(b.n_pages)),
                                 ws.free, part);
    for (int i = i0; i < i1; ++i) {
        const int st = ws.state[i];
        const int need = st < 0 ? 0 : st >> 1;
        const long long first = rank;
        rank += need;
        if (st < 0 || rank > n_free) {
            b.count_error();
            continue;
        }
        const int slot = b.slots ? b.slots[i] : i;
        const int len = b.kv_lens[slot], end = len + n_new[i];
        int32_t *row = b.row(slot);
        const int32_t *take = ws.free + first;
        if (st & 1) {
            const int col = len >> b.log2_ps, from = row[col], to = *take++;
            row[col] = to;
            b.refs[to] = 1;
            atomicSub(&b.refs[from], 1);
            const int m = atomicAdd(&moves, 1);
            ws.src[m] = from;
            ws.dst[m] = to;
        }
        for (int c = b.pages(len); c < b.pages(end); ++c) {
            const int to = *take++;
            row[c] = to;
            b.refs[to] = 1;
        }
        b.kv_lens[slot] = end;
    }
    __syncthreads();
    if (threadIdx.x == 0) ws.head[0] = moves;
}

__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const Books b, const int32_t *parents,
                                                          const int32_t *children, int n_forks,
                                                          Scratch ws) {
    __shared__ long long part[33];
    __shared__ int moves;
    if (threadIdx.x == 0) moves = 0;
    const int per = (n_forks + kPlan - 1) / kPlan;
    const int i0 = min(static_cast<int>(threadIdx.x) * per, n_forks), i1 = min(i0 + per, n_forks);
    const int ps_mask = (1 << b.log2_ps) - 1;
    long long sum = 0;
    for (int i = i0; i < i1; ++i) {
        int len, held;
        const bool ok = b.lookup(parents[i], len) && b.lookup(children[i], held) && held == 0 &&
                        parents[i] != children[i];
        ws.state[i] = ok ? len : -1;
        sum += ok && (len & ps_mask) != 0;
    }
    long long total;
    long long rank = block_prefix(sum, part, total);
    const int n_free = list_free(b.refs, b.n_pages, min(total, static_cast<long long>(b.n_pages)),
                                 ws.free, part);
    for (int i = i0; i < i1; ++i) {
        const int len = ws.state[i];
        const bool partial = len >= 0 && (len & ps_mask) != 0;
        const long long mine = rank;
        rank += partial;
        if (len < 0 || (partial && rank > n_free)) {
            ws.state[i] = -1;
            b.count_error();
            continue;
        }
        if (partial) {
            const int col = len >> b.log2_ps, from = b.row(parents[i])[col], to = ws.free[mine];
            b.row(children[i])[col] = to;
            b.refs[to] = 1;
            const int m = atomicAdd(&moves, 1);
            ws.src[m] = from;  // a bad id is skipped by the copy
            ws.dst[m] = to;
        }
        b.kv_lens[children[i]] = len;
    }
    __syncthreads();
    if (threadIdx.x == 0) ws.head[0] = moves;
}

// Live pages at or above the live count move into the holes below it, both in ascending
// order, so as few pages move as the dense pool allows and no page is both source and
// destination.
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Books b, Scratch ws,
                                                             int32_t *n_live_out) {
    __shared__ long long part[33];
    constexpr int kEach = 8;
    long long mine = 0;
    for (long long p = threadIdx.x; p < b.n_pages; p += kPlan) mine += b.refs[p] > 0;
    long long n_live;
    block_prefix(mine, part, n_live);
    long long done = 0;  // holes (low half) and movers (high half) so far
    for (long long base = 0; base < b.n_pages; base += kPlan * kEach) {
        const long long p0 = base + threadIdx.x * kEach;
        unsigned hole = 0, mover = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const long long p = p0 + i;
            if (p >= b.n_pages) break;
            const bool live = b.refs[p] > 0;
            if (!live && p < n_live) hole |= 1u << i;
            if (live && p >= n_live) mover |= 1u << i;
            if (!live && p >= n_live) ws.remap[p] = static_cast<int32_t>(p);
        }
        long long total;
        const long long rank = done + block_prefix(__popc(hole) + (static_cast<long long>(__popc(mover)) << 32),
                                                   part, total);
        long long h = rank & 0xFFFFFFFFll, m = rank >> 32;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if ((hole >> i) & 1u) ws.dst[h++] = static_cast<int32_t>(p0 + i);
            if ((mover >> i) & 1u) ws.src[m++] = static_cast<int32_t>(p0 + i);
        }
        done += total;
    }
    __syncthreads();
    const int moves = static_cast<int>(done >> 32);
    for (int i = threadIdx.x; i < moves; i += kPlan) {
        const int from = ws.src[i], to = ws.dst[i];
        ws.remap[from] = to;
        b.refs[to] = b.refs[from];
        b.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        ws.head[0] = moves;
        ws.head[1] = static_cast<int32_t>(n_live);
        if (n_live_out) *n_live_out = static_cast<int32_t>(n_live);
    }
}

// ------------------------------------------------------------------ the books' rows

// A forked child's row: the parent's full pages, each held once more.
__device__ __forceinline__ void fork_rows(const Books &b, const int32_t *parents,
                                          const int32_t *children, const int32_t *state,
                                          int n_forks) {
    const long long total = static_cast<long long>(n_forks) * b.max_pages;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
         x += step) {
        const int i = static_cast<int>(x / b.max_pages), c = static_cast<int>(x % b.max_pages);
        const int len = state[i];
        if (len < 0 || c >= (len >> b.log2_ps)) continue;
        const int page = b.row(parents[i])[c];
        b.row(children[i])[c] = page;
        if (b.page_ok(page)) atomicAdd(&b.refs[page], 1);
    }
}

// Entries of moved pages follow them.
__device__ __forceinline__ void compact_rows(const Books &b, const Scratch &ws) {
    const int n_live = ws.head[1];
    const long long total = static_cast<long long>(b.pool) * b.max_pages;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
         x += step) {
        const int slot = static_cast<int>(x / b.max_pages), c = static_cast<int>(x % b.max_pages);
        int len;
        if (!b.lookup(slot, len) || c >= b.pages(len)) continue;
        const int page = b.table[x];
        if (page >= n_live && page < b.n_pages) b.table[x] = ws.remap[page];
    }
}

// ------------------------------------------------------------------ page copies

struct MoveParams {
    uint4 *pages;
    const int32_t *src, *dst;
    const int32_t *count;  // NULL: n_moves
    int n_moves, n_planes, n_pages;
    size_t page_vec;  // 16-byte units of a page
    int32_t *err_count;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveEach = 8;  // 16-byte loads in flight per thread

// Pieces of 32 KB (a page of a plane, or part of one) dealt round-robin to the CTAs, all of a
// piece's loads ahead of its stores. HBM bounds it: 64 forks of a partly full page in 8 planes
// of 128 KB pages 24 us with their plan (0.8 of the copy rate); 0.53 GB of pages moved to make a
// pool dense 175 us (0.89).
__device__ __forceinline__ void move_pages(const MoveParams &p) {
    constexpr size_t kPiece = static_cast<size_t>(kMoveThreads) * kMoveEach;
    const int n = p.count ? *p.count : p.n_moves;
    const long long pieces = static_cast<long long>((p.page_vec + kPiece - 1) / kPiece);
    const long long total = pieces * n * p.n_planes;
    for (long long x = blockIdx.x; x < total; x += gridDim.x) {
        const int piece = static_cast<int>(x % pieces);
        const long long y = x / pieces;
        const int plane = static_cast<int>(y % p.n_planes), i = static_cast<int>(y / p.n_planes);
        const int from = p.src[i], to = p.dst[i];
        if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages) {
            if (piece == 0 && plane == 0 && threadIdx.x == 0 && p.err_count) atomicAdd(p.err_count, 1);
            continue;
        }
        const size_t plane0 = static_cast<size_t>(plane) * p.n_pages;
        const uint4 *a = p.pages + (plane0 + from) * p.page_vec;
        uint4 *b = p.pages + (plane0 + to) * p.page_vec;
        const size_t at = piece * kPiece + threadIdx.x;
        uint4 v[kMoveEach];
#pragma unroll
        for (int j = 0; j < kMoveEach; ++j)
            if (at + j * kMoveThreads < p.page_vec) v[j] = __ldcs(a + at + j * kMoveThreads);
#pragma unroll
        for (int j = 0; j < kMoveEach; ++j)
            if (at + j * kMoveThreads < p.page_vec) __stcs(b + at + j * kMoveThreads, v[j]);
    }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) { move_pages(p); }

__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const Books b, const int32_t *parents,
                                                            const int32_t *children, int n_forks,
                                                            Scratch ws, const MoveParams p) {
    fork_rows(b, parents, children, ws.state, n_forks);
    move_pages(p);
}

__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const Books b, Scratch ws,
                                                               const MoveParams p) {
    compact_rows(b, ws);
    move_pages(p);
}

// ------------------------------------------------------------------ truncation

constexpr int kTruncThreads = 128;

// One CTA per sequence: pages past the kept length lose a holder and leave the row.
__global__ void __launch_bounds__(kTruncThreads) truncate_kernel(const Books b,
                                                                 const int32_t *new_lens) {
    const int i = blockIdx.x;
    const int slot = b.slots ? b.slots[i] : i;
    int len = 0;
    const int keep = new_lens ? new_lens[i] : 0;
    const bool ok = b.lookup(slot, len) && keep >= 0 && keep <= len;
    __syncthreads();  // every thread has read the length
    if (!ok) {
        if (threadIdx.x == 0) b.count_error();
        return;
    }
    int32_t *row = b.row(slot);
    for (int c = b.pages(keep) + threadIdx.x; c < b.pages(len); c += kTruncThreads) {
        const int page = row[c];
        if (b.page_ok(page)) atomicSub(&b.refs[page], 1);
        row[c] = -1;
    }
    if (threadIdx.x == 0) b.kv_lens[slot] = keep;
}

// ------------------------------------------------------------------ host side

size_t pages_ws_bytes(int n_seqs, int n_pages) {
    return (16 + 4 * static_cast<size_t>(n_pages) + static_cast<size_t>(n_seqs)) * sizeof(int32_t);
}

gdn_status check_pages(const void *pages, int n_planes, int n_pages, size_t page_bytes) {
    if (!pages) return GDN_ERR_NULL;
    if (n_planes < 1 || n_pages < 1 || page_bytes < 16 || page_bytes % 16 != 0) return GDN_ERR_SHAPE;
    if (!aligned16(pages)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

gdn_status check_books(const int32_t *table, const int32_t *kv_lens, const int32_t *refs,
                       int page_size, int n_pages, int max_pages, int pool) {
    if (!table || !kv_lens || !refs) return GDN_ERR_NULL;
    if (page_size < 1 || n_pages < 1 || max_pages < 1 || pool < 1) return GDN_ERR_SHAPE;
    if (!supported_page_size(page_size) ||
        static_cast<long long>(max_pages) * page_size > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_ws(const void *ws, size_t bytes, int n_seqs, int n_pages) {
    if (!ws) return GDN_ERR_NULL;
    if (!aligned16(ws)) return GDN_ERR_ALIGN;
    return bytes < pages_ws_bytes(n_seqs, n_pages) ? GDN_ERR_SHAPE : GDN_OK;
}

MoveParams moves_from(void *pages, const Scratch &ws, int n_planes, int n_pages, size_t page_bytes) {
    return MoveParams{static_cast<uint4 *>(pages), ws.src, ws.dst, ws.head, 0, n_planes, n_pages,
                      page_bytes / 16, nullptr};
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_kv_append(const void *k, const void *v, void *k_pages, void *v_pages,
                         const int32_t *page_table, const int32_t *kv_lens,
                         const int32_t *cu_seqlens, int n_seqs, int total_tokens, int n_kv_heads,
                         int head_dim, int page_size, int n_pages, int max_pages, int k_stride,
                         int v_stride, int dtype, const int32_t *slots, int pool,
                         int32_t *err_count, gdn_stream_t stream) {
    if (!k || !v || !k_pages || !v_pages || !page_table || !kv_lens) return GDN_ERR_NULL;
    if (n_seqs < 0 || total_tokens < 0) return GDN_ERR_SHAPE;
    if (cu_seqlens == nullptr && n_seqs > 0 && total_tokens % n_seqs != 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_cache(n_kv_heads, head_dim, page_size, n_pages, max_pages, dtype));
    if (static_cast<long long>(n_kv_heads) * head_dim > 0x7fffffffLL ||
        k_stride < n_kv_heads * head_dim || v_stride < n_kv_heads * head_dim)
        return GDN_ERR_SHAPE;
    GDN_TRY(check_pool(n_seqs, slots, pool));
    const long long es = dtype_bytes(dtype);
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) ||
        k_stride * es % 16 != 0 || v_stride * es % 16 != 0)
        return GDN_ERR_ALIGN;
    if (n_seqs == 0 || total_tokens == 0) return GDN_OK;
    AppendParams p{};
    p.cache = PagedCache{page_table, kv_lens, slots, pool, max_pages, n_pages, n_kv_heads,
                         log2_of(page_size)};
    p.seqs = cu_seqlens ? SeqMap{cu_seqlens, total_tokens, total_tokens}
                        : uniform_seqs(n_seqs, total_tokens / n_seqs);
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.k_pages = static_cast<uint4 *>(k_pages);
    p.v_pages = static_cast<uint4 *>(v_pages);
    p.k_row = static_cast<size_t>(k_stride * es / 16);
    p.v_row = static_cast<size_t>(v_stride * es / 16);
    p.n_seqs = n_seqs;
    p.head_vec = static_cast<int>(head_dim * es / 16);
    p.err_count = err_count;
    p.log2_parts = total_tokens <= kSMs * 16 ? 2 : 0;
    const long long warps = static_cast<long long>(total_tokens > n_seqs ? total_tokens : n_seqs)
                            << p.log2_parts;
    const long long per = kAppendThreads / 32;
    kv_append_kernel<<<static_cast<unsigned>((warps + per - 1) / per), kAppendThreads, 0,
                       as_cuda(stream)>>>(p);
    return launch_status();
}

size_t gdn_pages_workspace_size(int n_seqs, int n_pages) {
    if (n_seqs < 0 || n_pages < 1) return 0;
    return pages_ws_bytes(n_seqs, n_pages);
}

gdn_status gdn_pages_copy(void *pages, const int32_t *src, const int32_t *dst, int n_copies,
                          int n_planes, int n_pages, size_t page_bytes, int32_t *err_count,
                          gdn_stream_t stream) {
    if (!src || !dst) return GDN_ERR_NULL;
    if (n_copies < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_pages(pages, n_planes, n_pages, page_bytes));
    if (n_copies == 0) return GDN_OK;
    const MoveParams p{static_cast<uint4 *>(pages), src, dst, nullptr, n_copies, n_planes, n_pages,
                       page_bytes / 16, err_count};
    move_kernel<<<kSMs * 8, kMoveThreads, 0, as_cuda(stream)>>>(p);
    return launch_status();
}

gdn_status gdn_pages_reserve(void *pages, int32_t *page_table, int32_t *kv_lens,
                             int32_t *page_refs, const int32_t *n_new, int n_seqs, int page_size,
                             int n_planes, int n_pages, size_t page_bytes, int max_pages,
                             const int32_t *slots, int pool, int32_t *err_count, void *workspace,
                             size_t workspace_bytes, gdn_stream_t stream) {
    if (!n_new) return GDN_ERR_NULL;
    if (n_seqs < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_pages(pages, n_planes, n_pages, page_bytes));
    GDN_TRY(check_books(page_table, kv_lens, page_refs, page_size, n_pages, max_pages, pool));
    GDN_TRY(check_pool(n_seqs, slots, pool));
    if (n_seqs == 0) return GDN_OK;
    GDN_TRY(check_ws(workspace, workspace_bytes, n_seqs, n_pages));
    const cudaStream_t s = as_cuda(stream);
    const Books b{page_table, kv_lens, page_refs, slots, pool, max_pages, n_pages,
                  log2_of(page_size), err_count};
    const Scratch ws = scratch_of(workspace, n_pages);
    reserve_plan_kernel<<<1, kPlan, 0, s>>>(b, n_new, n_seqs, ws);
    GDN_TRY(launch_status());
    move_kernel<<<kSMs * 8, kMoveThreads, 0, s>>>(
        moves_from(pages, ws, n_planes, n_pages, page_bytes));
    return launch_status();
}

gdn_status gdn_pages_fork(void *pages, int32_t *page_table, int32_t *kv_lens, int32_t *page_refs,
                          const int32_t *parents, const int32_t *children, int n_forks,
                          int page_size, int n_planes, int n_pages, size_t page_bytes,
                          int max_pages, int pool, int32_t *err_count, void *workspace,
                          size_t workspace_bytes, gdn_stream_t stream) {
    if (!parents || !children) return GDN_ERR_NULL;
    if (n_forks < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_pages(pages, n_planes, n_pages, page_bytes));
    GDN_TRY(check_books(page_table, kv_lens, page_refs, page_size, n_pages, max_pages, pool));
    if (n_forks == 0) return GDN_OK;
    GDN_TRY(check_ws(workspace, workspace_bytes, n_forks, n_pages));
    const cudaStream_t s = as_cuda(stream);
    const Books b{page_table, kv_lens, page_refs, nullptr, pool, max_pages, n_pages,
                  log2_of(page_size), err_count};
    const Scratch ws = scratch_of(workspace, n_pages);
    fork_plan_kernel<<<1, kPlan, 0, s>>>(b, parents, children, n_forks, ws);
    GDN_TRY(launch_status());
    fork_kernel<<<kSMs * 8, kMoveThreads, 0, s>>>(
        b, parents, children, n_forks, ws, moves_from(pages, ws, n_planes, n_pages, page_bytes));
    return launch_status();
}

gdn_status gdn_pages_truncate(int32_t *page_table, int32_t *kv_lens, int32_t *page_refs,
                              const int32_t *new_lens, int n_seqs, int page_size, int n_pages,
                              int max_pages, const int32_t *slots, int pool, int32_t *err_count,
                              gdn_stream_t stream) {
    if (n_seqs < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_books(page_table, kv_lens, page_refs, page_size, n_pages, max_pages, pool));
    GDN_TRY(check_pool(n_seqs, slots, pool));
    if (n_seqs == 0) return GDN_OK;
    const Books b{page_table, kv_lens, page_refs, slots, pool, max_pages, n_pages,
                  log2_of(page_size), err_count};
    truncate_kernel<<<n_seqs, kTruncThreads, 0, as_cuda(stream)>>>(b, new_lens);
    return launch_status();
}

gdn_status gdn_pages_compact(void *pages, int32_t *page_table, const int32_t *kv_lens,
                             int32_t *page_refs, int page_size, int n_planes, int n_pages,
                             size_t page_bytes, int max_pages, int pool, int32_t *n_live,
                             void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    GDN_TRY(check_pages(pages, n_planes, n_pages, page_bytes));
    GDN_TRY(check_books(page_table, kv_lens, page_refs, page_size, n_pages, max_pages, pool));
    GDN_TRY(check_ws(workspace, workspace_bytes, 0, n_pages));
    const cudaStream_t s = as_cuda(stream);
    const Books b{page_table, const_cast<int32_t *>(kv_lens), page_refs, nullptr, pool, max_pages,
                  n_pages, log2_of(page_size), nullptr};
    const Scratch ws = scratch_of(workspace, n_pages);
    compact_plan_kernel<<<1, kPlan, 0, s>>>(b, ws, n_live);
    GDN_TRY(launch_status());
    compact_kernel<<<kSMs * 8, kMoveThreads, 0, s>>>(
        b, ws, moves_from(pages, ws, n_planes, n_pages, page_bytes));
    return launch_status();
}

}  // extern "C"
