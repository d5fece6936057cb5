// gdn_attn_decode.cu -- attention of one new token, or a few draft tokens, of every
// sequence over its paged key/value cache (sm_103a).
//
//   s_j = scale q.k_j over the visible keys, o = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m}
//
// Every visible key and value is read once, so HBM bounds the call; the arithmetic has to
// stay out of the way. All query heads of a key head (times the draft tokens) form the rows
// of one small matrix product, so a key byte is read once for all of them.
//
// Work split. A unit is (sequence, key head, group of at most 16 rows); its keys are cut in
// tiles of 32 KB (64 KB for the widest heads). The units, in order, each weighing its tiles and
// one more for the turn to it, are dealt out evenly as one contiguous range per CTA, whatever
// the lengths: a ragged batch, one long sequence and many short ones all keep every SM equally
// busy, with no host knowledge of the lengths. (By tiles alone, the CTAs that got the short
// sequences were last: windowed fp32 pool 56 us, 48 with the turn weighed as one tile, 50 as two;
// 200 bf16 sequences of 16..2000 keys 149, 122, 129.) A unit that crosses a range boundary leaves
// partial results (m, l, o) in the workspace; the CTA that arrives last on it joins them in CTA
// order, so the bits do not depend on timing.
//
// Inside a CTA one warp walks the range and issues the TMA loads of the tiles' pages (and of
// q at a unit's first tile) into a ring of stages; four warps compute. Each of the four
// takes a quarter of a tile's keys for S = Q K^T, the row maxima are exchanged through
// shared memory, and each then takes a quarter of the head's columns for O += P V, so the
// running maximum is shared and O needs no join across warps.
//
// Measured (calls replayed back to back; the share is of the visible keys' and values' bytes
// at the copy rate): 64 sequences of 64..8192 bf16 keys, 16 key heads of 128: 168-172 us, 0.95
// to 0.97. Four of 60 to 131 thousand f16 keys, 2 key heads of 256: 99-100 us, 0.87. 64
// sequences with 4 draft tokens each, 4 key heads of 128: 60-64 us, 0.72 to 0.77. A pool of 256
// sequences with windows of 1024, 4 key heads of 64: fp32 48 us, 0.68; bf16 34 us, 0.48. One
// sequence of 1000 keys: 10 us. What lies above the bytes' time is 5 to 18 us in all of these,
// whatever that time is, and no pipe is busy in the short ones (tensor 23 %, issue 29 to 44 %),
// which points to a cost of a call -- lookups ahead of the first copy, the turn from unit to unit,
// joins, the spread of the CTAs' ends -- rather than to a rate. Its parts have not been measured
// apart.
#include <atomic>
#include <ctime>

#include "gdn_chunk_common.cuh"  // named_barrier_or
#include "gdn_paged.cuh"

namespace gdn {
namespace {

__device__ unsigned g_watchdog_attn_decode;

constexpr int kWarps = 4;                       // computing warps
constexpr int kCompute = 32 * kWarps;           // their threads
constexpr int kRows = 16;                       // rows of a unit
constexpr int kSMs = 152;
constexpr int kMaxCtas = 3 * kSMs;
constexpr int kJoin = 8;                        // partial results loaded together in a join
constexpr unsigned kTurn = 1;                   // what a unit weighs besides its tiles, in tiles

// kHead: the unit's first tile lies in this CTA's range. kEnd: the range's last tile.
enum : int { kFirst = 1, kLast = 2, kWhole = 4, kHead = 8, kEnd = 16 };  // kWhole, kHead: of a segment

// What the loading warp tells the computing warps: about a stage (the first key of its tile,
// and flags | blocks << 8, bit b of blocks: keys 8 b .. 8 b + 7 lie in a page that was
// loaded), and about a segment, the part of a unit in this CTA's range.
struct Segment {
    int seq, kvh, head_group, token_group, len, flags;
    int c0, c1;  // CTAs sharing the unit (when it is not whole here)

    // output row of the unit's (token, head), or -1 for one it has not
    template <typename P>
    __device__ __forceinline__ long long out_row(const P &p, int t, int h) const {
        const int token = token_group * p.tokens_per_unit + t, head = head_group * p.heads_per_unit + h;
        if (t >= p.tokens_per_unit || token >= p.n_tokens || head >= p.group) return -1;
        return (static_cast<long long>(seq) * p.n_tokens + token) * p.n_q_heads + kvh * p.group + head;
    }
};

struct Params {
    PagedCache cache;
    AttnMask mask;
    void *out;
    int n_seqs, n_tokens, n_q_heads, group;  // group: query heads of a key head
    int heads_per_unit, tokens_per_unit;     // rows of a unit: tokens x heads
    int head_groups, token_groups;
    float scale_log2;
    int32_t *err_count;
    float *partials;                 // [grid][2] records of kRows * (D + 2) floats
    unsigned long long *counters;    // [grid]
    unsigned long long nonce;
};

// RT: rows the arithmetic is laid out for (16-bit types: always 16, one matrix fragment).
template <typename T, int D, int RT>
struct Geometry {
    static constexpr bool kF32 = sizeof(T) == 4;
    // keys of a tile: 32 KB of K and V together, but for the widest heads (64 KB)
    static constexpr int KT = (D == 64 ? 2 : 1) * (kF32 ? 32 : 64);
    static constexpr int kCols = D * static_cast<int>(sizeof(T)) / 128;    // 128-byte columns
    static constexpr int kPlane = KT * D * static_cast<int>(sizeof(T));    // a K (or V) tile
    static constexpr int QR = RT < 8 ? 8 : RT;                             // q rows kept (whole swizzle atoms)
    static constexpr int kQ = QR * D * static_cast<int>(sizeof(T));
    static constexpr int kExtra = kF32 ? 2 * KT * RT * 4             // S, then P [key][row], two buffers
                                       : 2 * kRows * (KT + 8) * 2;   // P hi and lo [row][key]
    // CTAs per SM. A tile's chain of steps is latency: the more chains side by side the better,
    // as far as two stages and the registers of each allow. (fp32 heads of 64, three CTAs and
    // two: the windowed pool above 47.8 and 51.4 us, 200 sequences of 16..2000 keys 42.8 and 44.9,
    // 64 of up to 8192 49.6 both, four of 60 to 131 thousand 141 both.)
    static constexpr int kCtas = D == 256 ? 1 : kF32 && D == 64 && RT == 4 ? 3 : 2;
    // Threads: the computing warps, the loading warp and, where it costs no registers (three
    // CTAs of 5 warps fill the register file), a joining warp: it waits for the other CTAs of
    // the unit split at the range's start while the rest go on. (Windowed bf16 pool with heads of
    // 64: 33.6-34.2 us with it, 34.6 without; 200 ragged bf16 sequences of up to 2000 keys 121.8 and
    // 123.4.)
    static constexpr bool kJoinWarp = kCtas != 3;
    static constexpr int kThreads = kCompute + (kJoinWarp ? 64 : 32);
    // shared memory of a CTA, less alignment slack and the static part
    static constexpr int kBudget = (kCtas == 1 ? 232448 : kCtas == 2 ? 115712 : 76800) - 1024 - 2048;
    static constexpr int kStages = (kBudget - 2 * kQ - kExtra) / (2 * kPlane);
    static constexpr int kWarpKeys = KT / kWarps;
    static constexpr int kSmem = kStages * 2 * kPlane + 2 * kQ + kExtra + 1024;
    static_assert(kStages >= 2, "two stages at least");
};

// ------------------------------------------------------------------ waits

// False when a wait gave up: the warp leaves, and nothing of the units concerned is written.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *dead) {
    return gdn::warp_wait(bar, parity, dead, &g_watchdog_attn_decode);
}

// Counting the CTAs of a split unit that have stored their partial results. The word's upper
// 48 bits say whose count it is: this call's nonce, or anything else, which counts as 0 (so the
// workspace needs no initialisation). Every CTA tags a word that it sees untagged, then arrives
// with one addition. The CTA that completes the count clears the word. A captured call keeps its
// nonce over its replays; each leaves the words cleared, as a CTA that gave up a wait arrives at
// the units it has not finished all the same, with a partial result marked as none.
__device__ __forceinline__ bool tagged(unsigned long long word, unsigned long long nonce) {
    return (word >> 16) == nonce;
}

// `seen`: what the word held. (When it no longer does, another CTA has tagged it.)
__device__ __forceinline__ void tag(unsigned long long *word, unsigned long long seen,
                                    unsigned long long nonce) {
    if (!tagged(seen, nonce)) atomicCAS(word, seen, nonce << 16);
}

__device__ __forceinline__ bool last_arrival(unsigned long long *word, int n) {
    if (static_cast<int>(atomicAdd(word, 1ull) & 0xFFFFu) + 1 != n) return false;
    atomicExch(word, 0ull);
    return true;
}

// ------------------------------------------------------------------ matrix fragments

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared-memory tiles keep the pages' parts apart, each `rows` rows of 128 bytes for every
// 128-byte column ([part][column][row], the 128-byte swizzle within), as one copy per part
// brings them. Byte offset of row `row`, and of its 16-byte chunk `chunk`.
struct Tile {
    int log2_rows;   // rows of a part
    int part_bytes;  // of all columns of a part
    __device__ __forceinline__ uint32_t row(int r) const {
        return static_cast<uint32_t>((r >> log2_rows) * part_bytes + (r & ((1 << log2_rows) - 1)) * 128);
    }
    __device__ __forceinline__ uint32_t chunk(int r, int c) const {
        return static_cast<uint32_t>(((c >> 3) << (log2_rows + 7)) + (((c & 7) ^ (r & 7)) << 4));
    }
};

// A row's output from its sums; a row that saw nothing is 0.
__device__ __forceinline__ float finish(float o, float l, float inv) { return l == 0.0f ? 0.0f : o * inv; }

template <int LANES>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, o));
    return x;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(FULL_MASK, x, o);
    return x;
}

// ------------------------------------------------------------------ the join of a split unit

// By NT threads, once all of its CTAs have stored their partial results.
template <typename T, int D, int NT, typename Sync>
__device__ __forceinline__ void join_unit(const Params &p, const Segment &u, int tid, Sync sync,
                                          float (*part_of)[kRows], float *l_of) {
    constexpr int kRecord = kRows * (D + 2);
    const int c0 = u.c0, c1 = u.c1;
    T *out = static_cast<T *>(p.out);
    // The records' weights first: thread (g, r) takes every kGroups-th record of row r, and
    // leaves the weights in the records in place of the maxima. Then the rows, 4 columns a
    // thread, kJoin records' loads together.
    auto record_of = [&](int c) {
        // the first CTA holds the unit in its second record: it begins in its range
        return p.partials + static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * kRecord;
    };
    constexpr int kGroups = NT / kRows;
    {
        const int r = tid % kRows, g = tid / kRows;
        float top = -INFINITY;
#pragma unroll 4
        for (int c = c0 + g; c <= c1; c += kGroups)
            top = fmaxf(top, __ldcg(record_of(c) + kRows * D + r));
        part_of[g][r] = top;
        sync();
#pragma unroll
        for (int k = 0; k < kGroups; ++k) top = fmaxf(top, part_of[k][r]);
        const float base = top == -INFINITY ? 0.0f : top;
        float l = 0.0f;
        bool dead = false;
#pragma unroll 4
        for (int c = c0 + g; c <= c1; c += kGroups) {
            float *m = record_of(c) + kRows * D + r;
            const float w = fast_exp2(__ldcg(m) - base), part = __ldcg(m + kRows);
            __stcg(m, w);
            l = fmaf(w, part, l);
            dead |= part < 0.0f;
        }
        sync();  // the maxima have been read
        part_of[g][r] = dead ? -1.0f : l;
        __threadfence_block();
        sync();
        if (tid < kRows) {
            float sum_l = 0.0f;
            bool any_dead = false;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                any_dead |= part_of[k][tid] < 0.0f;
                sum_l += part_of[k][tid];
            }
            l_of[tid] = any_dead ? -1.0f : sum_l;
        }
        sync();
    }
    const int n_items = p.tokens_per_unit * p.heads_per_unit * (D / 4);
#pragma unroll 1
    for (int item = tid; item < n_items; item += NT) {
        const int r = item / (D / 4), col = (item % (D / 4)) * 4;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int c = c0; c <= c1; c += kJoin) {
            float4 x[kJoin];
            float w[kJoin];
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
                const bool in = c + k <= c1;
                const float *rec = record_of(in ? c + k : c1);
                x[k] = __ldcg(reinterpret_cast<const float4 *>(rec + r * D + col));
                w[k] = in ? __ldcg(rec + kRows * D + r) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
                if (w[k] == 0.0f) continue;  // a record that saw nothing may hold anything
                o.x = fmaf(w[k], x[k].x, o.x);
                o.y = fmaf(w[k], x[k].y, o.y);
                o.z = fmaf(w[k], x[k].z, o.z);
                o.w = fmaf(w[k], x[k].w, o.w);
            }
        }
        const long long row = u.out_row(p, r / p.heads_per_unit, r % p.heads_per_unit);
        const float l = l_of[r], inv = 1.0f / l;
        if (row < 0 || l < 0.0f) continue;
        const float4 y = make_float4(finish(o.x, l, inv), finish(o.y, l, inv), finish(o.z, l, inv),
                                     finish(o.w, l, inv));
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(out + row * D + col) = y;
        } else {
            *reinterpret_cast<uint2 *>(out + row * D + col) =
                make_uint2(Elem<T>::pack(y.x, y.y), Elem<T>::pack(y.z, y.w));
        }
    }
}

// ------------------------------------------------------------------ the kernel

template <typename T, int D, int RT>
__global__ void __launch_bounds__(Geometry<T, D, RT>::kThreads, Geometry<T, D, RT>::kCtas)
attn_decode_kernel(const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const Params p) {
    using G = Geometry<T, D, RT>;
    constexpr int KT = G::KT, kThreads = G::kThreads;
    constexpr int kRecord = kRows * (D + 2);  // floats of a partial result: o, then m, then l
    extern __shared__ uint8_t dyn[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *q_smem = smem + G::kStages * 2 * G::kPlane;
    uint8_t *extra = q_smem + 2 * G::kQ;

    __shared__ __align__(8) uint64_t full[G::kStages], empty[G::kStages], q_empty[2], early_ready;
    __shared__ int2 stages[G::kStages];
    __shared__ Segment segments[2], early;
    __shared__ unsigned warp_sum[kThreads / 32];
    __shared__ int sh_seq, sh_slot, sh_len, sh_dead, sh_join;
    __shared__ unsigned sh_seq_begin;
    __shared__ float red[kWarps][kRows];
    __shared__ __align__(16) float row_m[kRows], row_l[kRows];
    __shared__ float join_part[kCompute / kRows][kRows], early_part[2][kRows], early_l[kRows];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int subs = p.head_groups * p.token_groups;
    const unsigned units = static_cast<unsigned>(p.cache.n_kv_heads * subs);

    if (tid == kCompute) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        mbar_init(&q_empty[0], kWarps);
        mbar_init(&q_empty[1], kWarps);
        mbar_init(&early_ready, kWarps);
        fence_mbar_init();
        sh_dead = 0;
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }

    // Tiles of one unit of sequence n (1 when it sees nothing: its rows are zeros), 0 when
    // the sequence is skipped.
    auto tiles_of = [&](int n, int &slot, int &len) -> unsigned {
        if (!p.cache.lookup(n, slot, len)) return 0;
        return static_cast<unsigned>(max(1, walk_tiles<KT>(p.mask, len - p.n_tokens, len - 1).count));
    };

    // ---- this CTA's range of tiles: a thread's slab of sequences, the slabs' prefixes
    const int per = (p.n_seqs + kThreads - 1) / kThreads;
    const int n0 = min(tid * per, p.n_seqs), n1 = min(n0 + per, p.n_seqs);
    unsigned sum = 0;
    int slot0 = 0, len0 = 0;
    for (int n = n0; n < n1; ++n) {
        const unsigned t = tiles_of(n, slot0, len0);
        if (t == 0 && blockIdx.x == 0 && p.err_count) atomicAdd(p.err_count, 1);
        if (t != 0) sum += (t + kTurn) * units;
    }
    unsigned before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(FULL_MASK, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) warp_sum[warp] = before;
    before -= sum;
    __syncthreads();
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    // The ranges, in units' weights: a unit is kTurn places without a tile, then its tiles. No
    // range is without a tile, so the CTAs of a split unit are consecutive and all of them
    // arrive; the first `longer` are one place longer.
    const unsigned ranges = min(gridDim.x, total / (1 + kTurn));
    if (blockIdx.x >= ranges) return;
    const unsigned each = total / ranges, longer = total - each * ranges;
    auto range_begin = [&](unsigned c) { return c * each + min(c, longer); };
    const unsigned begin = range_begin(blockIdx.x), end = range_begin(blockIdx.x + 1);
    auto owner = [&](unsigned x) {  // of place x
        const unsigned split = longer * (each + 1);
        return static_cast<int>(x < split ? x / (each + 1) : longer + (x - split) / each);
    };
    if (begin >= before && begin < before + sum) {
        unsigned at = before;
        for (int n = n0; n < n1; ++n) {
            unsigned w = sum;
            if (per != 1) {
                const unsigned t = tiles_of(n, slot0, len0);
                w = t == 0 ? 0 : (t + kTurn) * units;
            }
            if (begin < at + w) {
                sh_seq = n;
                sh_slot = slot0;
                sh_len = len0;
                sh_seq_begin = at;
                break;
            }
            at += w;
        }
    }
    __syncthreads();

    auto k_tile = [&](int s) { return smem + s * 2 * G::kPlane; };
    auto v_tile = [&](int s) { return smem + s * 2 * G::kPlane + G::kPlane; };
    constexpr int kLog2KT = KT == 128 ? 7 : KT == 64 ? 6 : 5;
    const int log2_box = min(p.cache.log2_ps, kLog2KT);  // keys of a page's part of a tile
    const Tile tile{log2_box, D * static_cast<int>(sizeof(T)) << log2_box};

    if (warp == kWarps) {
        // ---------------------------------------------------------- the loading warp
        // The warp runs converged, one elected lane issuing.
        const bool leader = elect_one();
        const int ps = 1 << p.cache.log2_ps;
        const int box = 1 << log2_box, n_box = KT >> log2_box;
        const unsigned lane_blocks = ((1u << (box / 8)) - 1u) << ((lane * (box / 8)) & 31);
        int n = sh_seq, slot = sh_slot, len = sh_len;
        unsigned seq_begin = sh_seq_begin, at = begin;
        TileWalk walk = walk_tiles<KT>(p.mask, len - p.n_tokens, len - 1);
        unsigned tiles = static_cast<unsigned>(max(1, walk.count));
        unsigned unit = (at - seq_begin) / (tiles + kTurn);
        int st = 0, seg = 0;
        unsigned st_round = 0;
        while (at < end) {
            const unsigned unit_begin = seq_begin + unit * (tiles + kTurn) + kTurn;  // its first tile
            const unsigned unit_end = unit_begin + tiles;
            at = max(at, unit_begin);
            if (at >= end) break;
            const unsigned seg_end = min(unit_end, end);
            int kvh = static_cast<int>(unit), hg = 0, tg = 0;
            if (subs > 1) {
                kvh = static_cast<int>(unit) / subs;
                const int sub = static_cast<int>(unit) - kvh * subs;
                hg = sub / p.token_groups;
                tg = sub - hg * p.token_groups;
            }
            const bool whole = at == unit_begin && seg_end == unit_end;
            // the page of lane i's part of a tile, looked up one tile ahead of its load; -1 for a
            // part nobody sees (its id is not read: pages before the window may be gone)
            auto page_at = [&](int idx) -> int {
                if (walk.count == 0 || lane >= n_box) return -1;
                const int key = walk.tile(idx) * KT + lane * box;
                if (key > len - 1) return -1;
                if (!(len - p.n_tokens - (key + box - 1) < p.mask.window || key < p.mask.sinks)) return -1;
                const int page = p.cache.page_of(slot, key);
                if (unit == 0 && p.err_count && !p.cache.page_ok(page)) atomicAdd(p.err_count, 1);
                return page;
            };
            int i = static_cast<int>(at - unit_begin);
            int page = page_at(i);
            // the segment, and q
            if (seg >= 2 && !warp_wait(&q_empty[seg & 1], ((seg >> 1) - 1) & 1, &sh_dead)) goto leave;
            for (bool first = true; at < seg_end; ++at, ++i, first = false) {
                const int next_page = at + 1 < seg_end ? page_at(i + 1) : -1;
                if (st_round > 0 && !warp_wait(&empty[st], (st_round - 1) & 1, &sh_dead)) goto leave;
                const int key0 = walk.count ? walk.tile(i) * KT : 0;
                const bool ok = p.cache.page_ok(page);
                const unsigned have = __ballot_sync(FULL_MASK, ok);
                const unsigned blocks = __reduce_or_sync(FULL_MASK, ok ? lane_blocks : 0u);
                const int row = (page * p.cache.n_kv_heads + kvh) * ps + (key0 & (ps - 1));
                for (int b = 0; b < n_box; ++b) {
                    const int r = __shfl_sync(FULL_MASK, row, b);
                    if (leader && ((have >> b) & 1u)) {
                        tma_load_3d(k_tile(st) + b * tile.part_bytes, &k_map, 0, r, 0, &full[st]);
                        tma_load_3d(v_tile(st) + b * tile.part_bytes, &v_map, 0, r, 0, &full[st]);
                    }
                }
                if (leader) {
                    // The stage is full once the copies have landed and this thread has arrived:
                    // what there is to say of it is worked out while they are under way.
                    uint32_t bytes = (static_cast<uint32_t>(__popc(have)) << log2_box) * D * sizeof(T) * 2u;
                    if (first) {
                        const int head0 = kvh * p.group + hg * p.heads_per_unit;
                        const int token0 = n * p.n_tokens + tg * p.tokens_per_unit;
#pragma unroll
                        for (int cb = 0; cb < G::kCols; ++cb)
                            tma_load_3d(q_smem + (seg & 1) * G::kQ + cb * G::QR * 128, &q_map,
                                        cb * static_cast<int>(128 / sizeof(T)), head0, token0, &full[st]);
                        bytes += static_cast<uint32_t>(p.heads_per_unit * p.tokens_per_unit) * D * sizeof(T);
                        Segment sg;
                        sg.seq = n;
                        sg.kvh = kvh;
                        sg.head_group = hg;
                        sg.token_group = tg;
                        sg.len = len;
                        sg.flags = (whole ? kWhole : 0) | (unit_begin >= begin ? kHead : 0);
                        sg.c0 = whole ? 0 : owner(unit_begin);
                        sg.c1 = whole ? 0 : owner(unit_end - 1);
                        segments[seg & 1] = sg;
                    }
                    const bool last = at + 1 == seg_end, at_end = end <= unit_end + kTurn;
                    stages[st] = make_int2(key0, (first ? kFirst : 0) | (last ? kLast : 0) |
                                                     (last && at_end ? kEnd : 0) |
                                                     static_cast<int>(blocks << 8));
                    mbar_arrive_expect_tx(&full[st], bytes);
                }
                __syncwarp();
                if (++st == G::kStages) {
                    st = 0;
                    ++st_round;
                }
                page = next_page;
            }
            ++seg;
            if (at == unit_end && ++unit == units && at < end) {
                seq_begin = unit_end;
                unit = 0;
                do {
                    tiles = tiles_of(++n, slot, len);
                } while (tiles == 0 && n + 1 < p.n_seqs);
                if (tiles == 0) break;  // not reached: the range says tiles are left
                walk = walk_tiles<KT>(p.mask, len - p.n_tokens, len - 1);
            }
        }
    leave:
        if (*static_cast<volatile int *>(&sh_dead)) drain_in_flight();
        return;
    }
    if (G::kJoinWarp && warp == kWarps + 1) {
        // ---------------------------------------------------------- the joining warp
        // The computing warps come to this barrier whether a wait of theirs gave up or not, which
        // takes them a bounded wait or two; what they handed over before has to be counted.
        bool ready = warp_wait(&early_ready, 0, &sh_dead);
        for (int i = 0; i < 2 && !ready; ++i) ready = __all_sync(FULL_MASK, mbar_wait(&early_ready, 0));
        if (!ready || (early.flags & kWhole)) return;
        int last = 0;
        if (lane == 0) {
            __threadfence();
            last = last_arrival(p.counters + early.c0, early.c1 - early.c0 + 1);
            __threadfence();
        }
        if (__shfl_sync(FULL_MASK, last, 0))
            join_unit<T, D, 32>(p, early, lane, [] { __syncwarp(); }, early_part, early_l);
        return;
    }

    // -------------------------------------------------------------- the computing warps
    // 16-bit: NT tiles of 8 columns (a quarter of the head), rows lane/4 and lane/4 + 8
    constexpr int NT = D / 32;
    constexpr int KN = G::kWarpKeys / 8;  // 8-key tiles of S of a warp
    float o16[G::kF32 ? 1 : NT][4];
    uint32_t qf[G::kF32 ? 1 : D / 16][4];
    // fp32: LPR threads to a row in the softmax; in P V a lane holds 4 columns, C4 lanes
    // span the quarter and NKG groups of lanes split the keys
    constexpr int LPR = kCompute / RT;
    constexpr int C4 = D / 16;
    constexpr int NKG = 32 / C4;
    float o32[G::kF32 ? RT : 1][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    Segment sg{};
    // rows of this thread (16-bit: lane / 4 and lane / 4 + 8; fp32: the row of its scores):
    // token and head in the unit, position
    const int row0 = G::kF32 ? tid / LPR : lane >> 2, row1 = (lane >> 2) + 8;
    const int tok0 = row0 / p.heads_per_unit, tok1 = row1 / p.heads_per_unit;
    int pos0 = 0, pos1 = 0;
    unsigned long long word_seen = 0;
    bool had_early = false;
    int handed = 0;  // split units this CTA has stored its part of
    int seg = 0, s = 0;
    uint32_t phase = 0;

    bool more = true;  // tiles in this range
    bool gave_up = false;
    // A tile's first barrier also tells whether some warp's wait for it gave up: then all
    // computing warps leave together.
    auto left_alone = [&](int flags) {
        if (chunk::named_barrier_or(1, kCompute, false)) return true;
        if ((flags & kFirst) && tid == 0 && !(sg.flags & kWhole))
            word_seen = *reinterpret_cast<volatile unsigned long long *>(p.counters + sg.c0);
        return false;
    };
    for (int it = 0; more; ++it) {
        if (!warp_wait(&full[s], phase, &sh_dead)) {
            chunk::named_barrier_or(1, kCompute, true);
            gave_up = true;
            break;
        }
        const int2 stage = stages[s];
        const int key0 = stage.x, flags = stage.y;
        const unsigned blocks = static_cast<unsigned>(stage.y) >> 8;
        more = !(flags & kEnd);
        if (flags & kFirst) {
            sg = segments[seg & 1];
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.0f;
            const int base = sg.len - p.n_tokens + sg.token_group * p.tokens_per_unit;
            pos0 = base + tok0;
            pos1 = base + tok1;
        }
        const int p_first = sg.len - p.n_tokens, p_last = sg.len - 1;
        const bool clean = blocks == (1u << (KT / 8)) - 1u && key0 + KT - 1 <= p_first &&
                           (p_last - key0 < p.mask.window || key0 + KT <= p.mask.sinks);
        // The keys that P V takes, whole groups of kGroup: those between the first and the last
        // that some row sees.
        constexpr int kGroup = G::kF32 ? 8 : 16;
        int g_lo = 0, g_hi = KT / kGroup;
        if (!clean) {
            const int lo = p.mask.first(max(p_first, 0)) - key0;  // of the window
            int a = KT, b = 0;
            if (lo < KT) {
                a = max(lo, 0);
                b = min(p_last - key0 + 1, KT);
            }
            const int sinks = min(p.mask.sinks, p_last + 1) - key0;
            if (sinks > 0) {
                a = 0;
                b = max(b, min(sinks, KT));
            }
            g_lo = a / kGroup;
            g_hi = (b + kGroup - 1) / kGroup;
            // Keys of this warp's part of the tile, among those, that no row of the unit sees:
            // their V rows are cleared, so that whatever the page holds there (an infinity, a
            // NaN) cannot reach the sum through a weight of 0.
            const int i = warp * G::kWarpKeys + lane, key = key0 + i;
            const bool dead = lane < G::kWarpKeys && i / kGroup >= g_lo && i / kGroup < g_hi &&
                              (!((blocks >> ((i >> 3) & 31)) & 1u) || key > p_last ||
                               !(p_first - key < p.mask.window || key < p.mask.sinks));
            const unsigned left = __ballot_sync(FULL_MASK, dead);
            if (left != 0) {
                constexpr int kChunks = G::kCols * 8, kLanes = kChunks < 32 ? kChunks : 32;
                constexpr int kStep = 32 / kLanes;  // rows at a time
#pragma unroll 4
                for (int x = lane / kLanes; x < G::kWarpKeys; x += kStep) {
                    if (!((left >> x) & 1u)) continue;
                    const int r = warp * G::kWarpKeys + x;
                    uint8_t *row = v_tile(s) + tile.row(r);
#pragma unroll
                    for (int c = lane % kLanes; c < kChunks; c += kLanes)
                        *reinterpret_cast<uint4 *>(row + tile.chunk(r, c)) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();  // before the stage's next copy overwrites them
        }
        const uint8_t *q_here = q_smem + (seg & 1) * G::kQ;

        if constexpr (!G::kF32) {
            const uint32_t ks = smem_addr(k_tile(s)), vs = smem_addr(v_tile(s));
            if (flags & kFirst) {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
                const Tile q_tile{4, 0};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    ldsm4(qf[kk], smem_addr(q_here) + r * 128 + q_tile.chunk(r, 2 * kk + (lane >> 4)));
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_empty[seg & 1]);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o16[j][e] = 0.0f;
            }
            // S = Q K^T for this warp's keys, 16 at a time (two chains of products per 8 keys)
            float sc[KN][4];
#pragma unroll
            for (int h = 0; h < KN / 2; ++h) {
                float acc[2][2][4] = {};
                const int key = warp * G::kWarpKeys + h * 16 + (lane & 7) + (lane >> 4) * 8;
                const uint32_t kr = ks + tile.row(key);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b[4];
                    ldsm4(b, kr + tile.chunk(key, 2 * kk + ((lane >> 3) & 1)));
                    mma16816<T>(acc[kk & 1][0], qf[kk], b[0], b[1]);
                    mma16816<T>(acc[kk & 1][1], qf[kk], b[2], b[3]);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[2 * h + b][e] = (acc[0][b][e] + acc[1][b][e]) * p.scale_log2;
            }
            if (!clean) {
                // keys of the tile that a row sees: [lo, hi] and, up to hi, those below `sink`
                const int hi0 = pos0 - key0, hi1 = pos1 - key0, sink = p.mask.sinks - key0;
                const int lo0 = hi0 < p.mask.window ? 0 : hi0 - p.mask.window + 1;
                const int lo1 = hi1 < p.mask.window ? 0 : hi1 - p.mask.window + 1;
#pragma unroll
                for (int b = 0; b < KN; ++b) {
                    const int i0 = warp * G::kWarpKeys + b * 8;
                    const bool there = (blocks >> (i0 >> 3)) & 1u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = i0 + 2 * (lane & 3) + (e & 1);
                        const bool ok = there && i <= (e < 2 ? hi0 : hi1) && (i >= (e < 2 ? lo0 : lo1) || i < sink);
                        if (!ok) sc[b][e] = -INFINITY;
                    }
                }
            }
            const int r0 = row0;
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int b = 0; b < KN; ++b) {
                t0 = fmaxf(t0, fmaxf(sc[b][0], sc[b][1]));
                t1 = fmaxf(t1, fmaxf(sc[b][2], sc[b][3]));
            }
            t0 = group_max<4>(t0);
            t1 = group_max<4>(t1);
            if ((lane & 3) == 0) {
                red[warp][r0] = t0;
                red[warp][r0 + 8] = t1;
            }
            if (left_alone(flags)) {
                gave_up = true;
                break;
            }
            const float old0 = m0, old1 = m1;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                m0 = fmaxf(m0, red[w][r0]);
                m1 = fmaxf(m1, red[w][r0 + 8]);
            }
            // a row that has seen nothing yet keeps its weights at 2^-inf = 0
            float base0 = m0 == -INFINITY ? 0.0f : m0;
            float base1 = m1 == -INFINITY ? 0.0f : m1;
            const float corr0 = fast_exp2(old0 - base0), corr1 = fast_exp2(old1 - base1);
            // P is kept in two parts of the cache's type, hi + lo, so that rounding the
            // weights adds nothing to the output's own rounding; the tensor pipe has room.
            // (float16's steps end at 2^-24, so its weights go up to 2^14 instead of 1: what is
            // lost of a small one is 2^-39 of the largest. l carries the same factor.)
            base0 -= Elem<T>::kWeightBits;
            base1 -= Elem<T>::kWeightBits;
            uint8_t *ph = extra, *pl = extra + kRows * (KT + 8) * 2;
            l0 *= corr0;
            l1 *= corr1;
#pragma unroll
            for (int b = 0; b < KN; ++b) {
                const float x0 = fast_exp2(sc[b][0] - base0), x1 = fast_exp2(sc[b][1] - base0);
                const float y0 = fast_exp2(sc[b][2] - base1), y1 = fast_exp2(sc[b][3] - base1);
                l0 += x0 + x1;
                l1 += y0 + y1;
                const int col = warp * G::kWarpKeys + b * 8 + 2 * (lane & 3);
                const uint32_t oa = static_cast<uint32_t>(r0 * (KT + 8) + col) * 2u;
                const uint32_t ob = oa + 8 * (KT + 8) * 2u;
                const uint32_t xh = Elem<T>::pack(x0, x1), yh = Elem<T>::pack(y0, y1);
                const float2 xf = Elem<T>::unpack(xh), yf = Elem<T>::unpack(yh);
                *reinterpret_cast<uint32_t *>(ph + oa) = xh;
                *reinterpret_cast<uint32_t *>(ph + ob) = yh;
                *reinterpret_cast<uint32_t *>(pl + oa) = Elem<T>::pack(x0 - xf.x, x1 - xf.y);
                *reinterpret_cast<uint32_t *>(pl + ob) = Elem<T>::pack(y0 - yf.x, y1 - yf.y);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o16[j][0] *= corr0;
                o16[j][1] *= corr0;
                o16[j][2] *= corr1;
                o16[j][3] *= corr1;
            }
            named_barrier_sync(2, kCompute);
            const uint32_t poff = static_cast<uint32_t>(
                ((lane & 7) + ((lane >> 3) & 1) * 8) * (KT + 8) + (lane >> 4) * 8) * 2u;
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                if (kk < g_lo || kk >= g_hi) continue;
                uint32_t ah[4], al[4];
                ldsm4(ah, smem_addr(ph) + poff + kk * 32);
                ldsm4(al, smem_addr(pl) + poff + kk * 32);
                const int vrow = kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
                const uint32_t vr = vs + tile.row(vrow);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b[4];
                    ldsm4_trans(b, vr + tile.chunk(vrow, warp * NT + j + (lane >> 4)));
                    mma16816<T>(o16[j], ah, b[0], b[1]);
                    mma16816<T>(o16[j + 1], ah, b[2], b[3]);
                    mma16816<T>(o16[j], al, b[0], b[1]);
                    mma16816<T>(o16[j + 1], al, b[2], b[3]);
                }
            }
        } else {
            // fp32: the products on the FP32 pipes, every operand read once per warp
            // S, then P: [KT][RT]. Two buffers in turn: a warp may start on the next tile's
            // S while another still reads this tile's P
            float *sp = reinterpret_cast<float *>(extra) + (it & 1) * KT * RT;
            if (flags & kFirst) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o32[r][e] = 0.0f;
            }
            constexpr int KH = G::kWarpKeys / 8;  // keys of a lane
            {
                // lane: every 8th key of the warp's and a quarter of the dot product
                const int i0 = warp * G::kWarpKeys + (lane & 7), quarter = lane >> 3;
                // Chunk c of the quarter stands at its column's place (c & 7) ^ turn ^ (row & 7):
                // the swizzle, the quarter's half of a column (D = 64) and a turn of its own
                // that starts the quarters' lanes in different banks.
                const int turn = D >= 128 ? 2 * quarter : 4 * (quarter & 1) + (quarter >> 1);
                const uint32_t k_place = static_cast<uint32_t>(turn ^ (i0 & 7)) << 4;
                const uint32_t q_place = static_cast<uint32_t>(turn) << 4;
                constexpr int kQuarterCols = D >= 128 ? D / 128 : 1;  // 128-byte columns it touches
                const int col0 = D >= 128 ? quarter * kQuarterCols : quarter >> 1;
                const uint8_t *kr[KH];
#pragma unroll
                for (int h = 0; h < KH; ++h)
                    kr[h] = k_tile(s) + tile.row(i0 + 8 * h) + (col0 << (log2_box + 7));
                const uint8_t *qr = q_here + col0 * G::QR * 128;
                float acc[KH][RT];
#pragma unroll
                for (int h = 0; h < KH; ++h)
#pragma unroll
                    for (int r = 0; r < RT; ++r) acc[h][r] = 0.0f;
#pragma unroll
                for (int col = 0; col < kQuarterCols; ++col) {
#pragma unroll (RT == 16 ? 1 : RT == 8 ? 2 : 4)
                    for (int c = 0; c < (D >= 128 ? 8 : 4); ++c) {
                        float4 kv[KH];
#pragma unroll
                        for (int h = 0; h < KH; ++h)
                            kv[h] = *reinterpret_cast<const float4 *>(kr[h] + (col << (log2_box + 7)) +
                                                                      (k_place ^ (c << 4)));
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const float4 qv = *reinterpret_cast<const float4 *>(
                                qr + col * G::QR * 128 + r * 128 + (q_place ^ ((c ^ (r & 7)) << 4)));
#pragma unroll
                            for (int h = 0; h < KH; ++h) {
                                acc[h][r] = fmaf(qv.x, kv[h].x, acc[h][r]);
                                acc[h][r] = fmaf(qv.y, kv[h].y, acc[h][r]);
                                acc[h][r] = fmaf(qv.z, kv[h].z, acc[h][r]);
                                acc[h][r] = fmaf(qv.w, kv[h].w, acc[h][r]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < KH; ++h)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        acc[h][r] += __shfl_xor_sync(FULL_MASK, acc[h][r], 8);
                        acc[h][r] += __shfl_xor_sync(FULL_MASK, acc[h][r], 16);
                        if ((r & 3) == quarter) sp[(i0 + 8 * h) * RT + r] = acc[h][r] * p.scale_log2;
                    }
            }
            if (left_alone(flags)) {
                gave_up = true;
                break;
            }
            {
                const int r = tid / LPR, part = tid % LPR;
                float x[KT / LPR];
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < KT / LPR; ++i) {
                    const int k = part + i * LPR;
                    x[i] = sp[k * RT + r];
                    if (!clean && (!((blocks >> (k >> 3)) & 1u) || !p.mask.sees(pos0, key0 + k))) x[i] = -INFINITY;
                    top = fmaxf(top, x[i]);
                }
                const float old = m0;
                m0 = fmaxf(m0, group_max<LPR>(top));
                const float base = m0 == -INFINITY ? 0.0f : m0;
                const float corr = fast_exp2(old - base);
                l0 *= corr;
#pragma unroll
                for (int i = 0; i < KT / LPR; ++i) {
                    x[i] = fast_exp2(x[i] - base);
                    l0 += x[i];
                    sp[(part + i * LPR) * RT + r] = x[i];
                }
                if (part == 0) row_m[r] = corr;
            }
            named_barrier_sync(2, kCompute);
            {
                const int c4 = lane % C4, kg = lane / C4;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float corr = row_m[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o32[r][e] *= corr;
                }
#pragma unroll (RT == 16 ? 1 : RT == 8 ? 2 : 4)
                for (int j = g_lo * (8 / NKG); j < g_hi * (8 / NKG); ++j) {
                    // for D = 64 two keys share a quarter-warp's read: 4 apart, so that
                    // the swizzle keeps them in different banks
                    const int i = NKG == 8 ? (kg >> 1) + 4 * (kg & 1) + 8 * j : kg + NKG * j;
                    const float4 vv = *reinterpret_cast<const float4 *>(
                        v_tile(s) + tile.row(i) + tile.chunk(i, warp * C4 + c4));
#pragma unroll
                    for (int r = 0; r < RT; r += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(sp + i * RT + r);
                        const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            o32[r + a][0] = fmaf(ws[a], vv.x, o32[r + a][0]);
                            o32[r + a][1] = fmaf(ws[a], vv.y, o32[r + a][1]);
                            o32[r + a][2] = fmaf(ws[a], vv.z, o32[r + a][2]);
                            o32[r + a][3] = fmaf(ws[a], vv.w, o32[r + a][3]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        if ((flags & kFirst) && tid == 0 && !(sg.flags & kWhole)) tag(p.counters + sg.c0, word_seen, p.nonce);
        if (++s == G::kStages) {
            s = 0;
            phase ^= 1;
        }
        if (!(flags & kLast)) continue;

        // ---------------------------------------------------------- the segment's end
        if constexpr (G::kF32) {
            if (lane == 0) mbar_arrive(&q_empty[seg & 1]);
        }
        ++seg;
        named_barrier_sync(1, kCompute);  // the last tile's corrections have been read
        if constexpr (!G::kF32) {
            const float a = group_sum<4>(l0), b = group_sum<4>(l1);
            if ((lane & 3) == 0) {
                red[warp][lane >> 2] = a;
                red[warp][(lane >> 2) + 8] = b;
                if (warp == 0) {
                    row_m[lane >> 2] = m0;
                    row_m[(lane >> 2) + 8] = m1;
                }
            }
            named_barrier_sync(2, kCompute);
            if (tid < kRows) row_l[tid] = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
        } else {
            const float a = group_sum<LPR>(l0);
            if (tid % LPR == 0) {
                row_m[tid / LPR] = m0;
                row_l[tid / LPR] = a;
            }
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int o = C4; o < 32; o <<= 1)
                        o32[r][e] += __shfl_xor_sync(FULL_MASK, o32[r][e], o);
        }
        named_barrier_sync(1, kCompute);

        T *out = static_cast<T *>(p.out);
        const bool whole = sg.flags & kWhole;
        float *record = p.partials +
                        static_cast<size_t>(2 * blockIdx.x + ((sg.flags & kHead) ? 1 : 0)) * kRecord;
        if constexpr (!G::kF32) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = half ? row1 : row0, t = half ? tok1 : tok0;
                const long long row = sg.out_row(p, t, r - t * p.heads_per_unit);
                if (row < 0) continue;
                const float l = row_l[r], inv = 1.0f / l;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int col = (warp * NT + j) * 8 + 2 * (lane & 3);
                    const float x = o16[j][2 * half], y = o16[j][2 * half + 1];
                    if (whole) {
                        *reinterpret_cast<uint32_t *>(out + row * D + col) =
                            Elem<T>::pack(finish(x, l, inv), finish(y, l, inv));
                    } else {
                        __stcg(reinterpret_cast<float2 *>(record + r * D + col), make_float2(x, y));
                    }
                }
            }
        } else {
            if (lane / C4 == 0) {
                const int col = (warp * C4 + lane) * 4;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const long long row = sg.out_row(p, r / p.heads_per_unit, r % p.heads_per_unit);
                    if (row < 0) continue;
                    if (whole) {
                        const float l = row_l[r], inv = 1.0f / l;
                        *reinterpret_cast<float4 *>(out + row * D + col) =
                            make_float4(finish(o32[r][0], l, inv), finish(o32[r][1], l, inv),
                                        finish(o32[r][2], l, inv), finish(o32[r][3], l, inv));
                    } else {
                        __stcg(reinterpret_cast<float4 *>(record + r * D + col),
                               make_float4(o32[r][0], o32[r][1], o32[r][2], o32[r][3]));
                    }
                }
            }
        }
        if (whole) continue;
        ++handed;
        if (tid < kRows) {
            __stcg(record + kRows * D + tid, row_m[tid]);
            __stcg(record + kRows * D + kRows + tid, row_l[tid]);
        }
        // A range has at most two split units, its first and its last. The first one's arrival
        // (a fence takes thousands of cycles while copies are under way) and join are left to
        // the joining warp; the last one's are the CTA's last work.
        if (more && G::kJoinWarp) {
            if (tid == 0) early = sg;
            had_early = true;
            __syncwarp();
            if (lane == 0) mbar_arrive(&early_ready);
            continue;
        }
        named_barrier_sync(2, kCompute);
        if (tid == 0) {
            __threadfence();
            sh_join = last_arrival(p.counters + sg.c0, sg.c1 - sg.c0 + 1);
            __threadfence();
        }
        named_barrier_sync(1, kCompute);
        if (sh_join)
            join_unit<T, D, kCompute>(p, sg, tid, [] { named_barrier_sync(2, kCompute); }, join_part, row_l);
        named_barrier_sync(1, kCompute);  // row_l and join_part have been read
    }
    if (G::kJoinWarp && !had_early) {
        if (tid == 0) early.flags = kWhole;  // nothing to join
        __syncwarp();
        if (lane == 0) mbar_arrive(&early_ready);
    }
    if (!gave_up) return;
    if (tid == 0) {
        // The units shared with other CTAs -- the range's first and last at most -- that this one
        // has not stored its part of: their partial results are marked as none (a length below
        // zero), so that nobody writes these units' rows, and counted.
        int n = sh_seq, slot, len;
        unsigned seq_begin = sh_seq_begin, unit_begin, unit_end;
        auto find_unit = [&](unsigned place) {  // that holds this place, of this sequence or a later one
            unsigned each_unit = tiles_of(n, slot, len);
            while (each_unit == 0 || place - seq_begin >= (each_unit + kTurn) * units) {
                if (each_unit != 0) seq_begin += (each_unit + kTurn) * units;
                if (n + 1 == p.n_seqs) break;  // not reached: the range ends before the sequences do
                each_unit = tiles_of(++n, slot, len);
            }
            unit_begin = seq_begin + (place - seq_begin) / (each_unit + kTurn) * (each_unit + kTurn) + kTurn;
            unit_end = unit_begin + each_unit;
        };
        auto count_as_none = [&] {
            const int c0 = owner(unit_begin), c1 = owner(unit_end - 1);
            float *record = p.partials + static_cast<size_t>(2 * blockIdx.x + (unit_begin >= begin ? 1 : 0)) * kRecord;
            for (int r = 0; r < kRows; ++r) __stcg(record + kRows * D + kRows + r, -1.0f);
            unsigned long long *word = p.counters + c0;
            tag(word, *reinterpret_cast<volatile unsigned long long *>(word), p.nonce);
            __threadfence();
            last_arrival(word, c1 - c0 + 1);
        };
        find_unit(begin);
        const unsigned first = unit_begin;
        const bool first_split = unit_begin < begin || unit_end > end;
        if (first_split && handed == 0) count_as_none();
        find_unit(end - 1);
        if (unit_begin != first && unit_begin < end && unit_end > end && handed <= (first_split ? 1 : 0))
            count_as_none();
    }
    drain_in_flight();  // (the loading warp may have left before)
}

// ------------------------------------------------------------------ host side

// Rows of a unit: all query heads of a key head (groups of 16 when there are more), and as
// many draft tokens as fit beside them.
struct Split {
    int heads, tokens, head_groups, token_groups;
};

Split split_rows(int n_tokens, int group) {
    Split s;
    s.heads = group < kRows ? group : kRows;
    s.tokens = kRows / s.heads < n_tokens ? kRows / s.heads : n_tokens;
    s.head_groups = (group + s.heads - 1) / s.heads;
    s.token_groups = (n_tokens + s.tokens - 1) / s.tokens;
    return s;
}

constexpr size_t kCounterBytes = kMaxCtas * sizeof(unsigned long long);

size_t workspace_bytes_for(int head_dim) {
    return kCounterBytes + static_cast<size_t>(kMaxCtas) * 2 * kRows * (head_dim + 2) * sizeof(float);
}

// A value of its own for every call (48 bits, never 0).
unsigned long long next_nonce() {
    static std::atomic<unsigned long long> calls{0};
    static const unsigned long long seed = [] {
        timespec t{};
        clock_gettime(CLOCK_REALTIME, &t);
        return static_cast<unsigned long long>(t.tv_sec) * 1000000000ull + t.tv_nsec;
    }();
    unsigned long long z = seed + 0x9E3779B97F4A7C15ull * (calls.fetch_add(1) + 1);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;  // splitmix64
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return ((z ^ (z >> 31)) >> 16) | 1ull;
}

template <typename T, int D, int RT>
gdn_status launch(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p,
                  cudaStream_t s) {
    using G = Geometry<T, D, RT>;
    auto kernel = attn_decode_kernel<T, D, RT>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, G::kSmem, allowed));
    kernel<<<kSMs * G::kCtas, G::kThreads, G::kSmem, s>>>(q, k, v, p);
    return launch_status();
}

template <typename T, int D>
gdn_status launch_rows(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                       const Params &p, cudaStream_t s) {
    if constexpr (sizeof(T) == 4) {
        // the FP32 pipes' work grows with the rows laid out: 3 rows a unit in the windowed pool
        // take 48 us laid out for 4 and 124 for 16
        const int rows = p.heads_per_unit * p.tokens_per_unit;
        if (rows <= 4) return launch<T, D, 4>(q, k, v, p, s);
        if (rows <= 8) return launch<T, D, 8>(q, k, v, p, s);
    }
    return launch<T, D, 16>(q, k, v, p, s);
}

template <typename T>
gdn_status launch_dim(int d, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                      const Params &p, cudaStream_t s) {
    switch (d) {
        case 64: return launch_rows<T, 64>(q, k, v, p, s);
        case 128: return launch_rows<T, 128>(q, k, v, p, s);
        default: return launch_rows<T, 256>(q, k, v, p, s);
    }
}

}  // namespace

// The bounded-wait self-test on this unit's watchdog flag (gdn_selftest_attn_wait).
__global__ void wait_probe_kernel_attn_decode(int arm, unsigned long long limit_ns, float *out) {
    bounded_wait_probe(arm != 0, limit_ns, &g_watchdog_attn_decode, WD_STAGE_COPY, out);
}

gdn_status launch_wait_probe_attn_decode(bool arm, uint64_t limit_ns, float *out, cudaStream_t s) {
    wait_probe_kernel_attn_decode<<<1, 1, 0, s>>>(arm ? 1 : 0, limit_ns, out);
    return launch_status();
}

unsigned read_and_clear_watchdog_attn_decode(cudaStream_t s) {
    return read_and_clear_flag(g_watchdog_attn_decode, s);
}

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_attn_decode_workspace_size(int n_seqs, int n_tokens, int n_q_heads, int n_kv_heads,
                                      int head_dim) {
    if (n_seqs < 0 || n_tokens < 1 || n_kv_heads < 1 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads != 0 || !supported_head_dim(head_dim))
        return 0;
    return workspace_bytes_for(head_dim);
}

gdn_status gdn_attn_decode(const void *q, const void *k_pages, const void *v_pages,
                           const int32_t *page_table, const int32_t *kv_lens, void *out,
                           int n_seqs, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                           int page_size, int n_pages, int max_pages, int window, int n_sinks,
                           float scale, int q_stride, int dtype, const int32_t *slots, int pool,
                           int32_t *err_count, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream) {
    if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !out) return GDN_ERR_NULL;
    if (n_seqs < 0 || n_tokens < 1 || n_q_heads < 1 || window < 0 || n_sinks < 0) return GDN_ERR_SHAPE;
    GDN_TRY(check_cache(n_kv_heads, head_dim, page_size, n_pages, max_pages, dtype));
    if (n_q_heads % n_kv_heads != 0) return GDN_ERR_SHAPE;
    if (static_cast<long long>(n_q_heads) * head_dim > q_stride) return GDN_ERR_SHAPE;
    if (n_tokens > 64 || static_cast<long long>(n_seqs) * n_tokens > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    GDN_TRY(check_pool(n_seqs, slots, pool));
    const int es = dtype_bytes(dtype);
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
        (static_cast<long long>(q_stride) * es) % 16 != 0)
        return GDN_ERR_ALIGN;
    if (n_seqs == 0) return GDN_OK;
    if (!workspace) return GDN_ERR_NULL;
    if (!aligned16(workspace)) return GDN_ERR_ALIGN;
    if (workspace_bytes < workspace_bytes_for(head_dim)) return GDN_ERR_SHAPE;

    const int group = n_q_heads / n_kv_heads;
    const Split sp = split_rows(n_tokens, group);
    Params p{};
    p.cache = PagedCache{page_table, kv_lens, slots, pool, max_pages, n_pages, n_kv_heads,
                         log2_of(page_size)};
    p.mask = make_mask(window, n_sinks);
    p.out = out;
    p.n_seqs = n_seqs;
    p.n_tokens = n_tokens;
    p.n_q_heads = n_q_heads;
    p.group = group;
    p.heads_per_unit = sp.heads;
    p.tokens_per_unit = sp.tokens;
    p.head_groups = sp.head_groups;
    p.token_groups = sp.token_groups;
    p.scale_log2 = scale * kLog2E;
    p.err_count = err_count;
    p.counters = static_cast<unsigned long long *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes);
    p.nonce = next_nonce();

    // the ranges are counted in 32 bits (2^31 tiles are some 70 TB read in one call)
    const int kt = (head_dim == 64 ? 2 : 1) * (dtype == GDN_F32 ? 32 : 64);
    const long long widest = (static_cast<long long>(max_pages) * page_size + kt - 1) / kt + 2 + kTurn;
    if (widest * n_kv_heads * sp.head_groups * sp.token_groups > 0x7fffffffLL / n_seqs)
        return GDN_ERR_UNSUPPORTED;
    CUtensorMap q_map, k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(n_pages) * n_kv_heads * page_size;
    const int box = page_size < kt ? page_size : kt, cols = head_dim * es / 128;
    GDN_TRY(encode_heads_map(&q_map, q, dtype, head_dim, n_q_heads,
                             static_cast<uint64_t>(n_seqs) * n_tokens,
                             static_cast<uint64_t>(q_stride) * es, sp.heads, sp.tokens));
    GDN_TRY(encode_blocks_map(&k_map, k_pages, dtype, head_dim, rows,
                              static_cast<uint64_t>(head_dim) * es, box, cols));
    GDN_TRY(encode_blocks_map(&v_map, v_pages, dtype, head_dim, rows,
                              static_cast<uint64_t>(head_dim) * es, box, cols));
    const cudaStream_t s = as_cuda(stream);
    switch (dtype) {
        case GDN_F32: return launch_dim<float>(head_dim, q_map, k_map, v_map, p, s);
        case GDN_F16: return launch_dim<__half>(head_dim, q_map, k_map, v_map, p, s);
        default: return launch_dim<__nv_bfloat16>(head_dim, q_map, k_map, v_map, p, s);
    }
}

}  // extern "C"
