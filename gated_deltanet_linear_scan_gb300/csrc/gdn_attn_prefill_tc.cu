// gdn_attn_prefill_tc.cu -- prompt attention of 16-bit types on the tensor cores (sm_103a).
//
//   S = Q K^T      tcgen05, Q and K from shared memory, S in tensor memory
//   P = 2^(scale log2(e) S - m)   four warps per row tile, one thread per row: the row's
//                  maximum and sum need no exchange; P goes back to tensor memory over S,
//                  in the cache's type: half a unit of the type per weight, which adds a
//                  fifth to two fifths to the error of the output's own rounding
//   O += P V       tcgen05, P from tensor memory, V from shared memory as it lies there
//                  (rows are keys: the MN-major operand form, no transposition)
//
// O stays in tensor memory. It is rescaled only when a row's maximum has grown by more than
// 2^8 since the reference the weights use (they stay within 2^8 in bf16, 2^15 in f16).
//
// A row tile is 128 rows: tokens x the heads of a key head. Two row tiles (head_dim 64, 128)
// share every key tile of 128 keys and alternate: one tile's softmax runs while the tensor
// pipe works for the other. With head_dim 256 O fills half the tensor memory, so there is one
// row tile and two S buffers: S of the next key tile is computed during the softmax of this
// one. Within a key tile, only the 32-key chunks that some row of the row tile sees are
// multiplied and exponentiated.
//
// K and V stream through two rings of slots, each fed by a warp of its own (one warp's copies,
// barriers and page lookups would take longer than the products: a copy costs its warp about
// 60 cycles, a barrier 30 to 60). Pages are loaded one by one; a V slot keeps their rows apart
// ([page][128-byte column][row]), so that one copy brings all of a page's columns, and the
// MMA's descriptor strides say where they lie.
//
// CTAs are persistent: a scheduling warp takes the next pair of row tiles from the grid (the
// hardware cancels the launch of a CTA that has not begun and hands over its index), looks
// its sequence up and loads its Q, while the other warps are still busy with the one before.
// Sequences go longest first, their last tokens first, so the work left at the end is small.
//
// Measured, with the rate of the visible pairs' products and its share of a large bf16 matrix
// product's: 1500 tokens after 30000, 24 heads of 256, 720 us, 1575 TFLOP/s (0.84); 16384
// tokens of 39 ragged prompts, 32 heads of 128, 196 us, 884 TFLOP/s (0.47); 4 x 4096 tokens
// with a window of 1000, 16 heads of 64, 136 us, 435 TFLOP/s (0.23). Key tile by key tile, a
// pair of row tiles took 1.84 us at head_dim 128 and 1.55 at 64 (1 and 3 % less than now, before
// every wait became a warp's vote), where the tensor pipe is busy for 1.07 and 0.67: S, its softmax, and O are a chain per row tile, and when the warps of the
// two softmaxes run together, at different places of long unrolled code, they wait for
// instructions (a scheduler issues in 35 to 43 % of its cycles). A work's partial tiles,
// its first Q and its output add two to three tiles' time to each.
#include "gdn_attn_prefill.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace tc {

// ---- 128-byte swizzled operands, as tensor-map loads leave them: 1024-byte aligned blocks
// of rows of 128 bytes (64 16-bit elements), 16-byte chunk c of row r at chunk c ^ (r & 7).

// K-major: rows are M or N indices, the 64 elements run along K; a K step of 16 elements
// advances the start address by 32 bytes, 64 elements are the next block.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t start) {
    return static_cast<uint64_t>((start & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

// MN-major: rows are K indices, the 64 elements run along N; `block` bytes lie between one
// block of 64 N elements and the next, `group` between one group of 8 rows and the next.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t start, uint32_t block, uint32_t group) {
    return static_cast<uint64_t>((start & 0x3FFFFu) >> 4) |
           static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>((group >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

// Instruction descriptor of a dense kind::f16 MMA, f32 accumulator, A and B both bf16 or
// both f16, A K-major (or in tensor memory), B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit(bool bf16, int m, int n, bool b_mn_major) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

}  // namespace tc

namespace {

__device__ unsigned g_watchdog_attn_prefill;

constexpr int kTcKeys = 128;
constexpr int kTcRows = 128;
constexpr int kChunk = 32;     // keys of a chunk
constexpr int kNotes = 16;     // key tiles: more than K is ever ahead of the softmax
constexpr int kWorks = 3;      // entries of the work ring
constexpr float kLazy = 8.0f;  // log2 of the growth of a maximum that makes O rescale

template <int D>
struct Tc {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kBufs = D == 256 ? 2 : 1;              // S buffers of a row tile
    // Slots of a K (or V) tile, and of the rings. head_dim 256 has room for one and a half K
    // tiles: half of the next one arrives while this one is multiplied.
    static constexpr int kSubs = D == 256 ? 2 : 1;
    static constexpr int kKSlots = D == 64 ? 4 : D == 128 ? 2 : 3;
    static constexpr int kVSlots = D == 64 ? 4 : 2;
    static constexpr int kSlotBytes = kTcKeys * D * 2 / kSubs;
    static constexpr int kCols = D / 64 / kSubs;                // 128-byte columns of a K slot
    static constexpr int kVKeys = kTcKeys / kSubs;              // keys of a V slot
    static constexpr int kLog2VKeys = kSubs == 2 ? 6 : 7;
    static constexpr int kQBytes = kTcRows * D * 2;             // of a row tile
    static constexpr int kSmem = kTiles * kQBytes + (kKSlots + kVSlots) * kSlotBytes + 1024;
    static constexpr int kSoftmax = kTiles * 4;                 // softmax warps
    // then the MMA, the K, the V and the scheduling warp
    static constexpr int kMma = kSoftmax, kK = kMma + 1, kSched = kMma + 3;
    static constexpr int kThreads = (kSoftmax + 4) * 32;
    static constexpr int kS = 0, kO = 256;                      // tensor-memory columns
    // batches up to this many sequences run longest first (what shared memory has left): the 39
    // ragged prompts above took 193 us, in batch order 233; with heads of 256, 15 prompts of 12000
    // tokens 147 and 162, 9 of as many 160 and 171
    static constexpr int kTable = D == 256 ? 32 : kLongestFirstMaxSeqs;
};

// The sequences of a batch of up to N, in order of decreasing length.
template <int N>
struct SeqTable {
    int row0[N], new_tokens[N], slot[N], len[N];
    int order[N];      // sequence of rank r
    int first[N + 1];  // blocks (pairs of row tiles) before rank r
};

// A pair of row tiles to compute.
struct Work {
    int valid;
    int slot, row0, token0, tokens, kvh, head0, heads;
    int p_first, p_last;      // positions of its first and last token
    int n, n_sink, main0;     // its key tiles: a TileWalk
    // row tile i sees tiles 0 .. head - 1 (its sinks) and begin .. end - 1 (its window)
    int head[2], begin[2], end[2];

    __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : main0 + j - n_sink; }
    __device__ __forceinline__ bool active(int i, int j) const {
        return j < end[i] && (j < head[i] || j >= begin[i]);
    }
    // The next tile of row tile i from j on (end[i] or more: none).
    __device__ __forceinline__ int next(int i, int j) const {
        return j < head[i] || j >= begin[i] ? j : begin[i];
    }
};

// Positions of row tile i of a work item.
__device__ __forceinline__ int tile_first(const Work &w, int i, int per) { return w.p_first + i * per; }
__device__ __forceinline__ int tile_last(const Work &w, int i, int per) {
    return min(w.p_first + (i + 1) * per - 1, w.p_last);
}

// The chunks [x, y) of the key tile at key0 that hold every key a position in [lo_p, hi_p] sees.
__device__ __forceinline__ int2 chunks_seen(const AttnMask &mask, int key0, int lo_p, int hi_p) {
    int a = kTcKeys, b = 0;
    const int lo = mask.first(max(lo_p, 0));
    if (lo < key0 + kTcKeys) {
        a = max(lo - key0, 0);
        b = min(hi_p - key0 + 1, kTcKeys);
    }
    const int sinks = min(mask.sinks, hi_p + 1) - key0;
    if (sinks > 0) {
        a = 0;
        b = max(b, min(sinks, kTcKeys));
    }
    return make_int2(a / kChunk, (b + kChunk - 1) / kChunk);
}

// What the K warp notes about a key tile: bits 0..15 its 8-key blocks that were loaded, then
// eight bits for each row tile.
struct TileNote {
    uint32_t bits;
    __device__ __forceinline__ uint32_t of(int i) const { return bits >> (16 + 8 * i); }
    __device__ __forceinline__ bool active(int i) const { return of(i) & 1u; }
    __device__ __forceinline__ bool first(int i) const { return of(i) & 2u; }  // of the row tile's
    __device__ __forceinline__ bool last(int i) const { return of(i) & 4u; }
    __device__ __forceinline__ int begin(int i) const { return (of(i) >> 3) & 3u; }      // chunks
    __device__ __forceinline__ int end(int i) const { return ((of(i) >> 5) & 3u) + 1; }
    static __device__ __forceinline__ uint32_t make(bool first, bool last, int2 seen) {
        return 1u | (first ? 2u : 0u) | (last ? 4u : 0u) | static_cast<uint32_t>(seen.x) << 3 |
               static_cast<uint32_t>(seen.y - 1) << 5;
    }
};

// False when a wait gave up: the warp then leaves for the CTA's end.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *dead) {
    return gdn::warp_wait(bar, parity, dead, &g_watchdog_attn_prefill);
}

// Bits lo .. hi - 1 of a 32-bit word (any of them outside the word).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t skip = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below & ~skip;
}

// Asks for the index of a CTA of this grid that has not begun, in place of its launch; the
// answer (16 bytes) completes a phase of `bar`.
__device__ __forceinline__ void ask_next_cta(void *answer, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
        ::"r"(smem_addr(answer)), "r"(smem_addr(bar))
        : "memory");
}

// False when every CTA has begun.
__device__ __forceinline__ bool next_cta(const void *answer, int &x) {
    uint32_t ok, cx;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.b32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
        : "=r"(ok), "=r"(cx)
        : "r"(smem_addr(answer))
        : "memory");
    x = static_cast<int>(cx);
    return ok != 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(Tc<D>::kThreads, 1)
attn_prefill_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const PrefillParams p) {
    using C = Tc<D>;
    constexpr bool kBf16 = !__is_same(T, __half);
    constexpr uint32_t kIdescO = tc::idesc_16bit(kBf16, kTcRows, D, true);
    // log2 of the weight at the reference. float16's steps end at 2^-24: with 2^7, and the
    // allowance of 2^8 on top, its weights use the type's whole range, and what is lost of a
    // small one is 2^-32 of the largest. (l carries the same factor.)
    constexpr float kWeightBits = kBf16 ? 0.0f : 7.0f;
    extern __shared__ uint8_t dyn[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *k_ring = smem + C::kTiles * C::kQBytes;
    uint8_t *v_ring = k_ring + C::kKSlots * C::kSlotBytes;
    __shared__ __align__(8) uint64_t k_full[C::kKSlots], k_empty[C::kKSlots];
    __shared__ __align__(8) uint64_t v_full[C::kVSlots], v_empty[C::kVSlots];
    __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], o_done[2];
    __shared__ __align__(8) uint64_t work_full[kWorks], work_empty[kWorks], answer_full;
    __shared__ __align__(16) uint4 answer;
    __shared__ Work works[kWorks];
    __shared__ SeqTable<C::kTable> seqs;
    __shared__ uint32_t notes[kNotes];
    __shared__ uint32_t tmem_base;
    __shared__ int sh_dead;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = p.tokens_per_tile / C::kTiles;            // tokens of a row tile
    const int log2_bv = min(p.cache.log2_ps, C::kLog2VKeys);  // keys of a V load
    const int bv = 1 << log2_bv;
    const bool table = p.n_seqs <= C::kTable;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKSlots; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < C::kVSlots; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(&work_full[i], 1);
            mbar_init(&work_empty[i], 3 + C::kSoftmax);
        }
        mbar_init(&answer_full, 1);
        fence_mbar_init();
        sh_dead = 0;
    }
    if (warp == C::kMma) tc::tmem_alloc(&tmem_base, 512);
    // ---- the sequences, longest first
    for (int n = threadIdx.x; n < p.n_seqs; n += C::kThreads) {
        size_t row0 = 0;
        int m = 0, slot = 0, len = 0;
        const bool ok = p.seqs.range(n, row0, m) && p.cache.lookup(n, slot, len);
        if (!ok && blockIdx.x == 0 && p.err_count) atomicAdd(p.err_count, 1);
        if (table) {
            seqs.row0[n] = static_cast<int>(row0);
            seqs.new_tokens[n] = ok ? m : 0;
            seqs.slot[n] = slot;
            seqs.len[n] = ok ? len : 0;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base;
    if (table) {
        for (int n = threadIdx.x; n < p.n_seqs; n += C::kThreads) {
            const int mine = seqs.len[n];
            int rank = 0;
            for (int o = 0; o < p.n_seqs; ++o) rank += seqs.len[o] > mine || (seqs.len[o] == mine && o < n);
            seqs.order[rank] = n;
        }
        __syncthreads();
        if (warp == 0) {
            int run = 0;
            for (int r0 = 0; r0 < p.n_seqs; r0 += 32) {
                const int r = r0 + lane;
                const int own = r < p.n_seqs ? (seqs.new_tokens[seqs.order[r]] + p.tokens_per_tile - 1) / p.tokens_per_tile : 0;
                int x = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(FULL_MASK, x, o);
                    if (lane >= o) x += y;
                }
                if (r < p.n_seqs) seqs.first[r] = run + x - own;
                run += __shfl_sync(FULL_MASK, x, 31);
            }
            if (lane == 0) seqs.first[p.n_seqs] = run;
        }
        __syncthreads();
    }

    // Two row tiles: 384 threads of 168 registers; the softmax threads take 200 each, the
    // third warp group keeps 104 (2 * 200 + 104 = 3 * 168).
    if (warp >= C::kSoftmax) {
        if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // These warps run converged, with one elected lane issuing: the operands of a copy or
        // an MMA are then the same in every lane, as the hardware wants them.
        const bool leader = elect_one();
        if (warp == C::kSched) {
            // ------------------------------------------------------ the scheduling warp
            const int heads = p.cache.n_kv_heads * p.head_groups;
            int q_uses[2] = {0, 0};
            int id = blockIdx.x, ring = 0, round = 0, asked = 0;
            for (;;) {
                if (leader) {
                    mbar_arrive_expect_tx(&answer_full, 16);
                    ask_next_cta(&answer, &answer_full);
                }
                __syncwarp();
                const int x = id / heads, y = id % heads;
                int new_tokens = 0, row0 = 0, slot = 0, len = 0, block = 0;
                if (table) {
                    if (x < seqs.first[p.n_seqs]) {
                        int lo = 0, hi = p.n_seqs;  // the last rank with first[rank] <= x
                        while (hi - lo > 1) {
                            const int mid = (lo + hi) / 2;
                            if (seqs.first[mid] <= x) lo = mid;
                            else hi = mid;
                        }
                        const int n = seqs.order[lo];
                        new_tokens = seqs.new_tokens[n];
                        row0 = seqs.row0[n];
                        slot = seqs.slot[n];
                        len = seqs.len[n];
                        block = seqs.first[lo + 1] - 1 - x;
                    }
                } else {
                    size_t at;
                    const int n = warp_seq_of_slot(p.seqs.cu, p.n_seqs, p.tokens_per_tile, x);
                    if (n >= 0 && p.seqs.range(n, at, new_tokens) && p.cache.lookup(n, slot, len)) {
                        row0 = static_cast<int>(at);
                        block = x - (row0 / p.tokens_per_tile + n);
                    } else {
                        new_tokens = 0;
                    }
                }
                if (block * p.tokens_per_tile < new_tokens) {
                    Work w;
                    w.valid = 1;
                    w.slot = slot;
                    w.row0 = row0;
                    w.token0 = block * p.tokens_per_tile;
                    w.tokens = min(p.tokens_per_tile, new_tokens - w.token0);
                    w.kvh = y / p.head_groups;
                    const int hg = y % p.head_groups;
                    w.head0 = w.kvh * p.group + hg * p.heads_per_tile;
                    w.heads = min(p.heads_per_tile, p.group - hg * p.heads_per_tile);
                    w.p_first = len - new_tokens + w.token0;
                    w.p_last = w.p_first + w.tokens - 1;
                    const TileWalk walk = walk_tiles<kTcKeys>(p.mask, w.p_first, w.p_last);
                    w.n = walk.count;
                    w.n_sink = walk.n_sink;
                    w.main0 = walk.main0;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int first = tile_first(w, i, per), last = tile_last(w, i, per);
                        if (i >= C::kTiles || i * per >= w.tokens || last < 0) {
                            w.head[i] = w.begin[i] = w.end[i] = 0;
                        } else {
                            // (sinks past the walk's own sink tiles lie in its window part,
                            // where tile j has number j: n_sink is main0 then)
                            const int lo = p.mask.first(max(first, 0));
                            w.head[i] = (min(p.mask.sinks, lo) + kTcKeys - 1) / kTcKeys;
                            w.begin[i] = walk.n_sink + lo / kTcKeys - walk.main0;
                            w.end[i] = walk.n_sink + last / kTcKeys + 1 - walk.main0;
                        }
                    }
                    if (round > 0 && !warp_wait(&work_empty[ring], (round - 1) & 1, &sh_dead)) goto leave;
                    if (leader) {
                        works[ring] = w;
                        mbar_arrive(&work_full[ring]);
                    }
                    __syncwarp();
                    if (++ring == kWorks) {
                        ring = 0;
                        ++round;
                    }
                    // its Q, as the row tiles before let go of theirs
#pragma unroll
                    for (int i = 0; i < C::kTiles; ++i) {
                        if (w.end[i] == 0) continue;
                        if (q_uses[i] > 0 && !warp_wait(&q_empty[i], (q_uses[i] - 1) & 1, &sh_dead)) goto leave;
                        ++q_uses[i];
                        if (leader) {
                            mbar_arrive_expect_tx(&q_full[i], static_cast<uint32_t>(p.heads_per_tile * per) * D * 2u);
                            for (int cb = 0; cb < D / 64; ++cb)
                                tma_load_3d(smem + i * C::kQBytes + cb * kTcRows * 128, &q_map, cb * 64,
                                            w.head0, w.row0 + w.token0 + i * per, &q_full[i]);
                        }
                        __syncwarp();
                    }
                }
                if (!warp_wait(&answer_full, asked & 1, &sh_dead)) goto leave;
                ++asked;
                const bool more = next_cta(&answer, id);
                fence_proxy_async_smem();  // read before the next answer overwrites it
                __syncwarp();
                if (!more) break;
            }
            if (round > 0 && !warp_wait(&work_empty[ring], (round - 1) & 1, &sh_dead)) goto leave;
            if (leader) {
                works[ring].valid = 0;
                mbar_arrive(&work_full[ring]);
            }
            __syncwarp();
        } else if (warp == C::kMma) {
            // ------------------------------------------------------ the MMA warp
            const uint64_t q_desc = tc::smem_desc_sw128(smem_addr(smem));
            const uint64_t k_desc = tc::smem_desc_sw128(smem_addr(k_ring));
            // V lies page by page, every page's 128-byte columns one behind the other: 16 keys
            // are two groups of 8 rows, in one page (bv >= 16) or in two
            const uint64_t v_desc = tc::smem_desc_sw128_mn(smem_addr(v_ring), bv * 128, bv >= 16 ? 1024 : D * 16);
            uint32_t v_step[C::kVKeys / 16];  // from 16 keys to the next, in 16-byte units
#pragma unroll
            for (int x = 0; x < C::kVKeys / 16; ++x)
                v_step[x] = (((x * 16) >> log2_bv) * (bv * D * 2) + ((x * 16) & (bv - 1)) * 128) >> 4;
            int s_count = 0, o_count = 0;         // products issued (one row tile: its buffer)
            uint32_t o_phase = 0, q_phase = 0;    // bit i: of row tile i's p_ready, q_full
            // (The functions below return false when a wait gave up.)
            // The note of key tile g (numbered over all work), once its K is there.
            auto note_of = [&](int g, TileNote &note) {
                const int slot = (g * C::kSubs) % C::kKSlots;
                if (!warp_wait(&k_full[slot], (g * C::kSubs / C::kKSlots) & 1, &sh_dead)) return false;
                note.bits = static_cast<volatile uint32_t *>(notes)[g % kNotes];
                return true;
            };
            // S of row tile i over key tile g. (This code and issue_o's stand once, in rolled loops:
            // unrolled for both row tiles the warp spent its time fetching instructions.)
            auto issue_s = [&](int i, int g, TileNote note) {
                const int buf = C::kBufs == 2 ? s_count & 1 : i;
                ++s_count;
                if (note.first(i)) {
                    if (!warp_wait(&q_full[i], (q_phase >> i) & 1, &sh_dead)) return false;
                    q_phase ^= 1u << i;
                }
                const bool release = i == 1 || !note.active(1), last = note.last(i);
                const int from = note.begin(i) * kChunk;
                const uint32_t to = tmem + C::kS + buf * kTcKeys + from;
                const uint32_t idesc = tc::idesc_16bit(kBf16, kTcRows, 0, false) |
                                       static_cast<uint32_t>(note.end(i) - note.begin(i)) << (17 + 2);
                const uint64_t q0 = q_desc + ((i * C::kQBytes) >> 4);
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int slot = (g * C::kSubs + s) % C::kKSlots;
                    if (s > 0 && !warp_wait(&k_full[slot], ((g * C::kSubs + s) / C::kKSlots) & 1, &sh_dead)) return false;
                    tc::fence_after_sync();
                    const uint64_t k = k_desc + ((slot * C::kSlotBytes + from * 128) >> 4);
                    const uint64_t q = q0 + ((s * C::kCols * kTcRows * 128) >> 4);
                    if (leader) {
#pragma unroll
                        for (int c = 0; c < C::kCols; ++c)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                tc::mma_bf16(to, q + ((c * kTcRows * 128 + x * 32) >> 4),
                                             k + ((c * kTcKeys * 128 + x * 32) >> 4), idesc, s + c + x > 0);
                        if (release) tc::mma_commit(&k_empty[slot]);
                        if (s == C::kSubs - 1) {
                            tc::mma_commit(&s_full[buf]);
                            if (last) tc::mma_commit(&q_empty[i]);
                        }
                    }
                    __syncwarp();
                }
                return true;
            };
            // O of row tile i += P V over key tile g
            auto issue_o = [&](int i, int g, TileNote note) {
                const int buf = C::kBufs == 2 ? o_count & 1 : i;
                const uint32_t phase = C::kBufs == 2 ? (o_count >> 1) & 1 : (o_phase >> i) & 1;
                ++o_count;
                o_phase ^= 1u << i;
                const bool release = i == 1 || !note.active(1), first = note.first(i);
                const int from = note.begin(i) * (kChunk / 16), to = note.end(i) * (kChunk / 16);
                if (!warp_wait(&p_ready[buf], phase, &sh_dead)) return false;
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int slot = (g * C::kSubs + s) % C::kVSlots;
                    if (!warp_wait(&v_full[slot], ((g * C::kSubs + s) / C::kVSlots) & 1, &sh_dead)) return false;
                    tc::fence_after_sync();
                    const uint64_t v = v_desc + ((slot * C::kSlotBytes) >> 4);
                    const uint32_t pw = tmem + C::kS + buf * kTcKeys + s * C::kVKeys / 2, o = tmem + C::kO + i * D;
                    if (leader) {
                        if (from == 0 && to == kTcKeys / 16) {
#pragma unroll
                            for (int x = 0; x < C::kVKeys / 16; ++x)
                                tc::mma_bf16_ts(o, pw + x * 8, v + v_step[x], kIdescO, !first || s + x > 0);
                        } else {
                            const int x0 = max(from - s * (C::kVKeys / 16), 0), x1 = min(to - s * (C::kVKeys / 16), C::kVKeys / 16);
#pragma unroll 1
                            for (int x = x0; x < x1; ++x) {
                                const uint32_t at = (((x * 16) >> log2_bv) * (bv * D * 2) + ((x * 16) & (bv - 1)) * 128) >> 4;
                                tc::mma_bf16_ts(o, pw + x * 8, v + at, kIdescO, !first || s * (C::kVKeys / 16) + x > from);
                            }
                        }
                        if (release) tc::mma_commit(&v_empty[slot]);
                        if (s == C::kSubs - 1) tc::mma_commit(&o_done[i]);
                    }
                    __syncwarp();
                }
                return true;
            };
            int base = 0;         // key tiles of the work before
            TileNote carried{0};  // of the work's first tile, when its S is already issued
            for (int ring = 0, round = 0;;) {
                if (!warp_wait(&work_full[ring], round & 1, &sh_dead)) goto leave;
                const int n = works[ring].n;
                if (!works[ring].valid) break;
                const int next_ring = ring + 1 == kWorks ? 0 : ring + 1;
                const int next_round = ring + 1 == kWorks ? round + 1 : round;
                // Key tile by key tile, row tile 0 ahead of row tile 1 (the last of them that
                // sees a tile lets its slots go), O of a tile and S of the next together: while
                // one row tile multiplies, the other computes its weights. Two row tiles: the
                // last step's S is the next work's first, so that its softmax can begin while the
                // other row tile finishes here. One row tile: S goes ahead of O, into the other
                // buffer.
                TileNote note = carried, next{0};
                carried.bits = 0;
#pragma unroll 1
                for (int j = note.bits != 0 || n == 0 ? 0 : -1; j < n; ++j) {
                    auto look_ahead = [&] {
                        if (j + 1 < n) return note_of(base + j + 1, next);
                        if (C::kTiles == 2) {
                            if (!warp_wait(&work_full[next_ring], next_round & 1, &sh_dead)) return false;
                            if (works[next_ring].valid && works[next_ring].n > 0 && !note_of(base + n, carried))
                                return false;
                        }
                        next = carried;  // (one row tile: nothing)
                        return true;
                    };
                    if constexpr (C::kTiles == 1) {
                        if (!look_ahead()) goto leave;
                        if (next.active(0) && !issue_s(0, base + j + 1, next)) goto leave;
                        if (j >= 0 && !issue_o(0, base + j, note)) goto leave;
                    } else {
#pragma unroll 1
                        for (int i = 0; i < 2; ++i) {
                            if (note.active(i) && !issue_o(i, base + j, note)) goto leave;
                            if (i == 0 && !look_ahead()) goto leave;
                            if (next.active(i) && !issue_s(i, base + j + 1, next)) goto leave;
                        }
                    }
                    note = next;
                }
                base += n;
                if (leader) mbar_arrive(&work_empty[ring]);
                __syncwarp();
                ring = next_ring;
                round = next_round;
            }
        } else if (warp < C::kSched) {
            // ------------------------------------------------------ the K and the V warp
            const bool is_k = warp == C::kK;
            const int ps = 1 << p.cache.log2_ps;
            const int log2_bk = min(p.cache.log2_ps, 7);  // keys of a page's part of a key tile
            const int bk = 1 << log2_bk, n_bk = kTcKeys >> log2_bk;
            if (leader) tma_prefetch_map(is_k ? &k_map : &v_map);
            int base = 0, slot = 0, slot_round = 0;
            for (int ring = 0, round = 0;;) {
                if (!warp_wait(&work_full[ring], round & 1, &sh_dead)) goto leave;
                const Work w = works[ring];
                if (!w.valid) break;
                const int n = w.n, p_first = w.p_first, p_last = w.p_last, kvh = w.kvh;
                // Whether someone sees keys of lane i's part of key tile j; its page if so (the
                // ids of pages before the window, which may be gone, are not read).
                auto seen = [&](int j) {
                    const int key = w.tile(j) * kTcKeys + lane * bk;
                    return lane < n_bk && key <= p_last &&
                           (p_first - (key + bk - 1) < p.mask.window || key < p.mask.sinks);
                };
                auto page_at = [&](int j) {
                    return j < n && seen(j) ? p.cache.page_of(w.slot, w.tile(j) * kTcKeys + lane * bk) : -1;
                };
                // what there is to say of tile j, whose parts `have` pages (one lane's business)
                auto note_of = [&](int j, unsigned have) {
                    unsigned note = 0;
                    if (is_k && leader && j < n) {
                        const int key0 = w.tile(j) * kTcKeys;
                        for (int i = 0; i < kTcKeys / 8; ++i)
                            if ((have >> ((i * 8) >> log2_bk)) & 1u) note |= 1u << i;
#pragma unroll
                        for (int i = 0; i < C::kTiles; ++i)
                            if (w.active(i, j))
                                note |= TileNote::make(j == w.next(i, 0), w.next(i, j + 1) >= w.end[i],
                                                       chunks_seen(p.mask, key0, tile_first(w, i, per),
                                                                   tile_last(w, i, per)))
                                        << (16 + 8 * i);
                    }
                    __syncwarp();
                    return note;
                };
                int page = page_at(0);
                unsigned have = __ballot_sync(FULL_MASK, p.cache.page_ok(page));
                unsigned note = note_of(0, have);
                for (int j = 0; j < n; ++j) {
                    const int next_page = page_at(j + 1);
                    const int key0 = w.tile(j) * kTcKeys;
                    const int row = (page * p.cache.n_kv_heads + kvh) * ps + (key0 & (ps - 1));
                    if (is_k) {
                        if (!p.cache.page_ok(page) && seen(j) && kvh == 0 && p.err_count) atomicAdd(p.err_count, 1);
                        if (leader) notes[(base + j) % kNotes] = note;
                        __syncwarp();
                    }
                    for (int s = 0; s < C::kSubs; ++s) {
                        uint64_t *full = is_k ? &k_full[slot] : &v_full[slot];
                        if (slot_round > 0 &&
                            !warp_wait(is_k ? &k_empty[slot] : &v_empty[slot], (slot_round - 1) & 1, &sh_dead))
                            goto leave;
                        if (is_k) {
                            uint8_t *to = k_ring + slot * C::kSlotBytes;
                            if (leader)
                                mbar_arrive_expect_tx(full, (static_cast<uint32_t>(__popc(have)) << (log2_bk + 7)) * C::kCols);
                            if (n_bk == 1) {  // one page: its columns in one copy
                                const int r = __shfl_sync(FULL_MASK, row, 0);
                                if (leader && have) tma_load_3d(to, &k_map, 0, r, s * C::kCols, full);
                            } else {
                                for (int i = 0; i < n_bk; ++i) {
                                    const int r = __shfl_sync(FULL_MASK, row, i);
                                    if (leader && ((have >> i) & 1u)) {
#pragma unroll
                                        for (int c = 0; c < C::kCols; ++c)
                                            tma_load_3d(to + c * kTcKeys * 128 + (i << (log2_bk + 7)), &k_map, 0, r,
                                                        s * C::kCols + c, full);
                                    }
                                }
                            }
                        } else {
                            // this slot's copies of bv keys, from the parts they lie in
                            uint8_t *to = v_ring + slot * C::kSlotBytes;
                            const int i0 = s << (C::kLog2VKeys - log2_bv), i1 = (s + 1) << (C::kLog2VKeys - log2_bv);
                            const bool here = lane >= i0 && lane < i1 && ((have >> ((lane << log2_bv) >> log2_bk)) & 1u);
                            const unsigned loads = __popc(__ballot_sync(FULL_MASK, here));
                            if (leader) mbar_arrive_expect_tx(full, loads * static_cast<uint32_t>(bv) * D * 2u);
                            for (int i = i0; i < i1; ++i) {
                                const int part = (i << log2_bv) >> log2_bk;
                                const int r = __shfl_sync(FULL_MASK, row, part) + ((i << log2_bv) & (bk - 1));
                                if (leader && ((have >> part) & 1u))
                                    tma_load_3d(to + (i - i0) * (bv * D * 2), &v_map, 0, r, 0, full);
                            }
                        }
                        __syncwarp();
                        if (++slot == (is_k ? C::kKSlots : C::kVSlots)) {
                            slot = 0;
                            ++slot_round;
                        }
                    }
                    page = next_page;
                    have = __ballot_sync(FULL_MASK, p.cache.page_ok(page));
                    note = note_of(j + 1, have);  // while the copies are on their way
                }
                base += n;
                if (leader) mbar_arrive(&work_empty[ring]);
                __syncwarp();
                if (++ring == kWorks) {
                    ring = 0;
                    ++round;
                }
            }
        }
    } else {
        if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------------------------------------------------- softmax, one row a thread
        const int i = warp / 4, row = threadIdx.x & 127;
        const int row_token = row / p.heads_per_tile, row_head = row % p.heads_per_tile;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + lanes + C::kO + i * D;
        const bool positive = p.scale_log2 > 0.0f;
        const float mult = positive ? p.scale_log2 : 1.0f;
        int base = 0, count = 0;  // key tiles of the work before, tiles of this row tile so far
        for (int ring = 0, round = 0;;) {
            if (!warp_wait(&work_full[ring], round & 1, &sh_dead)) goto leave;
            const Work &w = works[ring];
            if (!w.valid) break;
            const int head_tiles = w.head[i], begin_tile = w.begin[i], end_tile = w.end[i];
            const int n_sink = w.n_sink, main0 = w.main0;
            auto next_tile = [&](int j) { return j < head_tiles || j >= begin_tile ? j : begin_tile; };
            const int token = i * per + row_token;
            const int pos = w.p_first + token;
            const int p_first = tile_first(w, i, per), p_last = tile_last(w, i, per);
            const int all_first = w.p_first, all_last = w.p_last;
            float m = -INFINITY, l = 0.0f;
            bool begun = false;
            for (int j = next_tile(0); j < end_tile; j = next_tile(j + 1)) {
                const int buf = C::kBufs == 2 ? count & 1 : i;
                const uint32_t s_addr = tmem + lanes + C::kS + buf * kTcKeys;
                const int key0 = (j < n_sink ? j : main0 + j - n_sink) * kTcKeys;
                if (!warp_wait(&s_full[buf], (C::kBufs == 2 ? count >> 1 : count) & 1, &sh_dead)) goto leave;
                tc::fence_after_sync();
                // written before K was loaded, and K has been multiplied
                const TileNote note{static_cast<volatile uint32_t *>(notes)[(base + j) % kNotes]};
                const unsigned blocks = note.bits & 0xFFFFu;
                const int2 seen = make_int2(note.begin(i), note.end(i));
                // every row of the work sees every key of the tile
                const bool alive = blocks == 0xFFFFu && key0 + kTcKeys - 1 <= all_last &&
                                   (all_first - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                if (!alive) {
                    // V rows that no row of the work sees are cleared (by both row tiles, each
                    // ahead of its own product), so that whatever the page holds there (an
                    // infinity, a NaN) cannot reach O through a weight of 0.
                    // (Two S buffers: once the O product before this tile's is complete, the
                    // ring slots of V are at most one phase from the one waited for.)
                    if (C::kBufs == 2 && begun && !warp_wait(&o_done[0], (count - 1) & 1, &sh_dead)) goto leave;
                    const int key = key0 + row;
                    const bool dead = !((blocks >> (row >> 3)) & 1u) || key > all_last ||
                                      !(all_first - key < p.mask.window || key < p.mask.sinks);
                    for (int y = 0; y < C::kSubs; ++y) {
                        const int g = (base + j) * C::kSubs + y, slot = g % C::kVSlots;
                        if (!warp_wait(&v_full[slot], (g / C::kVSlots) & 1, &sh_dead)) goto leave;
                        if (dead && (row >> C::kLog2VKeys) == y) {
                            const int r = row & (C::kVKeys - 1);
                            uint8_t *at = v_ring + slot * C::kSlotBytes + (r >> log2_bv) * (bv * D * 2) + (r & (bv - 1)) * 128;
                            for (int x = 0; x < D / 8; ++x)  // (the lanes' 16 bytes in different banks)
                                *reinterpret_cast<uint4 *>(at + (x >> 3) * bv * 128 + ((x + row) & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                }
                // The reference of the weights, from the tile's maximum; O is rescaled when it
                // moves by more than the allowance. (False when a wait gave up.)
                auto settle = [&](float mx) {
                    if (!begun) {
                        m = mx;
                        return true;
                    }
                    const bool grow = (mx - m) * mult > kLazy;
                    if (__any_sync(FULL_MASK, grow)) {
                        // O is complete up to the tile before: S of this tile was issued after
                        // it (two S buffers: after the one before that)
                        if (C::kBufs == 2) {
                            if (!warp_wait(&o_done[0], (count - 1) & 1, &sh_dead)) return false;
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
                    return true;
                };
                float2 sum[4] = {};
                // weights of 32 scores, and their place in P
                auto weigh = [&](const uint32_t (&s)[32], float2 mul2, float2 sub2, uint32_t to) {
                    uint32_t pw[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 a = __ffma2_rn(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
                                              mul2, sub2);
                        a.x = fast_exp2(a.x);
                        a.y = fast_exp2(a.y);
                        sum[x & 3] = __fadd2_rn(sum[x & 3], a);
                        pw[x] = Elem<T>::pack(a.x, a.y);
                    }
                    tc::tmem_st16(to, pw);
                };
                auto top_of = [&](const uint32_t (&s)[32], float (&top)[4]) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            top[y] = fmaxf(fmaxf(top[y], __uint_as_float(s[x + 2 * y])), __uint_as_float(s[x + 2 * y + 1]));
                };
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const bool clean = positive && blocks == 0xFFFFu && key0 + kTcKeys - 1 <= p_first &&
                                   (p_last - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                if (clean) {
                    // every row sees every key: the whole tile in registers
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_ld32_nowait(s_addr + c * kChunk, s[c]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) top_of(s[c], top);
                    if (!settle(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])))) goto leave;
                    const float off = (m == -INFINITY ? 0.0f : m * mult) - kWeightBits;
                    const float2 mul2 = make_float2(mult, mult), sub2 = make_float2(-off, -off);
#pragma unroll
                    for (int c = 0; c < 4; ++c) weigh(s[c], mul2, sub2, s_addr + c * (kChunk / 2));
                } else {
                    // chunk by chunk, twice: the maximum, then the weights (a chunk's P lies over
                    // scores that have been read)
                    auto chunk = [&](int c, uint32_t (&s)[32]) {
                        tc::tmem_ld32_nowait(s_addr + c * kChunk, s);
                        const int at = key0 + c * kChunk;
                        // the keys this row sees: from its window's first to itself, and the sinks
                        const int hi = pos - at + 1;
                        const int lo = pos - at < p.mask.window ? 0 : pos - p.mask.window + 1 - at;
                        uint32_t see = bits_between(lo, hi) | bits_between(0, min(p.mask.sinks - at, hi));
                        uint32_t there = 0;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if ((blocks >> (4 * c + x)) & 1u) there |= 0xFFu << (8 * x);
                        see &= there;
                        tc::tmem_ld_wait();
                        if (!positive) {
#pragma unroll
                            for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * p.scale_log2);
                        }
                        if (__any_sync(FULL_MASK, see != 0xFFFFFFFFu)) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!(see & (1u << x))) s[x] = __float_as_uint(-INFINITY);
                        }
                    };
                    uint32_t s[32];
#pragma unroll 1
                    for (int c = seen.x; c < seen.y; ++c) {
                        chunk(c, s);
                        top_of(s, top);
                    }
                    if (!settle(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])))) goto leave;
                    const float off = (m == -INFINITY ? 0.0f : m * mult) - kWeightBits;
                    const float2 mul2 = make_float2(mult, mult), sub2 = make_float2(-off, -off);
#pragma unroll 1
                    for (int c = seen.x; c < seen.y; ++c) {
                        chunk(c, s);
                        weigh(s, mul2, sub2, s_addr + c * (kChunk / 2));
                    }
                }
                sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += sum[0].x + sum[0].y;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                // keeps this thread at most one phase behind o_done
                if (C::kBufs == 2 && begun && !warp_wait(&o_done[0], (count - 1) & 1, &sh_dead)) goto leave;
                if (lane == 0) mbar_arrive(&p_ready[buf]);
                begun = true;
                ++count;
            }
            // ------------------------------------------------------ O out
            if (i * per < w.tokens) {
                const bool mine = token < w.tokens && row_token < per && row_head < w.heads;
                const long long at = mine ? static_cast<long long>(w.row0 + w.token0 + token) * p.n_q_heads + w.head0 + row_head : -1;
                // Four lanes write a row's 64 bytes together, row after row of their four:
                // eight lines a store instead of 32.
                long long rows[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) rows[r] = __shfl_sync(FULL_MASK, at, (lane & ~3) + r);
                T *out = static_cast<T *>(p.out) + (lane & 3) * 8;
                if (begun) {
                    if (!warp_wait(&o_done[i], (count - 1) & 1, &sh_dead)) goto leave;
                    tc::fence_after_sync();
                }
                const float inv = 1.0f / l;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32_nowait(o_addr + c, o);
                    tc::tmem_ld_wait();
                    uint32_t pw[4][4];  // 16 bytes of this row at a time; then of the four lanes' rows
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        pw[x / 4][x % 4] = l == 0.0f ? 0u
                                                     : Elem<T>::pack(__uint_as_float(o[2 * x]) * inv,
                                                                     __uint_as_float(o[2 * x + 1]) * inv);
#pragma unroll
                    for (int bit = 1; bit < 4; bit *= 2) {
                        const bool upper = lane & bit;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (r & bit) continue;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t got = __shfl_xor_sync(FULL_MASK, upper ? pw[r][y] : pw[r | bit][y], bit);
                                if (upper) pw[r][y] = got;
                                else pw[r | bit][y] = got;
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (rows[r] >= 0)
                            *reinterpret_cast<uint4 *>(out + rows[r] * D + c) =
                                make_uint4(pw[r][0], pw[r][1], pw[r][2], pw[r][3]);
                }
                tc::fence_before_sync();
            }
            base += w.n;
            __syncwarp();
            if (lane == 0) mbar_arrive(&work_empty[ring]);
            if (++ring == kWorks) {
                ring = 0;
                ++round;
            }
        }
    }
leave:
    __syncthreads();
    if (sh_dead) drain_in_flight();
    if (warp == C::kMma) {
        tc::fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D>
gdn_status launch(PrefillParams p, int dtype, cudaStream_t s) {
    using C = Tc<D>;
    const int ps = 1 << p.cache.log2_ps;
    p.heads_per_tile = p.group < kTcRows ? p.group : kTcRows;
    p.head_groups = (p.group + p.heads_per_tile - 1) / p.heads_per_tile;
    const int per = kTcRows / p.heads_per_tile;
    p.tokens_per_tile = per * C::kTiles;
    // every sequence's last block may be short: one block more than full ones each
    const long long blocks = p.seqs.total / p.tokens_per_tile + p.n_seqs;
    const long long grid = blocks * p.cache.n_kv_heads * p.head_groups;
    if (grid > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    CUtensorMap q_map, k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(p.cache.n_pages) * p.cache.n_kv_heads * ps;
    GDN_TRY(encode_heads_map(&q_map, p.q, dtype, D, p.n_q_heads, static_cast<uint64_t>(p.seqs.total),
                             static_cast<uint64_t>(p.q_stride) * 2, p.heads_per_tile, per));
    GDN_TRY(encode_blocks_map(&k_map, p.k_pages, dtype, D, rows, D * 2, ps < kTcKeys ? ps : kTcKeys,
                              ps < kTcKeys ? 1 : C::kCols));
    GDN_TRY(encode_blocks_map(&v_map, p.v_pages, dtype, D, rows, D * 2, ps < C::kVKeys ? ps : C::kVKeys,
                              D / 64));
    auto kernel = attn_prefill_tc_kernel<T, D>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, C::kSmem, allowed));
    kernel<<<static_cast<unsigned>(grid), C::kThreads, C::kSmem, s>>>(q_map, k_map, v_map, p);
    return launch_status();
}

template <typename T>
gdn_status launch_dim(int d, const PrefillParams &p, int dtype, cudaStream_t s) {
    switch (d) {
        case 64: return launch<T, 64>(p, dtype, s);
        case 128: return launch<T, 128>(p, dtype, s);
        default: return launch<T, 256>(p, dtype, s);
    }
}

}  // namespace

gdn_status launch_attn_prefill_tc(const PrefillParams &p, int dtype, int head_dim, cudaStream_t s) {
    return dtype == GDN_F16 ? launch_dim<__half>(head_dim, p, dtype, s)
                            : launch_dim<__nv_bfloat16>(head_dim, p, dtype, s);
}

// The bounded-wait self-test on this unit's watchdog flag (gdn_selftest_attn_wait).
__global__ void wait_probe_kernel_attn_prefill(int arm, unsigned long long limit_ns, float *out) {
    bounded_wait_probe(arm != 0, limit_ns, &g_watchdog_attn_prefill, WD_STAGE_COPY, out);
}

gdn_status launch_wait_probe_attn_prefill(bool arm, uint64_t limit_ns, float *out, cudaStream_t s) {
    wait_probe_kernel_attn_prefill<<<1, 1, 0, s>>>(arm ? 1 : 0, limit_ns, out);
    return launch_status();
}

unsigned read_and_clear_watchdog_attn_prefill(cudaStream_t s) {
    return read_and_clear_flag(g_watchdog_attn_prefill, s);
}

}  // namespace gdn
