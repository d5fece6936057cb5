// gdn_attn_tree_tc.cu -- attention of trees of drafts over the paged cache on the tensor cores
// (16-bit types, more rows of (node, head of a key head) than one matrix fragment; sm_103a).
//
//   S = Q K^T on tcgen05, P = 2^(scale log2(e) S - m) by four warps per lane, O += P V on tcgen05, as the
//   prompt attention does it (gdn_attn_prefill_tc.cu): S, P and O in tensor memory, P in the cache's
//   type, O rescaled only when a maximum has grown by more than 2^8. (P rounded to the type: half a unit a
//   weight, which random signs average out over the keys: errors of 0.0020 of the outputs' norm against 64 bits in
//   bf16, where rounding the outputs alone leaves 0.0017; 0.00029 and 0.00021 in f16. Two parts of P would be half as
//   many products again.)
//
// Every visible key and value is read once per 256 rows (128 for heads of 256), so HBM bounds the call:
// the keys of the whole batch are dealt out evenly over the SMs, whatever the lengths, as the decode
// attention deals them (a unit: sequence, key head, block of rows; a range of key tiles per CTA), and
// what a unit that crosses a range's end leaves behind is joined by a second kernel.
//
// Two lanes (head_dim 64, 128) share the tensor pipe, each with its S, P and O, one's softmax running
// while the pipe works for the other. With more than 128 rows in a block a lane has rows of its own
// and both take every key tile; with at most 128 the lanes have the same rows and take the tiles in
// turn, and the one whose turn was last adds the two up. Heads of 256 leave room for one lane with two S buffers.
//
// Measured (calls replayed back to back; shares of the visible keys' and values' bytes at the copy
// rate): 64 trees of 16 over 64..8192 bf16 keys, 16 key heads of 128: 189-193 us, 0.88 to 0.9. Eight of 64 with 6
// heads a key head over 16001..40000: 200-205, 0.39: two units a key head, of 256 and 128 rows, 2.1 us a
// tile in both, of which the products are 1.1; neither fewer instructions, nor keys from L2, nor other weights in
// the dealing changed that. One of 24 over 4000, heads of 256: 28, of which the join's launch is 4.
#include "gdn_attn_again.cuh"
#include "gdn_attn_tc.cuh"
#include "gdn_attn_tree.cuh"
#include "gdn_tree.cuh"

namespace gdn {
namespace {

constexpr int kSMs = 152;
constexpr unsigned kTurn = 2;  // what a unit weighs besides its tiles, in tiles
constexpr int kJoinParts = 16;

// EXTRA: with few rows, what their Q does not need of shared memory goes to the rings.
template <int D, bool EXTRA>
struct TreeTc {
    static constexpr int kLanes = D == 256 ? 1 : 2;
    static constexpr int kBufs = D == 256 ? 2 : 1;  // S buffers of a lane
    // Slots of a K (or V) tile, and of the rings, as the prompt attention's.
    static constexpr int kSubs = D == 256 ? 2 : 1;
    static constexpr int kKSlots = D == 64 ? (EXTRA ? 6 : 4) : D == 128 ? (EXTRA ? 3 : 2) : 3;
    static constexpr int kVSlots = D == 64 ? (EXTRA ? 6 : 4) : EXTRA ? 3 : 2;
    static constexpr int kSlotBytes = kTcKeys * D * 2 / kSubs;
    static constexpr int kCols = D / 64 / kSubs;  // 128-byte columns of a K slot
    static constexpr int kVKeys = kTcKeys / kSubs;
    static constexpr int kLog2VKeys = kSubs == 2 ? 6 : 7;
    static constexpr int kRings = (kKSlots + kVSlots) * kSlotBytes;
    static constexpr int kRoom = 232448 - 1024 - (D == 256 ? 2048 : 5632) - kRings;  // for Q
    static constexpr int kSoftmax = kLanes * 4;
    static constexpr int kMma = kSoftmax, kK = kMma + 1, kSched = kMma + 3;
    static constexpr int kThreads = (kSoftmax + 4) * 32;
    static constexpr int kS = 0, kO = 256;  // tensor-memory columns
    static constexpr int kWorks = D == 256 ? 2 : 4;  // entries of the work ring (what shared memory has left)
};

// A segment: the part of a unit in this CTA's range.
struct Work {
    int valid;
    int seq, slot, kvh, head0, heads, node0, nodes;  // nodes: of the block
    int base, len;                                   // position of a root; cache rows
    int n_sink, main0;                               // the unit's key tiles: a TileWalk
    int j0, j1;                                      // those of the segment
    int g0, t0;                                      // numbers of the first tile, and lane's turn, over all segments
    int turns;                                       // the lanes take the tiles in turn
    int q_buf[2];                                    // the lanes' Q buffers
    int whole, head;                                 // nothing of the unit elsewhere; it begins in this range

    __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : main0 + j - n_sink; }
    // lane i's first tile (the lanes' turns go on from one segment to the next), and from one to the next
    __device__ __forceinline__ int first(int i) const { return turns ? j0 + ((t0 + i) & 1) : j0; }
    __device__ __forceinline__ int step() const { return turns ? 2 : 1; }
    // whose turn the last tile is: that lane adds the other's sums to its own
    __device__ __forceinline__ int adder() const { return (t0 + j1 - 1 - j0) & 1; }
};

template <typename T, int D, bool EXTRA>
__global__ void __launch_bounds__(TreeTc<D, EXTRA>::kThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const TreeAttnParams p) {
    using C = TreeTc<D, EXTRA>;
    constexpr int kWorks = C::kWorks;
    constexpr bool kBf16 = !__is_same(T, __half);
    constexpr uint32_t kIdescO = tc::idesc_16bit(kBf16, kTcRows, D, true);
    // log2 of the weight at the reference (float16 uses its range, as in the prompt attention)
    constexpr float kWeightBits = kBf16 ? 0.0f : 7.0f;
    extern __shared__ uint8_t dyn[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    const int q_bytes = p.q_rows * D * 2;  // of a Q buffer: [128-byte column][row]
    uint8_t *const q_smem = smem;  // (a product reads 128 rows: past a smaller Q whatever lies behind it)
    uint8_t *k_ring = smem + p.q_bufs * q_bytes;
    uint8_t *v_ring = k_ring + C::kKSlots * C::kSlotBytes;
    __shared__ __align__(8) uint64_t k_full[C::kKSlots], k_empty[C::kKSlots];
    __shared__ __align__(8) uint64_t v_full[C::kVSlots], v_empty[C::kVSlots];
    __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], o_done[2];
    __shared__ __align__(8) uint64_t work_full[kWorks], work_empty[kWorks], half_done[2], half_free[2];
    __shared__ Work works[kWorks];
    __shared__ unsigned long long trees[kWorks][kMaxNodes];  // the nodes' paths
    __shared__ int up_of[kMaxNodes];
    __shared__ uint32_t notes[kNotes];
    __shared__ float2 half_ml[2][C::kLanes == 2 ? kTcRows : 1];
    __shared__ unsigned warp_sum[C::kThreads / 32];
    __shared__ unsigned sh_seq_begin;
    __shared__ int sh_seq, sh_slot, sh_len;
    __shared__ uint32_t tmem_base;
    __shared__ int sh_dead;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = p.tokens_per_tile;                        // nodes of a lane
    const int log2_bv = min(p.cache.log2_ps, C::kLog2VKeys);  // keys of a V load
    const int bv = 1 << log2_bv;
    const unsigned units = static_cast<unsigned>(p.cache.n_kv_heads * p.head_groups * p.blocks);  // of a sequence

    if (tid == 0) {
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
        for (int i = 0; i < 2; ++i) {  // from lane i
            mbar_init(&half_done[i], 4);
            mbar_init(&half_free[i], 4);
        }
        fence_mbar_init();
        sh_dead = 0;
        p.joins[blockIdx.x].c1 = -1;
    }
    // The records are none (a length below zero) until they are written, so that nobody joins what
    // was left by an earlier call, or by a CTA whose wait gave up.
    for (int x = tid; x < 2 * p.record_rows; x += C::kThreads)
        p.record(blockIdx.x, x / p.record_rows, D)[p.record_rows * (D + 1) + x % p.record_rows] = -1.0f;
    if (warp == C::kMma) tc::tmem_alloc(&tmem_base, 512);

    // ---- this CTA's range, in places: a unit is kTurn places without a tile, then its tiles (as in
    // the decode attention)
    auto tiles_of = [&](int n, int &slot, int &len) -> unsigned {
        if (!p.cache.lookup(n, slot, len) || len < p.n_nodes) return 0;
        return static_cast<unsigned>(walk_tiles<kTcKeys>(p.mask, len - p.n_nodes, len - 1).count);
    };
    const int slab = (p.n_seqs + C::kThreads - 1) / C::kThreads;
    const int n0 = min(tid * slab, p.n_seqs), n1 = min(n0 + slab, p.n_seqs);
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
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base;
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    // (no range is without a tile)
    const unsigned ranges = min(gridDim.x, total / (1 + kTurn));
    const bool idle = blockIdx.x >= ranges;
    const unsigned each = idle ? 0 : total / ranges, longer = idle ? 0 : total - each * ranges;
    auto range_begin = [&](unsigned c) { return c * each + min(c, longer); };
    const unsigned begin = range_begin(blockIdx.x), end = idle ? begin : range_begin(blockIdx.x + 1);
    auto owner = [&](unsigned x) {  // of place x
        const unsigned split = longer * (each + 1);
        return static_cast<int>(x < split ? x / (each + 1) : longer + (x - split) / each);
    };
    if (!idle && begin >= before && begin < before + sum) {
        unsigned at = before;
        for (int n = n0; n < n1; ++n) {
            const unsigned t = tiles_of(n, slot0, len0), w = t == 0 ? 0 : (t + kTurn) * units;
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

    // Two lanes: 384 threads of 168 registers; the softmax threads take 200 each, the third warp group
    // keeps 104 (2 * 200 + 104 = 3 * 168).
    if (warp >= C::kSoftmax) {
        if constexpr (C::kLanes == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const bool leader = elect_one();  // these warps run converged, one elected lane issuing
        if (warp == C::kSched) {
            // ------------------------------------------------------ the scheduling warp
            int ring = 0, round = 0, q_uses[2] = {0, 0}, next_buf = 0, g = 0, t = 0;
            int n = sh_seq, slot = sh_slot, len = sh_len, tree_of = -1;
            unsigned seq_begin = sh_seq_begin, at = begin;
            TileWalk walk{0, 0, 0};
            unsigned tiles = 1, unit = 0;
            unsigned long long paths[2] = {0, 0};
            if (!idle) {
                walk = walk_tiles<kTcKeys>(p.mask, len - p.n_nodes, len - 1);
                tiles = static_cast<unsigned>(walk.count);
                unit = (at - seq_begin) / (tiles + kTurn);
            }
            while (at < end) {
                const unsigned unit_begin = seq_begin + unit * (tiles + kTurn) + kTurn;  // its first tile
                const unsigned unit_end = unit_begin + tiles;
                at = max(at, unit_begin);
                if (at >= end) break;
                const unsigned seg_end = min(unit_end, end);
                Work w;
                w.valid = 1;
                w.seq = n;
                w.slot = slot;
                const int block = static_cast<int>(unit) % p.blocks, head = static_cast<int>(unit) / p.blocks;
                w.kvh = head / p.head_groups;
                const int hg = head % p.head_groups;
                w.head0 = w.kvh * p.group + hg * p.heads_per_tile;
                w.heads = min(p.heads_per_tile, p.group - hg * p.heads_per_tile);
                w.node0 = block * C::kLanes * per;
                w.nodes = min(C::kLanes * per, p.n_nodes - w.node0);
                w.base = len - p.n_nodes;
                w.len = len;
                w.n_sink = walk.n_sink;
                w.main0 = walk.main0;
                w.j0 = static_cast<int>(at - unit_begin);
                w.j1 = static_cast<int>(seg_end - unit_begin);
                w.turns = C::kLanes == 2 && w.nodes <= per;
                w.g0 = g;
                w.t0 = t;
                g += w.j1 - w.j0;
                t += (w.j1 - w.j0) * (C::kLanes == 2 && !w.turns ? 2 : 1);
                w.whole = at == unit_begin && seg_end == unit_end;
                w.head = unit_begin >= begin;
                // rows of its own for each lane, or one Q for both: the buffers in turn
                w.q_buf[0] = C::kLanes == 1 ? 0 : w.turns ? next_buf : 0;
                w.q_buf[1] = C::kLanes == 1 ? 0 : w.turns ? next_buf : 1;
                if (w.turns && p.q_bufs == 2) next_buf ^= 1;
                if (round > 0 && !warp_wait(&work_empty[ring], (round - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                if (tree_of != n) {
                    tree_of = n;
                    const bool bad = tree_paths(p.parents + static_cast<size_t>(n) * p.n_nodes, p.n_nodes, paths,
                                                trees[ring], up_of);
                    // (counted where the sequence's first tile is)
                    if (bad && unit == 0 && w.j0 == 0 && lane == 0 && p.err_count) atomicAdd(p.err_count, 1);
                } else {
                    trees[ring][lane] = paths[0];
                    trees[ring][lane + 32] = paths[1];
                }
                __syncwarp();
                if (leader) {
                    works[ring] = w;
                    if (!w.whole && w.head) {
                        TreeJoin join;
                        join.seq = n;
                        join.head0 = w.head0;
                        join.heads = w.heads;
                        join.node0 = w.node0;
                        join.nodes = w.nodes;
                        join.turns = w.turns;
                        join.c1 = owner(unit_end - 1);
                        p.joins[blockIdx.x] = join;
                    }
                    mbar_arrive(&work_full[ring]);
                }
                __syncwarp();
                if (++ring == kWorks) {
                    ring = 0;
                    ++round;
                }
                // its Q, as the work before lets go of its buffers
#pragma unroll
                for (int i = 0; i < C::kLanes; ++i) {
                    if (i > 0 && w.turns) continue;
                    const int b = w.q_buf[i];
                    const int uses = b == 0 ? q_uses[0] : q_uses[1];
                    if (uses > 0 && !warp_wait(&q_empty[b], (uses - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                    if (b == 0) ++q_uses[0];
                    else ++q_uses[1];
                    if (leader) {
                        mbar_arrive_expect_tx(&q_full[b], static_cast<uint32_t>(p.heads_per_tile * per) * D * 2u);
                        for (int cb = 0; cb < D / 64; ++cb)
                            tma_load_3d(q_smem + b * q_bytes + cb * p.q_rows * 128, &q_map, cb * 64, w.head0,
                                        n * p.n_nodes + w.node0 + i * per, &q_full[b]);
                    }
                    __syncwarp();
                }
                at = seg_end;
                if (at == unit_end && ++unit == units && at < end) {
                    seq_begin = unit_end;
                    unit = 0;
                    do {
                        tiles = tiles_of(++n, slot, len);
                    } while (tiles == 0 && n + 1 < p.n_seqs);
                    if (tiles == 0) break;  // not reached: the range says tiles are left
                    walk = walk_tiles<kTcKeys>(p.mask, len - p.n_nodes, len - 1);
                }
            }
            if (round > 0 && !warp_wait(&work_empty[ring], (round - 1) & 1, &sh_dead, p.watchdog)) goto leave;
            if (leader) {
                works[ring].valid = 0;
                mbar_arrive(&work_full[ring]);
            }
            __syncwarp();
        } else if (warp == C::kMma) {
            // ------------------------------------------------------ the MMA warp
            const uint64_t q_desc = tc::smem_desc_sw128(smem_addr(q_smem));
            const uint64_t k_desc = tc::smem_desc_sw128(smem_addr(k_ring));
            // V lies page by page, every page's 128-byte columns one behind the other: 16 keys are two
            // groups of 8 rows, in one page (bv >= 16) or in two
            const uint64_t v_desc = tc::smem_desc_sw128_mn(smem_addr(v_ring), bv * 128, bv >= 16 ? 1024 : D * 16);
            uint32_t v_step[C::kVKeys / 16];  // from 16 keys to the next, in 16-byte units
#pragma unroll
            for (int x = 0; x < C::kVKeys / 16; ++x)
                v_step[x] = (((x * 16) >> log2_bv) * (bv * D * 2) + ((x * 16) & (bv - 1)) * 128) >> 4;
            // The products run through all segments' tiles in one order, lane by lane in turn (a tile of rows
            // of its own for each lane has a turn of both); with one lane, S buffer by S buffer. S runs
            // kLanes turns ahead of O: a lane's next S is issued right behind its O.
            struct Place {
                int n, j, j1, g;    // segments begun; tile, the segment's end, the tile's number
                int left;           // turns left of the tile
                int turns, t;       // of the segment; the turn's number
                bool over;
            };
            Place sp{0, 0, 0, 0, 0, 0, 0, false}, op{0, 0, 0, 0, 0, 0, 0, false};
            uint32_t q_new = 0, q_phase = 0;  // bit b: Q buffer b's contents are still to be waited for; its phase
            int q_bufs = 0, o_first = 0;      // bit i: lane i's buffer; tiles of the segment before op's
            // (The functions below return false when a wait gave up.) Opens the next segment; over when none.
            auto open = [&](Place &at) {
                if (!warp_wait(&work_full[at.n % kWorks], (at.n / kWorks) & 1, &sh_dead, p.watchdog)) return false;
                const Work &w = works[at.n % kWorks];
                at.over = !w.valid;
                at.j = w.j0;
                at.j1 = w.j1;
                at.g = w.g0;
                at.turns = w.turns;
                at.left = C::kLanes == 2 && !at.turns ? 2 : 1;
                ++at.n;
                return true;
            };
            auto step = [&](Place &at) {
                ++at.t;
                if (--at.left == 0) {
                    ++at.j;
                    ++at.g;
                    at.left = C::kLanes == 2 && !at.turns ? 2 : 1;
                }
            };
            auto next_s = [&] {
                if (sp.over) return true;
                if (sp.j == sp.j1) {
                    if (!open(sp)) return false;
                    if (sp.over) return true;
                    const Work &w = works[(sp.n - 1) % kWorks];
                    q_bufs = w.q_buf[0] | w.q_buf[1] << 1;
                    q_new = C::kLanes == 1 ? 1u : sp.turns ? 1u << w.q_buf[0] : 3u;
                }
                const int i = C::kLanes == 1 ? 0 : sp.t & 1, buf = sp.t & 1, g = sp.g;
                const int q_buf = (q_bufs >> i) & 1;
                const int slot0 = (g * C::kSubs) % C::kKSlots;
                if (!warp_wait(&k_full[slot0], (g * C::kSubs / C::kKSlots) & 1, &sh_dead, p.watchdog)) return false;
                const TileNote note{static_cast<volatile uint32_t *>(notes)[g % kNotes]};
                if ((q_new >> q_buf) & 1u) {
                    if (!warp_wait(&q_full[q_buf], (q_phase >> q_buf) & 1, &sh_dead, p.watchdog)) return false;
                    q_phase ^= 1u << q_buf;
                    q_new &= ~(1u << q_buf);
                }
                // the tile's last turn lets K go, the segment's last tile (of the lane, where it has a Q of its
                // own) Q
                const bool release = sp.left == 1, last = sp.j + 1 == sp.j1;
                const int from = note.begin(0) * kChunk;
                const uint32_t to = tmem + C::kS + buf * kTcKeys + from;
                const uint32_t idesc = tc::idesc_16bit(kBf16, kTcRows, 0, false) |
                                       static_cast<uint32_t>(note.end(0) - note.begin(0)) << (17 + 2);
                const uint64_t q0 = q_desc + ((q_buf * q_bytes) >> 4);
                const uint32_t q_col = p.q_rows * 8;  // 128-byte columns of Q, in 16-byte units
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int slot = (g * C::kSubs + s) % C::kKSlots;
                    if (s > 0 && !warp_wait(&k_full[slot], ((g * C::kSubs + s) / C::kKSlots) & 1, &sh_dead, p.watchdog)) return false;
                    tc::fence_after_sync();
                    const uint64_t k = k_desc + ((slot * C::kSlotBytes + from * 128) >> 4);
                    const uint64_t q = q0 + s * C::kCols * q_col;
                    if (leader) {
#pragma unroll
                        for (int c = 0; c < C::kCols; ++c)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                tc::mma_bf16(to, q + (c * q_col + x * 2), k + ((c * kTcKeys * 128 + x * 32) >> 4), idesc,
                                             s + c + x > 0);
                        if (release) tc::mma_commit(&k_empty[slot]);
                        if (s == C::kSubs - 1) {
                            tc::mma_commit(&s_full[buf]);
                            if (last) tc::mma_commit(&q_empty[q_buf]);
                        }
                    }
                    __syncwarp();
                }
                step(sp);
                return true;
            };
            auto next_o = [&] {
                const int i = C::kLanes == 1 ? 0 : op.t & 1, buf = op.t & 1, g = op.g;
                const bool first = op.turns ? o_first < 2 : o_first == 0, release = op.left == 1;
                const TileNote note{static_cast<volatile uint32_t *>(notes)[g % kNotes]};
                const int from = note.begin(0) * (kChunk / 16), to = note.end(0) * (kChunk / 16);
                if (!warp_wait(&p_ready[buf], (op.t >> 1) & 1, &sh_dead, p.watchdog)) return false;
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    const int slot = (g * C::kSubs + s) % C::kVSlots;
                    if (!warp_wait(&v_full[slot], ((g * C::kSubs + s) / C::kVSlots) & 1, &sh_dead, p.watchdog)) return false;
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
                if (op.left == 1) ++o_first;
                step(op);
                return true;
            };
#pragma unroll 1
            for (int i = 0; i < C::kLanes; ++i)
                if (!next_s()) goto leave;
            for (;;) {
                if (op.j == op.j1) {
                    if (op.n > 0) {
                        if (leader) mbar_arrive(&work_empty[(op.n - 1) % kWorks]);
                        __syncwarp();
                    }
                    o_first = 0;
                    if (!open(op)) goto leave;
                    if (op.over) break;
                }
                if constexpr (C::kLanes == 1) {
                    if (!next_s() || !next_o()) goto leave;  // into the other buffer, ahead of this tile's O
                } else {
                    if (!next_o() || !next_s()) goto leave;
                }
            }
        } else {
            // ------------------------------------------------------ the K and the V warp
            const bool is_k = warp == C::kK;
            const int ps = 1 << p.cache.log2_ps;
            const int log2_bk = min(p.cache.log2_ps, 7);  // keys of a page's part of a key tile
            const int bk = 1 << log2_bk, n_bk = kTcKeys >> log2_bk;
            if (leader) tma_prefetch_map(is_k ? &k_map : &v_map);
            int slot = 0, slot_round = 0;
            for (int ring = 0, round = 0;;) {
                if (!warp_wait(&work_full[ring], round & 1, &sh_dead, p.watchdog)) goto leave;
                const Work w = works[ring];
                if (!w.valid) break;
                // Whether someone sees keys of lane i's part of key tile j; its page if so (the ids of pages
                // before the window, which may be gone, are not read).
                auto seen = [&](int j) {
                    const int key = w.tile(j) * kTcKeys + lane * bk;
                    return lane < n_bk && key < w.len &&
                           (w.base - (key + bk - 1) < p.mask.window || key < p.mask.sinks);
                };
                auto page_at = [&](int j) {
                    return j < w.j1 && seen(j) ? p.cache.page_of(w.slot, w.tile(j) * kTcKeys + lane * bk) : -1;
                };
                // what there is to say of tile j, whose parts `have` pages (one lane's business)
                auto note_of = [&](int j, unsigned have) {
                    unsigned note = 0;
                    if (is_k && leader && j < w.j1) {
                        for (int i = 0; i < kTcKeys / 8; ++i)
                            if ((have >> ((i * 8) >> log2_bk)) & 1u) note |= 1u << i;
                        note |= TileNote::make(false, false, chunks_seen(p.mask, w.tile(j) * kTcKeys, w.base, w.len - 1)) << 16;
                    }
                    __syncwarp();
                    return note;
                };
                int page = page_at(w.j0);
                unsigned have = __ballot_sync(FULL_MASK, p.cache.page_ok(page));
                unsigned note = note_of(w.j0, have);
                for (int j = w.j0; j < w.j1; ++j) {
                    const int next_page = page_at(j + 1);
                    const int key0 = w.tile(j) * kTcKeys;
                    const int row = (page * p.cache.n_kv_heads + w.kvh) * ps + (key0 & (ps - 1));
                    if (is_k) {
                        // (a page is counted where the sequence's first unit loads it)
                        if (!p.cache.page_ok(page) && seen(j) && w.kvh == 0 && w.node0 == 0 && w.head0 == 0 && p.err_count)
                            atomicAdd(p.err_count, 1);
                        if (leader) notes[(w.g0 + j - w.j0) % kNotes] = note;
                        __syncwarp();
                    }
                    for (int s = 0; s < C::kSubs; ++s) {
                        uint64_t *full = is_k ? &k_full[slot] : &v_full[slot];
                        if (slot_round > 0 &&
                            !warp_wait(is_k ? &k_empty[slot] : &v_empty[slot], (slot_round - 1) & 1, &sh_dead, p.watchdog))
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
                if (leader) mbar_arrive(&work_empty[ring]);
                __syncwarp();
                if (++ring == kWorks) {
                    ring = 0;
                    ++round;
                }
            }
        }
    } else {
        if constexpr (C::kLanes == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------------------------------------------------- softmax, one row a thread
        const int i = warp / 4, row = tid & 127;
        const int row_token = row / p.heads_per_tile, row_head = row % p.heads_per_tile;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + lanes + C::kO + i * D;
        const bool positive = p.scale_log2 > 0.0f;
        const float mult = positive ? p.scale_log2 : 1.0f;
        int count = 0;         // tiles of this lane so far
        int given = 0, taken = 0;  // times this lane's sums went to the other lane, and the other's came here
        bool owed = false;         // the other lane may still be reading this one's O
        for (int ring = 0, round = 0;;) {
            if (!warp_wait(&work_full[ring], round & 1, &sh_dead, p.watchdog)) goto leave;
            const Work &w = works[ring];
            if (!w.valid) break;
            const int j1 = w.j1, step = w.step(), first = w.first(i), n_sink = w.n_sink, main0 = w.main0;
            const int base = w.base, len = w.len, g0 = w.g0 - w.j0, turns = w.turns;
            const int token = (turns ? 0 : i * per) + row_token;  // of the block
            const bool mine = row_token < per && token < w.nodes && row_head < w.heads;
            const bool busy = __any_sync(FULL_MASK, mine);  // (else the warp only keeps the lane's steps)
            const unsigned long long path = mine ? trees[ring][w.node0 + token] : 0;
            // nodes that the row sees; nodes that are there
            unsigned long long tree = path;
            {
                const int depth = __popcll(path) - 1;
                if (depth >= p.mask.window) {
                    tree = 0;
                    for (unsigned long long left = path; left != 0; left &= left - 1) {
                        const int a = __ffsll(static_cast<long long>(left)) - 1, at = __popcll(trees[ring][a]) - 1;
                        if (depth - at < p.mask.window || base + at < p.mask.sinks) tree |= 1ull << a;
                    }
                }
            }
            const bool any_node = __any_sync(FULL_MASK, (trees[ring][lane] | trees[ring][lane + 32]) != 0);
            const int pos = base + __popcll(path) - 1;
            float m = -INFINITY, l = 0.0f;
            bool begun = false;
            for (int j = first; j < j1; j += step) {
                const int buf = C::kBufs == 2 ? count & 1 : i;
                const uint32_t s_addr = tmem + lanes + C::kS + buf * kTcKeys;
                const int key0 = (j < n_sink ? j : main0 + j - n_sink) * kTcKeys;
                if (!warp_wait(&s_full[buf], (C::kBufs == 2 ? count >> 1 : count) & 1, &sh_dead, p.watchdog)) goto leave;
                tc::fence_after_sync();
                // written before K was loaded, and K has been multiplied
                const TileNote note{static_cast<volatile uint32_t *>(notes)[(g0 + j) % kNotes]};
                const unsigned blocks = note.bits & 0xFFFFu;
                const int2 seen = make_int2(note.begin(0), note.end(0));
                // every row sees every key of the tile
                const bool clean = blocks == 0xFFFFu && key0 + kTcKeys - 1 < base &&
                                   (len - 1 - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                // every key is seen by some row of the tree
                const bool alive = blocks == 0xFFFFu && key0 + kTcKeys - 1 < base && any_node &&
                                   (base - key0 < p.mask.window || key0 + kTcKeys <= p.mask.sinks);
                if (!alive) {
                    // V rows that no row of the tree sees are cleared (by both lanes where both multiply
                    // them, each ahead of its own product), so that whatever the page holds there (an
                    // infinity, a NaN) cannot reach O through a weight of 0. (Two S buffers: once the O
                    // product before this tile's is complete, the ring slots of V are at most one phase
                    // from the one waited for.)
                    if (C::kBufs == 2 && begun && !warp_wait(&o_done[0], (count - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                    const int key = key0 + row;
                    const bool dead = !((blocks >> (row >> 3)) & 1u) || key >= len || !any_node ||
                                      !(base - key < p.mask.window || key < p.mask.sinks) ||
                                      (key >= base && trees[ring][(key - base) & 63] == 0);
                    for (int y = 0; y < C::kSubs; ++y) {
                        const int g = (g0 + j) * C::kSubs + y, slot = g % C::kVSlots;
                        if (!warp_wait(&v_full[slot], (g / C::kVSlots) & 1, &sh_dead, p.watchdog)) goto leave;
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
                // The reference of the weights, from the tile's maximum; O is rescaled when it moves by more
                // than the allowance. (False when a wait gave up.)
                auto settle = [&](float mx) {
                    if (!begun) {
                        m = mx;
                        return true;
                    }
                    const bool grow = (mx - m) * mult > kLazy;
                    if (__any_sync(FULL_MASK, grow)) {
                        // O is complete up to the tile before: S of this tile was issued after it (two S
                        // buffers: after the one before that)
                        if (C::kBufs == 2) {
                            if (!warp_wait(&o_done[0], (count - 1) & 1, &sh_dead, p.watchdog)) return false;
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
                if (busy) {
                    if (!EXTRA && positive && clean) {
                        // the whole tile in registers
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
                        // chunk by chunk, twice: the maximum, then the weights (a chunk's P lies over scores
                        // that have been read). With few rows every tile goes this way: the one warp that has
                        // rows waits for its instructions more than for its data, and this code stays near.
                        auto chunk = [&](int c, uint32_t (&s)[32]) {
                            tc::tmem_ld32_nowait(s_addr + c * kChunk, s);
                            if (positive && clean) {
                                tc::tmem_ld_wait();
                                return;
                            }
                            const int at = key0 + c * kChunk;
                            // the keys this row sees: before the tree from its window's first on and the sinks,
                            // then of the tree
                            const int hi = min(pos + 1, base) - at;
                            const int lo = pos - at < p.mask.window ? 0 : pos - p.mask.window + 1 - at;
                            uint32_t see = bits_between(lo, hi) | bits_between(0, min(p.mask.sinks - at, hi));
                            const int shift = at - base;
                            if (shift >= 0) see |= shift < 64 ? static_cast<uint32_t>(tree >> shift) : 0u;
                            else if (shift > -32) see |= static_cast<uint32_t>(tree << -shift);
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
                }
                sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += sum[0].x + sum[0].y;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                // keeps this thread at most one phase behind o_done
                if (C::kBufs == 2 && begun && !warp_wait(&o_done[0], (count - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                if (owed) {
                    if (!warp_wait(&half_free[i], (given - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                    owed = false;
                }
                if (lane == 0) mbar_arrive(&p_ready[buf]);
                begun = true;
                ++count;
            }
            // ------------------------------------------------------ O out
            if (begun) {
                if (!warp_wait(&o_done[i], (count - 1) & 1, &sh_dead, p.watchdog)) goto leave;
                tc::fence_after_sync();
            }
            if (tree == 0) {  // a node that is not there sees nothing
                m = -INFINITY;
                l = 0.0f;
            }
            float f0 = 1.0f, f1 = 0.0f;
            const bool both = C::kLanes == 2 && turns && j1 - w.j0 > 1;  // both lanes have had tiles
            const bool adds = !(C::kLanes == 2 && turns) || i == w.adder();
            if (both && !adds) {
                if (owed && !warp_wait(&half_free[i], (given - 1) & 1, &sh_dead, p.watchdog)) goto leave;  // (not reached: it has had a tile)
                half_ml[i][row] = make_float2(m, l);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&half_done[i]);
                owed = true;
                ++given;
            } else if (both) {
                if (!warp_wait(&half_done[i ^ 1], taken & 1, &sh_dead, p.watchdog)) goto leave;
                tc::fence_after_sync();
                ++taken;
                const float2 ml = half_ml[i ^ 1][row];
                const float top = fmaxf(m, ml.x);
                f0 = m == -INFINITY ? 0.0f : fast_exp2((m - top) * mult);
                f1 = ml.x == -INFINITY ? 0.0f : fast_exp2((ml.x - top) * mult);
                m = top;
                l = l * f0 + ml.y * f1;
            }
            if (adds && busy) {
                const bool add = both && __any_sync(FULL_MASK, f1 != 0.0f);
                const uint32_t other_addr = tmem + lanes + C::kO + (i ^ 1) * D;
                // this lane's sums and the other's, 32 columns at a time, by factors
                const float inv = w.whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
                const float2 mine2 = make_float2(f0 * inv, f0 * inv), other2 = make_float2(f1 * inv, f1 * inv);
                T *out = static_cast<T *>(p.out) +
                         ((static_cast<long long>(w.seq) * p.n_nodes + w.node0 + token) * p.n_q_heads + w.head0 + row_head) * D;
                float *record = p.record(blockIdx.x, w.head ? 1 : 0, D);
                const int r = (turns ? 0 : i * kTcRows) + row;
                float *sums = record + static_cast<size_t>(r) * D;
                const bool nothing = l == 0.0f;
                bool nan = false;  // (for infinities of both signs, too)
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32], y[32];
                    tc::tmem_ld32_nowait(o_addr + c, o);
                    if (add) tc::tmem_ld32_nowait(other_addr + c, y);
                    tc::tmem_ld_wait();
                    float2 z[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        z[x] = __fmul2_rn(make_float2(__uint_as_float(o[2 * x]), __uint_as_float(o[2 * x + 1])), mine2);
                    if (add) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            z[x] = __ffma2_rn(make_float2(__uint_as_float(y[2 * x]), __uint_as_float(y[2 * x + 1])), other2, z[x]);
                    }
                    if (!mine) continue;
                    float2 check = z[0];
#pragma unroll
                    for (int x = 1; x < 16; ++x) check = __fadd2_rn(check, z[x]);
                    nan |= check.x + check.y != check.x + check.y;
                    if (w.whole) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint4 pw;
                            pw.x = nothing ? 0u : Elem<T>::pack(z[4 * x].x, z[4 * x].y);
                            pw.y = nothing ? 0u : Elem<T>::pack(z[4 * x + 1].x, z[4 * x + 1].y);
                            pw.z = nothing ? 0u : Elem<T>::pack(z[4 * x + 2].x, z[4 * x + 2].y);
                            pw.w = nothing ? 0u : Elem<T>::pack(z[4 * x + 3].x, z[4 * x + 3].y);
                            *reinterpret_cast<uint4 *>(out + c + 8 * x) = pw;
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *reinterpret_cast<float4 *>(sums + c + 4 * x) =
                                make_float4(z[2 * x].x, z[2 * x].y, z[2 * x + 1].x, z[2 * x + 1].y);
                    }
                }
                if (!w.whole && mine) {
                    record[p.record_rows * D + r] = m == -INFINITY ? -INFINITY : m * mult;
                    record[p.record_rows * (D + 1) + r] = l;
                }
                __syncwarp();
                for (unsigned odd = __ballot_sync(FULL_MASK, nan && l > 0.0f); odd != 0; odd &= odd - 1) {
                    const int from = __ffs(odd) - 1;
                    const int node = w.node0 + __shfl_sync(FULL_MASK, token, from), head = w.head0 + __shfl_sync(FULL_MASK, row_head, from);
                    AgainRow<T> x;
                    x.q = static_cast<const T *>(p.q) + (static_cast<size_t>(w.seq) * p.n_nodes + node) * p.q_stride + static_cast<size_t>(head) * D;
                    x.k_pages = static_cast<const T *>(p.k_pages);
                    x.v_pages = static_cast<const T *>(p.v_pages);
                    x.parents = p.parents + static_cast<size_t>(w.seq) * p.n_nodes;
                    x.out = static_cast<T *>(p.out) + ((static_cast<long long>(w.seq) * p.n_nodes + node) * p.n_q_heads + head) * D;
                    x.ml = nullptr;
                    x.record = w.whole ? nullptr : record + static_cast<size_t>(__shfl_sync(FULL_MASK, r, from)) * D;
                    x.slot = w.slot;
                    x.kvh = w.kvh;
                    x.node = node;
                    x.base = base;
                    x.len = len;
                    x.from = w.tile(w.j0) * kTcKeys;  // (nobody sees what lies between the sinks' tiles and the window's)
                    x.to = (w.tile(j1 - 1) + 1) * kTcKeys;
                    x.scale_log2 = p.scale_log2;
                    x.l = __shfl_sync(FULL_MASK, l, from);
                    again<T, D, D, false>(p.cache, p.mask, x, 0);
                }
                tc::fence_before_sync();
            }
            if (both && adds) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&half_free[i ^ 1]);
            }
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

// Adds up the parts of the units that crossed a range's end. Grid: (CTA in whose range the unit began,
// share of its rows); a warp takes a row at a time: the parts' weights by lane, then their sums.
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_tree_join_kernel(const TreeAttnParams p) {
    constexpr int kCols = D / 32;  // columns of a lane
    __shared__ float weights[4][kSMs];
    const TreeJoin join = p.joins[blockIdx.x];
    const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (join.c1 < 0) return;
    const int per = p.tokens_per_tile;
    const int rows = join.turns || join.nodes <= per ? kTcRows : 2 * kTcRows;
    for (int r = blockIdx.y * 4 + warp; r < rows; r += kJoinParts * 4) {
        const int in = r & (kTcRows - 1), token = (r / kTcRows) * per + in / p.heads_per_tile, head = in % p.heads_per_tile;
        if (in / p.heads_per_tile >= per || token >= join.nodes || head >= join.heads) continue;
        auto record = [&](int c) { return p.record(c, c == c0 ? 1 : 0, D); };
        float top = -INFINITY;
        bool none = false;
        for (int c = c0 + lane; c <= join.c1; c += 32) {
            const float *rec = record(c);
            none |= rec[p.record_rows * (D + 1) + r] < 0.0f;
            top = fmaxf(top, rec[p.record_rows * D + r]);
        }
        __syncwarp();
        if (__any_sync(FULL_MASK, none)) continue;  // a wait gave up there
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        float l = 0.0f;
        for (int c = c0 + lane; c <= join.c1; c += 32) {
            const float *rec = record(c);
            const float m = rec[p.record_rows * D + r], f = m == -INFINITY ? 0.0f : fast_exp2(m - top);
            weights[warp][c - c0] = f;
            l = fmaf(f, rec[p.record_rows * (D + 1) + r], l);
        }
        __syncwarp();
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(FULL_MASK, l, o);
        float o[kCols] = {};
        // (all parts' loads on their way together; one that saw nothing may hold anything)
#pragma unroll 8
        for (int c = c0; c <= join.c1; ++c) {
            const float f = weights[warp][c - c0];
            float x[kCols];
            load_vec<kCols>(x, record(c) + static_cast<size_t>(r) * D + lane * kCols);
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[e] = f == 0.0f ? o[e] : fmaf(f, x[e], o[e]);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T *out = static_cast<T *>(p.out) +
                 ((static_cast<long long>(join.seq) * p.n_nodes + join.node0 + token) * p.n_q_heads + join.head0 + head) * D + lane * kCols;
#pragma unroll
        for (int e = 0; e < kCols; e += 2)
            *reinterpret_cast<uint32_t *>(out + e) = Elem<T>::pack(o[e] * inv, o[e + 1] * inv);
        __syncwarp();  // the weights have been read
    }
}

// ------------------------------------------------------------------ host side

struct Rows {
    int heads, nodes, blocks, record;  // of a lane: heads x nodes; blocks of a key head's nodes; rows of a record
};

Rows rows_of(int n_nodes, int group, int head_dim) {
    Rows r;
    r.heads = group < kTcRows ? group : kTcRows;
    r.nodes = kTcRows / r.heads < n_nodes ? kTcRows / r.heads : n_nodes;
    const int lanes = head_dim == 256 ? 1 : 2;
    r.blocks = (n_nodes + lanes * r.nodes - 1) / (lanes * r.nodes);
    r.record = lanes == 2 && n_nodes > r.nodes ? 2 * kTcRows : kTcRows;
    return r;
}

constexpr size_t kJoinBytes = (kSMs * sizeof(TreeJoin) + 255) / 256 * 256;

template <typename T, int D, bool EXTRA>
gdn_status launch(TreeAttnParams p, int dtype, cudaStream_t s) {
    using C = TreeTc<D, EXTRA>;
    const int ps = 1 << p.cache.log2_ps;
    const int q_bytes = p.q_rows * D * 2;
    p.q_bufs = C::kLanes == 1 || 2 * q_bytes > C::kRoom ? 1 : 2;
    CUtensorMap q_map, k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(p.cache.n_pages) * p.cache.n_kv_heads * ps;
    GDN_TRY(encode_heads_map(&q_map, p.q, dtype, D, p.n_q_heads, static_cast<uint64_t>(p.n_seqs) * p.n_nodes,
                             static_cast<uint64_t>(p.q_stride) * 2, p.heads_per_tile, p.tokens_per_tile));
    GDN_TRY(encode_blocks_map(&k_map, p.k_pages, dtype, D, rows, D * 2, ps < kTcKeys ? ps : kTcKeys,
                              ps < kTcKeys ? 1 : C::kCols));
    GDN_TRY(encode_blocks_map(&v_map, p.v_pages, dtype, D, rows, D * 2, ps < C::kVKeys ? ps : C::kVKeys, D / 64));
    auto kernel = attn_tree_tc_kernel<T, D, EXTRA>;
    static std::atomic<unsigned long long> allowed{0};
    GDN_TRY(allow_smem(kernel, C::kRings + C::kRoom + 1024, allowed));
    kernel<<<kSMs, C::kThreads, C::kRings + p.q_bufs * q_bytes + 1024, s>>>(q_map, k_map, v_map, p);
    GDN_TRY(launch_status());
    attn_tree_join_kernel<T, D><<<dim3(kSMs, kJoinParts), 128, 0, s>>>(p);
    return launch_status();
}

template <typename T, int D>
gdn_status launch_rows(const TreeAttnParams &p, int dtype, cudaStream_t s) {
    static_assert(TreeTc<D, false>::kRoom >= TreeTc<D, false>::kLanes * kTcRows * D * 2, "a whole Q for each lane");
    const bool extra = p.blocks == 1 && p.record_rows == kTcRows && p.q_rows * D * 2 <= TreeTc<D, true>::kRoom;
    return extra ? launch<T, D, true>(p, dtype, s) : launch<T, D, false>(p, dtype, s);
}

template <typename T>
gdn_status launch_dim(int d, const TreeAttnParams &p, int dtype, cudaStream_t s) {
    switch (d) {
        case 64: return launch_rows<T, 64>(p, dtype, s);
        case 128: return launch_rows<T, 128>(p, dtype, s);
        default: return launch_rows<T, 256>(p, dtype, s);
    }
}

}  // namespace

// More rows than a fragment of the decode attention's: from there on each 16 would read the keys again.
bool tree_on_tensor_cores(int dtype, int n_nodes, int group) { return dtype != GDN_F32 && n_nodes * group > 16; }

size_t attn_tree_tc_workspace(int n_nodes, int group, int head_dim) {
    return kJoinBytes + static_cast<size_t>(kSMs) * 2 * rows_of(n_nodes, group, head_dim).record * (head_dim + 2) * sizeof(float);
}

gdn_status launch_attn_tree_tc(TreeAttnParams p, int dtype, int head_dim, void *workspace, cudaStream_t s) {
    const Rows r = rows_of(p.n_nodes, p.group, head_dim);
    p.heads_per_tile = r.heads;
    p.tokens_per_tile = r.nodes;
    p.head_groups = (p.group + r.heads - 1) / r.heads;
    p.blocks = r.blocks;
    p.record_rows = r.record;
    p.q_rows = (r.heads * r.nodes + 7) / 8 * 8;
    // the ranges are counted in 32 bits
    const long long widest = ((static_cast<long long>(p.cache.max_pages) << p.cache.log2_ps) + kTcKeys - 1) / kTcKeys + 2 + kTurn;
    if (widest * p.cache.n_kv_heads * p.head_groups * p.blocks > 0x7fffffffLL / p.n_seqs) return GDN_ERR_UNSUPPORTED;
    p.joins = static_cast<TreeJoin *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kJoinBytes);
    return dtype == GDN_F16 ? launch_dim<__half>(head_dim, p, dtype, s) : launch_dim<__nv_bfloat16>(head_dim, p, dtype, s);
}

}  // namespace gdn
