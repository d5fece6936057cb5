// gdn_attn_tree.cuh -- what the tree attention's call and its tensor-core kernel share.
#pragma once

#include "gdn_paged.cuh"

namespace gdn {

// A unit (sequence, key head, block of rows) that crosses the end of the range it begins in: what the
// joining kernel needs to know of it. c1: the last CTA that has a part of it; -1: none.
struct TreeJoin {
    int seq, head0, heads, node0, nodes, turns, c1;
};

struct TreeAttnParams {
    PagedCache cache;
    AttnMask mask;
    const int32_t *parents;
    const void *q, *k_pages, *v_pages;
    void *out;
    int n_seqs, n_nodes, n_q_heads, group, q_stride;
    int heads_per_tile, tokens_per_tile;  // rows of a lane: nodes x heads
    int head_groups, blocks;              // of a key head
    int record_rows;                      // rows of a partial result: 128 or 256
    int q_rows, q_bufs;                   // rows of a Q buffer; buffers
    float scale_log2;
    int32_t *err_count;
    unsigned *watchdog;
    TreeJoin *joins;   // [grid]
    float *partials;   // [grid][2] records: rows of sums, then maxima, then lengths

    // CTA c's part of the unit split at its range's start (0) or end (1).
    __device__ __forceinline__ float *record(int c, int which, int d) const {
        return partials + static_cast<size_t>(2 * c + which) * record_rows * (d + 2);
    }
};

// Whether a call's rows are the tensor cores' (16-bit types), and the workspace it then needs.
bool tree_on_tensor_cores(int dtype, int n_nodes, int group);
size_t attn_tree_tc_workspace(int n_nodes, int group, int head_dim);
gdn_status launch_attn_tree_tc(TreeAttnParams p, int dtype, int head_dim, void *workspace, cudaStream_t s);

}  // namespace gdn
