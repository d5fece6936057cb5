// gdn_attn_prefill.cuh -- what the prompt attention's two paths (fp32 on the FP32 pipes, 16-bit
// types on the tensor cores) share.
#pragma once

#include "gdn_paged.cuh"

namespace gdn {

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

// 16-bit types (dtype GDN_F16 or GDN_BF16).
gdn_status launch_attn_prefill_tc(const PrefillParams &p, int dtype, int head_dim, cudaStream_t s);

}  // namespace gdn
