// gdn_attn_tree.cu -- attention of a tree of drafted tokens over the paged cache: the call, and the
// decode attention's kernel (gdn_attn_decode.cuh) in its tree form, for fp32 and for few rows. (Each 16
// rows of (node, head) read the keys again there: more of them, in 16-bit types, are the tensor cores'
// of gdn_attn_tree_tc.cu. In fp32 the products bound the call, not the reading.)
#include "gdn_attn_decode.cuh"
#include "gdn_attn_tree.cuh"

using namespace gdn;

extern "C" {

size_t gdn_attn_tree_workspace_size(int n_seqs, int n_nodes, int n_q_heads, int n_kv_heads, int head_dim) {
    if (n_seqs < 0 || n_nodes < 1 || n_nodes > kMaxNodes || n_kv_heads < 1 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads != 0 || !supported_head_dim(head_dim))
        return 0;
    // (the type is not known here)
    const size_t small = workspace_bytes_for(head_dim);
    const size_t large = attn_tree_tc_workspace(n_nodes, n_q_heads / n_kv_heads, head_dim);
    return tree_on_tensor_cores(GDN_BF16, n_nodes, n_q_heads / n_kv_heads) && large > small ? large : small;
}

gdn_status gdn_attn_tree(const void *q, const void *k_pages, const void *v_pages,
                         const int32_t *page_table, const int32_t *kv_lens, void *out,
                         const int32_t *parents, int n_seqs, int n_nodes, int n_q_heads,
                         int n_kv_heads, int head_dim, int page_size, int n_pages, int max_pages,
                         int window, int n_sinks, float scale, int q_stride, int dtype,
                         const int32_t *slots, int pool, int32_t *err_count, void *workspace,
                         size_t workspace_bytes, gdn_stream_t stream) {
    GDN_TRY(check_tree(parents, n_seqs, n_nodes));
    const size_t need = gdn_attn_tree_workspace_size(n_seqs, n_nodes, n_q_heads, n_kv_heads, head_dim);
    GDN_TRY(check_decode(q, k_pages, v_pages, page_table, kv_lens, out, n_seqs, n_nodes, n_q_heads, n_kv_heads,
                         head_dim, page_size, n_pages, max_pages, window, n_sinks, q_stride, dtype, slots, pool,
                         workspace, workspace_bytes, need));
    if (n_seqs == 0) return GDN_OK;
    if (tree_on_tensor_cores(dtype, n_nodes, n_q_heads / n_kv_heads)) {
        TreeAttnParams p{};
        p.cache = PagedCache{page_table, kv_lens, slots, pool, max_pages, n_pages, n_kv_heads, log2_of(page_size)};
        p.mask = make_mask(window, n_sinks);
        p.parents = parents;
        p.q = q;
        p.k_pages = k_pages;
        p.v_pages = v_pages;
        p.out = out;
        p.n_seqs = n_seqs;
        p.n_nodes = n_nodes;
        p.n_q_heads = n_q_heads;
        p.group = n_q_heads / n_kv_heads;
        p.q_stride = q_stride;
        p.scale_log2 = scale * kLog2E;
        p.err_count = err_count;
        p.watchdog = watchdog_attn_decode();
        if (p.watchdog == nullptr) return GDN_ERR_LAUNCH;
        return launch_attn_tree_tc(p, dtype, head_dim, workspace, as_cuda(stream));
    }
    return attn_decode_call<true>(q, k_pages, v_pages, page_table, kv_lens, out, parents, n_seqs, n_nodes,
                                  n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, window,
                                  n_sinks, scale, q_stride, dtype, slots, pool, err_count, workspace,
                                  workspace_bytes, stream);
}

}  // extern "C"
