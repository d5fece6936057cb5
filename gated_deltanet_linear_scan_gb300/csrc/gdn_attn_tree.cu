// gdn_attn_tree.cu -- attention of a tree of drafted tokens over the paged cache: the call, and the
// decode attention's kernel (gdn_attn_decode.cuh) in its tree form.
#include "gdn_attn_decode.cuh"

using namespace gdn;

extern "C" {

size_t gdn_attn_tree_workspace_size(int n_seqs, int n_nodes, int n_q_heads, int n_kv_heads, int head_dim) {
    if (n_seqs < 0 || n_nodes < 1 || n_nodes > kMaxNodes || n_kv_heads < 1 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads != 0 || !supported_head_dim(head_dim))
        return 0;
    return workspace_bytes_for(head_dim);
}

gdn_status gdn_attn_tree(const void *q, const void *k_pages, const void *v_pages,
                         const int32_t *page_table, const int32_t *kv_lens, void *out,
                         const int32_t *parents, int n_seqs, int n_nodes, int n_q_heads,
                         int n_kv_heads, int head_dim, int page_size, int n_pages, int max_pages,
                         int window, int n_sinks, float scale, int q_stride, int dtype,
                         const int32_t *slots, int pool, int32_t *err_count, void *workspace,
                         size_t workspace_bytes, gdn_stream_t stream) {
    GDN_TRY(check_tree(parents, n_seqs, n_nodes));
    return attn_decode_call<true>(q, k_pages, v_pages, page_table, kv_lens, out, parents, n_seqs, n_nodes,
                                  n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, window,
                                  n_sinks, scale, q_stride, dtype, slots, pool, err_count, workspace,
                                  workspace_bytes, stream);
}

}  // extern "C"
