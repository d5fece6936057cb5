// gdn_attn_decode.cu -- decode attention's entry points; the kernel is gdn_attn_decode.cuh's.
#include "gdn_attn_decode.cuh"

namespace gdn {

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

unsigned *watchdog_attn_decode() {
    static std::atomic<unsigned *> known[64];
    return flag_address(g_watchdog_attn_decode, known);
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
    return attn_decode_call<false>(q, k_pages, v_pages, page_table, kv_lens, out, nullptr, n_seqs, n_tokens,
                                   n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, window,
                                   n_sinks, scale, q_stride, dtype, slots, pool, err_count, workspace,
                                   workspace_bytes, stream);
}

}  // extern "C"
