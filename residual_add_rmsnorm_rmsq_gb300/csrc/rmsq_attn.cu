// Attention over the paged NVFP4 cache: C entries.
#include "rmsq_attn_launch.cuh"

namespace rmsq {
cudaError_t take_prompt_fault(unsigned int* out) { return take_fault_of_unit(out); }
}  // namespace rmsq

extern "C" {

size_t rmsq_paged_attention_workspace_bytes(int64_t n_tokens, int64_t num_requests, int num_heads, int num_kv_heads,
                                            int head_dim) {
    if (rmsq::attn_shape(n_tokens, num_requests, num_heads, num_kv_heads, head_dim) != RMSQ_OK) return 0;
    // for the most row blocks of any call, so that a workspace serves every smaller one
    const int nb = head_dim <= 128 ? 2 : 1;
    return static_cast<size_t>(rmsq::kAttnMaxWorkers) * (sizeof(rmsq::CutItem) + 2 * rmsq::part_floats(head_dim, nb) * 4);
}

int rmsq_paged_attention_nvfp4(const void* q, int64_t q_stride, const void* kv_cache, int64_t num_pages, int64_t page_size,
                               const int32_t* block_table, int64_t table_width, const int32_t* query_start,
                               const int32_t* seq_lens, const float* k_global_scale, const float* v_global_scale,
                               float softmax_scale, int64_t window, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int64_t n_tokens, int64_t num_requests, int num_heads,
                               int num_kv_heads, int head_dim, int dtype, void* stream, int variant) {
    return rmsq_paged_attention_nvfp4_ex(q, q_stride, kv_cache, num_pages, page_size, block_table, table_width, query_start,
                                         seq_lens, k_global_scale, v_global_scale, softmax_scale, window, out, lse, workspace,
                                         workspace_bytes, n_tokens, num_requests, num_heads, num_kv_heads, head_dim, dtype,
                                         stream, variant, 0);
}

int rmsq_paged_attention_nvfp4_ex(const void* q, int64_t q_stride, const void* kv_cache, int64_t num_pages,
                                  int64_t page_size, const int32_t* block_table, int64_t table_width,
                                  const int32_t* query_start, const int32_t* seq_lens, const float* k_global_scale,
                                  const float* v_global_scale, float softmax_scale, int64_t window, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, int64_t n_tokens, int64_t num_requests,
                                  int num_heads, int num_kv_heads, int head_dim, int dtype, void* stream, int variant,
                                  int64_t max_query) {
    const rmsq::AttnCall c = {q, q_stride, kv_cache, nullptr, num_pages, page_size, block_table, table_width, query_start,
                              seq_lens, k_global_scale, v_global_scale, softmax_scale, window, out, lse, workspace,
                              workspace_bytes, n_tokens, num_requests, num_heads, num_kv_heads, head_dim, dtype, stream,
                              variant, max_query};
    return rmsq::attend<rmsq::Nvfp4Cache, rmsq::Nvfp4Prompt>(c, head_dim * 9 / 16);
}

}  // extern "C"
