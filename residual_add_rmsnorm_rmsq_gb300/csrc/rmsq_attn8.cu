// Attention over the paged FP8 cache: C entry.
#include "rmsq_attn8.cuh"
#include "rmsq_attn_launch.cuh"

namespace rmsq {
cudaError_t take_prompt_fault_fp8(unsigned int* out) { return take_fault_of_unit(out); }
}  // namespace rmsq

extern "C" int rmsq_paged_attention_fp8(const void* q, int64_t q_stride, const void* cache, const uint8_t* scales,
                                        int64_t num_pages, int64_t page_size, const int32_t* block_table,
                                        int64_t table_width, const int32_t* query_start, const int32_t* seq_lens,
                                        float softmax_scale, int64_t window, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, int64_t n_tokens, int64_t num_requests, int num_heads,
                                        int num_kv_heads, int head_dim, int dtype, void* stream, int variant,
                                        int64_t max_query) {
    const rmsq::AttnCall c = {q, q_stride, cache, scales, num_pages, page_size, block_table, table_width, query_start,
                              seq_lens, nullptr, nullptr, softmax_scale, window, out, lse, workspace, workspace_bytes,
                              n_tokens, num_requests, num_heads, num_kv_heads, head_dim, dtype, stream, variant, max_query};
    return rmsq::attend<rmsq::Fp8Cache, rmsq::Fp8Prompt>(c, head_dim);
}
