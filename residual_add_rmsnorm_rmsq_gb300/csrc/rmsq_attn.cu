// Attention over the paged NVFP4 cache: argument checks and launches.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_attn.cuh"
#include "rmsq_attn_prompt.cuh"
#include "rmsq_host.cuh"

namespace rmsq {

cudaError_t take_prompt_fault(unsigned int* out) {
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_prompt_fault, sizeof(unsigned int));
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_prompt_fault, &zero, sizeof(zero));
    return e;
}

namespace {

// Row blocks of 8: two (16 rows share a pass over the keys) where a request
// has more than 8 rows on average; one for D = 256, whose accumulators for 16
// rows would not fit the registers.  Beside the prompt kernel the average says
// nothing about the requests that are left, and they are taken for decodes of
// one token: one block for a group of up to 8.  The other mistake is the
// smaller one: 127 decodes of 8 x 4 heads on 2000 keys beside a prompt of 300
// tokens take 58 us with one block and 78 with two (on 8000 keys beside 2000
// tokens 225 and 273; one of 4 x 8 heads on 4000 keys beside 1500 70 and 79), but
// 250 requests of four queries of 4 x 8 heads on 1000 keys 139 and 132, and two
// prompts alone 3 us more, for the larger empty launch.
int row_blocks(int64_t tokens, int64_t requests, int group, int head_dim, bool beside_prompts) {
    return head_dim <= 128 && (beside_prompts ? group > 8 : tokens * group > 8 * requests) ? 2 : 1;
}

size_t part_floats(int head_dim, int nb) { return static_cast<size_t>(8) * nb * (head_dim + 4); }    // kPartRow

template <class E, int D, int NB>
cudaError_t launch_split(AttnArgs a, int64_t max_tiles, cudaStream_t stream) {
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess) return e;
    const void* split = (const void*)&attn_split_kernel<E, D, NB>;
    const void* join = (const void*)&attn_join_kernel<E, D, NB>;
    // the scanned tile counts, in steps of 1 KB (so that few launch shapes occur)
    const int counts = ((a.requests + 1) * 8 + 1023) / 1024 * 1024, smem = kAttnMem<D, NB> + counts;
    constexpr int kMostCounts = ((RMSQ_MAX_REQUESTS + 1) * 8 + 1023) / 1024 * 1024;
    e = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnMem<D, NB> + kMostCounts);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(split, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    const int per_sm = occupancy_blocks(split, kAttnThreads, smem, &e);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    int64_t workers = static_cast<int64_t>(per_sm) * sms;
    if (workers > kAttnMaxWorkers) workers = kAttnMaxWorkers;
    if (workers > max_tiles) workers = max_tiles;
    a.workers = static_cast<int>(workers);
    void* params[] = {&a};
    e = launch_kernel(split, dim3(a.workers), dim3(kAttnThreads), params, smem, stream);
    if (e != cudaSuccess) return e;
    // few items: each is cut into many parts
    const int64_t items = (static_cast<int64_t>(a.tokens) * a.group / (8 * NB) + a.requests) * a.kv_heads;
    const unsigned shares = items * 8 <= workers ? kJoinShares : 1;
    return launch_kernel(join, dim3(a.workers, shares), dim3(kJoinThreads), params, 0, stream);
}

template <class E, int D>
cudaError_t launch_prompt(AttnArgs a, cudaStream_t stream) {
    const void* fn = (const void*)&attn_prompt_kernel<E, D>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptTile<D>::smem);
    if (e != cudaSuccess) return e;
    // as many 256-row items as these sizes can hold; those without one return at once
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.group;
    const int64_t few = rows / (a.most_rows + 1);
    const int64_t items = rows / 256 + (few < a.requests ? few : a.requests);
    void* params[] = {&a};
    return launch_kernel(fn, dim3(static_cast<unsigned>(items * a.kv_heads)), dim3(kPromptThreads), params,
                         PromptTile<D>::smem, stream);
}

// What the kernels take for 128 keys, in us: the split kernel for 48 (row, kv
// head) per SM, the prompt kernel for a CTA's 256 rows on every SM.  Measured on
// 20000 to 100000 keys: 1.92 to 2.07 and 1.80 to 1.92 (D = 128), 1.16 to 1.27 and
// 1.44 to 1.52 (64).
struct Cost {
    double split, prompt;
};
Cost cost_of(int head_dim) { return head_dim <= 64 ? Cost{1.21, 1.48} : Cost{1.97, 1.86}; }

// Requests of more than kPromptRows rows go to the prompt kernel (AUTO: if they
// are worth it there, see prompt_takes), the others to the split kernel, whichever
// they are: the lengths are the device's.
//
// The prompt kernel is launched (AUTO) where it is expected sooner.  It gives a
// CTA 256 rows and all their keys; the split kernel gives equal runs of keys, for
// 16 rows at a time, to the CTAs of the whole card.  So few rows on a long context
// belong to the split kernel, although it reads the keys once per 16 rows.  Both
// costs are proportional to the length, which the host does not know, so that
// what decides is the rows.  Measured with one request of 8 x 8 heads of 128 and
// 20000 keys, split and prompt: 88 queries 250 and 300 us, 104 292 and 301, 112
// 313 and 300, 128 355 and 301 (on 2000 keys already 96 queries 49 and 42); heads
// of 64, 128 queries: 218 and 237.  8 queries of 16 x 8 heads on 50000 keys 124
// and 675; 8 requests of 50 queries (8 x 4 heads) on 2000 82 and 46; 4 of 200 (4 x
// 8) on 500 66 and 23.
//
// It is not launched where no request can be its: the caller's bound on the
// queries of a request says so, or, without one, that there are no more than one
// token per request and the rows of one prompt (requests without queries count
// as having one: only the time is lost if a longer one is among them).  Its
// empty CTAs are not free: 260 and 1000 decodes of 4 x 8 heads on 1000 keys took
// 77 and 261 us behind them, 73 and 253 without, 1000 requests of four queries
// on 200 keys 273 and 243.
template <class E>
cudaError_t launch_attn(AttnArgs a, int head_dim, int64_t max_query, int64_t max_tiles, int variant, cudaStream_t stream) {
    cudaError_t err;
    const int sms = sm_count(&err);
    if (err != cudaSuccess) return err;
    const int64_t tokens = max_query > 0 && max_query < a.tokens / a.requests ? max_query * a.requests : a.tokens;
    const int64_t rows = tokens * a.group;
    const int64_t items = (rows / 256 + 1) * a.kv_heads;
    const Cost cost = cost_of(head_dim);
    const bool sooner = cost.split * static_cast<double>(rows * a.kv_heads) / (48.0 * sms) >
                        cost.prompt * static_cast<double>((items + sms - 1) / sms);
    const int64_t rest = a.tokens >= a.requests ? a.tokens - a.requests + 1 : 1;    // left for one request
    const int64_t longest = max_query > 0 ? (max_query < a.tokens ? max_query : a.tokens)
                            : variant == kVariantPipelined ? a.tokens : rest;
    const bool prompt = head_dim <= 128 && longest * a.group > kPromptRows && variant != kVariantDirect &&
                        (variant == kVariantPipelined || sooner);
    // (a single request is the prompt kernel's whatever its length)
    a.most_rows = !prompt ? INT32_MAX : a.requests == 1 ? 0 : kPromptRows;
    if (prompt && variant == kVariantAuto && a.requests > 1)
        a.share = static_cast<int64_t>(cost.prompt / cost.split * 48.0 * sms / a.kv_heads) + 1;
    if (prompt) {
        const cudaError_t e = head_dim == 64 ? launch_prompt<E, 64>(a, stream) : launch_prompt<E, 128>(a, stream);
        if (e != cudaSuccess || a.requests == 1) return e;
    }
    const int nb = row_blocks(a.tokens, a.requests, a.group, head_dim, prompt);
    switch (head_dim) {
    case 64: return nb == 2 ? launch_split<E, 64, 2>(a, max_tiles, stream) : launch_split<E, 64, 1>(a, max_tiles, stream);
    case 128: return nb == 2 ? launch_split<E, 128, 2>(a, max_tiles, stream) : launch_split<E, 128, 1>(a, max_tiles, stream);
    default: return launch_split<E, 256, 1>(a, max_tiles, stream);
    }
}

int attn_shape(int64_t tokens, int64_t requests, int heads, int kv_heads, int head_dim) {
    if (tokens < 0 || requests < 0 || heads <= 0 || kv_heads <= 0) return RMSQ_ERR_INVALID_ARG;
    if (heads % kv_heads != 0 || heads > 4096 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        requests > RMSQ_MAX_REQUESTS || tokens > INT32_MAX / heads)
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    return RMSQ_OK;
}

}  // namespace
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
    using rmsq_abi::aligned;
    using rmsq_abi::overlaps;
    using rmsq_abi::Span;
    using rmsq_abi::span;
    if (dtype != RMSQ_BF16 && dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    if (variant != RMSQ_VARIANT_AUTO && variant != RMSQ_VARIANT_DIRECT && variant != RMSQ_VARIANT_PIPELINED)
        return RMSQ_ERR_INVALID_ARG;
    int st = rmsq::attn_shape(n_tokens, num_requests, num_heads, num_kv_heads, head_dim);
    if (st != RMSQ_OK) return st;
    if (!std::isfinite(softmax_scale) || softmax_scale <= 0.0f || window < 0 || num_pages < 0 || table_width < 0 ||
        max_query < 0)
        return RMSQ_ERR_INVALID_ARG;
    int shift = -1;
    for (int s = 4; s <= 8; ++s)
        if (page_size == (1 << s)) shift = s;
    if (shift < 0 || num_pages > INT32_MAX || table_width > (INT32_MAX >> (shift + 1))) return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int64_t row = static_cast<int64_t>(num_heads) * head_dim;
    if (q_stride < row || q_stride > INT32_MAX) return RMSQ_ERR_INVALID_ARG;
    if (n_tokens == 0 || num_requests == 0) return RMSQ_OK;
    if (!q || !query_start || !seq_lens || !k_global_scale || !v_global_scale || !out || !workspace ||
        (num_pages > 0 && !kv_cache) || (table_width > 0 && !block_table))
        return RMSQ_ERR_INVALID_ARG;
    const size_t need = rmsq_paged_attention_workspace_bytes(n_tokens, num_requests, num_heads, num_kv_heads, head_dim);
    if (workspace_bytes < need) return RMSQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(query_start, 4) ||
        !aligned(seq_lens, 4) || !aligned(k_global_scale, 4) || !aligned(v_global_scale, 4) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return RMSQ_ERR_ALIGNMENT;
    const size_t tile = static_cast<size_t>(head_dim) * 9 / 16 << shift;
    const Span ins[7] = {span(q, (static_cast<size_t>(n_tokens - 1) * q_stride + row) * 2),
                         span(kv_cache, static_cast<size_t>(num_pages) * 2 * num_kv_heads * tile),
                         span(block_table, static_cast<size_t>(num_requests) * table_width * 4),
                         span(query_start, static_cast<size_t>(num_requests + 1) * 4),
                         span(seq_lens, static_cast<size_t>(num_requests) * 4), span(k_global_scale, 4),
                         span(v_global_scale, 4)};
    const Span outs[3] = {span(out, static_cast<size_t>(n_tokens) * row * 2),
                          span(lse, static_cast<size_t>(n_tokens) * num_heads * 4), span(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& in : ins)
            if (overlaps(outs[i], in)) return RMSQ_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outs[j])) return RMSQ_ERR_ALIAS;
    }
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    rmsq::AttnArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(kv_cache);
    a.table = block_table;
    a.q_start = query_start;
    a.seq_lens = seq_lens;
    a.k_gs = k_global_scale;
    a.v_gs = v_global_scale;
    a.out = out;
    a.lse = lse;
    a.cut = static_cast<rmsq::CutItem*>(workspace);
    a.part = reinterpret_cast<float*>(a.cut + rmsq::kAttnMaxWorkers);
    a.requests = static_cast<int>(num_requests);
    a.width = static_cast<int>(table_width);
    a.tokens = static_cast<int>(n_tokens);
    a.heads = num_heads;
    a.kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.page_shift = shift;
    a.num_pages = static_cast<int>(num_pages);
    a.window = window > INT32_MAX / 2 ? 0 : static_cast<int>(window);
    a.scale_log2 = softmax_scale * 1.44269504088896341f;
    // most (row tile, kv head, key tile) tiles these sizes can hold
    const int64_t ktiles = (static_cast<int64_t>(table_width) << shift) / rmsq::kAttnKeyTile + 1;
    constexpr int64_t kMaxTiles = int64_t(1) << 40;
    const int64_t qtiles = n_tokens * a.group / 8 + num_requests;
    const int64_t max_tiles = qtiles > kMaxTiles / ktiles / num_kv_heads ? kMaxTiles : qtiles * ktiles * num_kv_heads;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = variant == RMSQ_VARIANT_DIRECT ? rmsq::kVariantDirect
                  : variant == RMSQ_VARIANT_PIPELINED ? rmsq::kVariantPipelined : rmsq::kVariantAuto;
    const cudaError_t e = dtype == RMSQ_BF16 ? rmsq::launch_attn<rmsq::Bf16T>(a, head_dim, max_query, max_tiles, v, s)
                                             : rmsq::launch_attn<rmsq::Fp16T>(a, head_dim, max_query, max_tiles, v, s);
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

}  // extern "C"
