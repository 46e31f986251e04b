// Launches of the attention kernels over a paged cache and the checks of their
// arguments, for the cache's readers C (split kernel) and P<D> (prompt kernel).
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_attn.cuh"
#include "rmsq_attn_prompt.cuh"
#include "rmsq_host.cuh"

namespace rmsq {

// Reads and clears this unit's fault flag.  Static as the flag is: one copy for all
// units would read one unit's.
static cudaError_t take_fault_of_unit(unsigned int* out) {
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_prompt_fault, sizeof(unsigned int));
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_prompt_fault, &zero, sizeof(zero));
    return e;
}

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
inline int row_blocks(int64_t tokens, int64_t requests, int group, int head_dim, bool beside_prompts) {
    return head_dim <= 128 && (beside_prompts ? group > 8 : tokens * group > 8 * requests) ? 2 : 1;
}

inline size_t part_floats(int head_dim, int nb) { return static_cast<size_t>(8) * nb * (head_dim + 4); }    // kPartRow

template <class C, class E, int D, int NB>
cudaError_t launch_split(AttnArgs a, int64_t max_tiles, cudaStream_t stream) {
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess) return e;
    const void* split = (const void*)&attn_split_kernel<C, E, D, NB>;
    const void* join = (const void*)&attn_join_kernel<C, E, D, NB>;
    // the scanned tile counts, in steps of 1 KB (so that few launch shapes occur)
    const int counts = ((a.requests + 1) * 8 + 1023) / 1024 * 1024, smem = kAttnMem<C, D, NB> + counts;
    constexpr int kMostCounts = ((RMSQ_MAX_REQUESTS + 1) * 8 + 1023) / 1024 * 1024;
    e = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnMem<C, D, NB> + kMostCounts);
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

template <class P, class E, int D>
cudaError_t launch_prompt(AttnArgs a, cudaStream_t stream) {
    const void* fn = (const void*)&attn_prompt_kernel<P, E, D>;
    constexpr int smem = PromptTile<D>::with_ring(P::ring);
    static_assert(smem <= 230400, "the rest is the kernel's static shared memory");
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // as many items of 256 rows as these sizes can hold, and of 128 as they and the card
    // can; those without one return at once
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.group;
    int64_t few = rows / (a.most_rows + 1);
    if (few > a.requests) few = a.requests;
    int64_t items = rows / 256 + few;
    const int64_t halves = rows / 128 + few < a.half_items ? rows / 128 + few : a.half_items;
    if (halves > items) items = halves;
    void* params[] = {&a};
    return launch_kernel(fn, dim3(static_cast<unsigned>(items * a.kv_heads)), dim3(kPromptThreads), params,
                         smem, stream);
}

// What the kernels take for 128 keys, in us: the split kernel for 48 (row, kv
// head) per SM, the prompt kernel for a CTA's 256 rows on every SM.  Measured on
// 20000 to 100000 keys of the NVFP4 cache: 1.92 to 2.07 and 1.80 to 1.92 (D = 128),
// 1.16 to 1.27 and 1.44 to 1.52 (64).  The prompt kernel's steps have become shorter
// since, 1.67 at D = 128: it would be sooner from 96 queries of 8 x 8 heads on (270
// us split and 261, 104 290 and 261) and is taken from 108.  The border has stayed,
// and with it what calls in between give to the last bit.
// On 20000 keys of the FP8 cache 2.31 and 1.98, 1.50 and 1.54, with 128 rows per CTA
// 1.82 and 1.39, up to 5 % more than the constants; the two kernels meet where these
// say: 88 queries of 8 x 8 heads of 128 279 us split and 283, 96 304 and 285, heads of
// 64 104 213 and 218, 112 228 and 216.
struct Cost {
    double split, prompt, half;
};
template <class C>
Cost cost_of(int head_dim) {
    if (C::block_scales) return head_dim <= 64 ? Cost{1.43, 1.52, 1.38} : Cost{2.21, 1.97, 1.78};
    return head_dim <= 64 ? Cost{1.21, 1.48, 1.48} : Cost{1.97, 1.86, 1.86};
}

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
// 20000 keys of the NVFP4 cache, split and prompt: 88 queries 249 and 262 us, 96 270
// and 261, 112 311 and 261, 128 353 and 261 (on 2000 keys 96 queries 48 and 36);
// heads of 64, 128 queries: 214 and 225.  8 queries of 16 x 8 heads on 50000 keys 123
// and 603; 8 requests of 50 queries (8 x 4 heads) on 2000 82 and 40; 4 of 200 (4 x
// 8) on 500 65 and 21.
//
// It is not launched where no request can be its: the caller's bound on the
// queries of a request says so, or, without one, that there are no more than one
// token per request and the rows of one prompt (requests without queries count
// as having one: only the time is lost if a longer one is among them).  Its
// empty CTAs are not free: 260 and 1000 decodes of 4 x 8 heads on 1000 keys took
// 77 and 261 us behind them, 73 and 253 without, 1000 requests of four queries
// on 200 keys 273 and 243.
template <class C, template <int> class P, class E>
cudaError_t launch_attn(AttnArgs a, int head_dim, int64_t max_query, int64_t max_tiles, int variant, cudaStream_t stream) {
    cudaError_t err;
    const int sms = sm_count(&err);
    if (err != cudaSuccess) return err;
    const int64_t tokens = max_query > 0 && max_query < a.tokens / a.requests ? max_query * a.requests : a.tokens;
    const int64_t rows = tokens * a.group;
    const int64_t items = (rows / 256 + 1) * a.kv_heads;
    const Cost cost = cost_of<C>(head_dim);
    const double step = (rows / 128 + 1) * a.kv_heads <= sms ? cost.half : cost.prompt;
    const bool sooner = cost.split * static_cast<double>(rows * a.kv_heads) / (48.0 * sms) >
                        step * static_cast<double>((items + sms - 1) / sms);
    const int64_t rest = a.tokens >= a.requests ? a.tokens - a.requests + 1 : 1;    // left for one request
    const int64_t longest = max_query > 0 ? (max_query < a.tokens ? max_query : a.tokens)
                            : variant == kVariantPipelined ? a.tokens : rest;
    const bool prompt = head_dim <= 128 && longest * a.group > kPromptRows && variant != kVariantDirect &&
                        (variant == kVariantPipelined || sooner);
    // (a single request is the prompt kernel's whatever its length)
    a.most_rows = !prompt ? INT32_MAX : a.requests == 1 ? 0 : kPromptRows;
    if (prompt && variant == kVariantAuto && a.requests > 1)
        a.share = static_cast<int64_t>(step / cost.split * 48.0 * sms / a.kv_heads) + 1;
    a.half_items = C::block_scales ? sms / a.kv_heads : 0;      // (over the NVFP4 cache items have 256 rows)
    if (prompt) {
        const cudaError_t e = head_dim == 64 ? launch_prompt<P<64>, E, 64>(a, stream) : launch_prompt<P<128>, E, 128>(a, stream);
        if (e != cudaSuccess || a.requests == 1) return e;
    }
    const int nb = row_blocks(a.tokens, a.requests, a.group, head_dim, prompt);
    switch (head_dim) {
    case 64: return nb == 2 ? launch_split<C, E, 64, 2>(a, max_tiles, stream) : launch_split<C, E, 64, 1>(a, max_tiles, stream);
    case 128: return nb == 2 ? launch_split<C, E, 128, 2>(a, max_tiles, stream) : launch_split<C, E, 128, 1>(a, max_tiles, stream);
    default: return launch_split<C, E, 256, 1>(a, max_tiles, stream);
    }
}

inline int attn_shape(int64_t tokens, int64_t requests, int heads, int kv_heads, int head_dim) {
    if (tokens < 0 || requests < 0 || heads <= 0 || kv_heads <= 0) return RMSQ_ERR_INVALID_ARG;
    if (heads % kv_heads != 0 || heads > 4096 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        requests > RMSQ_MAX_REQUESTS || tokens > INT32_MAX / heads)
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    return RMSQ_OK;
}

// An attention call: the arguments of the C entries, checked and launched.
// scales is the FP8 cache's, the global scales are the NVFP4 cache's; `per_token`
// is the bytes of a token, side and head in the cache.
struct AttnCall {
    const void* q;
    int64_t q_stride;
    const void* cache;
    const uint8_t* scales;
    int64_t num_pages, page_size;
    const int32_t* table;
    int64_t width;
    const int32_t *query_start, *seq_lens;
    const float *k_gs, *v_gs;
    float softmax_scale;
    int64_t window;
    void* out;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int64_t tokens, requests;
    int heads, kv_heads, head_dim, dtype;
    void* stream;
    int variant;
    int64_t max_query;
};

template <class C, template <int> class P>
int attend(const AttnCall& c, int per_token) {
    using rmsq_abi::aligned;
    using rmsq_abi::overlaps;
    using rmsq_abi::Span;
    using rmsq_abi::span;
    if (c.dtype != RMSQ_BF16 && c.dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    if (c.variant != RMSQ_VARIANT_AUTO && c.variant != RMSQ_VARIANT_DIRECT && c.variant != RMSQ_VARIANT_PIPELINED)
        return RMSQ_ERR_INVALID_ARG;
    int st = attn_shape(c.tokens, c.requests, c.heads, c.kv_heads, c.head_dim);
    if (st != RMSQ_OK) return st;
    if (!std::isfinite(c.softmax_scale) || c.softmax_scale <= 0.0f || c.window < 0 || c.num_pages < 0 || c.width < 0 ||
        c.max_query < 0)
        return RMSQ_ERR_INVALID_ARG;
    int shift = -1;
    for (int s = 4; s <= 8; ++s)
        if (c.page_size == (1 << s)) shift = s;
    if (shift < 0 || c.num_pages > INT32_MAX || c.width > (INT32_MAX >> (shift + 1))) return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int64_t row = static_cast<int64_t>(c.heads) * c.head_dim;
    if (c.q_stride < row || c.q_stride > INT32_MAX) return RMSQ_ERR_INVALID_ARG;
    if (c.tokens == 0 || c.requests == 0) return RMSQ_OK;
    if (!c.q || !c.query_start || !c.seq_lens || !c.out || !c.workspace || (c.num_pages > 0 && !c.cache) ||
        (c.width > 0 && !c.table) || (C::block_scales ? c.num_pages > 0 && !c.scales : !c.k_gs || !c.v_gs))
        return RMSQ_ERR_INVALID_ARG;
    const size_t need = rmsq_paged_attention_workspace_bytes(c.tokens, c.requests, c.heads, c.kv_heads, c.head_dim);
    if (c.workspace_bytes < need) return RMSQ_ERR_INVALID_ARG;
    if (!aligned(c.q, 16) || c.q_stride % 8 || !aligned(c.cache, 16) || !aligned(c.table, 4) || !aligned(c.query_start, 4) ||
        !aligned(c.seq_lens, 4) || !aligned(c.k_gs, 4) || !aligned(c.v_gs, 4) || !aligned(c.out, 16) ||
        !aligned(c.lse, 4) || !aligned(c.workspace, 16))
        return RMSQ_ERR_ALIGNMENT;
    const size_t sides = static_cast<size_t>(c.num_pages) * 2 * c.kv_heads;
    const Span ins[8] = {span(c.q, (static_cast<size_t>(c.tokens - 1) * c.q_stride + row) * 2),
                         span(c.cache, sides * per_token << shift), span(c.scales, sides << (shift - 4)),
                         span(c.table, static_cast<size_t>(c.requests) * c.width * 4),
                         span(c.query_start, static_cast<size_t>(c.requests + 1) * 4),
                         span(c.seq_lens, static_cast<size_t>(c.requests) * 4), span(c.k_gs, 4),
                         span(c.v_gs, 4)};
    const Span outs[3] = {span(c.out, static_cast<size_t>(c.tokens) * row * 2),
                          span(c.lse, static_cast<size_t>(c.tokens) * c.heads * 4), span(c.workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& in : ins)
            if (overlaps(outs[i], in)) return RMSQ_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outs[j])) return RMSQ_ERR_ALIAS;
    }
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    AttnArgs a = {};
    a.q = c.q;
    a.q_stride = c.q_stride;
    a.cache = static_cast<const uint8_t*>(c.cache);
    a.scales = c.scales;
    a.table = c.table;
    a.q_start = c.query_start;
    a.seq_lens = c.seq_lens;
    a.k_gs = c.k_gs;
    a.v_gs = c.v_gs;
    a.out = c.out;
    a.lse = c.lse;
    a.cut = static_cast<CutItem*>(c.workspace);
    a.part = reinterpret_cast<float*>(a.cut + kAttnMaxWorkers);
    a.requests = static_cast<int>(c.requests);
    a.width = static_cast<int>(c.width);
    a.tokens = static_cast<int>(c.tokens);
    a.heads = c.heads;
    a.kv_heads = c.kv_heads;
    a.group = c.heads / c.kv_heads;
    a.page_shift = shift;
    a.num_pages = static_cast<int>(c.num_pages);
    a.window = c.window > INT32_MAX / 2 ? 0 : static_cast<int>(c.window);
    a.scale_log2 = c.softmax_scale * 1.44269504088896341f;
    // most (row tile, kv head, key tile) tiles these sizes can hold
    const int64_t ktiles = (static_cast<int64_t>(c.width) << shift) / kAttnKeyTile + 1 + C::piece;
    constexpr int64_t kMaxTiles = int64_t(1) << 40;
    const int64_t qtiles = c.tokens * a.group / 8 + c.requests;
    const int64_t max_tiles = qtiles > kMaxTiles / ktiles / c.kv_heads ? kMaxTiles : qtiles * ktiles * c.kv_heads;
    const cudaStream_t s = static_cast<cudaStream_t>(c.stream);
    const int v = c.variant == RMSQ_VARIANT_DIRECT ? kVariantDirect
                  : c.variant == RMSQ_VARIANT_PIPELINED ? kVariantPipelined : kVariantAuto;
    const cudaError_t e = c.dtype == RMSQ_BF16 ? launch_attn<C, P, Bf16T>(a, c.head_dim, c.max_query, max_tiles, v, s)
                                               : launch_attn<C, P, Fp16T>(a, c.head_dim, c.max_query, max_tiles, v, s);
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

}  // namespace rmsq
