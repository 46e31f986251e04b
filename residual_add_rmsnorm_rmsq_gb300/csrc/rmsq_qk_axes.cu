// QK-norm + RoPE with three positions per token (time, height, width):
// argument checks, the axis of each angle, launches.  The kernels are the
// one-axis op's (rmsq_qk.cuh), told where each angle's row is.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_qk.cuh"

namespace rmsq {

cudaError_t take_pipe_fault_qk_axes(unsigned int* out) { return take_pipe_fault(out); }

namespace {

// Axis of angle i of `half`: the sections one after the other, or alternating
// (every third angle height's and width's, up to their number).
int axis_of(int i, int t, int h, int w, bool interleaved) {
    if (interleaved) return i % 3 == 1 && i < 3 * h ? 1 : i % 3 == 2 && i < 3 * w ? 2 : 0;
    return i < t ? 0 : i < t + h ? 1 : 2;
}

// Sets the angles' axes; true if every aligned group of four has one axis.
bool set_axes(QkArgs* a, int half, int t, int h, int w, bool interleaved) {
    bool quads = true;
    for (int i = 0; i < half; ++i) {
        const int axis = axis_of(i, t, h, w, interleaved);
        if (axis == 1) a->axis_h[i >> 5] |= 1u << (i & 31);
        if (axis == 2) a->axis_w[i >> 5] |= 1u << (i & 31);
        quads = quads && axis == axis_of(i & ~3, t, h, w, interleaved);
    }
    return quads;
}

template <class E>
cudaError_t launch_axes(const QkArgs& a, int head_dim, bool neox, bool quads, int variant, cudaStream_t stream) {
    return quads ? launch_qk<E, kQuadAxes>(a, head_dim, neox, variant, stream)
                 : launch_qk<E, kAnyAxes>(a, head_dim, neox, variant, stream);
}

}  // namespace
}  // namespace rmsq

extern "C" int rmsq_qk_norm_mrope(void* qkv, void* out, const int64_t* positions, const float* cos_sin_cache,
                                  int64_t max_positions, const void* q_weight, const void* k_weight, float eps,
                                  int64_t n_tokens, int num_q_heads, int num_kv_heads, int head_dim, int section_t,
                                  int section_h, int section_w, int interleaved, int is_neox, int dtype, void* stream,
                                  int variant) {
    using rmsq_abi::aligned;
    using rmsq_abi::overlaps;
    using rmsq_abi::Span;
    using rmsq_abi::span;
    if (dtype != RMSQ_BF16 && dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    if (variant != RMSQ_VARIANT_AUTO && variant != RMSQ_VARIANT_DIRECT && variant != RMSQ_VARIANT_PIPELINED)
        return RMSQ_ERR_INVALID_ARG;
    if (n_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || max_positions <= 0 || (is_neox != 0 && is_neox != 1) ||
        (interleaved != 0 && interleaved != 1) || section_t < 0 || section_h < 0 || section_w < 0)
        return RMSQ_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f) return RMSQ_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return RMSQ_ERR_UNSUPPORTED_SHAPE;
    if (num_q_heads > 4096 || num_kv_heads > 4096) return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int heads = num_q_heads + num_kv_heads;
    if (heads == 0) return RMSQ_ERR_INVALID_ARG;
    if (n_tokens > INT32_MAX / heads || max_positions > INT64_MAX / (4 * head_dim)) return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int half = head_dim / 2;
    if (static_cast<int64_t>(section_t) + section_h + section_w != half) return RMSQ_ERR_INVALID_ARG;
    // the last of the height's (width's) alternating angles has to exist
    if (interleaved && ((section_h > 0 && 3 * section_h - 1 > half) || 3 * section_w > half)) return RMSQ_ERR_INVALID_ARG;
    if ((q_weight == nullptr) != (k_weight == nullptr)) return RMSQ_ERR_INVALID_ARG;
    if (n_tokens == 0) return RMSQ_OK;
    if (!qkv || !positions || !cos_sin_cache) return RMSQ_ERR_INVALID_ARG;
    if (!aligned(qkv, 16) || !aligned(out, 16) || !aligned(positions, 8) || !aligned(cos_sin_cache, 16) ||
        !aligned(q_weight, 16) || !aligned(k_weight, 16))
        return RMSQ_ERR_ALIGNMENT;
    const int64_t width = static_cast<int64_t>(heads + num_kv_heads) * head_dim;
    const Span in = span(qkv, static_cast<size_t>(n_tokens) * width * 2);
    const Span dst = out ? span(out, static_cast<size_t>(n_tokens) * heads * head_dim * 2) : in;
    const Span ins[4] = {span(positions, static_cast<size_t>(n_tokens) * 24),
                         span(cos_sin_cache, static_cast<size_t>(max_positions) * head_dim * 4),
                         span(q_weight, static_cast<size_t>(head_dim) * 2), span(k_weight, static_cast<size_t>(head_dim) * 2)};
    for (const Span& i : ins)
        if (overlaps(dst, i)) return RMSQ_ERR_ALIAS;
    if (out && overlaps(dst, in)) return RMSQ_ERR_ALIAS;
    const int st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    rmsq::QkArgs a = {};
    a.qkv = static_cast<uint32_t*>(qkv);
    a.pos = positions;
    a.cs = cos_sin_cache;
    a.max_pos = max_positions;
    a.qw = static_cast<const uint32_t*>(q_weight);
    a.kw = static_cast<const uint32_t*>(k_weight);
    a.eps = eps;
    a.inv_d = 1.0f / static_cast<float>(head_dim);
    a.n = static_cast<int>(n_tokens);
    a.nq = num_q_heads;
    a.nkv = num_kv_heads;
    a.out = static_cast<uint32_t*>(out ? out : qkv);
    a.out_words = out ? static_cast<int64_t>(heads) * half : width / 2;
    const bool quads = rmsq::set_axes(&a, half, section_t, section_h, section_w, interleaved == 1);
    const int v = variant == RMSQ_VARIANT_DIRECT ? rmsq::kVariantDirect
                  : variant == RMSQ_VARIANT_PIPELINED ? rmsq::kVariantPipelined : rmsq::kVariantAuto;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSQ_FP16 ? rmsq::launch_axes<rmsq::Fp16T>(a, head_dim, is_neox == 1, quads, v, s)
                                             : rmsq::launch_axes<rmsq::Bf16T>(a, head_dim, is_neox == 1, quads, v, s);
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}
