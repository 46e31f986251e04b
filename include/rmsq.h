/*
 * librmsq — fused residual-add + RMSNorm + activation quantisation on GB300 (sm_103a).
 *
 * The operation is the one vLLM's RMSNorm + quantisation fusion puts in place
 * of a separate (fused-add) RMSNorm kernel and a quantisation kernel:
 *   vLLM docs, "Fusion torch.compile passes", section
 *   "RMSNorm + Quantization (fuse_norm_quant)": rms_norm(x) -> quant_fp8(y) and
 *   fused_add_rms_norm(x, residual) -> quant_fp8(y), the residual updated in
 *   place; schemes FP8 static per-tensor, FP8 dynamic per-token and FP8
 *   dynamic per-token-group (128/64);
 *   blog "[vLLM] Compilation Fusion Passes", sections "Pattern matching
 *   structure" (result, input, weight, scale, epsilon), "Fused Add + RMSNorm +
 *   Group Quantization" (the fused-op table keyed by quant scheme and fused
 *   add), "Type validation" (input and weight share one dtype) and "Why this
 *   design" (column-major scales);
 *   vLLM PR #51925 summary (prhub), "Motivation" and "Key source snippets":
 *   residual update + RMSNorm followed by NVFP4 block scales and FP4 values,
 *   with an fp32 activation (global) scale given as an input.
 *
 * Per row t of an [n_tokens, hidden] activation (T = bf16 or fp16):
 *   h    = T(fp32(x) + fp32(residual))       (h = x when residual is NULL)
 *   residual_out = h
 *   S    = pairwise-tree sum of fp32(h)^2     (zero-pad to a power of two,
 *                                              add adjacent pairs level by level)
 *   inv  = 1 / sqrt(S / hidden + eps)         (IEEE division and square root)
 *   y    = (fp32(h) * inv) * fp32(weight)     (fp32, not rounded to T)
 *   then one of the quantisation modes below.  All fp32 arithmetic rounds to
 *   nearest even; results are bit-identical to that definition.
 *
 * Besides that op (rmsq_fused_add_rmsnorm_quant and its variants) the library
 * has: NVFP4 with the global scale taken from the data
 * (rmsq_fused_add_rmsnorm_nvfp4_dynamic); scale options E8M0 and TMA-aligned
 * column-major (RMSQ_QUANT_*); SiLU+Mul + quantisation (rmsq_silu_mul_quant,
 * the same docs page's "SiLU+Mul + Quantization (fuse_act_quant)"); and the
 * unfused two-op sequence the fusion replaces (rmsq_fused_add_rmsnorm,
 * rmsq_quant); and QK-norm + RoPE on the attention input
 * (rmsq_qk_norm_rope, the docs page's "QK Norm + RoPE
 * (enable_qk_norm_rope_fusion)").  Around that input it has the serving
 * operators of an attention block: slot maps from request lengths
 * (rmsq_build_slot_map), a paged key / value cache in NVFP4
 * (rmsq_kv_cache_store_nvfp4, rmsq_kv_cache_load_nvfp4) and causal attention
 * over it (rmsq_paged_attention_nvfp4); and the FP8 matrix product that
 * consumes the group-128 modes' outputs (rmsq_fp8_block_matmul).  For models of
 * images and video, and for caches in 8 bits, the same block has QK-norm + RoPE
 * with three positions per token (rmsq_qk_norm_mrope), a paged FP8 cache with a
 * power-of-two scale per 16 tokens and head (rmsq_kv_cache_store_fp8,
 * rmsq_kv_cache_load_fp8) and attention over it (rmsq_paged_attention_fp8).
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" must be addressable by the current CUDA device
 *     (cudaMalloc / torch CUDA tensors, or managed memory).  The caller owns
 *     every buffer; the library allocates no device memory and keeps no
 *     per-call state.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls are
 *     asynchronous with respect to the host and do not synchronise.
 *   - Argument errors are reported synchronously, before any launch, and leave
 *     every output untouched.  A failed launch returns RMSQ_ERR_CUDA; the CUDA
 *     error code is then available from rmsq_last_cuda_error().
 *   - Device code is built for sm_103a only; any other device gives
 *     RMSQ_ERR_UNSUPPORTED_DEVICE and there is no CPU fallback.
 */
#ifndef RMSQ_H
#define RMSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RMSQ_VERSION 10000        /* 1.0.0 */
#define RMSQ_MAX_HIDDEN 16384

typedef enum {
    RMSQ_OK = 0,
    RMSQ_ERR_INVALID_ARG = 1,        /* NULL where a pointer is required, bad enum, bad eps */
    RMSQ_ERR_ALIGNMENT = 2,          /* a pointer misses the alignment stated below */
    RMSQ_ERR_ALIAS = 3,              /* outputs overlap inputs other than as allowed */
    RMSQ_ERR_UNSUPPORTED_SHAPE = 4,  /* hidden not a multiple of 8 / the group / 16, or too large */
    RMSQ_ERR_UNSUPPORTED_DEVICE = 5, /* current device is not compute capability 10.3 */
    RMSQ_ERR_NO_DEVICE = 6,          /* no CUDA device / driver */
    RMSQ_ERR_CUDA = 7                /* a CUDA runtime call or launch failed */
} rmsq_status;

typedef enum { RMSQ_BF16 = 0, RMSQ_FP16 = 1 } rmsq_dtype;

/*
 * Quantisation modes (blog "[vLLM] Compilation Fusion Passes", section
 * "Fused Add + RMSNorm + Group Quantization": static per-tensor, dynamic
 * per-token and dynamic 128-group symmetric FP8; vLLM docs "Fusion
 * torch.compile passes", fuse_norm_quant: group 128 or 64; PR #51925: NVFP4).
 * E4M3 is OCP FP8 E4M3FN: round to nearest even, magnitudes above 448
 * (including infinities) saturate to 448, sign kept (-0 -> 0x80).
 *
 *  RMSQ_FP8_STATIC        s = scale_in[0];                q = e4m3(y / s)
 *  RMSQ_FP8_PER_TOKEN     s_t = max(amax_t(|y|) / 448, 1e-12), fp32 [n_tokens]
 *  RMSQ_FP8_GROUP{128,64}_ROW  s_{t,g} over G contiguous elements, fp32 [n_tokens, hidden/G]
 *  RMSQ_FP8_GROUP{128,64}_COL  same values stored [hidden/G, n_tokens] (column-major)
 *                         q = e4m3(y / s), one byte per element, [n_tokens, hidden]
 *  RMSQ_NVFP4             per 16-element block b: sb = e4m3((amax_b / 6) * gs),
 *                         gs = scale_in[0]; d = decode(sb); r = d ? gs / d : 0;
 *                         q = e2m1(y * r) (values {0,.5,1,1.5,2,3,4,6}, round to
 *                         nearest even, saturate at 6, sign kept); element 2j in
 *                         the low nibble of byte j: q is u8 [n_tokens, hidden/2],
 *                         block scales u8 (E4M3) [n_tokens, hidden/16], row-major.
 * The divisions y / s are correctly rounded fp32 divisions.
 */
typedef enum {
    RMSQ_FP8_STATIC = 0,
    RMSQ_FP8_PER_TOKEN = 1,
    RMSQ_FP8_GROUP128_ROW = 2,
    RMSQ_FP8_GROUP128_COL = 3,
    RMSQ_FP8_GROUP64_ROW = 4,
    RMSQ_FP8_GROUP64_COL = 5,
    RMSQ_NVFP4 = 6
} rmsq_quant_mode;

/*
 * Scale options, OR-ed into a quant_mode argument (blog "[vLLM] Compilation
 * Fusion Passes", section "Why this design", item 3: E8M0 scales,
 * column-major scales and TMA alignment registered as combinable options).
 *  RMSQ_QUANT_E8M0         the dynamic scale (per-token and group modes only)
 *                          is rounded up to a power of two,
 *                          s = 2^ceil(log2 max(amax / 448, 1e-12)); it is
 *                          still stored as fp32 (its E8M0 byte is the
 *                          exponent field, bits 30..23), q = e4m3(y / s).
 *  RMSQ_QUANT_UE8M0        the same power-of-two scale, stored as one byte
 *                          (per-token and group modes only): the UE8M0
 *                          encoding, byte e standing for 2^(e - 127) (the
 *                          biased exponent of the fp32 scale).  out_scales is
 *                          then u8 with the layouts below (1-byte aligned);
 *                          implies RMSQ_QUANT_E8M0, codes are the same.
 *  RMSQ_QUANT_TMA_ALIGNED  column-major group scales (_COL modes only) use a
 *                          stride of n_tokens rounded up to 16 bytes of scales
 *                          between groups: [hidden/G, round4(n)] fp32 scales,
 *                          or [hidden/G, round16(n)] UE8M0 bytes; the padding
 *                          entries are not written.
 * Any other bit, or an option with a mode it does not apply to, is
 * RMSQ_ERR_INVALID_ARG.
 */
#define RMSQ_QUANT_MODE_MASK 0x0f
#define RMSQ_QUANT_E8M0 0x10
#define RMSQ_QUANT_TMA_ALIGNED 0x20
#define RMSQ_QUANT_UE8M0 0x40

/*
 * rmsq_fused_add_rmsnorm_quant — one launch of the fused op over n_tokens rows.
 *
 *  x            device, T[n_tokens, hidden], row-major, 16-byte aligned.
 *  residual     device, T[n_tokens, hidden], 16-byte aligned, or NULL (plain
 *               RMSNorm + quant: h = x, nothing is written to residual_out).
 *  weight       device, T[hidden], 16-byte aligned (same dtype as x).
 *  eps          finite, >= 0 (1e-5 and 1e-6 are the values the pages use).
 *  quant_mode   an rmsq_quant_mode, optionally OR-ed with RMSQ_QUANT_* options.
 *  scale_in     device, one fp32: the static scale s (FP8_STATIC) or the global
 *               scale gs (NVFP4); ignored (may be NULL) for the dynamic FP8
 *               modes.  Its value must be finite and > 0; it is not checked.
 *  out_q        device, u8[n_tokens, hidden] (FP8) or u8[n_tokens, hidden/2]
 *               (NVFP4), 16-byte aligned.
 *  out_scales   device; fp32 per-token / per-group scales (4-byte aligned),
 *               their UE8M0 bytes (RMSQ_QUANT_UE8M0), or u8 NVFP4 block
 *               scales; ignored (may be NULL) for FP8_STATIC.
 *               rmsq_query_sizes gives the byte sizes.
 *  residual_out device, T[n_tokens, hidden], 16-byte aligned; NULL exactly when
 *               residual is NULL.  It may be the same pointer as residual (the
 *               in-place update of fused_add_rms_norm) or as x.
 *  n_tokens     >= 0 and < 2^31; 0 returns RMSQ_OK without a launch.
 *  hidden       > 0, a multiple of 8 (16 for NVFP4, G for the group modes),
 *               <= RMSQ_MAX_HIDDEN.
 *  dtype        an rmsq_dtype: the type of x, residual, weight, residual_out.
 *  stream       cudaStream_t to launch on.
 * Aliasing: besides residual_out == residual or residual_out == x, no output
 * may overlap any input or another output, and x / residual / residual_out
 * must be identical or disjoint.
 * Returns an rmsq_status.
 */
int rmsq_fused_add_rmsnorm_quant(const void *x, const void *residual, const void *weight,
                                 float eps, int quant_mode, const float *scale_in,
                                 void *out_q, void *out_scales, void *residual_out,
                                 int64_t n_tokens, int64_t hidden, int dtype, void *stream);

/*
 * Kernel variants.  Both compute bit-identical results; AUTO picks by batch
 * size.  DIRECT: one CTA per row, loads straight into registers (lowest
 * latency for a few rows).  PIPELINED: persistent CTAs with several rows per
 * CTA in flight as bulk asynchronous copies into shared memory (highest
 * bandwidth for large batches).
 */
typedef enum { RMSQ_VARIANT_AUTO = 0, RMSQ_VARIANT_DIRECT = 1, RMSQ_VARIANT_PIPELINED = 2 } rmsq_variant;

/*
 * rmsq_fused_add_rmsnorm_quant_ex — rmsq_fused_add_rmsnorm_quant with an
 * explicit rmsq_variant (RMSQ_ERR_INVALID_ARG for any other value).  Same
 * arguments, rules and results otherwise.
 */
int rmsq_fused_add_rmsnorm_quant_ex(const void *x, const void *residual, const void *weight,
                                    float eps, int quant_mode, const float *scale_in,
                                    void *out_q, void *out_scales, void *residual_out,
                                    int64_t n_tokens, int64_t hidden, int dtype, void *stream,
                                    int variant);

/*
 * rmsq_fused_add_rmsnorm_nvfp4_dynamic — the NVFP4 mode with the global scale
 * taken from the data instead of scale_in: gs = 448 * 6 / amax(|y|) over the
 * whole batch (the NVFP4 workload's definition of the global scale; gs = 1
 * when that amax is 0), then exactly the RMSQ_NVFP4 quantisation with that gs
 * (vLLM PR #51925 summary, "Motivation": residual update + RMSNorm, block
 * scales, FP4 values, fp32 global scale).  Two kernels: the first computes
 * the residual, and the per-row inv_rms and per-CTA maxima of |y| into
 * `workspace`; the second takes the batch amax from those maxima, re-reads h
 * (residual_out, or x without a residual) and quantises.
 *  out_global_scale  device, one fp32 (4-byte aligned): receives gs.
 *  workspace         device, 16-byte aligned, at least
 *                    rmsq_nvfp4_dynamic_workspace_bytes(n_tokens) bytes of
 *                    caller-owned scratch; its contents on entry do not
 *                    matter and are overwritten.  Two calls in flight at the
 *                    same time must not share one workspace.
 *  variant           an rmsq_variant for the first pass.
 * Every other argument as in rmsq_fused_add_rmsnorm_quant with quant_mode
 * RMSQ_NVFP4 (out_block_scales = its out_scales).  RMSQ_ERR_INVALID_ARG also
 * for a NULL or too small workspace; no output may overlap the workspace.
 */
int rmsq_fused_add_rmsnorm_nvfp4_dynamic(const void *x, const void *residual, const void *weight,
                                         float eps, void *out_q, void *out_block_scales,
                                         float *out_global_scale, void *residual_out,
                                         void *workspace, size_t workspace_bytes,
                                         int64_t n_tokens, int64_t hidden, int dtype, void *stream,
                                         int variant);

/* Bytes of workspace rmsq_fused_add_rmsnorm_nvfp4_dynamic needs for n_tokens
 * rows: 256 + 8 * n_tokens (one fp32 inverse RMS per row and at most one
 * fp32 partial maximum per row), rounded up to a multiple of 256 (0 for
 * n < 0). */
size_t rmsq_nvfp4_dynamic_workspace_bytes(int64_t n_tokens);

/* Largest batch rmsq_fused_add_rmsnorm_nvfp4_dynamic_noalloc accepts. */
#define RMSQ_NOALLOC_MAX_TOKENS 65536

/*
 * rmsq_fused_add_rmsnorm_nvfp4_dynamic_noalloc — rmsq_fused_add_rmsnorm_nvfp4_dynamic
 * without a caller workspace and without any device allocation.  The pages
 * have no counterpart to this entry point: it exists for callers that cannot
 * allocate device memory themselves — for instance a plugin inside an engine
 * that owns all device memory through its own pool and hands the plugin none,
 * or latency-critical code that must not call cudaMalloc because it can
 * synchronise the device.  The caller still passes every input and output.
 *
 * The workspace lives in a fixed device array inside the library (256 + 8 *
 * RMSQ_NOALLOC_MAX_TOKENS bytes, about 513 KiB), present on every device that
 * loads the library until the process exits.  n_tokens above
 * RMSQ_NOALLOC_MAX_TOKENS returns RMSQ_ERR_UNSUPPORTED_SHAPE (use the entry
 * point with a workspace for larger batches).  Every call looks up the
 * array's device address in the current device's context
 * (cudaGetSymbolAddress), so a reset of the device's primary context between
 * calls is followed; the first call on a device may load the library's device
 * code there: make that first call before any stream capture.  Every call on a
 * device shares the one array and leaves its contents behind; nothing in it
 * has to start at zero (every call writes what it reads).  Calls whose work overlaps on
 * the GPU (other streams, or other host threads) race on the array: order them.
 * Arguments, results and every other rule are those of
 * rmsq_fused_add_rmsnorm_nvfp4_dynamic; without a CUDA device it returns
 * RMSQ_ERR_NO_DEVICE.
 */
int rmsq_fused_add_rmsnorm_nvfp4_dynamic_noalloc(const void *x, const void *residual,
                                                 const void *weight, float eps, void *out_q,
                                                 void *out_block_scales, float *out_global_scale,
                                                 void *residual_out, int64_t n_tokens,
                                                 int64_t hidden, int dtype, void *stream,
                                                 int variant);

/*
 * The unfused two-op sequence the fused op replaces (vLLM docs "Fusion
 * torch.compile passes", fuse_norm_quant: fused_add_rms_norm / rms_norm
 * followed by the quantisation op), for comparison and for callers that need
 * the normalised activations themselves.
 *
 * rmsq_fused_add_rmsnorm — steps 1-4 of rmsq_fused_add_rmsnorm_quant (residual
 * add and write-back, RMSNorm with the same canonical sum), then y rounded to
 * the activation type (nearest even) into y_out: device [n_tokens, hidden],
 * same type as x, 16-byte aligned, overlapping no input or residual_out.
 * Arguments and errors otherwise as rmsq_fused_add_rmsnorm_quant.
 *
 * rmsq_quant — the quantisation step of rmsq_fused_add_rmsnorm_quant applied
 * to a [n_tokens, hidden] tensor y of the activation type (widened exactly to
 * fp32): every quant_mode and scale option, same outputs and layouts.
 * Running the two in sequence gives the unfused result, which differs from
 * the fused op's in that y is rounded to the activation type in between.
 */
int rmsq_fused_add_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                           void *y_out, void *residual_out, int64_t n_tokens, int64_t hidden, int dtype,
                           void *stream);
int rmsq_quant(const void *y, int quant_mode, const float *scale_in, void *out_q, void *out_scales,
               int64_t n_tokens, int64_t hidden, int dtype, void *stream);

/*
 * rmsq_qk_norm_rope — QK-norm + RoPE in one kernel (vLLM docs "Fusion
 * torch.compile passes", section "QK Norm + RoPE (enable_qk_norm_rope_fusion)":
 * split QKV, per-head RMSNorm of Q and K, rotary embedding), in place.
 *  qkv            device, T[n_tokens, (num_q_heads + 2 num_kv_heads) head_dim]:
 *                 per token the q heads, then the k heads, then the v heads;
 *                 16-byte aligned; updated in place (v heads untouched).
 *  positions      device, int64[n_tokens], 8-byte aligned: each token's position.
 *  cos_sin_cache  device, fp32[max_positions, head_dim], 16-byte aligned: at
 *                 row p, cos of the head_dim/2 angles then their sin.
 *  q_weight, k_weight  device, T[head_dim], 16-byte aligned: the norm weights.
 * Per q / k head: S = canonical pairwise sum of x^2 over the head,
 * inv = 1 / sqrt(S / head_dim + eps), y = (x * inv) * w in fp32 (the norm op's
 * steps); then with c_i, s_i from row positions[t] of the table, each pair
 * (a, b) becomes (a c - b s, b c + a s) (every product and sum rounded to
 * fp32 separately), rounded once to T.  is_neox = 1 pairs element i with
 * i + head_dim/2, 0 pairs 2i with 2i + 1 (GPT-J); angle index i either way.
 * A token whose position is outside [0, max_positions) is left unchanged.
 * head_dim 64, 128 or 256 (else RMSQ_ERR_UNSUPPORTED_SHAPE); eps finite,
 * >= 0; no input may overlap qkv.  Asynchronous on `stream`.
 */
int rmsq_qk_norm_rope(void *qkv, const int64_t *positions, const float *cos_sin_cache,
                      int64_t max_positions, const void *q_weight, const void *k_weight, float eps,
                      int64_t n_tokens, int num_q_heads, int num_kv_heads, int head_dim, int is_neox,
                      int dtype, void *stream);

/*
 * rmsq_qk_norm_rope_ex — rmsq_qk_norm_rope with an explicit rmsq_variant
 * (RMSQ_ERR_INVALID_ARG for any other value); bit-identical results either
 * way.  DIRECT: each warp loads its heads straight into registers (lowest
 * latency for a few tokens).  PIPELINED: persistent CTAs keep the q and k
 * heads and the cos / sin rows of several tokens in flight as bulk
 * asynchronous copies into shared memory; it needs two tokens' q and k heads
 * plus their cos / sin rows within the shared-memory ring (about 110 KB per
 * CTA) and runs as DIRECT where they do not fit.  AUTO: PIPELINED from eight
 * tokens per SM up.
 */
int rmsq_qk_norm_rope_ex(void *qkv, const int64_t *positions, const float *cos_sin_cache,
                         int64_t max_positions, const void *q_weight, const void *k_weight, float eps,
                         int64_t n_tokens, int num_q_heads, int num_kv_heads, int head_dim, int is_neox,
                         int dtype, void *stream, int variant);

/*
 * rmsq_qk_norm_mrope — rmsq_qk_norm_rope_ex with three positions per token
 * (time, height, width: images and video in the text), the norm optional and
 * the result in place or in a buffer of its own.
 *  qkv            as there; read only if out is given.
 *  out            device, T[n_tokens, (num_q_heads + num_kv_heads) head_dim],
 *                 16-byte aligned: the q heads, then the k heads; overlapping no
 *                 input.  NULL: in place on qkv.
 *  positions      device, int64[3, n_tokens], 8-byte aligned: the times, the
 *                 heights, the widths.  A token with one of its three outside
 *                 [0, max_positions) is left unchanged (its row of out is not
 *                 written).
 *  cos_sin_cache  as there.  Angle i takes its cos and sin from the row of its
 *                 axis's position.
 *  q_weight, k_weight  as there, or both NULL: no norm, the heads are rotated
 *                 only (eps is then not used, but checked).
 *  section_t, section_h, section_w  number of angles of each axis, together
 *                 head_dim / 2.
 *  interleaved    0: the first section_t angles are the time's, the next
 *                 section_h the height's, the others the width's.  1: angles 1,
 *                 4, 7, .. (section_h of them) are the height's, 2, 5, 8, ..
 *                 (section_w) the width's, all others the time's; they have to
 *                 exist, 3 section_h - 1 and 3 section_w at most head_dim / 2.
 * The arithmetic is that of rmsq_qk_norm_rope: three equal positions give its
 * bits.  Both variants give the same bits.  Sections that do not add up, or do
 * not fit, are RMSQ_ERR_INVALID_ARG.
 */
int rmsq_qk_norm_mrope(void *qkv, void *out, const int64_t *positions, const float *cos_sin_cache,
                       int64_t max_positions, const void *q_weight, const void *k_weight, float eps,
                       int64_t n_tokens, int num_q_heads, int num_kv_heads, int head_dim, int section_t,
                       int section_h, int section_w, int interleaved, int is_neox, int dtype, void *stream,
                       int variant);

/* Most requests of rmsq_build_slot_map and of the attention over a paged cache. */
#define RMSQ_MAX_REQUESTS 8192

/* Bits of rmsq_build_slot_map's status. */
#define RMSQ_SLOT_NO_PAGES 1         /* the free list is shorter than the pages needed */
#define RMSQ_SLOT_TABLE_FULL 2       /* a request needs more than table_width pages */
#define RMSQ_SLOT_TOO_MANY_TOKENS 4  /* the query lengths add up to more than max_tokens */
#define RMSQ_SLOT_BAD_LENGTH 8       /* a negative length, or num_free outside [0, free_capacity] */

/*
 * rmsq_build_slot_map — block tables and slot map of one step, from the
 * requests' lengths, on the device (no length has to be known to the host, so
 * a captured graph can be replayed for every step).  Request r has
 * context_lens[r] tokens in the cache and brings query_lens[r] new ones.
 * Pages are taken from the end of the free list, in request order, and
 * appended to the request's row of the block table; token i of request r gets
 *   position = context_lens[r] + i,
 *   slot     = block_table[r, position / page_size] * page_size + position % page_size
 * (slot -1 where the table holds a negative page).
 *  context_lens, query_lens  device, int32[num_requests].
 *  block_table   device, int32[num_requests, table_width], updated in place:
 *                only the entries of the new pages are written.
 *  free_pages    device, int32[free_capacity]; the first num_free[0] are free.
 *  num_free      device, int32[1].
 *  page_size     16, 32, 64, 128 or 256 tokens.
 *  slot_map, positions  device, int64[max_tokens]: tokens in request order;
 *                entries behind the last token are -1 (the store skips such a
 *                slot, rmsq_qk_norm_rope such a position).
 *  query_start   device, int32[num_requests + 1]: first token of each request,
 *                and their number.
 *  seq_lens      device, int32[num_requests]: context + query length.
 *  num_free_out  device, int32[1]: pages still free (the next call's num_free).
 *  status        device, int32[1]: 0, or RMSQ_SLOT_* bits.  Then nothing was
 *                assigned: every slot and position is -1, query_start 0,
 *                seq_lens the context lengths, num_free_out num_free, the
 *                table unchanged.
 * int32 buffers 4-byte, int64 buffers 8-byte aligned.  num_requests at most
 * RMSQ_MAX_REQUESTS, max_tokens below 2^30; 0 requests are allowed.  No output
 * may overlap an input or another output.  Asynchronous on `stream`.
 */
int rmsq_build_slot_map(const int32_t *context_lens, const int32_t *query_lens, int32_t *block_table,
                        int64_t table_width, const int32_t *free_pages, int64_t free_capacity,
                        const int32_t *num_free, int64_t page_size, int64_t num_requests, int64_t max_tokens,
                        int64_t *slot_map, int64_t *positions, int32_t *query_start, int32_t *seq_lens,
                        int32_t *num_free_out, int32_t *status, void *stream);

/*
 * The paged NVFP4 cache: device, u8 [num_pages, 2, num_kv_heads, tile],
 * 16-byte aligned, with keys at index 0 and values at index 1 of the second
 * axis and tiles of page_size * head_dim * 9 / 16 bytes: first the codes
 * [page_size, head_dim / 2] (E2M1, element 2j in the low nibble of byte j),
 * then the E4M3 scales of the 16-element blocks [page_size, head_dim / 16].
 * Slot s is token s % page_size of page s / page_size.  An element stands for
 * code * scale / global scale; the scale's NaN codes, which the store never
 * writes, read as 448.
 *
 * rmsq_kv_cache_store_nvfp4 — quantises the key and value heads of n_tokens
 * tokens into the cache, bit for bit as RMSQ_NVFP4 does (rmsq_quant).
 * rmsq_kv_cache_load_nvfp4 — reads tokens back: T((code * scale) / global
 * scale), one fp32 division, rounded once to T.
 *  k, v          device, T[n_tokens, num_kv_heads, head_dim], heads contiguous,
 *                tokens k_stride / v_stride elements apart (so k and v may be
 *                column ranges of a qkv buffer); 16-byte aligned, strides
 *                multiples of 8, at least num_kv_heads * head_dim.
 *  slot_map      device, int64[n_tokens].  A token whose slot lies outside
 *                [0, num_pages * page_size) is skipped by the store and read
 *                as zeros by the load.  The store's slots must differ: of two
 *                tokens with one slot either may be kept, block by block.
 *  k_global_scale, v_global_scale  device, one fp32 each, finite and > 0
 *                (not checked): 448 * 6 / the largest magnitude expected.
 *  head_dim      64, 128 or 256; page_size 16, 32, 64, 128 or 256.
 *  n_tokens      >= 0 (0 returns RMSQ_OK without a launch).
 * No output may overlap an input; the load's k and v rows may interleave in
 * one buffer.  Asynchronous on `stream`.
 */
int rmsq_kv_cache_store_nvfp4(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                              const int64_t *slot_map, const float *k_global_scale, const float *v_global_scale,
                              void *kv_cache, int64_t num_pages, int64_t page_size, int64_t n_tokens,
                              int num_kv_heads, int head_dim, int dtype, void *stream);
int rmsq_kv_cache_load_nvfp4(const void *kv_cache, int64_t num_pages, int64_t page_size, const int64_t *slot_map,
                             const float *k_global_scale, const float *v_global_scale, void *k, int64_t k_stride,
                             void *v, int64_t v_stride, int64_t n_tokens, int num_kv_heads, int head_dim, int dtype,
                             void *stream);

/*
 * rmsq_paged_attention_nvfp4 — causal attention of ragged queries over the
 * paged NVFP4 cache, grouped query heads (num_heads a multiple of
 * num_kv_heads: query head h reads kv head h / (num_heads / num_kv_heads)).
 * Request r has the query tokens query_start[r] .. query_start[r+1] - 1, the
 * last of them at position seq_lens[r] - 1; their keys must be in the cache
 * already.  Query token i of request r, at position p = seq_lens[r] -
 * query_len + i, attends keys 0 .. p, with window > 0 only the last `window`
 * of them (p included):
 *   out = sum_j softmax_j(softmax_scale * q.k_j) v_j,
 *   lse = ln sum_j exp(softmax_scale * q.k_j).
 * A query that sees no key (an empty request, p < 0) gets zeros and -inf.
 * A key on a page outside [0, num_pages) is left out.  A NaN among a query
 * head's elements gives NaN in its out and lse, and nowhere else.
 *  q             device, T[n_tokens, num_heads, head_dim], tokens q_stride
 *                elements apart (a multiple of 8), 16-byte aligned.
 *  kv_cache, num_pages, page_size, head_dim, global scales: as above.
 *  block_table   device, int32[num_requests, table_width]; page of key j of
 *                request r: block_table[r, j / page_size].
 *  query_start   device, int32[num_requests + 1], ascending from 0;
 *  seq_lens      device, int32[num_requests].  Values outside the buffers
 *                (rows beyond n_tokens, lengths beyond the table) are clamped.
 *  softmax_scale finite, > 0.   window >= 0, 0 for none.
 *  out           device, T[n_tokens, num_heads, head_dim], 16-byte aligned;
 *                rows behind query_start[num_requests] are left as they were.
 *  lse           device, fp32[n_tokens, num_heads], or NULL.
 *  workspace     device, 16-byte aligned, at least
 *                rmsq_paged_attention_workspace_bytes(...) bytes of scratch;
 *                contents on entry do not matter.  Two calls in flight at the
 *                same time must not share one.
 *  variant       an rmsq_variant.  DIRECT: the kernel for few queries, which
 *                divides the keys of each request over the device.  PIPELINED:
 *                a tensor-core kernel for requests of more than 64 (query, head
 *                of the group) pairs, DIRECT for the others (and for head_dim
 *                256).  AUTO: whichever is expected sooner, for each request
 *                by its own length and those beside it.  The two agree within
 *                the rounding of their sums.
 * Sums, maxima and the log-sum-exp are fp32, and logits may have any magnitude
 * that fp32 has; probabilities are rounded to f16 before they meet the values
 * (fp16 outputs are off by 2.9e-4 instead of 2.1e-4 on long contexts; bf16
 * outputs hide it).  Results are deterministic.  n_tokens * num_heads below 2^31;
 * 0 tokens or requests return RMSQ_OK without a launch.  No output may overlap an
 * input.  Asynchronous on `stream`; a launch that gives up waiting shows in
 * rmsq_take_fault_flags.
 */
int rmsq_paged_attention_nvfp4(const void *q, int64_t q_stride, const void *kv_cache, int64_t num_pages,
                               int64_t page_size, const int32_t *block_table, int64_t table_width,
                               const int32_t *query_start, const int32_t *seq_lens, const float *k_global_scale,
                               const float *v_global_scale, float softmax_scale, int64_t window, void *out,
                               float *lse, void *workspace, size_t workspace_bytes, int64_t n_tokens,
                               int64_t num_requests, int num_heads, int num_kv_heads, int head_dim, int dtype,
                               void *stream, int variant);

/* rmsq_paged_attention_nvfp4 told the most queries any request has: max_query
 * (0: not known).  It is for AUTO's choice alone, which cannot see the lengths:
 * with it no step without a prompt pays for the kernel of prompts.  A request
 * that is longer all the same gets its result too. */
int rmsq_paged_attention_nvfp4_ex(const void *q, int64_t q_stride, const void *kv_cache, int64_t num_pages,
                                  int64_t page_size, const int32_t *block_table, int64_t table_width,
                                  const int32_t *query_start, const int32_t *seq_lens, const float *k_global_scale,
                                  const float *v_global_scale, float softmax_scale, int64_t window, void *out,
                                  float *lse, void *workspace, size_t workspace_bytes, int64_t n_tokens,
                                  int64_t num_requests, int num_heads, int num_kv_heads, int head_dim, int dtype,
                                  void *stream, int variant, int64_t max_query);

/*
 * The paged FP8 cache: codes, device, u8 (E4M3) [num_pages, 2, num_kv_heads,
 * page_size, head_dim], 16-byte aligned, keys at index 0 and values at index 1
 * of the second axis; and scales, device, u8 [num_pages, 2, num_kv_heads,
 * page_size / 16], one for each block of 16 tokens and head: byte b stands for
 * 2^(b - 127) (bytes are read as if they were at least 1 and at most 187, 2^60).
 * Slot s is token s % page_size of page s / page_size; an element stands for
 * code * scale.
 *
 * rmsq_kv_cache_store_fp8 — quantises the key and value heads of n_tokens tokens
 * into the cache.  For each block of 16 slots and head that receives tokens, with
 * amax their largest finite magnitude,
 *   s = 2^ceil(log2 max(amax / 448, 1e-12))       (at most 2^60)
 * as RMSQ_QUANT_E8M0 has it.  Codes are e4m3(x / s).  A block whose first slot is
 * among those received is begun anew: what its other slots held is lost (their codes
 * stay and are read with the new scale).  Else it is one that is partly filled, s is
 * at least the scale it has, and its other slots keep their values: if the scale has
 * grown their codes are rounded to it (exact unless they become subnormal).
 * Magnitudes above 448 * 2^60 saturate.  An element that is not
 * finite is stored as NaN, and so are then all key codes of that token and head,
 * so that every query that attends to the token gives NaN, and no other.
 * rmsq_kv_cache_load_fp8 — reads tokens back: T(code * scale), rounded once.
 *  k, v, their strides, head_dim, page_size, n_tokens: as for the NVFP4 cache.
 *  slot_map      device, int64[n_tokens].  A token whose slot lies outside
 *                [0, num_pages * page_size) is skipped by the store and read as
 *                zeros by the load.  Of the store's, those of one block of 16
 *                have to ascend (each slot once) within 16 consecutive entries,
 *                with none but skipped ones between them: as rmsq_build_slot_map
 *                writes them, whichever of them are then taken out.  What a
 *                block holds after a call where they do not is not specified
 *                (other blocks are not concerned).  The load takes any slots.
 * Deterministic with such a map.  No output may overlap an input; the load's k and v rows may
 * interleave in one buffer.  Asynchronous on `stream`.
 */
int rmsq_kv_cache_store_fp8(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const int64_t *slot_map, void *cache, uint8_t *scales, int64_t num_pages,
                            int64_t page_size, int64_t n_tokens, int num_kv_heads, int head_dim, int dtype,
                            void *stream);
int rmsq_kv_cache_load_fp8(const void *cache, const uint8_t *scales, int64_t num_pages, int64_t page_size,
                           const int64_t *slot_map, void *k, int64_t k_stride, void *v, int64_t v_stride,
                           int64_t n_tokens, int num_kv_heads, int head_dim, int dtype, void *stream);

/*
 * rmsq_paged_attention_fp8 — the same attention over the paged FP8 cache (codes
 * and scales as above), with rmsq_paged_attention_nvfp4_ex's arguments, rules,
 * variants, workspace and errors otherwise.  The products with the codes are
 * exact and summed in fp32; a block's key scale multiplies its 16 logits in fp32,
 * its value scale its 16 weights, relative to the largest weight times value scale
 * among the keys that the query sees, before those are rounded to f16.  With w the
 * weights (sum 1), S_j the value scale of key j's block and U = max w_j S_j over the
 * n keys seen, that rounding puts an output off by at most 2^-11 sum w_j |v_j| +
 * n 2^-30 448 U (n 2^-24 448 U for prompts in the pipelined variant, where blocks of
 * one tile of 128 keys whose value scales are up to 2^7 apart share the largest),
 * whatever the scales of keys that it does not see.  fp16 outputs of ordinary
 * values are off by 2.5e-4 of their magnitude where 32-bit weights give 2.1e-4,
 * bf16 ones by 1.7e-3 either way.
 * A NaN among a key's elements gives NaN in the out and lse of the queries that
 * attend to it, and of no others (the store marks a token whose value has one in
 * this way); NaN codes of values read as 448.  What unwritten slots and scales
 * behind a request's last token hold does not matter.
 *  cache         16-byte aligned;  scales  no alignment.
 */
int rmsq_paged_attention_fp8(const void *q, int64_t q_stride, const void *cache, const uint8_t *scales,
                             int64_t num_pages, int64_t page_size, const int32_t *block_table, int64_t table_width,
                             const int32_t *query_start, const int32_t *seq_lens, float softmax_scale,
                             int64_t window, void *out, float *lse, void *workspace, size_t workspace_bytes,
                             int64_t n_tokens, int64_t num_requests, int num_heads, int num_kv_heads, int head_dim,
                             int dtype, void *stream, int variant, int64_t max_query);

/* Bytes of workspace rmsq_paged_attention_nvfp4 and _fp8 need (0 for arguments it
 * refuses; else the same for every number of tokens and requests, 10 to 21
 * MB: one workspace serves the calls of a program that follow one another). */
size_t rmsq_paged_attention_workspace_bytes(int64_t n_tokens, int64_t num_requests, int num_heads,
                                            int num_kv_heads, int head_dim);

/* Most ranks rmsq_allreduce_add_rmsnorm_quant sums. */
#define RMSQ_MAX_ALLREDUCE_RANKS 8

/*
 * rmsq_allreduce_add_rmsnorm_quant — the tensor-parallel all-reduce fused with
 * the residual add, RMSNorm and quantisation (vLLM docs "Fusion torch.compile
 * passes", section "AllReduce + RMSNorm (fuse_allreduce_rms)": all-reduce ->
 * RMSNorm (+ residual add) (-> FP8 static or NVFP4 quantisation), worth it at
 * small token counts).  One-shot, by loads: for every row the kernel reads
 * the row of each rank's partial sums, adds them in rank order in fp32 and
 * rounds the sum once to T:
 *   x = T(fp32(partials[0]) + fp32(partials[1]) + ... + fp32(partials[n_ranks-1]))
 * and then computes exactly rmsq_fused_add_rmsnorm_quant on that x (every
 * quant_mode and option; the same outputs and layouts).
 *  partials     HOST array of n_ranks (1 .. RMSQ_MAX_ALLREDUCE_RANKS) device
 *               pointers, each T[n_tokens, hidden], 16-byte aligned, that
 *               the current device can read: its own memory, or another
 *               GPU's memory mapped into this device's address space (CUDA
 *               IPC or peer access, set up by the caller; the library maps
 *               nothing).  The pointer values are copied at the call.
 *  Every other argument as in rmsq_fused_add_rmsnorm_quant (residual may be
 *  NULL; residual_out == residual is the in-place update).
 * Ordering: the kernel does not wait for other GPUs.  Every rank's partials
 * must be complete before the launch in `stream`'s order (for instance a
 * stream wait on an event each producer recorded, or a host barrier after
 * the producers synchronised); with peer buffers the caller also keeps them
 * alive and unmodified until the call completes.  Each rank that needs the
 * result calls this on its own device with the same partials (a one-shot
 * all-reduce), or on its own slice of rows (pointers and n_tokens of that
 * slice) followed by an all-gather of the outputs (a two-shot one).
 * No output may overlap a partial; RMSQ_ERR_INVALID_ARG for a NULL array or
 * pointer or a bad n_ranks.  Asynchronous on `stream`.
 */
int rmsq_allreduce_add_rmsnorm_quant(const void *const *partials, int n_ranks, const void *residual,
                                     const void *weight, float eps, int quant_mode,
                                     const float *scale_in, void *out_q, void *out_scales,
                                     void *residual_out, int64_t n_tokens, int64_t hidden,
                                     int dtype, void *stream);

/* Largest d (activation width) of rmsq_silu_mul_quant. */
#define RMSQ_ACT_MAX_D 32768

/*
 * rmsq_silu_mul_quant — SiLU+Mul + activation quantisation in one kernel (vLLM
 * docs "Fusion torch.compile passes", section "SiLU+Mul + Quantization
 * (fuse_act_quant)": silu_and_mul on the gated up-projection followed by the
 * quantisation, without the full-precision activation tensor in between).
 * Per row t: a_i = silu(g_i) * u_i in fp32, silu(g) = g / (1 + e^-g) with
 * g_i = gate_up[t, i] and u_i = gate_up[t, d + i]; then exactly the
 * quantisation step of rmsq_fused_add_rmsnorm_quant with a in place of y
 * (every quant_mode; scales and codes laid out the same way with hidden = d).
 * e^x follows W. J. Cody and W. Waite's argument reduction, then the
 * hardware's approximate 2^x on the reduced argument (within about 2.4 ulp
 * of e^x over the normal range); the quotient is g times the hardware's
 * approximate reciprocal of 1 + e^-g (within one ulp), so a is within
 * 9.8 * 2^-24 relative of the exact silu(g) * u (results are deterministic:
 * the same inputs always give the same bytes).  Where e^-g
 * overflows (g < -88.72) silu is -0.  The quantisation of a is exact, as in
 * the norm op.
 *  gate_up     device, [n_tokens, 2 d] bf16/fp16, row-major, 16-byte aligned.
 *  quant_mode  an rmsq_quant_mode, optionally OR-ed with RMSQ_QUANT_* options.
 *  scale_in    device fp32: FP8 static scale or NVFP4 global scale (else
 *              ignored, may be NULL).
 *  out_q       device: [n, d] E4M3 bytes, or [n, d/2] E2M1 pairs for NVFP4.
 *  out_scales  device: as for rmsq_fused_add_rmsnorm_quant with hidden = d.
 *  n_tokens    >= 0 (0 returns RMSQ_OK without a launch);
 *  d           > 0, a multiple of 8 (16 for NVFP4, the group for group
 *              modes), at most RMSQ_ACT_MAX_D (else
 *              RMSQ_ERR_UNSUPPORTED_SHAPE).
 * Errors as for rmsq_fused_add_rmsnorm_quant (no output may overlap an input
 * or another output).  Asynchronous on `stream`; the caller owns all memory.
 */
int rmsq_silu_mul_quant(const void *gate_up, int quant_mode, const float *scale_in, void *out_q,
                        void *out_scales, int64_t n_tokens, int64_t d, int dtype, void *stream);

/*
 * rmsq_fp8_block_matmul — the matrix product that consumes what the FP8
 * group-128 modes write: a linear layer with E4M3 activations (one scale per
 * row and 128 columns) and E4M3 weights (one scale per 128 x 128 block):
 *   out[i, j] = T( sum_kb sa[i, kb] * sb[j / 128, kb] * sum_{l in block kb} a[i, l] * b[j, l] )
 *  a_codes      device, u8 (E4M3) [m, k], 16-byte aligned.
 *  a_scales     device, as rmsq_fused_add_rmsnorm_quant / rmsq_silu_mul_quant
 *               write them for
 *  quant_mode   RMSQ_FP8_GROUP128_ROW or RMSQ_FP8_GROUP128_COL with their
 *               options (hidden = k, n_tokens = m); any other mode is
 *               RMSQ_ERR_INVALID_ARG.
 *  b_codes      device, u8 (E4M3) [n, k], 16-byte aligned.
 *  b_scales     device, fp32 [ceil(n / 128), k / 128], 4-byte aligned.
 *  out          device, T[m, n], 16-byte aligned, overlapping no input.
 *  m            >= 0 (0 returns RMSQ_OK without a launch);
 *  n            > 0, a multiple of 8;  k > 0, a multiple of 128, at most
 *               RMSQ_ACT_MAX_D (else RMSQ_ERR_UNSUPPORTED_SHAPE).
 * The 128 products of a block are summed by the tensor cores in fp32, the
 * blocks in fp32 registers, times sa * sb, which is formed first, in fp32; out
 * is rounded once.  Deterministic.  NaN codes give NaN in their row or column.
 * Asynchronous on `stream`; a launch that gives up waiting shows in
 * rmsq_take_fault_flags.
 */
int rmsq_fp8_block_matmul(const void *a_codes, const void *a_scales, int quant_mode, const void *b_codes,
                          const float *b_scales, void *out, int64_t m, int64_t n, int64_t k, int dtype,
                          void *stream);

/*
 * rmsq_set_pipeline_config — process-wide tuning of the PIPELINED variant:
 * chunks_per_thread (16-byte chunks of a row per thread: 1, 2, 4 or 8),
 * stages (rows in flight per CTA: 1..8) and ctas_per_sm (cap on resident
 * CTAs per SM: 1..32).  rows_per_iter (0, 1 or 2) is accepted and has no
 * effect: the norm kernels work on one row per CTA iteration.  0 keeps the
 * automatic choice for that parameter.  The pipelined QK-norm + RoPE kernel takes stages (tokens
 * in flight per CTA, 2..8) and ctas_per_sm from the same settings.  A choice
 * that does not fit (more than 512 threads, or a ring larger than the shared
 * memory budget) falls back to the automatic one.  Results do not depend on
 * these settings.  Not synchronised with launches running concurrently on
 * other host threads.
 */
int rmsq_set_pipeline_config(int chunks_per_thread, int stages, int ctas_per_sm, int rows_per_iter);

/*
 * rmsq_set_programmatic_launch — process-wide: 1 (the default) launches every
 * kernel with programmatic stream serialisation (programmatic dependent
 * launch), 0 with plain stream order.  With it, a kernel may be scheduled
 * while the previous kernel in the stream is still finishing, which hides the
 * launch gap between back-to-back calls (in a CUDA graph as well); each
 * kernel still waits for the previous one to complete, with its memory
 * visible, before its first global memory access, so stream semantics and
 * results are unchanged.  The pages have no counterpart: it is a launch
 * detail of this implementation.  Returns RMSQ_ERR_INVALID_ARG for a value
 * other than 0 or 1.  Not synchronised with launches on other host threads.
 */
int rmsq_set_programmatic_launch(int enable);

/*
 * rmsq_take_fault_flags — reads and clears, on the current device, the flag a
 * pipelined launch (norm, QK-norm + RoPE, all-reduce), a matrix product
 * (rmsq_fp8_block_matmul) or the attention's kernel of prompts sets if it ever
 * gives up waiting (after 100 ms) for its own shared-memory copies, its matrix
 * instructions or its other warps; the outputs of such a launch are incomplete,
 * although the call that launched it has returned RMSQ_OK.
 * *flags = 0 when no launch gave up.  Synchronous with respect to the device:
 * call it after the launches of interest have completed.
 */
int rmsq_take_fault_flags(uint32_t *flags);

/*
 * rmsq_query_sizes — bytes of out_q and out_scales for a mode and shape (host
 * only, no device needed).  scale_bytes is 0 for FP8_STATIC.
 */
int rmsq_query_sizes(int quant_mode, int64_t n_tokens, int64_t hidden, size_t *q_bytes,
                     size_t *scale_bytes);

/*
 * rmsq_query_launch — the launch rmsq_fused_add_rmsnorm_quant_ex would make on
 * the current device for a mode, shape, residual (0/1), dtype and variant,
 * without launching anything: out[0] = 1 for the pipelined kernel, 0 for the
 * direct one; out[1] = 16-byte chunks per thread; out[2] = ring stages (0
 * for the direct kernel); out[3] = CTAs; out[4] = threads per CTA (all 0 for
 * n_tokens = 0).  The pages have no counterpart: it reports this
 * implementation's choice (for profiling and tuning).  out: host, 5 int32.
 * Errors as for rmsq_fused_add_rmsnorm_quant_ex's mode, shape, dtype and
 * variant; RMSQ_ERR_NO_DEVICE / RMSQ_ERR_UNSUPPORTED_DEVICE without a
 * suitable device.
 */
int rmsq_query_launch(int quant_mode, int64_t n_tokens, int64_t hidden, int has_residual, int dtype,
                      int variant, int32_t *out);

/*
 * rmsq_debug_convert — the library's own fp32 -> 8-bit / 4-bit conversions on
 * a device array, so that tests can pin them against a reference encoder.
 * kind 0: out[i] = e4m3(in[i]) (E4M3FN, nearest even, saturating);
 * kind 1: out[i] = e2m1(in[i]) in the low nibble (high nibble 0).
 * in: device fp32[n]; out: device u8[n]; no alignment requirement.
 */
int rmsq_debug_convert(int kind, const float *in, uint8_t *out, int64_t n, void *stream);

/*
 * rmsq_debug_activation — the library's own e^x and SiLU steps (those of
 * rmsq_silu_mul_quant) on device arrays, so that tests can compare them with
 * a reference element by element.  kind 0: out[i] = e^in[i]; kind 1:
 * out[i] = silu(in[i]); kind 2: out[i] = silu(in[i]) * in2[i] (in2 is
 * ignored otherwise and may be NULL); kind 3: e^in[i] by the shorter steps
 * the kernel takes when |in[i]| <= 87 (defined only there).  Device fp32 arrays of n elements,
 * 4-byte aligned; out must not overlap the inputs.
 */
int rmsq_debug_activation(int kind, const float *in, const float *in2, float *out, int64_t n,
                          void *stream);

/*
 * rmsq_debug_bounded_wait — failure detection without a fault: one CTA waits
 * on a shared-memory barrier that nothing ever completes, with the same
 * bounded wait the pipelined kernels use on their copies, here limited to
 * limit_ns (1 .. 1e9).  *gave_up = 1 when every thread gave up and the kernel
 * returned normally (the expected outcome), 0 if none did, 2 if only some
 * did.  Synchronous (waits for the device); the context stays usable.
 */
int rmsq_debug_bounded_wait(int64_t limit_ns, int *gave_up);

/* Text for an rmsq_status (static storage, never NULL). */
const char *rmsq_status_string(int status);

/* CUDA error code (cudaError_t) of the last RMSQ_ERR_CUDA on this thread. */
int rmsq_last_cuda_error(void);

/* RMSQ_VERSION of the built library. */
int rmsq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RMSQ_H */
