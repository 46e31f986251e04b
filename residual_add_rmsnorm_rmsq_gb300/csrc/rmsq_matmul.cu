// FP8 block-scaled matrix product: argument checks, tensor maps, launches.
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_host.cuh"
#include "rmsq_matmul.cuh"

namespace rmsq {

cudaError_t take_mm_fault(unsigned int* out) {
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_mm_fault, sizeof(unsigned int));
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_mm_fault, &zero, sizeof(zero));
    return e;
}

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A row-major [rows, cols] matrix, rows `pitch` elements apart, in boxes of
// box_rows x 128 bytes, swizzled.
bool make_map(CUtensorMap* map, const void* p, bool codes, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const int elem = codes ? 1 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * elem};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
    return enc(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p), dims,
               strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch in clusters of `size` CTAs along x.
cudaError_t launch_cluster(const void* fn, dim3 grid, dim3 block, void** params, int smem, int size, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic_launch() ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, params);
}

// Pairs of CTAs of `fn` that can run at once (cached per device): not more are
// launched, since their tiles are dealt out in advance.
int resident_pairs(const void* fn, int smem, std::atomic<int>* cached, cudaError_t* err) {
    int dev = 0;
    *err = cudaGetDevice(&dev);
    if (*err != cudaSuccess || dev < 0 || dev >= 128) return 0;
    int n = cached[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *err = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
    if (*err == cudaSuccess && n < 1) *err = cudaErrorInvalidConfiguration;
    if (*err != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_release);
    return n;
}

struct MmCall {
    const void *a, *b;
    int64_t m, n, k;
    MmArgs args;
};

// CTAs of a cluster that divide K: doubled while there are not more than two
// CTAs per SM and each keeps two blocks.
int token_splits(int64_t ctas, int64_t kb, int sms) {
    int splits = 1;
    while (splits < 8 && ctas * splits * 2 <= 2 * sms && kb >= splits * 4) splits *= 2;
    return splits;
}

// Columns n0 .. n0 + n - 1 (n0 a multiple of 128) by the kernel for many rows.
template <class E, int BN>
cudaError_t launch_rows(const MmCall& c, int64_t n0, int64_t n, cudaStream_t stream) {
    using Tile = RowsTile<BN>;
    const void* fn = (const void*)&mm_rows_kernel<E, BN>;
    static std::atomic<int> cached[128];
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile::smem);
    if (e != cudaSuccess) return e;
    const int64_t pairs = resident_pairs(fn, Tile::smem, cached, &e);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mb, mo;
    MmArgs args = c.args;
    args.sb += n0 / 128 * args.kb;
    args.out = static_cast<uint16_t*>(args.out) + n0;
    args.n = static_cast<int>(n);
    if (!make_map(&ma, c.a, true, c.m, c.k, c.k, 128) ||
        !make_map(&mb, static_cast<const uint8_t*>(c.b) + n0 * c.k, true, n, c.k, c.k, BN / 2) ||
        !make_map(&mo, args.out, false, c.m, n, c.n, 128))
        return cudaErrorInvalidValue;
    const int64_t tiles = (c.m + 255) / 256 * ((n + BN - 1) / BN);
    void* params[] = {&ma, &mb, &mo, &args};
    return launch_cluster(fn, dim3(2 * static_cast<unsigned>(tiles < pairs ? tiles : pairs)), dim3(kRowsThreads), params,
                          Tile::smem, 2, stream);
}

template <class E, int NT>
cudaError_t launch_tokens(const MmCall& c, int sms, cudaStream_t stream) {
    using Tile = TokTile<NT>;
    const void* fn = (const void*)&mm_tokens_kernel<E, NT>;
    const int64_t blocks = (c.n + 127) / 128, mt = (c.m + NT - 1) / NT, kb = c.k / 128;
    int splits = token_splits(blocks * mt, kb, sms);
    const int64_t most_kb = (kb + splits - 1) / splits;
    int stages = static_cast<int>((kTokSmem - 1024 - most_kb * NT * 4) / Tile::stage_bytes);
    if (stages > Tile::max_stages) stages = Tile::max_stages;
    // a long run of K leaves too little room for the ring: half as many tokens per CTA
    if constexpr (NT > 16) {
        if (stages < 3) return launch_tokens<E, NT / 2>(c, sms, stream);
    }
    if (stages < 2) return cudaErrorInvalidConfiguration;
    CUtensorMap ma, mb;
    if (!make_map(&ma, c.a, true, c.m, c.k, c.k, NT) || !make_map(&mb, c.b, true, c.n, c.k, c.k, 128)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTokSmem);
    if (e != cudaSuccess) return e;
    MmArgs args = c.args;
    void* params[] = {&ma, &mb, &args, &splits, &stages};
    return launch_cluster(fn, dim3(static_cast<unsigned>(blocks * splits), static_cast<unsigned>(mt)), dim3(kTokThreads),
                          params, kTokSmem, splits, stream);
}

template <class E>
cudaError_t launch_matmul(const MmCall& c, cudaStream_t stream) {
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess) return e;
    // Up to 64 rows the tokens kernel, which reads b at 4.5 TB/s then.  Above,
    // whichever of it and the two row tiles is expected sooner.  The estimates
    // (us) are straight lines through what was measured at n = 2048 .. 14336,
    // k = 2048 .. 7168 and m = 96 .. 2048: a round of 256 x 128 (256 x 256) tiles
    // takes 0.27 (0.36) per block of K, a tokens CTA 0.85 per block of its part
    // of K.  At 128 x 4096 x 4096 the tokens kernel takes 11.5 and the narrow row
    // tiles 12.8, at 256 rows 14.9 and 13.0, at 128 x 7168 x 2048 10.7 and 8.9; at
    // 768 x 4096 x 4096 the narrow tiles take 22.9 (two rounds), the wide ones
    // 18.2, at 512 rows 13.4 and 17.7.
    if (c.m > 64) {
        const int64_t mt = (c.m + 255) / 256, pairs = sms / 2, kb = c.k / 128;
        const int64_t narrow = (mt * ((c.n + 127) / 128) + pairs - 1) / pairs, wide = (mt * ((c.n + 255) / 256) + pairs - 1) / pairs;
        const double us_narrow = 3.9 + 0.27 * static_cast<double>(narrow * kb), us_wide = 3.9 + 0.36 * static_cast<double>(wide * kb);
        const int64_t ctas = (c.n + 127) / 128 * ((c.m + 127) / 128), splits = token_splits(ctas, kb, sms);
        const int64_t rounds = (ctas * splits + 2 * sms - 1) / (2 * sms);
        const double us_tokens = 8.0 + 0.85 * static_cast<double>((kb + splits - 1) / splits * rounds);
        // Or full rounds of wide tiles and, in a second launch (3 us: it waits for
        // the first one's last tile), narrow ones for the columns left over: 300 x
        // 10240 x 8192 takes 51.5 us so and 55.6 in two wide rounds, 768 x 7168 x
        // 7168 46.8 and 49.2; at k = 4096 the second launch costs what it saves.
        const int64_t full = wide > 1 ? (wide - 1) * pairs / mt * 256 : 0;
        if (full > 0 && full < c.n) {
            const int64_t last = (mt * ((c.n - full + 127) / 128) + pairs - 1) / pairs;
            const int64_t first = (mt * (full / 256) + pairs - 1) / pairs;
            const double us_both = 6.9 + (0.36 * static_cast<double>(first) + 0.27 * static_cast<double>(last)) * static_cast<double>(kb);
            if (us_both < us_wide && us_both < us_narrow && us_both < us_tokens) {
                e = launch_rows<E, 256>(c, 0, full, stream);
                return e == cudaSuccess ? launch_rows<E, 128>(c, full, c.n - full, stream) : e;
            }
        }
        if (us_wide <= us_narrow && us_wide <= us_tokens) return launch_rows<E, 256>(c, 0, c.n, stream);
        if (us_narrow <= us_tokens) return launch_rows<E, 128>(c, 0, c.n, stream);
    }
    if (c.m <= 16) return launch_tokens<E, 16>(c, sms, stream);
    if (c.m <= 32) return launch_tokens<E, 32>(c, sms, stream);
    if (c.m <= 64) return launch_tokens<E, 64>(c, sms, stream);
    return launch_tokens<E, 128>(c, sms, stream);
}

}  // namespace
}  // namespace rmsq

extern "C" int rmsq_fp8_block_matmul(const void* a_codes, const void* a_scales, int quant_mode, const void* b_codes,
                                     const float* b_scales, void* out, int64_t m, int64_t n, int64_t k, int dtype,
                                     void* stream) {
    using rmsq_abi::aligned;
    using rmsq_abi::overlaps;
    using rmsq_abi::Span;
    using rmsq_abi::span;
    if (dtype != RMSQ_BF16 && dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    const int mode = quant_mode & RMSQ_QUANT_MODE_MASK;
    if (quant_mode < 0 || (mode != RMSQ_FP8_GROUP128_ROW && mode != RMSQ_FP8_GROUP128_COL)) return RMSQ_ERR_INVALID_ARG;
    if (m < 0 || n <= 0 || k <= 0) return RMSQ_ERR_INVALID_ARG;
    // the scale options are the quantisation's; K is its hidden size
    size_t q_bytes = 0, sa_bytes = 0;
    int st = rmsq_query_sizes(quant_mode, m, k <= RMSQ_MAX_HIDDEN ? k : 128, &q_bytes, &sa_bytes);
    if (st != RMSQ_OK) return st;
    if (k % 128 != 0 || k > RMSQ_ACT_MAX_D || n % 8 != 0 || n > INT32_MAX / 2 || m > INT32_MAX / 2 ||
        (m + 127) / 128 * ((n + 127) / 128) > INT32_MAX / 2)
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    if (m == 0) return RMSQ_OK;
    if (!a_codes || !a_scales || !b_codes || !b_scales || !out) return RMSQ_ERR_INVALID_ARG;
    const bool ue8m0 = (quant_mode & RMSQ_QUANT_UE8M0) != 0, col = mode == RMSQ_FP8_GROUP128_COL;
    if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(out, 16) || !aligned(a_scales, ue8m0 ? 1 : 4) ||
        !aligned(b_scales, 4))
        return RMSQ_ERR_ALIGNMENT;
    const int64_t kb = k / 128, per16 = ue8m0 ? 16 : 4;
    const int64_t stride = (quant_mode & RMSQ_QUANT_TMA_ALIGNED) ? (m + per16 - 1) / per16 * per16 : m;
    const size_t width = ue8m0 ? 1 : 4;
    const Span ins[4] = {span(a_codes, static_cast<size_t>(m) * k),
                         span(a_scales, static_cast<size_t>(col ? kb * stride : m * kb) * width),
                         span(b_codes, static_cast<size_t>(n) * k), span(b_scales, static_cast<size_t>((n + 127) / 128) * kb * 4)};
    const Span O = span(out, static_cast<size_t>(m) * n * 2);
    for (const Span& in : ins)
        if (overlaps(O, in)) return RMSQ_ERR_ALIAS;
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    rmsq::MmCall c = {a_codes, b_codes, m, n, k, {}};
    c.args.sa = a_scales;
    c.args.sb = b_scales;
    c.args.out = out;
    c.args.sa_row = col ? 1 : kb;
    c.args.sa_kb = col ? stride : 1;
    c.args.m = static_cast<int>(m);
    c.args.n = static_cast<int>(n);
    c.args.kb = static_cast<int>(kb);
    c.args.ue8m0 = ue8m0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSQ_BF16 ? rmsq::launch_matmul<rmsq::Bf16T>(c, s) : rmsq::launch_matmul<rmsq::Fp16T>(c, s);
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}
