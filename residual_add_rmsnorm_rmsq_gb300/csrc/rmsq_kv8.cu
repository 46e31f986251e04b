// Paged FP8 cache with a power-of-two scale per block of 16 tokens and head:
// store and load.
#include <cstdint>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_device.cuh"
#include "rmsq_host.cuh"
#include "rmsq_kv.cuh"
#include "rmsq_kv8.cuh"

namespace rmsq {

struct Cache8Args {
    const uint4* k;            // source (store) / destination (load) of the keys
    const uint4* v;
    int64_t k_stride, v_stride;   // 16-byte chunks per token
    const int64_t* slots;
    uint8_t* codes;
    uint8_t* scales;
    int64_t slots_total;       // pages * page size
    int n, heads;
    int page_shift;
    int range_shift;           // store: log2 of the tokens a warp looks after
};

// Index of a (page, keys or values, head) in the cache.
__device__ __forceinline__ int64_t side_index(const Cache8Args& a, int64_t slot, int side, int head) {
    return ((slot >> a.page_shift) * 2 + side) * a.heads + head;
}
__device__ __forceinline__ uint8_t* scale_at(const Cache8Args& a, int64_t slot, int side, int head) {
    const int block = (static_cast<int>(slot) & ((1 << a.page_shift) - 1)) / kBlockTokens;
    return a.scales + (side_index(a, slot, side, head) << (a.page_shift - 4)) + block;
}

// ---------------------------------------------------------------------------
// Store.  With X the magnitudes that one block of 16 slots gets in this call,
//   s = 2^ceil(log2(max(max X / 448, 1e-12))),
// and, if the block's first slot is not among those it gets, at least the scale
// it has; codes e4m3(x / s).  Slots that the call does not write keep their value:
// if the scale has grown, their codes are rounded to it.
//
// A warp looks after a range of tokens (a power of two up to 16) of one kv head,
// and takes the runs of tokens of one block that start there.  The slots of a run
// ascend within 16 consecutive entries of the slot map, with none but skipped ones
// between them, so that 16 entries before the range and 16 behind it show which
// runs start in it, and all of them to their end; no token is looked after twice and
// no warp waits for another.  A lane holds 8 elements of a token, D / 8 lanes a
// token, all of a run's tokens are in registers before the maximum is taken: one
// pass.  Prompts are bound by HBM and, as much, by the chain of a run (slots, tokens,
// maximum, codes) that a warp walks a side after the other with 80 registers a
// thread; 16000 tokens of 4 + 4 heads of 128, 49 MB, take 9.6 us (5.1 TB/s), 256
// decodes of 8 + 8 heads 4.0 us (latency: slots, then tokens and the old scale).
//
// Not finite elements do not count for the scale.  They become NaN, and so do all
// of the token's key codes of that head: the attention's reader can then leave
// NaN out of the values (it reads the codes as 448), so that no masked or unwritten
// place reaches a sum, and a query that sees the token gets NaN all the same.
// ---------------------------------------------------------------------------
template <class E>
struct Magnitude {
    static constexpr uint32_t inf = E::kBits87 == Bf16T::kBits87 ? 0x7f80u : 0x7c00u;
    static __device__ __forceinline__ float value(uint32_t bits) { return E::lo(bits); }
};

// max of two pairs of unsigned 16-bit numbers
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Codes of 8 elements times f.
template <class E>
__device__ __forceinline__ uint2 codes8(const uint4& u, float f) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = mul2_rn(make_float2(E::lo(word(u, i)), E::hi(word(u, i))), make_float2(f, f));
        c[i] = e4m3x2(x.x, x.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A pair of elements: both, or those that are not finite, as NaN.
constexpr uint32_t kNanPair = 0x7fff7fffu;
template <class E>
__device__ __forceinline__ uint32_t nan_unless_finite(uint32_t w) {
    const uint32_t m = w & 0x7fff7fffu;
    if ((m & 0xffffu) >= Magnitude<E>::inf) w |= 0x7fffu;
    if ((m >> 16) >= Magnitude<E>::inf) w |= 0x7fff0000u;
    return w;
}

// Rounds the codes of a block's slots that are not in `taken` to a scale 2^up
// times as large.
template <int D>
__device__ __forceinline__ void round_anew(uint8_t* block, uint32_t taken, int up, int lane) {
    constexpr int PER = D / 16;     // lanes of a slot
    const float f = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
    for (int s = lane / PER; s < kBlockTokens; s += 32 / PER) {
        if (taken >> s & 1u) continue;
        uint4* p = reinterpret_cast<uint4*>(block + s * D) + lane % PER;
        const uint4 u = *p;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = e4m3x2_to_f16x2(word(u, i)), b = e4m3x2_to_f16x2(word(u, i) >> 16);
            w[i] = e4m3x2(Fp16T::lo(a) * f, Fp16T::hi(a) * f) | e4m3x2(Fp16T::lo(b) * f, Fp16T::hi(b) * f) << 16;
        }
        *p = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <class E, int D>
__global__ void __launch_bounds__(256, D == 64 ? 4 : D == 128 ? 3 : 2) cache8_store_kernel(Cache8Args a) {
    constexpr int LT = D / 8, TP = 32 / LT;         // lanes of a token, tokens of a pass
    constexpr int PASSES = kBlockTokens / TP;
    allow_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    const int head = static_cast<int>(w % a.heads);
    const int64_t base = w / a.heads << a.range_shift;
    if (base >= a.n) return;
    // lane i: entry base - 1 + i of the slot map; -1: skipped
    auto entry = [&](int64_t i) {
        const int64_t s = i >= 0 && i < a.n ? __ldg(reinterpret_cast<const long long*>(a.slots) + i) : -1;
        return s < a.slots_total ? s : -1;
    };
    // A token goes on a run if the entry before it that is not skipped, at most 15
    // away, is a smaller slot of its block.
    auto goes_on = [](int64_t s, int64_t before) {
        return s >= 0 && before >= 0 && s > before && s / kBlockTokens == before / kBlockTokens;
    };
    const int64_t slot = entry(base - 1 + lane);
    const uint32_t valid = __ballot_sync(kFull, slot >= 0);
    int64_t before = __shfl_up_sync(kFull, slot, 1);
    if (__any_sync(kFull, slot < 0 && base - 1 + lane >= 0 && base - 1 + lane < a.n)) {
        // something is skipped: the one before may be further off, or before these
        const int64_t prior = (valid & 1u) == 0u && lane < kBlockTokens ? entry(base - kBlockTokens + lane) : -1;
        const uint32_t below = valid & ((1u << lane) - 1u), valid_prior = __ballot_sync(kFull, prior >= 0);
        const int last = 31 - __clz(below), last_prior = 31 - __clz(valid_prior);       // -1: none
        const int64_t near = __shfl_sync(kFull, slot, max(last, 0)), far = __shfl_sync(kFull, prior, max(last_prior, 0));
        before = last >= 0 ? near : last_prior >= 0 ? far : -1;
        if ((last >= 0 ? lane - last : lane + kBlockTokens - 1 - last_prior) >= kBlockTokens) before = -1;
    }
    const uint32_t begins = valid & ~__ballot_sync(kFull, lane > 0 && goes_on(slot, before));
    uint32_t starts = begins & (((1u << (1 << a.range_shift)) - 1u) << 1);
    const int sub = lane / LT, chunk = lane % LT;
    while (starts != 0) {
        const int first = __ffs(starts) - 1;
        starts &= starts - 1;
        // bit j: the j-th entry from there is the run's, up to the next one that begins another
        const uint32_t next = begins >> first & ~1u;
        const uint32_t members = valid >> first & 0xffffu & ((next & (0u - next)) - 1u);
        const int len = 32 - __clz(members);
        const int64_t slot0 = __shfl_sync(kFull, slot, first);
        // lane j: where the j-th entry's slot lies in its block
        const int offset = __shfl_sync(kFull, static_cast<int>(slot) & (kBlockTokens - 1), (first + lane) & 31);
        // The values, then the keys; the keys' first tokens are loaded with the
        // values' (a decode has no others), the rest only when the values'
        // registers are free.
        const int64_t tok0 = base - 1 + first;
        auto load = [&](int i, int p) {
            const int j = p * TP + sub;
            if (j >= len) return make_uint4(0u, 0u, 0u, 0u);
            const int64_t t = tok0 + j;
            return ld_act((i == 0 ? a.v + t * a.v_stride : a.k + t * a.k_stride) + head * LT + chunk);
        };
        const uint4 front[2] = {load(0, 0), load(1, 0)};
        const int o0 = static_cast<int>(slot0) & (kBlockTokens - 1);
        uint8_t* const sp[2] = {scale_at(a, slot0, 1, head), scale_at(a, slot0, 0, head)};
        uint32_t old[2] = {0u, 0u};
        if (o0 > 0) {
            old[0] = *sp[0];
            old[1] = *sp[1];
        }
        // offsets that the run takes
        const uint32_t taken = __reduce_or_sync(kFull, members >> lane & 1u ? 1u << offset : 0u);
        uint32_t poison = 0u;       // tokens of the run with an element that is not finite
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            uint4 in[PASSES];
            in[0] = i == 0 ? front[0] : front[1];
#pragma unroll
            for (int p = 1; p < PASSES; ++p) in[p] = load(i, p);
            if ((members & (members + 1u)) != 0u) {     // tokens between the run's that are skipped
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    if (!(members >> (p * TP + sub) & 1u)) in[p] = make_uint4(0u, 0u, 0u, 0u);
            }
            uint32_t m = 0u;
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) m = max_u16x2(m, word(in[p], j) & 0x7fff7fffu);
            uint32_t top = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
            if (top >= Magnitude<E>::inf) {
                m = 0u;
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    bool bad = false;
                    uint32_t x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j] = nan_unless_finite<E>(word(in[p], j));
                        const uint32_t lo = x[j] & 0x7fffu, hi = x[j] >> 16 & 0x7fffu;
                        bad |= lo == 0x7fffu || hi == 0x7fffu;
                        m = max(m, max(lo == 0x7fffu ? 0u : lo, hi == 0x7fffu ? 0u : hi));
                    }
                    in[p] = make_uint4(x[0], x[1], x[2], x[3]);
                    const uint32_t lanes = __ballot_sync(kFull, bad);
#pragma unroll
                    for (int t = 0; t < TP; ++t)
                        if (lanes >> (t * LT) & (LT == 32 ? 0xffffffffu : (1u << (LT & 31)) - 1u)) poison |= 1u << (p * TP + t);
                }
                top = __reduce_max_sync(kFull, m);
            }
            if (i == 1 && poison != 0u) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    if (poison >> (p * TP + sub) & 1u) in[p] = make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
            }
            const float s = fmaxf(__fdiv_rn(Magnitude<E>::value(top), 448.0f), 1e-12f);
            uint32_t e = min((__float_as_uint(s) + 0x7fffffu) >> 23, kScaleMost);
            uint8_t* block = a.codes + ((side_index(a, slot0, 1 - i, head) << a.page_shift) +
                                        ((slot0 & ((1 << a.page_shift) - 1)) - o0)) * D;
            if (o0 > 0) {
                const uint32_t had = cache_scale_code(i == 0 ? old[0] : old[1]);
                if (e > had) round_anew<D>(block, taken, min(static_cast<int>(e - had), 126), lane);
                e = max(e, had);
            }
            const float f = __uint_as_float((254u - e) << 23);      // 2^-(e - 127)
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (p * TP >= len) break;
                const int j = p * TP + sub;
                const int at = __shfl_sync(kFull, offset, j);
                const uint2 c = codes8<E>(in[p], f);
                if (members >> j & 1u) *reinterpret_cast<uint2*>(block + at * D + chunk * 8) = c;
            }
            if (lane == 0) *(i == 0 ? sp[0] : sp[1]) = static_cast<uint8_t>(e);
        }
    }
}

// ---------------------------------------------------------------------------
// Load: T(code * scale), exact before its rounding; zeros for a slot outside the
// cache.  One thread per 16 elements, a token's (keys, then values) on a power of
// two of lanes up to 32, as in the NVFP4 load.  Bound by HBM: 16016 tokens of 4 + 4
// heads of 128, 49 MB, take 10.0 us (4.9 TB/s), 2134 of 8 + 8 heads 6.4 us.
// ---------------------------------------------------------------------------
template <class E, int D>
__global__ void __launch_bounds__(256) cache8_load_kernel(Cache8Args a) {
    constexpr int B = D / 16;
    allow_dependents();
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = i >> a.range_shift;
    if (t >= a.n) return;
    const int64_t slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
    const bool inside = slot >= 0 && slot < a.slots_total;
    const int blocks = 2 * a.heads * B, step = 1 << a.range_shift;
    for (int c = static_cast<int>(i) & (step - 1); c < blocks; c += 2 * step) {
        // two pieces' loads before either's arithmetic
        uint4 u[2];
        uint32_t e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u[h] = make_uint4(0u, 0u, 0u, 0u);
            e[h] = 127u;
            const int x = c + h * step, side = x >= a.heads * B, rest = x - side * a.heads * B;
            if (inside && x < blocks) {
                const int64_t row = (side_index(a, slot, side, rest / B) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
                u[h] = __ldg(reinterpret_cast<const uint4*>(a.codes + row * D) + rest % B);
                e[h] = *scale_at(a, slot, side, rest / B);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int x = c + h * step, side = x >= a.heads * B, rest = x - side * a.heads * B;
            if (x >= blocks) break;
            uint4* dst = const_cast<uint4*>(side ? a.v + t * a.v_stride : a.k + t * a.k_stride) + 2 * rest;
            const float s = cache_scale_value(cache_scale_code(e[h]));
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t p = e4m3x2_to_f16x2(word(u[h], j / 2) >> (16 * (j & 1)));
                const float2 y = mul2_rn(make_float2(Fp16T::lo(p), Fp16T::hi(p)), make_float2(s, s));
                w[j] = E::pack(y.x, y.y);
            }
            st_stream(dst, make_uint4(w[0], w[1], w[2], w[3]));
            st_stream(dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
        }
    }
}

namespace {

// The checks the store and the load share; fills the launch arguments.
int cache8_args(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slot_map,
                const void* cache, const void* scales, int64_t num_pages, int64_t page_size, int64_t n, int heads,
                int head_dim, int dtype, Cache8Args* a) {
    if (dtype != RMSQ_BF16 && dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    if (n < 0 || heads <= 0 || num_pages <= 0) return RMSQ_ERR_INVALID_ARG;
    int shift = -1;
    for (int s = 4; s <= 8; ++s)
        if (page_size == (1 << s)) shift = s;
    if (shift < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256) || heads > 4096 || n > INT32_MAX ||
        num_pages > INT32_MAX)
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    if (k_stride < row || v_stride < row || k_stride > INT32_MAX || v_stride > INT32_MAX) return RMSQ_ERR_INVALID_ARG;
    if (n == 0) return RMSQ_OK;
    if (!k || !v || !slot_map || !cache || !scales) return RMSQ_ERR_INVALID_ARG;
    using rmsq_abi::aligned;
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8 || !aligned(slot_map, 8) || !aligned(cache, 16))
        return RMSQ_ERR_ALIGNMENT;
    a->k = static_cast<const uint4*>(k);
    a->v = static_cast<const uint4*>(v);
    a->k_stride = k_stride / 8;
    a->v_stride = v_stride / 8;
    a->slots = slot_map;
    a->codes = static_cast<uint8_t*>(const_cast<void*>(cache));
    a->scales = static_cast<uint8_t*>(const_cast<void*>(scales));
    a->slots_total = num_pages * page_size;
    a->n = static_cast<int>(n);
    a->heads = heads;
    a->page_shift = shift;
    return RMSQ_OK;
}

// Spans of the token rows [n, stride], of the cache and of the slots.
struct Cache8Spans {
    rmsq_abi::Span k, v, codes, scales, slots;
};
Cache8Spans cache8_spans(const Cache8Args& a, int head_dim) {
    const size_t row = static_cast<size_t>(a.heads) * head_dim;
    auto rows = [&](const uint4* p, int64_t stride) {
        return rmsq_abi::span(p, static_cast<size_t>(a.n - 1) * stride * 16 + row * 2);
    };
    const size_t slots = static_cast<size_t>(a.slots_total) * 2;
    return {rows(a.k, a.k_stride), rows(a.v, a.v_stride), rmsq_abi::span(a.codes, slots * row),
            rmsq_abi::span(a.scales, slots * a.heads / kBlockTokens), rmsq_abi::span(a.slots, static_cast<size_t>(a.n) * 8)};
}

template <class E>
const void* cache8_kernel(bool store, int head_dim) {
    switch (head_dim) {
    case 64: return store ? (const void*)&cache8_store_kernel<E, 64> : (const void*)&cache8_load_kernel<E, 64>;
    case 128: return store ? (const void*)&cache8_store_kernel<E, 128> : (const void*)&cache8_load_kernel<E, 128>;
    default: return store ? (const void*)&cache8_store_kernel<E, 256> : (const void*)&cache8_load_kernel<E, 256>;
    }
}

cudaError_t launch_cache8(bool store, int head_dim, int dtype, Cache8Args& a, cudaStream_t stream) {
    const void* fn = dtype == RMSQ_FP16 ? cache8_kernel<Fp16T>(store, head_dim) : cache8_kernel<Bf16T>(store, head_dim);
    int64_t threads;
    if (store) {
        // Tokens of a warp: one for a decode (each token starts a run: a warp of
        // several takes them one after the other), more for a prompt (most of its
        // tokens start none).  The host sees only how many there are.  Measured, in
        // us for 1, 2, 4, 8, 16: 256 decodes of 8 heads of 128 4.2 6.0 8.2 14.1 26.4, a
        // prompt of 1000 6.7 6.2 6.1 5.3 6.3; 1000 decodes 8.7 9.5 12.4 18.9 28.3, a
        // prompt of 2000 8.9 7.9 7.5 7.2 7.3; 3000 decodes 21.4 20.2 20.1 23.7 42.1, a
        // prompt of 4000 13.1 10.3 8.7 8.1 8.5; 8000 decodes 53 50 49 51 62, a prompt of
        // 8000 21.7 16.6 13.9 12.4 11.6; a prompt of 30000 70 50 40 36 34.
        const int64_t warps = static_cast<int64_t>(a.n) * a.heads;
        a.range_shift = warps < 8192 ? 0 : warps < 24576 ? 1 : warps < 49152 ? 2 : warps < 131072 ? 3 : 4;
        const int64_t ranges = (static_cast<int64_t>(a.n) + (1 << a.range_shift) - 1) >> a.range_shift;
        threads = ranges * a.heads * 32;
    } else {
        a.range_shift = 3;   // the smallest token: one head of 64, keys and values
        while (a.range_shift < 5 && (1 << a.range_shift) < 2 * a.heads * head_dim / 16) ++a.range_shift;
        threads = static_cast<int64_t>(a.n) << a.range_shift;
    }
    const int64_t grid = (threads + 255) / 256;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    void* params[] = {&a};
    return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(256), params, 0, stream);
}

}  // namespace
}  // namespace rmsq

extern "C" {

int rmsq_kv_cache_store_fp8(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slot_map,
                            void* cache, uint8_t* scales, int64_t num_pages, int64_t page_size, int64_t n_tokens,
                            int num_kv_heads, int head_dim, int dtype, void* stream) {
    using rmsq_abi::overlaps;
    rmsq::Cache8Args a = {};
    int st = rmsq::cache8_args(k, k_stride, v, v_stride, slot_map, cache, scales, num_pages, page_size, n_tokens,
                               num_kv_heads, head_dim, dtype, &a);
    if (st != RMSQ_OK || n_tokens == 0) return st;
    const rmsq::Cache8Spans s = rmsq::cache8_spans(a, head_dim);
    if (overlaps(s.codes, s.scales)) return RMSQ_ERR_ALIAS;
    for (const rmsq_abi::Span& in : {s.k, s.v, s.slots})
        if (overlaps(s.codes, in) || overlaps(s.scales, in)) return RMSQ_ERR_ALIAS;
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    const cudaError_t e = rmsq::launch_cache8(true, head_dim, dtype, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

int rmsq_kv_cache_load_fp8(const void* cache, const uint8_t* scales, int64_t num_pages, int64_t page_size,
                           const int64_t* slot_map, void* k, int64_t k_stride, void* v, int64_t v_stride, int64_t n_tokens,
                           int num_kv_heads, int head_dim, int dtype, void* stream) {
    using rmsq_abi::overlaps;
    rmsq::Cache8Args a = {};
    int st = rmsq::cache8_args(k, k_stride, v, v_stride, slot_map, cache, scales, num_pages, page_size, n_tokens,
                               num_kv_heads, head_dim, dtype, &a);
    if (st != RMSQ_OK || n_tokens == 0) return st;
    const rmsq::Cache8Spans s = rmsq::cache8_spans(a, head_dim);
    // k and v may be two column ranges of one token-major buffer
    const bool columns = a.k_stride == a.v_stride && rmsq::disjoint_columns(a.k, a.v, a.k_stride, num_kv_heads * head_dim / 8);
    if (overlaps(s.k, s.v) && !columns) return RMSQ_ERR_ALIAS;
    for (const rmsq_abi::Span& in : {s.codes, s.scales, s.slots})
        if (overlaps(s.k, in) || overlaps(s.v, in)) return RMSQ_ERR_ALIAS;
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    const cudaError_t e = rmsq::launch_cache8(false, head_dim, dtype, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

}  // extern "C"
