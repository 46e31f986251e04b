// Paged key / value cache: slot maps from request lengths, and the NVFP4
// cache's store and load.
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_abi.h"
#include "rmsq_device.cuh"
#include "rmsq_host.cuh"
#include "rmsq_kv.cuh"

namespace rmsq {

// ---------------------------------------------------------------------------
// Slot map.  With q_r new and c_r cached tokens of request r, page size P:
//   start_r = q_0 + .. + q_{r-1},   held_r = ceil(c_r / P),
//   new_r = ceil((c_r + q_r) / P) - held_r,   off_r = new_0 + .. + new_{r-1}
//   table[r][held_r + k] = free[num_free - 1 - off_r - k]       (k < new_r)
//   token i of r: position c_r + i, slot = table[r][pos / P] * P + pos % P.
//
// Bound by latency: 8 bytes read per request and 16 written per token; 3.2 us for
// 64 requests of one token, 4.3 us for 1000 requests with 16000 tokens.  Every CTA scans all lengths itself
// (an L2-resident array, two loads per request), so one launch is enough and
// no CTA waits for another; then the CTAs share out the tokens and the new
// pages, each finding its request by binary search in the scanned offsets in
// shared memory.  A token on a new page takes the page from the free list
// itself, not from the table entry another CTA may not have written yet; the
// table entries read (pages held before) are written by nobody.
// ---------------------------------------------------------------------------
struct SlotArgs {
    const int* ctx;
    const int* qlen;
    int* table;
    const int* free_pages;
    const int* num_free;
    int64_t* slots;
    int64_t* positions;
    int* q_start;
    int* seq_lens;
    int* num_free_out;
    int* status;
    int requests, width, free_capacity, page_shift, tokens;
};

constexpr int kSlotThreads = 512;

// Exclusive scan of one pair of 64-bit values per thread over the CTA;
// total_* receive the sums.
__device__ __forceinline__ void block_scan_pair(int64_t& a, int64_t& b, int64_t& total_a, int64_t& total_b) {
    __shared__ int64_t wa[kSlotThreads / 32], wb[kSlotThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(kFull, ia, o), ub = __shfl_up_sync(kFull, ib, o);
        if (lane >= o) {
            ia += ua;
            ib += ub;
        }
    }
    if (lane == 31) {
        wa[warp] = ia;
        wb[warp] = ib;
    }
    __syncthreads();
    int64_t pa = 0, pb = 0;
    total_a = total_b = 0;
#pragma unroll
    for (int w = 0; w < kSlotThreads / 32; ++w) {
        if (w == warp) {
            pa = total_a;
            pb = total_b;
        }
        total_a += wa[w];
        total_b += wb[w];
    }
    a = pa + ia - a;
    b = pb + ib - b;
}

// Largest r in [0, n) with start[r] <= x, for start[0] = 0 <= x < start[n]
// and ascending starts.
__device__ __forceinline__ int find_request(const int* start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(SlotArgs a) {
    extern __shared__ int smem[];
    int* start = smem;                     // [requests + 1]
    int* page_off = smem + a.requests + 1; // [requests + 1]
    __shared__ int err_sh;
    const int tid = threadIdx.x, R = a.requests, P = 1 << a.page_shift;
    allow_dependents();
    grid_dependency_wait();
    if (tid == 0) err_sh = 0;
    __syncthreads();

    // Thread t owns `per` consecutive requests: local sums, one scan over the
    // CTA, then the offsets.  Lengths are staged through the offset arrays so
    // that the global reads are coalesced.
    for (int r = tid; r < R; r += kSlotThreads) {
        start[r] = __ldg(a.qlen + r);
        page_off[r] = __ldg(a.ctx + r);
    }
    const int nf = __ldg(a.num_free);
    __syncthreads();
    const int per = (R + kSlotThreads - 1) / kSlotThreads;
    const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
    int64_t sq = 0, sp = 0;
    int err = 0;
    for (int r = r0; r < r1; ++r) {
        const int q = start[r], c = page_off[r];
        if (q < 0 || c < 0) {
            err |= RMSQ_SLOT_BAD_LENGTH;
            continue;
        }
        const int64_t want = (static_cast<int64_t>(c) + q + P - 1) >> a.page_shift;
        if (want > a.width) err |= RMSQ_SLOT_TABLE_FULL;
        sq += q;
        sp += want - ((static_cast<int64_t>(c) + P - 1) >> a.page_shift);
    }
    int64_t tq, tp;
    block_scan_pair(sq, sp, tq, tp);
    if (tid == 0) {
        if (nf < 0 || nf > a.free_capacity) err |= RMSQ_SLOT_BAD_LENGTH;
        else if (tp > nf) err |= RMSQ_SLOT_NO_PAGES;
        if (tq > a.tokens) err |= RMSQ_SLOT_TOO_MANY_TOKENS;
    }
    if (err) atomicOr(&err_sh, err);
    __syncthreads();
    err = err_sh;
    const int stride = gridDim.x * kSlotThreads, first = blockIdx.x * kSlotThreads + tid;
    if (first == 0) {
        *a.status = err;
        *a.num_free_out = err ? nf : nf - static_cast<int>(tp);
    }
    if (err) {   // nothing is assigned; every output is still defined
        for (int t = first; t < a.tokens; t += stride) a.slots[t] = a.positions[t] = -1;
        for (int r = first; r <= R; r += stride) {
            a.q_start[r] = 0;
            if (r < R) a.seq_lens[r] = __ldg(a.ctx + r);
        }
        return;
    }
    // Totals fit int32 here: tokens <= a.tokens, pages <= nf.
    for (int r = r0; r < r1; ++r) {
        const int q = start[r], c = page_off[r];
        start[r] = static_cast<int>(sq);
        page_off[r] = static_cast<int>(sp);
        sq += q;
        sp += ((c + q + P - 1) >> a.page_shift) - ((c + P - 1) >> a.page_shift);
    }
    if (tid == 0) {
        start[R] = static_cast<int>(tq);
        page_off[R] = static_cast<int>(tp);
    }
    __syncthreads();
    for (int t = first; t < a.tokens; t += stride) {
        int64_t slot = -1, pos = -1;
        if (t < start[R]) {
            const int r = find_request(start, R, t);
            const int c = __ldg(a.ctx + r);
            const int held = (c + P - 1) >> a.page_shift;
            const int p = c + (t - start[r]), idx = p >> a.page_shift;
            const int page = idx < held ? a.table[static_cast<int64_t>(r) * a.width + idx]
                                        : __ldg(a.free_pages + (nf - 1 - page_off[r] - (idx - held)));
            pos = p;
            slot = page < 0 ? -1 : (static_cast<int64_t>(page) << a.page_shift) + (p & (P - 1));
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int k = first; k < page_off[R]; k += stride) {
        const int r = find_request(page_off, R, k);
        const int held = (__ldg(a.ctx + r) + P - 1) >> a.page_shift;
        a.table[static_cast<int64_t>(r) * a.width + held + (k - page_off[r])] = __ldg(a.free_pages + (nf - 1 - k));
    }
    for (int r = first; r <= R; r += stride) {
        a.q_start[r] = start[r];
        if (r < R) a.seq_lens[r] = __ldg(a.ctx + r) + (start[r + 1] - start[r]);
    }
}

// ---------------------------------------------------------------------------
// Store and load.  One thread per 16-element block; a token's blocks (keys,
// then values) take `lanes` lanes of a warp, a power of two up to 32, so that
// neither a token nor a head is found by division, and a token with more
// blocks several rounds, two at a time with their loads together (256 tokens of
// 8 + 8 heads of 128 3.0 us stored and 2.8 loaded; 3.4 and 3.1 with one after the
// other, where the second round's loads waited for the first's arithmetic).
// Bound by HBM: 2 bytes of T and 9/16 of codes and scales per element; 16001
// tokens of 4 + 4 heads of 128, 42 MB each way, take 9.3 us stored (4.5 TB/s)
// and 12.1 loaded into buffers larger than L2 (3.5 TB/s, about half of the issue
// slots).  What it took for both together: 40 us with a 64-bit division
// per block to find its place and sixteen divisions to decode it.  A warp reads
// (store) or writes (load) up to 1 KB of T in one piece and whole 32-byte
// sectors of codes; the scale bytes of a head are adjacent bytes of one access.
//
// The store takes the same steps as the RMSQ_NVFP4 quantisation of the row ops
// and so gives the same bits.
// ---------------------------------------------------------------------------
struct CacheArgs {
    const uint4* k;            // source (store) / destination (load) of the keys
    const uint4* v;
    int64_t k_stride, v_stride;   // 16-byte chunks per token
    const int64_t* slots;
    const float* k_gs;
    const float* v_gs;
    uint8_t* cache;
    int64_t slots_total;       // pages * page size
    int n, heads, blocks;      // tokens, kv heads, 16-element blocks per head
    int page_shift;
    int lane_shift;            // log2 of the lanes per token
};

template <class E>
__device__ __forceinline__ void unpack16(const uint4& lo, const uint4& hi, float (&a)[8], float (&b)[8]) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] = E::lo(w[i]);
        a[2 * i + 1] = E::hi(w[i]);
        b[2 * i] = E::lo(w[4 + i]);
        b[2 * i + 1] = E::hi(w[4 + i]);
    }
}

// Byte offset of a (page, key or value, head) tile in the cache.
__device__ __forceinline__ int64_t tile_offset(const CacheArgs& a, int64_t page, int side, int head) {
    const int64_t tile = (static_cast<int64_t>(a.blocks) * 9) << a.page_shift;
    return ((page * 2 + side) * a.heads + head) * tile;
}

// The token of a thread and its first block; false beyond the last token.
__device__ __forceinline__ bool cache_place(const CacheArgs& a, int& t, int& c) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    c = static_cast<int>(i) & ((1 << a.lane_shift) - 1);
    const int64_t token = i >> a.lane_shift;
    t = static_cast<int>(token);
    return token < a.n;
}

// A block of a token: its place in the token's rows and in the cache.
template <int B>
struct BlockPlace {
    int side, rest;      // keys or values; 16-element block within the token's heads
    uint8_t *codes, *scale;
    __device__ __forceinline__ BlockPlace(const CacheArgs& a, int c, int64_t slot) {
        const int per_side = a.heads * B;
        side = c >= per_side;
        rest = c - side * per_side;
        const int head = rest / B, blk = rest % B;      // B is a power of two
        const int in_page = static_cast<int>(slot) & ((1 << a.page_shift) - 1);
        uint8_t* tile = a.cache + tile_offset(a, slot >> a.page_shift, side, head);
        codes = tile + (in_page * B + blk) * 8;
        scale = tile + ((B * 8) << a.page_shift) + in_page * B + blk;
    }
};

// (bf16 at 48 registers, five CTAs per SM: 9.3 us instead of 10.1 for 16001
// tokens; fp16 would spill there, 10.4 instead of 9.9)
template <class E, int B>
__global__ void __launch_bounds__(256, std::is_same<E, Bf16T>::value ? 5 : 4) cache_store_kernel(CacheArgs a) {
    allow_dependents();
    grid_dependency_wait();
    int t, c;
    if (!cache_place(a, t, c)) return;
    const int64_t slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
    if (slot < 0 || slot >= a.slots_total) return;
    const float gs[2] = {__ldg(a.k_gs), __ldg(a.v_gs)};
    const int blocks = 2 * a.heads * B, step = 1 << a.lane_shift;
    for (; c < blocks; c += 2 * step) {
        // two blocks' loads before either's arithmetic
        uint4 in[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c + i * step < blocks) {
                const BlockPlace<B> p(a, c + i * step, slot);
                const uint4* src = (p.side ? a.v + t * a.v_stride : a.k + t * a.k_stride) + 2 * p.rest;
                in[i][0] = ld_act(src);
                in[i][1] = ld_act(src + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c + i * step >= blocks) break;
            const BlockPlace<B> p(a, c + i * step, slot);
            float x[8], y[8];
            unpack16<E>(in[i][0], in[i][1], x, y);
            const float amax = max_abs8(max_abs8(0.0f, x), y);
            const float g = p.side ? gs[1] : gs[0];
            const uint32_t sb = e4m3x2(__fmul_rn(__fdiv_rn(amax, 6.0f), g), 0.0f) & 0x7fu;
            const float r = sb == 0u ? 0.0f : __fdiv_rn(g, e4m3_value_nonneg(sb));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __fmul_rn(x[j], r);
                y[j] = __fmul_rn(y[j], r);
            }
            *reinterpret_cast<uint2*>(p.codes) = make_uint2(e2m1x8(x), e2m1x8(y));
            *p.scale = static_cast<uint8_t>(sb);
        }
    }
}

// Load: value = T((q * d) / gs) with q * d exact in fp32; zero for a token
// whose slot is outside the cache.  The correctly rounded quotient lies
// between the products with the two ends of a bracket around 1 / gs (2^-18
// wide, far above the roundings involved), and rounding to T is monotone, so
// where both ends round to the same T that is the result; otherwise (about
// one block in a thousand) the block is divided out.
template <class E, int B>
__global__ void __launch_bounds__(256, 4) cache_load_kernel(CacheArgs a) {
    allow_dependents();
    grid_dependency_wait();
    int t, c;
    if (!cache_place(a, t, c)) return;
    const int64_t slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
    const bool inside = slot >= 0 && slot < a.slots_total;
    const float gs[2] = {__ldg(a.k_gs), __ldg(a.v_gs)};
    const Fp8Recips rc[2] = {fp8_recips(gs[0]), fp8_recips(gs[1])};
    const int blocks = 2 * a.heads * B, step = 1 << a.lane_shift;
    for (; c < blocks; c += 2 * step) {
        // two blocks' loads before either's arithmetic
        uint2 codes[2];
        uint32_t scale[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            codes[i] = make_uint2(0u, 0u);
            scale[i] = 0u;
            if (inside && c + i * step < blocks) {
                const BlockPlace<B> p(a, c + i * step, slot);
                codes[i] = __ldg(reinterpret_cast<const uint2*>(p.codes));
                scale[i] = __ldg(p.scale);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c + i * step >= blocks) break;
            const int side = c + i * step >= a.heads * B, rest = c + i * step - side * a.heads * B;
            uint4* dst = const_cast<uint4*>(side ? a.v + t * a.v_stride : a.k + t * a.k_stride) + 2 * rest;
            const float d = nvfp4_scale_value(scale[i]), g = side ? gs[1] : gs[0];
            const float dn = side ? rc[1].rdn : rc[0].rdn, up = side ? rc[1].rup : rc[0].rup;
            // outside this range the bracket's ends would be subnormal or infinite
            uint32_t w[8], pair[8], diff = !(g >= 7.8886091e-31f && g <= 1.2676506e30f);
            e2m1x8_f16x2(codes[i].x, *reinterpret_cast<uint32_t(*)[4]>(&pair[0]));
            e2m1x8_f16x2(codes[i].y, *reinterpret_cast<uint32_t(*)[4]>(&pair[4]));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = mul2_rn(make_float2(Fp16T::lo(pair[j]), Fp16T::hi(pair[j])), make_float2(d, d));
                const float2 lo = mul2_rn(v, make_float2(dn, dn)), hi = mul2_rn(v, make_float2(up, up));
                w[j] = E::pack(lo.x, lo.y);
                diff |= w[j] ^ E::pack(hi.x, hi.y);
            }
            if (diff) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = E::pack(__fdiv_rn(__fmul_rn(Fp16T::lo(pair[j]), d), g),
                                   __fdiv_rn(__fmul_rn(Fp16T::hi(pair[j]), d), g));
            }
            if (!inside) {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0u;
            }
            st_stream(dst, make_uint4(w[0], w[1], w[2], w[3]));
            st_stream(dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
        }
    }
}

namespace {

int page_shift_of(int64_t page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == (1 << s)) return s;
    return -1;
}

// The checks the store and the load share; fills the launch arguments.
int cache_args(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slot_map, const float* k_gs,
               const float* v_gs, const void* cache, int64_t num_pages, int64_t page_size, int64_t n, int heads,
               int head_dim, int dtype, CacheArgs* a) {
    if (dtype != RMSQ_BF16 && dtype != RMSQ_FP16) return RMSQ_ERR_INVALID_ARG;
    if (n < 0 || heads <= 0 || num_pages <= 0) return RMSQ_ERR_INVALID_ARG;
    if (page_shift_of(page_size) < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256) || heads > 4096 ||
        n > INT32_MAX || num_pages > INT32_MAX)
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    if (k_stride < row || v_stride < row || k_stride > INT32_MAX || v_stride > INT32_MAX) return RMSQ_ERR_INVALID_ARG;
    if (n == 0) return RMSQ_OK;
    if (!k || !v || !slot_map || !k_gs || !v_gs || !cache) return RMSQ_ERR_INVALID_ARG;
    using rmsq_abi::aligned;
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8 || !aligned(slot_map, 8) || !aligned(k_gs, 4) ||
        !aligned(v_gs, 4) || !aligned(cache, 16))
        return RMSQ_ERR_ALIGNMENT;
    a->k = static_cast<const uint4*>(k);
    a->v = static_cast<const uint4*>(v);
    a->k_stride = k_stride / 8;
    a->v_stride = v_stride / 8;
    a->slots = slot_map;
    a->k_gs = k_gs;
    a->v_gs = v_gs;
    a->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
    a->slots_total = num_pages * page_size;
    a->n = static_cast<int>(n);
    a->heads = heads;
    a->blocks = head_dim / 16;
    a->page_shift = page_shift_of(page_size);
    return RMSQ_OK;
}

// Spans of the token rows [n, stride], of the cache and of the small inputs.
struct CacheSpans {
    rmsq_abi::Span k, v, cache, small[3];
};
CacheSpans cache_spans(const CacheArgs& a, const float* k_gs, const float* v_gs) {
    const size_t row = static_cast<size_t>(a.heads) * a.blocks * 32;
    auto rows = [&](const uint4* p, int64_t stride) {
        return rmsq_abi::span(p, static_cast<size_t>(a.n - 1) * stride * 16 + row);
    };
    const size_t tile = static_cast<size_t>(a.blocks) * 9 << a.page_shift;
    return {rows(a.k, a.k_stride), rows(a.v, a.v_stride),
            rmsq_abi::span(a.cache, (a.slots_total >> a.page_shift) * 2 * a.heads * tile),
            {rmsq_abi::span(a.slots, static_cast<size_t>(a.n) * 8), rmsq_abi::span(k_gs, 4), rmsq_abi::span(v_gs, 4)}};
}

cudaError_t launch_cache(bool store, bool fp16, CacheArgs& a, cudaStream_t stream) {
    const void* fn;
#define RMSQ_CACHE_KERNEL(B)                                                                                     \
    (store ? (fp16 ? (const void*)&cache_store_kernel<Fp16T, B> : (const void*)&cache_store_kernel<Bf16T, B>)    \
           : (fp16 ? (const void*)&cache_load_kernel<Fp16T, B> : (const void*)&cache_load_kernel<Bf16T, B>))
    switch (a.blocks) {
    case 4: fn = RMSQ_CACHE_KERNEL(4); break;
    case 8: fn = RMSQ_CACHE_KERNEL(8); break;
    default: fn = RMSQ_CACHE_KERNEL(16); break;
    }
#undef RMSQ_CACHE_KERNEL
    a.lane_shift = 3;   // the smallest token: one head of 64, keys and values
    while (a.lane_shift < 5 && (1 << a.lane_shift) < 2 * a.heads * a.blocks) ++a.lane_shift;
    const int64_t grid = ((static_cast<int64_t>(a.n) << a.lane_shift) + 255) / 256;
    void* params[] = {&a};
    return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(256), params, 0, stream);
}

}  // namespace
}  // namespace rmsq

extern "C" {

int rmsq_build_slot_map(const int32_t* context_lens, const int32_t* query_lens, int32_t* block_table, int64_t table_width,
                        const int32_t* free_pages, int64_t free_capacity, const int32_t* num_free, int64_t page_size,
                        int64_t num_requests, int64_t max_tokens, int64_t* slot_map, int64_t* positions,
                        int32_t* query_start, int32_t* seq_lens, int32_t* num_free_out, int32_t* status, void* stream) {
    using rmsq_abi::aligned;
    using rmsq_abi::overlaps;
    using rmsq_abi::Span;
    using rmsq_abi::span;
    if (num_requests < 0 || max_tokens < 0 || table_width < 0 || free_capacity < 0) return RMSQ_ERR_INVALID_ARG;
    const int shift = rmsq::page_shift_of(page_size);
    // positions and slots inside a request stay below 2^31
    if (shift < 0 || num_requests > RMSQ_MAX_REQUESTS || max_tokens > INT32_MAX / 2 || free_capacity > INT32_MAX ||
        table_width > (INT32_MAX >> shift))
        return RMSQ_ERR_UNSUPPORTED_SHAPE;
    if (!num_free || !query_start || !num_free_out || !status) return RMSQ_ERR_INVALID_ARG;
    if (num_requests > 0 && (!context_lens || !query_lens || !seq_lens || (table_width > 0 && !block_table)))
        return RMSQ_ERR_INVALID_ARG;
    if ((free_capacity > 0 && !free_pages) || (max_tokens > 0 && (!slot_map || !positions))) return RMSQ_ERR_INVALID_ARG;
    if (!aligned(context_lens, 4) || !aligned(query_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
        !aligned(num_free, 4) || !aligned(slot_map, 8) || !aligned(positions, 8) || !aligned(query_start, 4) ||
        !aligned(seq_lens, 4) || !aligned(num_free_out, 4) || !aligned(status, 4))
        return RMSQ_ERR_ALIGNMENT;
    const size_t R = static_cast<size_t>(num_requests), T = static_cast<size_t>(max_tokens);
    const Span ins[4] = {span(context_lens, R * 4), span(query_lens, R * 4),
                         span(free_pages, static_cast<size_t>(free_capacity) * 4), span(num_free, 4)};
    const Span outs[7] = {span(block_table, R * static_cast<size_t>(table_width) * 4), span(slot_map, T * 8),
                          span(positions, T * 8), span(query_start, (R + 1) * 4), span(seq_lens, R * 4),
                          span(num_free_out, 4), span(status, 4)};
    for (int i = 0; i < 7; ++i) {
        for (const Span& in : ins)
            if (overlaps(outs[i], in)) return RMSQ_ERR_ALIAS;
        for (int j = i + 1; j < 7; ++j)
            if (overlaps(outs[i], outs[j])) return RMSQ_ERR_ALIAS;
    }
    const int st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    rmsq::SlotArgs a = {context_lens, query_lens, block_table, free_pages, num_free, slot_map, positions, query_start,
                        seq_lens, num_free_out, status, static_cast<int>(num_requests), static_cast<int>(table_width),
                        static_cast<int>(free_capacity), shift, static_cast<int>(max_tokens)};
    const void* fn = (const void*)&rmsq::slot_map_kernel;
    const int smem = static_cast<int>(2 * (num_requests + 1) * 4);
    cudaError_t e;
    const int sms = rmsq::sm_count(&e);
    if (e == cudaSuccess && smem > 40 * 1024)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * (RMSQ_MAX_REQUESTS + 1) * 4);
    if (e != cudaSuccess) return rmsq_abi::fail_cuda(e);
    const int64_t most = max_tokens > num_requests + 1 ? max_tokens : num_requests + 1;
    int64_t grid = (most + rmsq::kSlotThreads - 1) / rmsq::kSlotThreads;
    if (grid > sms) grid = sms;
    void* params[] = {&a};
    e = rmsq::launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(rmsq::kSlotThreads), params, smem,
                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

int rmsq_kv_cache_store_nvfp4(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slot_map,
                              const float* k_global_scale, const float* v_global_scale, void* kv_cache, int64_t num_pages,
                              int64_t page_size, int64_t n_tokens, int num_kv_heads, int head_dim, int dtype,
                              void* stream) {
    rmsq::CacheArgs a = {};
    int st = rmsq::cache_args(k, k_stride, v, v_stride, slot_map, k_global_scale, v_global_scale, kv_cache, num_pages,
                              page_size, n_tokens, num_kv_heads, head_dim, dtype, &a);
    if (st != RMSQ_OK || n_tokens == 0) return st;
    const rmsq::CacheSpans s = rmsq::cache_spans(a, k_global_scale, v_global_scale);
    if (rmsq_abi::overlaps(s.cache, s.k) || rmsq_abi::overlaps(s.cache, s.v)) return RMSQ_ERR_ALIAS;
    for (const rmsq_abi::Span& in : s.small)
        if (rmsq_abi::overlaps(s.cache, in)) return RMSQ_ERR_ALIAS;
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    const cudaError_t e = rmsq::launch_cache(true, dtype == RMSQ_FP16, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

int rmsq_kv_cache_load_nvfp4(const void* kv_cache, int64_t num_pages, int64_t page_size, const int64_t* slot_map,
                             const float* k_global_scale, const float* v_global_scale, void* k, int64_t k_stride, void* v,
                             int64_t v_stride, int64_t n_tokens, int num_kv_heads, int head_dim, int dtype, void* stream) {
    rmsq::CacheArgs a = {};
    int st = rmsq::cache_args(k, k_stride, v, v_stride, slot_map, k_global_scale, v_global_scale, kv_cache, num_pages,
                              page_size, n_tokens, num_kv_heads, head_dim, dtype, &a);
    if (st != RMSQ_OK || n_tokens == 0) return st;
    const rmsq::CacheSpans s = rmsq::cache_spans(a, k_global_scale, v_global_scale);
    // k and v may be two column ranges of one token-major buffer: their rows
    // interleave without sharing an element
    const bool columns = a.k_stride == a.v_stride && rmsq::disjoint_columns(a.k, a.v, a.k_stride, a.heads * a.blocks * 2);
    if (rmsq_abi::overlaps(s.k, s.v) && !columns) return RMSQ_ERR_ALIAS;
    const rmsq_abi::Span outs[2] = {s.k, s.v};
    for (const rmsq_abi::Span& o : outs) {
        if (rmsq_abi::overlaps(o, s.cache)) return RMSQ_ERR_ALIAS;
        for (const rmsq_abi::Span& in : s.small)
            if (rmsq_abi::overlaps(o, in)) return RMSQ_ERR_ALIAS;
    }
    st = rmsq_abi::check_device();
    if (st != RMSQ_OK) return st;
    const cudaError_t e = rmsq::launch_cache(false, dtype == RMSQ_FP16, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RMSQ_OK : rmsq_abi::fail_cuda(e);
}

}  // extern "C"
