// Attention over a paged cache for many queries per request (prompts), on the
// fifth-generation tensor cores; the NVFP4 cache's reader (the FP8 cache's is in
// rmsq_attn8.cuh).  The mathematics, the f16 operands and
// the scaling of queries and probabilities are those of rmsq_attn.cuh.
//
// A CTA takes 256 rows (query token, head of the group) of a request and kv
// head as two tiles of 128 (or one, see find_item), and walks the keys 128 at a time:
//   S = Q . K^T (128 x 128 x D)  ->  P = 2^(f (S - m))  ->  O += P . V (128 x D x 128)
// with S, P (f16, in S's place) and O in tensor memory, a thread per row in the
// softmax.  While one tile is in its softmax the matrix unit works for the
// other.  Four warps turn the cache's codes into f16 operand tiles in shared
// memory, once for both tiles: a key per thread for K; 8 keys x D/8 dims per
// thread for V, whose nibbles are interleaved pairwise so that eight keys of a
// dim come out as one 16-byte piece of V^T, the layout the product wants.
//
// Bound by the matrix unit in the limit (4 D flop per row and key; 16 products
// of 72 clocks per tile and 128 keys at D = 128), and at present by two things.
// One is the chain of a tile: its products (1150 clocks), the hand-over (200), its
// softmax (2100: 520 to read the logits, 330 for the maximum, 1040 for the
// weights, the rest hand-over) and the next products; two tiles hide half of
// that.  128 keys take 1.66 us on a context of 20000 (1.70 with all products of a
// tile unrolled).  The other
// is what lies outside it: a CTA has all of tensor memory, so the next one's
// request, queries and first conversion, and the last one's output, overlap with
// nothing (8 to 10 us a CTA: 128 queries of 8 x 8 heads take 12 us on 128 keys and
// 74 on 4000).  2478 and 2445 queries of 32 heads on contexts of 732 and 1574
// keys: 198 us, 192 GFLOP (0.97 PFLOP/s; half the measured bf16 rate, 101 us), of
// which the 80 steps of an SM are 133 and the starts and ends of its 4.1 CTAs and
// the last round the rest.  Heads of 64: 2000 queries of 32 heads on 4000 keys 88
// us, of 128 115.  Measured and not kept (against
// 212 to 215 us): two threads per row (326: 88 registers a thread spill), one
// issuing warp per tile (260, the two fall into step), the logits of 64 keys
// in two buffers so that products run ahead (268: a product of 64 columns takes as
// long as one of 128), weights handed over in halves (226), weights taken before
// the maximum is known and again where it moves (231), logits read twice instead
// of held (259), the next tile's codes in registers of their own (215, spilling).
//
// Every wait is bounded, as in the matrix product.
#pragma once

#include <type_traits>

#include "rmsq.h"
#include "rmsq_attn.cuh"
#include "rmsq_tc.cuh"

namespace rmsq {

static __device__ unsigned int g_prompt_fault;

// Four warpgroups: two for the softmax, one converting, one whose first two
// warps issue.  They are launched with 128 registers a thread and share them out
// anew: 176 + 176 + 120 + 40 = 4 x 128.
constexpr int kPromptThreads = 512;
constexpr int kSoftmaxGroups = 2;
constexpr int kSoftmaxRegs = 176, kConvertRegs = 120, kIssueRegs = 40;
static_assert(2 * kSoftmaxRegs + kConvertRegs + kIssueRegs == 4 * 128, "the shares are the launch's registers");

template <int D>
struct PromptTile {
    static constexpr int q = 128 * D * 2, k = 128 * D * 2, v = 128 * D * 2;    // bytes of one operand tile
    // one CTA per SM in any case: it takes all of tensor memory
    static constexpr int with_ring(int ring) { return 1024 + (6 * q + ring > 120 * 1024 ? 6 * q + ring : 120 * 1024); }
    static constexpr int smem = 1024 + (6 * q > 120 * 1024 ? 6 * q : 120 * 1024);
    static_assert(smem - 1024 - 2 * q >= (RMSQ_MAX_REQUESTS + 1) * 8, "the scan fits behind the queries");
};

// Instruction descriptor: f16 x f16 -> fp32, both K-major, 128 x N.
template <int N>
constexpr uint32_t kF16Idesc = (1u << 4) | (static_cast<uint32_t>(N / 8) << 17) | ((128u / 16u) << 24);

// D = A . B^T over STEPS steps of 16 along K; A and B in swizzled tiles (low
// descriptor words) whose 64-element column blocks are A_BLOCK / B_BLOCK bytes
// apart.
template <int N, int STEPS, int A_BLOCK, int B_BLOCK>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll 4
    for (int i = 0; i < STEPS; ++i)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                     :: "r"(d), "r"(a + (i >> 2) * (A_BLOCK >> 4) + (i & 3) * 2),
                        "r"(b + (i >> 2) * (B_BLOCK >> 4) + (i & 3) * 2), "r"(kF16Idesc<N>), "r"(i), "n"(kTileDescHigh)
                     : "memory");
}

// D (+)= A . B^T with A in tensor memory (8 columns per step).
template <int N, int STEPS, int B_BLOCK>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, bool add) {
#pragma unroll 4
    for (int i = 0; i < STEPS; ++i)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
                     :: "r"(d), "r"(a + 8 * i), "r"(b + (i >> 2) * (B_BLOCK >> 4) + (i & 3) * 2), "r"(kF16Idesc<N>),
                        "r"(i > 0 || add ? 1 : 0), "n"(kTileDescHigh)
                     : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A converting thread's share of a 128-key tile, as it lies in the cache.
template <int D>
struct RawTile {
    static constexpr int KW = D / 8;        // words of the thread's key
    static constexpr int VW = D / 64;       // words of each of its 8 keys' values (D/8 dims)
    uint32_t k[KW], ks[D / 64], v[8][VW], vs[8];
};

template <int D>
__device__ __forceinline__ void load_keys(RawTile<D>& x, const AttnArgs& a, int key, int kpage, int head) {
    const int64_t tile = static_cast<int64_t>(D / 16 * 9) << a.page_shift;
    if (kpage >= 0) {
        const uint8_t* t = a.cache + (static_cast<int64_t>(kpage) * 2 * a.kv_heads + head) * tile;
        const int in = key & ((1 << a.page_shift) - 1);
        const uint4* p = reinterpret_cast<const uint4*>(t + in * (D / 2));
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const uint4 u = __ldg(p + j);
            x.k[4 * j] = u.x; x.k[4 * j + 1] = u.y; x.k[4 * j + 2] = u.z; x.k[4 * j + 3] = u.w;
        }
        const uint32_t* s = reinterpret_cast<const uint32_t*>(t + ((D / 2) << a.page_shift) + in * (D / 16));
#pragma unroll
        for (int j = 0; j < D / 64; ++j) x.ks[j] = __ldg(s + j);
    } else {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) x.k[j] = 0u;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) x.ks[j] = 0u;
    }
}

template <int D>
__device__ __forceinline__ void load_values(RawTile<D>& x, const AttnArgs& a, int key, int vpage, int head, int unit) {
    const int64_t tile = static_cast<int64_t>(D / 16 * 9) << a.page_shift;
    const uint8_t* t = a.cache + ((static_cast<int64_t>(max(vpage, 0)) * 2 + 1) * a.kv_heads + head) * tile;
    const int in = key & ((1 << a.page_shift) - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (vpage >= 0) {
            const uint8_t* p = t + (in + i) * (D / 2) + unit * (D / 16);
            if constexpr (D == 128) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
                x.v[i][0] = u.x; x.v[i][1] = u.y;
            } else {
                x.v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            }
            x.vs[i] = __ldg(t + ((D / 2) << a.page_shift) + (in + i) * (D / 16) + unit * (D / 8) / 16);
        } else {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) x.v[i][j] = 0u;
            x.vs[i] = 0u;
        }
    }
}

// K of the thread's key as a row of the operand tile.
template <int D>
__device__ __forceinline__ void write_keys(unsigned char* dst, const RawTile<D>& x, int row) {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        uint32_t lo[4], hi[4];
        e2m1x8_f16x2(x.k[2 * j], lo);
        e2m1x8_f16x2(x.k[2 * j + 1], hi);
        const uint32_t s = dup_half(e4m3x2_f16x2(x.ks[j / 4] >> (8 * (j & 2))), j & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = mul_f16x2(lo[i], s);
            hi[i] = mul_f16x2(hi[i], s);
        }
        unsigned char* r = dst + (j >> 2) * (128 * 128) + row * 128;
        const int c = (j & 3) * 2;
        *reinterpret_cast<uint4*>(r + ((c ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(r + (((c + 1) ^ (row & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// V of the thread's 8 keys and D/8 dims as 16-byte pieces of V^T's rows.
template <int D>
__device__ __forceinline__ void write_values(unsigned char* dst, const RawTile<D>& x, int octet, int unit) {
    uint32_t sc[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) sc[p] = e4m3x2_f16x2(x.vs[2 * p] | (x.vs[2 * p + 1] << 8));
    unsigned char* base = dst + (octet >> 3) * (D * 128);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        uint32_t even[4][4], odd[4][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t A = x.v[2 * p][j], B = x.v[2 * p + 1][j];
            e2m1x8_f16x2((A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u), even[p]);
            e2m1x8_f16x2(((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u), odd[p]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                even[p][c] = mul_f16x2(even[p][c], sc[p]);
                odd[p][c] = mul_f16x2(odd[p][c], sc[p]);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = unit * (D / 8) + 8 * j + 2 * c;
            *reinterpret_cast<uint4*>(base + row * 128 + (((octet & 7) ^ (row & 7)) << 4)) =
                make_uint4(even[0][c], even[1][c], even[2][c], even[3][c]);
            *reinterpret_cast<uint4*>(base + (row + 1) * 128 + (((octet & 7) ^ ((row + 1) & 7)) << 4)) =
                make_uint4(odd[0][c], odd[1][c], odd[2][c], odd[3][c]);
        }
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// What a reader with block_scales tells of a step: the 128 keys it is about and
// which of them it takes, the factor of their logits and the byte of their values'
// scale (as a number; 0: there is none), whether it is the last one, and the eight blocks'
// pages (-1: not taken) and the f16 factors of their keys and values.
struct StepInfo {
    uint32_t valid[4];
    float k, v;
    int key0, last;
    int page[8];
    uint32_t fk[8], fv[8];
};

template <int D>
struct Nvfp4Prompt : Nvfp4Cache {
    static constexpr int ring = 0;      // it loads into registers
};

// A row's 128 logits.  They stay in registers from the maximum to the weights:
// read from tensor memory twice, 16 at a time, the two passes waited out
// sixteen load latencies per tile (260 us for the prompt step of 147 GFLOP).
using Row = float[8][16];

// A stage that is not a constant.
struct StageOf {
    int value;
};

// Half h (0, 1) of a row: 64 logits.
__device__ __forceinline__ void start_half(Row& d, uint32_t s_at, int h) {
#pragma unroll
    for (int c = 0; c < 4; c += 2) tmem_ld32(d[4 * h + c], d[4 * h + c + 1], s_at + (4 * h + c) * 16);
}
__device__ __forceinline__ void finish_half(Row& d, int h) {
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_wait(d[4 * h + c]);    // the first one waits for all
}

// Logits whose bit is not set in `see` to -inf.
__device__ __forceinline__ void mask_half(Row& d, int h, const uint32_t (&see)[4]) {
#pragma unroll
    for (int c = 4 * h; c < 4 * h + 4; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (!(see[c >> 1] >> ((c & 1) * 16 + j) & 1u)) d[c][j] = -INFINITY;
}

__device__ __forceinline__ float max_half(const Row& d, int h) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 4 * h; c < 4 * h + 4; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) top[j & 3] = max3(top[j & 3], d[c][2 * j], d[c][2 * j + 1]);
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// The half's weights 2^(f s + shift) in f16, in the place of the row's logits
// in tensor memory; returns their sum.
__device__ __forceinline__ float weigh_half(const Row& d, int h, uint32_t s_at, float f, float shift) {
    const float2 f2 = make_float2(f, f), s2 = make_float2(shift, shift);
    float2 sum[2] = {};
#pragma unroll
    for (int c = 2 * h; c < 2 * h + 2; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float(&x16)[16] = d[2 * c + (j >> 3)];
            float2 x = fma2_rn(make_float2(x16[2 * (j & 7)], x16[2 * (j & 7) + 1]), f2, s2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            sum[j & 1] = add2_rn(sum[j & 1], x);
            p[j] = Fp16T::pack(x.x, x.y);
        }
        tmem_st16(s_at + c * 16, p);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The CTA's item, counted from its request's first one, and the request; -1 if
// there are not that many.  Up to 32 requests every warp finds it for itself, a
// lane per request; more are scanned in `scratch` (the key and value tiles' space,
// which is theirs on return).
//
// An item has 256 rows, or 128 where all items of 128 fit the card's SMs at once: a
// CTA then has one row tile, whose step is shorter, and a prompt twice the CTAs.  In
// us for 256 and 128 (FP8, heads of 128): 452 queries of 4 x 4 heads on 1510 keys (60
// CTAs of 128 rows) 34.6 28.3, 600 of 8 x 4 on 2000 (152) 42.5 36.2, 900 (228) 42.5
// 55.7, 280 of 8 x 8 on 20000 (144) 309 284, 320 (160) 309 529; heads of 64, 1100 of 4 x
// 4 on 1500 (140) 25.9 22.7, 320 of 8 x 8 on 20000 240 418 (the taken ones are up to
// 1.5 % longer now: 28.8, 36.7, 290).  More than 32 requests are scanned by all
// threads with a barrier each time, for items of 256 rows first; a second scan, for
// 128, is made only where it is sure to fit, at most twice as many: between half of
// the card's SMs and all of them a batch of so many requests keeps its 256.  `shift`:
// log2 of the rows.
__device__ __forceinline__ int64_t find_item(const AttnArgs& a, int64_t* scratch, int& req, int& shift) {
    const int skip = static_cast<int>(blockIdx.x) / a.kv_heads;
    if (a.requests <= 32) {
        const int lane = threadIdx.x & 31;
        int rows = 0, own = 0, n = 0;
        if (lane < a.requests) {
            const Req x = load_request(a, lane);
            rows = x.qlen * a.group;
            own = 31 - __clz(x.ktiles);
        }
        const bool open = rows > a.most_rows;
        const uint32_t all = __ballot_sync(kFull, open);
        if (a.share != 0)
#pragma unroll 1
            for (uint32_t rest = all; rest != 0; rest &= rest - 1) n += __shfl_sync(kFull, own, __ffs(rest) - 1) >= own;
        if (!open || (a.share != 0 && static_cast<int64_t>(rows) * n < a.share)) rows = 0;
        const int halves = (rows + 127) >> 7;
        shift = __reduce_add_sync(kFull, min(halves, 1 << 24)) <= a.half_items ? 7 : 8;
        const int items = shift == 7 ? halves : (halves + 1) >> 1;
        int inc = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        const int item = __shfl_sync(kFull, inc, 31) - 1 - skip;
        if (item < 0) return -1;
        req = __ffs(__ballot_sync(kFull, inc > item)) - 1;
        return item - __shfl_sync(kFull, inc - items, req);
    }
    auto scan = [&](int rows) {
        scan_requests<kPromptThreads, false, 0>(a, scratch, [rows](int64_t r, bool taken) { return taken ? (r + rows - 1) / rows : 0; });
    };
    shift = 8;
#pragma unroll 1
    for (;;) {
        scan(1 << shift);
        const int64_t total = scratch[a.requests];
        if (shift == 7 || total == 0 || 2 * total > a.half_items) break;    // (at most twice as many of 128)
        shift = 7;
        __syncthreads();    // the total has been read
    }
    int64_t item = scratch[a.requests] - 1 - skip;
    if (item >= 0) {
        int hi = a.requests;
        while (hi - req > 1) {
            const int mid = (req + hi) >> 1;
            if (scratch[mid] <= item) req = mid;
            else hi = mid;
        }
        item -= scratch[req];
    }
    __syncthreads();    // the scan has been read
    return item < 0 ? -1 : item;
}

template <class P, class E, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) attn_prompt_kernel(AttnArgs a) {
    using Tile = PromptTile<D>;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t qfull[2], kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pready[2],
        ofull[2], drained;
    __shared__ __align__(16) uint32_t valid[4][4];  // which keys of a tile lie on a page, four tiles deep
    __shared__ __align__(16) StepInfo info[P::block_scales ? 8 : 1];
    __shared__ __align__(8) uint64_t rawfull[2], rawempty[2];     // block_scales: the ring of raw keys
    __shared__ uint32_t tmem_base;
    unsigned char* qs = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    unsigned char* ks = qs + 2 * Tile::q;
    unsigned char* vs = ks + 2 * Tile::k;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 4);
            mbar_init(&kfull[i], 4);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], 4);
            mbar_init(&vempty[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 4);
            mbar_init(&ofull[i], 1);
        }
        mbar_init(&drained, 1);
        if constexpr (P::block_scales) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&rawfull[i], 1);
                mbar_init(&rawempty[i], 4);
            }
        }
        fence_mbar_init();
    }
    grid_dependency_wait();

    // The item of this CTA: tiles of a request from the last rows (most keys)
    // to the first, kv heads innermost.
    const int head = blockIdx.x % a.kv_heads;
    int req = 0, shift = 8;
    const int64_t item = find_item(a, reinterpret_cast<int64_t*>(ks), req, shift);
    const int row0 = static_cast<int>(item) << shift;
    if (item < 0) {
        allow_dependents();
        return;
    }
    if (warp == 12) tmem_alloc(&tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    allow_dependents();
    const uint32_t tmem = tmem_base;

    const Req rq = load_request(a, req);
    const int rows = rq.qlen * a.group, first_pos = rq.seq - rq.qlen;
    const int end_row = min(rows - row0, 1 << shift) + row0;
    const int tiles = end_row - row0 > 128 ? 2 : 1;
    const int last_pos = first_pos + (end_row - 1) / a.group;
    const int low_pos = first_pos + row0 / a.group;
    const int low_key = a.window > 0 ? max(low_pos - a.window + 1, 0) : 0;
    const int key_begin = low_key / 128 * 128;
    const int tiles128 = last_pos < key_begin ? 0 : (last_pos - key_begin) / 128 + 1;
    // With block_scales a tile may take several steps, and their number is known
    // when the last one comes.
    int steps = P::block_scales && tiles128 > 0 ? INT32_MAX - 1 : tiles128;
    bool ok = true;

    if (warp >= 12) {
        fewer_registers<kIssueRegs>();
        if (warp == 12 && steps > 0) {
            // The whole warp walks the loop, so that its addresses stay
            // uniform, and twice a round, so that its stages are constants
            // (with block_scales once, and a tile after the other: the roles' code
            // together does not fit the instruction cache there, and a step of
            // 128 keys took 2.49 us with all SMs at work and 1.89 with a fifth of
            // them, so 1.96 either way); one lane issues.  Tile by tile: O += P . V of the step before, then
            // S = Q . K^T of this one.  (One issuing warp per tile let the two
            // fall into step, both tiles' softmax at once and then both tiles'
            // products: 260 us instead of 212 for the prompt step.)
            const bool issuer = elect_one();
            const uint32_t q_desc = tile_desc(smem_u32(qs)), k_desc = tile_desc(smem_u32(ks)), v_desc = tile_desc(smem_u32(vs));
            for (int i = 0; i < tiles && ok; ++i) ok = mbar_wait(&qfull[i], 0);
            ok = __all_sync(kFull, ok);
            auto step = [&](auto stage, int n) {
                const int s = stage.value, z = s ^ 1;
                if (n < steps) ok = ok && mbar_wait(&kfull[s], (n >> 1) & 1);
                if (n > 0) ok = ok && mbar_wait(&vfull[z], ((n - 1) >> 1) & 1);
#pragma unroll (P::block_scales ? 1 : 2)
                for (int i = 0; i < 2; ++i) {
                    if (i >= tiles) break;
                    const uint32_t s_at = tmem + i * 128, o_at = tmem + 256 + i * D;
                    if (n > 0) {
                        ok = ok && mbar_wait(&pready[i], z);
                    }
                    ok = __all_sync(kFull, ok);
                    if (!ok) return;
                    tc_fence_after();
                    if (issuer) {
                        if (n > 0) mma_f16_ts<D, 8, D * 128>(o_at, s_at, v_desc + z * (Tile::v >> 4), n > 1);
                        if (n < steps) {
                            mma_f16_ss<128, D / 16, 128 * 128, 128 * 128>(s_at, q_desc + i * (Tile::q >> 4),
                                                                          k_desc + s * (Tile::k >> 4));
                            mma_commit(&sfull[i]);
                        } else {
                            mma_commit(&ofull[i]);
                        }
                        if (i == tiles - 1) {
                            if (n > 0) mma_commit(&vempty[z]);
                            if (n < steps) mma_commit(&kempty[s]);
                        }
                    }
                }
            };
            if constexpr (P::block_scales) {
#pragma unroll 1
                for (int n = 0; n <= steps && ok; ++n) {
                    step(StageOf{n & 1}, n);
                    if (ok && n < steps && info[n & 7].last) steps = n + 1;     // (read behind the products)
                }
            } else {
                for (int n = 0; n <= steps && ok; n += 2) {
                    step(std::integral_constant<int, 0>{}, n);
                    if (ok && n < steps) step(std::integral_constant<int, 1>{}, n + 1);
                }
            }
            if (!ok && issuer) {
                mma_commit(&drained);
                mbar_wait(&drained, 0);
            }
        }
        if constexpr (P::block_scales) {
            if (warp == 13 && steps > 0)
                ok = P::fetch(a, req, head, key_begin, last_pos, tiles128, qs + 6 * Tile::q, rawfull, rawempty, info);
        }
    } else if (warp >= 8) {
        fewer_registers<kConvertRegs>();
        if constexpr (P::block_scales) {
            if (steps > 0)
                ok = P::convert(a, head, qs + 6 * Tile::q, ks, vs, rawfull, rawempty, kfull, kempty, vfull, vempty, info);
        } else {
            // Conversion.  The codes of the next tile are loaded into the registers
            // that this one's have just left, the pages a tile before that.
            const int t = tid - 128 * kSoftmaxGroups, w = warp - 4 * kSoftmaxGroups;
            const int octet = (w & 1) * 8 + (lane & 7), unit = (w >> 1) * 4 + (lane >> 3);
            const int* table = a.table + static_cast<int64_t>(req) * a.width;
            // A page is compared with their number only when it is used: next to
            // the load the comparison would make the warp wait for it every time.
            auto page_of = [&](int key) { return key > last_pos ? -1 : __ldg(table + (key >> a.page_shift)); };
            auto checked = [&](int p) { return p < a.num_pages ? p : -1; };
            RawTile<D> raw;
            int kkey = key_begin + t, vkey = key_begin + octet * 8;
            bool here = checked(page_of(kkey)) >= 0;
            load_keys<D>(raw, a, kkey, checked(page_of(kkey)), head);
            load_values<D>(raw, a, vkey, checked(page_of(vkey)), head, unit);
            int kp = page_of(kkey + 128), vp = page_of(vkey + 128);
            for (int n = 0; n < steps; ++n) {
                const int s = n & 1;
                kkey += 128;
                vkey += 128;
                ok = warp_wait(&kempty[s], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                const uint32_t there = __ballot_sync(kFull, here);
                if (lane == 0) valid[n & 3][w] = there;
                write_keys<D>(ks + s * Tile::k, raw, t);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&kfull[s]);
                kp = checked(kp);
                here = kp >= 0;
                load_keys<D>(raw, a, kkey, kp, head);
                kp = page_of(kkey + 128);
                ok = warp_wait(&vempty[s], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                write_values<D>(vs + s * Tile::v, raw, octet, unit);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&vfull[s]);
                load_values<D>(raw, a, vkey, checked(vp), head, unit);
                vp = page_of(vkey + 128);
            }
        }
    } else {
        more_registers<kSoftmaxRegs>();
        const int i = warp >> 2, quad = warp & 3, local = quad * 32 + lane, row = row0 + i * 128 + local;
        if (i < tiles) {
            // The row's query: scaled into f16's range, into its operand row.
            const int token = row / a.group, qh = head * a.group + row % a.group;
            const bool live = row < rows;
            uint32_t q[D / 2];
#pragma unroll
            for (int j = 0; j < D / 2; ++j) q[j] = 0u;
            if (live) {
                const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                (rq.q0 + token) * a.q_stride + qh * D);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const uint4 u = __ldg(p + j);
                    q[4 * j] = u.x; q[4 * j + 1] = u.y; q[4 * j + 2] = u.z; q[4 * j + 3] = u.w;
                }
            }
            float f = P::block_scales ? a.scale_log2 : a.scale_log2 / __ldg(a.k_gs);
            if constexpr (E::kBits87 == Bf16T::kBits87) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 2; ++j) top = max_abs3(top, E::lo(q[j]), E::hi(q[j]));
                const int e = min(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                f *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int j = 0; j < D / 2; ++j) q[j] = Fp16T::pack(E::lo(q[j]) * up, E::hi(q[j]) * up);
            }
            f = clamp_factor(f);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<uint4*>(qs + i * Tile::q + (j >> 3) * (128 * 128) + local * 128 +
                                          (((j & 7) ^ (local & 7)) << 4)) =
                    make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[i]);

            const int pos = live ? first_pos + token : -1, lo = a.window > 0 ? pos - a.window + 1 : 0;
            const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
            const uint32_t s_at = tmem + i * 128 + lanes, o_at = tmem + 256 + i * D + lanes;
            // (block_scales: limit is what the weighted values may pass the reference by)
            Peak peak = {-INFINITY, 0.0f};
            float l = 0.0f, limit = P::block_scales ? P::lazy : -INFINITY, shift = 0.0f;
            for (int n = 0; n < steps; ++n) {
                ok = warp_wait(&sfull[i], n & 1);
                if (!ok) break;
                tc_fence_after();
                Row d;
                start_half(d, s_at, 0);
                // (read together, beside the logits: shared memory is busy with the
                // products' operands, a read takes up to 400 clocks)
                const StepInfo& at = info[P::block_scales ? n & 7 : 0];
                const uint4 have = *reinterpret_cast<const uint4*>(P::block_scales ? at.valid : valid[n & 3]);
                const uint4 rest = P::block_scales ? *reinterpret_cast<const uint4*>(&at.k) : make_uint4(0u, 0u, 0u, 0u);
                const float tile_k = __uint_as_float(rest.x);
                const float tile_v = __uint_as_float(rest.y);
                const int key0 = P::block_scales ? static_cast<int>(rest.z) : key_begin + n * 128;
                if (P::block_scales && rest.w != 0u) steps = n + 1;
                const uint32_t hv[4] = {have.x, have.y, have.z, have.w};
                const bool whole = (have.x & have.y & have.z & have.w) == 0xffffffffu;
                // keys this row may see, as bits, where not every row of the warp sees all of them
                const bool full = __all_sync(kFull, whole && (!live || (key0 + 127 <= pos && key0 >= lo)));
                uint32_t see[4] = {};
                if (!full) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k = key0 + 32 * c;
                        const int upto = min(max(pos - k + 1, 0), 32), from = min(max(lo - k, 0), 32);
                        const uint32_t below = upto == 32 ? 0xffffffffu : (1u << upto) - 1u;
                        const uint32_t above = from == 32 ? 0u : 0xffffffffu << from;
                        see[c] = below & above & hv[c];
                    }
                }
                finish_half(d, 0);
                start_half(d, s_at, 1);
                if (!full) mask_half(d, 0, see);
                float top = max_half(d, 0);
                finish_half(d, 1);
                if (!full) mask_half(d, 1, see);
                top = fmaxf(top, max_half(d, 1));
                // block_scales: log2 of the largest weighted value relative to the row's; all of
                // them far below what f16 holds
                float gain = 0.0f;
                bool high = top > limit, low = false;
                if constexpr (P::block_scales) {
                    top *= tile_k;
                    gain = above<P>({top, tile_v}, peak, f);    // (nothing yet, nothing here: NaN)
                    high = (limit == -INFINITY ? top : gain) > limit;
                    low = gain < -30.0f - P::p_shift;
                }
                float up = 0.0f;        // block_scales: what these weights are raised by
                float move = 1.0f;      // factor of the row's O
                bool moved = false;
                bool done = false;      // the factors are in the logits
                if (__any_sync(kFull, high || low)) {
                    // sfull of this step says that the previous P . V has
                    // completed too: O may be rescaled here
                    const Peak was = peak;
                    if (high) peak = higher<P>(peak, {top, tile_v}, f);     // whatever shares the warp
                    const float x = peak.m == -INFINITY ? 0.0f : above<P>(was, peak, f);
                    limit = P::block_scales ? P::lazy : lag_limit<P>(peak.m, f);
                    shift = weight_shift<P>(peak.m, f);
                    l = lowered<P>(l, x);
                    move = exp2_approx(x);
                    moved = n > 0 && (!P::block_scales || __any_sync(kFull, high));
                    // They are brought just below what f16 holds, so that the sum of the
                    // weights, in which they may be the largest, has them whole.
                    if (low) up = fminf(ceilf(-30.0f - P::p_shift - gain), 100.0f);
                    // A row that is far out comes here at every step (its limit
                    // is passed by any logit); the others subtract zero.
                    if (__any_sync(kFull, is_far(shift))) {
                        const bool own = is_far(shift);
                        const float t = own ? peak.m : 0.0f;
                        if (own) {
                            shift = P::p_shift;
                            limit = -INFINITY;
                        }
#pragma unroll
                        for (int c = 0; c < 8; ++c)
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                if constexpr (P::block_scales) d[c][j] *= tile_k;
                                d[c][j] -= t;
                            }
                        done = P::block_scales;
                    }
                }
                if constexpr (P::block_scales) {
                    // Weights times their values' scale, a power of two that only changes
                    // the addend; the sum of the weights from theirs.  (The factor within the
                    // normal numbers: a masked logit times zero would be NaN.)
                    const float fk = done ? f : clamp_factor(f * tile_k);
                    float sum = 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) sum += weigh_half(d, h, s_at, fk, shift + (tile_v - peak.e + up));
                    // 2^(middle - v - up); 0 below the normal numbers
                    const int unit = 127 + P::middle - static_cast<int>(tile_v + up);
                    l = fmaf(sum, __uint_as_float(static_cast<uint32_t>(max(unit, 0)) << 23), l);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) l += weigh_half(d, h, s_at, f, shift);
                }
                // O to the new maximum, now that the logits' registers are free: 64
                // columns at a time (16 at a time, beside the logits, was 14 us of 283 for
                // prompts of 2478 and 2445 tokens over the FP8 cache)
                if (moved) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
                        Row& o = d;
                        start_half(o, o_at + c, 0);
                        finish_half(o, 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t u[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[k][j] * move);
                            tmem_st16(o_at + c + k * 16, u);
                        }
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready[i]);
            }
            // O / l, in T
            if (ok && steps > 0) {
                ok = warp_wait(&ofull[i], 0);
                tc_fence_after();
            }
            const float inv = l > 0.0f ? 1.0f / (P::block_scales ? l : l * __ldg(a.v_gs)) : (l == 0.0f ? 0.0f : l);
            const int64_t oh = static_cast<int64_t>(rq.q0 + token) * a.heads + qh;
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + oh * D);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                float o[16];
                if (steps > 0) {
                    __syncwarp();   // the lanes come from the stores below, which not all of them make
                    tmem_ld16(o, o_at + c * 16);
                    tmem_wait(o);
                    if constexpr (P::block_scales) {    // O is in units of 2^(e - 127), l of 2^(e - middle)
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= pow2(P::middle - 127);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0.0f;
                }
                if (live && ok) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        out[2 * c + h] = make_uint4(E::pack(o[8 * h] * inv, o[8 * h + 1] * inv),
                                                    E::pack(o[8 * h + 2] * inv, o[8 * h + 3] * inv),
                                                    E::pack(o[8 * h + 4] * inv, o[8 * h + 5] * inv),
                                                    E::pack(o[8 * h + 6] * inv, o[8 * h + 7] * inv));
                }
            }
            if (live && ok && a.lse) a.lse[oh] = row_lse<P>(peak, l, f);
        }
    }
    if (!ok) atomicOr(&g_prompt_fault, 1u);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_free(tmem, 512);
}

}  // namespace rmsq
