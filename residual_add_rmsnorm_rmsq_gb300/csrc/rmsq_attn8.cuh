// The FP8 cache's readers for the attention kernels (rmsq_attn.cuh,
// rmsq_attn_prompt.cuh).
//
// Decode is bound by HBM: 128 requests of 2048 to 8192 keys, 8 heads on each of 4 kv
// heads of 128, take 115 us for 697 MB (6.0 TB/s, 46 % of the issue slots; the NVFP4
// cache's 390 MB 81 us), 3 requests of up to 131071 keys on 8 kv heads 104 us for 635
// MB (6.1 TB/s).
//
// An E4M3 code is exact in f16, so that a code is converted and nothing else: the
// scale of a block of 16 tokens, which is a step's half and a chunk of a logit
// row in the two kernels, is a factor of the block's logits (keys) and of its
// weights (values; relative to what, see WarpState), and costs nothing per
// element.  NaN codes of values read as 448: a masked place meets a weight of 0,
// which a NaN would survive (the store turns the token's keys to NaN as well, so
// that queries that see it are told).
//
// Weights relative to the largest value scale met, as they were, cost 1 to 3 % less
// (113 us for the 128 requests) and lost what lay beside a large scale of no weight.
#pragma once

#include "rmsq_attn_prompt.cuh"
#include "rmsq_kv8.cuh"

namespace rmsq {

// A lane's share of 16 keys.
template <int D>
struct KeyRegs8 {
    static constexpr int KW = D / 16;           // words of K codes per key (D/4 dims)
    static constexpr int VW = D / 32;           // words of V codes per key (D/8 dims)
    uint32_t k[2][KW], v[4][VW];
};

// A step of a warp: 32 keys, two halves of 16; a half is its keys' rows, then its
// values' rows, of D bytes, with their 16-byte chunks swapped so that the reads
// below are free of bank conflicts.
template <int D>
struct Step8 {
    static constexpr int codes = 16 * D;                      // bytes of a half, keys or values
    static constexpr int half = 2 * codes;
    // 8, 16 or 16 KB in flight per warp (128 requests of up to 8192 keys, items cut by
    // their tiles alone: 122 us with two stages of D = 128, which let three CTAs on an
    // SM, 118 with three and two)
    static constexpr int stages = D == 256 ? 2 : 3;
    static constexpr int ring = stages * 2 * half;            // per warp
    // Keys are read by lanes (g, t) at row kappa(g), which for eight lanes are two
    // rows four apart, 64 bytes each: those go to different halves of the banks.
    static __device__ __forceinline__ int key_swap(int row) { return (row >> 2 & 1) << 6; }
    // Values are read at row t + 4 i, four rows at once, 32 bytes (D = 64: 8 bytes
    // of sixteen lanes) each.
    static __device__ __forceinline__ int value_swap(int row) {
        return D == 64 ? (row >> 1 & 1) << 5 : D == 128 ? (row & 3) << 5 : ((row & 1) | (row & 2) << 1) << 4;
    }
};

struct Fp8Cache {
    static constexpr bool block_scales = true;
    // Weights, times their values' scale, are held as 2^6 at the row's largest (2^5 where
    // that was taken for larger, see attend32; prompts: see kNarrowValues), up to 2^9 more while it lags: moving it
    // costs a pass over O (it had to move at one step in nine with 2^9 and 2^6, on tokens
    // of uneven strength).  Those below 2^-19 of the largest are subnormal f16, off by
    // 2^-30 of it.
    static constexpr float p_shift = 6.0f, lazy = 9.0f, close = 1.0f;
    // Scale bytes v are 1 to 187 as they are read.  A weight in units of 2^(e - middle) is
    // 2^(middle - v) times its weighted value: from 2^(5 - 107) for a row's largest at v =
    // 187, with 24 bits below it within fp32, to 2^(15 + 79) at 1.
    static constexpr int middle = 80;
    // Tiles that starting and ending an item counts for, where there are more tiles
    // than CTAs.  For 0, 1, 2, 3, 4, 6, in us: 32 decodes of 100 to 2000 keys, 4 x 8
    // heads of 128, 26.0 20.9 19.7 17.7 18.6 20.5, 128 of 16 to 2000 66.5 51.7 47.1 42.6
    // 41.6 44.8, 256 of 100 to 1000 104 88 81 74 72 73, 128 of 2000 to 8192 (8 x 4)
    // 103.9 103.5 100.8 100.4 99.9 100.1; heads of 64, 128 of 16 to 2000 34.6 31.5 29.0
    // 26.1 26.7 27.6; of 256 41.5 30.2 28.8 26.9 26.4 28.2.  (One tile per CTA is
    // the best cut there is: 8 decodes of up to 500 keys 9.5, with 4 more 10.7.)
    static constexpr int piece = 4;
    template <int D> using Step = Step8<D>;
    template <int D> using Regs = KeyRegs8<D>;
    // first of the lane's j-th eight dims: 16 of every 64
    template <int D>
    static __device__ __forceinline__ int q_dim(int t, int j) { return (j >> 1) * 64 + t * 16 + (j & 1) * 8; }
    // scale bytes of a block's keys and values, as they are used
    static __device__ __forceinline__ uint32_t scale_codes(uint32_t k, uint32_t v) {
        return cache_scale_code(k) | cache_scale_code(v) << 8;
    }
    // Starts the copies of a half from row `in` of a page: 16 lanes, lane l takes
    // every 16th 16-byte chunk.
    template <int D>
    static __device__ __forceinline__ void copy_half(unsigned char* dst, const AttnArgs& a, int in, int page, int head, int l) {
        using S = Step8<D>;
        const int64_t tile = static_cast<int64_t>(D) << a.page_shift;
        const uint8_t* kt = a.cache + (static_cast<int64_t>(page) * 2 * a.kv_heads + head) * tile + in * D + l * 16;
        const uint8_t* vt = kt + a.kv_heads * tile;
#pragma unroll
        for (int i = 0; i < S::codes / 256; ++i) {
            const int at = l * 16 + i * 256;
            copy16(dst + (at ^ S::key_swap(at / D)), kt + i * 256);
        }
#pragma unroll
        for (int i = 0; i < S::codes / 256; ++i) {
            const int at = l * 16 + i * 256;
            copy16(dst + S::codes + (at ^ S::value_swap(at / D)), vt + i * 256);
        }
    }
};

__device__ __forceinline__ void set4(uint32_t* d, uint4 u) {
    d[0] = u.x; d[1] = u.y; d[2] = u.z; d[3] = u.w;
}

template <int D>
__device__ __forceinline__ void read_keys(KeyRegs8<D>& x, const unsigned char* st, int g, int t) {
    const int kappa = (g >> 1) + ((g & 1) << 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            set4(&x.k[i][4 * j], *reinterpret_cast<const uint4*>(
                                     st + (((kappa + 8 * i) * D + j * 64 + t * 16) ^ Step8<D>::key_swap(kappa))));
}

template <int D>
__device__ __forceinline__ void read_values(KeyRegs8<D>& x, const unsigned char* st, int g, int t) {
    const unsigned char* v = st + Step8<D>::codes;
    const int swap = Step8<D>::value_swap(t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (t + 4 * i) * D + g * (D / 8);
        if constexpr (D == 64) {
            const uint2 u = *reinterpret_cast<const uint2*>(v + (at ^ swap));
            x.v[i][0] = u.x; x.v[i][1] = u.y;
        } else {
#pragma unroll
            for (int j = 0; j < D / 128; ++j)
                set4(&x.v[i][4 * j], *reinterpret_cast<const uint4*>(v + ((at + 16 * j) ^ swap)));
        }
    }
}

// S^T of 16 keys, without their scale.
template <int D, int NB>
__device__ __forceinline__ void scores16(float (&s)[NB][4], const KeyRegs8<D>& x, const uint32_t (&qf)[D / 16][NB][2]) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[b][j] = 0.0f;
#pragma unroll
    for (int j = 0; j < KeyRegs8<D>::KW; ++j) {     // a word of codes: 4 dims, a k-step
        const uint32_t a0 = e4m3x2_to_f16x2(x.k[0][j]), a1 = e4m3x2_to_f16x2(x.k[1][j]);
        const uint32_t a2 = e4m3x2_to_f16x2(x.k[0][j] >> 16), a3 = e4m3x2_to_f16x2(x.k[1][j] >> 16);
#pragma unroll
        for (int b = 0; b < NB; ++b) mma_f16(s[b], a0, a1, a2, a3, qf[j][b][0], qf[j][b][1]);
    }
}

// Four dims of two keys' values, the same dim of both in a pair.
__device__ __forceinline__ void pair_values(uint32_t a, uint32_t b, uint32_t (&r)[4]) {
    const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
    r[0] = e4m3x2_f16x2(lo);
    r[1] = e4m3x2_f16x2(lo >> 16);
    r[2] = e4m3x2_f16x2(hi);
    r[3] = e4m3x2_f16x2(hi >> 16);
}

// O^T += V^T . P of 16 keys; the weights have the values' scale in them.
template <int D, int NB>
__device__ __forceinline__ void values16(WarpState<D, NB>& w, const KeyRegs8<D>& x, const uint32_t (&pf)[NB][2]) {
#pragma unroll
    for (int j = 0; j < KeyRegs8<D>::VW; ++j) {     // 4 dims: two m-tiles
        uint32_t v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) pair_values(x.v[2 * i][j], x.v[2 * i + 1][j], v[i]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                mma_f16(w.o[2 * j + c][b], v[0][2 * c], v[0][2 * c + 1], v[1][2 * c], v[1][2 * c + 1], pf[b][0], pf[b][1]);
    }
}

// The prompt kernel's tiles of 128 keys.  A warp of their own (`fetch`) finds the
// pages and scales of a tile's eight blocks and copies their keys, D * 16
// contiguous bytes each, into a ring of two raw tiles; four warps (`convert`) turn
// those into operand rows, and values from registers that are loaded a tile
// ahead.
//
// The prompt step of rmsq_attn_prompt.cuh's figures (2478 and 2445 queries of 32
// heads, 192 GFLOP) takes 234 us, over the NVFP4 cache 198; 128 keys 1.96 us on a
// context of 20000 (1.66).  What it is sensitive to is the size of the roles' code
// (see the issuing loop) and the latency of reads.  Tried on the way: keys loaded into
// registers, a row per thread, with a factor for each 16 logits in the softmax 278;
// the same with lines read whole 295; the blocks that are far apart handled in the
// softmax, which then holds code for both, 305; keys converted by two warps of the
// issuing group 283; values converted in a rolled loop 246 where it was 251.
template <int D>
struct RawValues {
    static constexpr int VW = D / 32;           // words of a key's values (D/8 dims)
    uint32_t v[8][VW];
};

// First byte of a key (side 0) or value (1) of a page.
template <int D>
__device__ __forceinline__ const uint8_t* row_of(const AttnArgs& a, int page, int side, int head, int key) {
    const int64_t at = (static_cast<int64_t>(page) * 2 + side) * a.kv_heads + head;
    return a.cache + ((at << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * D;
}

template <int D>
__device__ __forceinline__ void load_values(RawValues<D>& x, const AttnArgs& a, int key, int page, int head, int unit) {
    const uint8_t* p = row_of<D>(a, max(page, 0), 1, head, key) + unit * (D / 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (page >= 0) {
            if constexpr (D == 128) {
                set4(x.v[i], __ldg(reinterpret_cast<const uint4*>(p + i * D)));
            } else {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + i * D));
                x.v[i][0] = u.x; x.v[i][1] = u.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < RawValues<D>::VW; ++j) x.v[i][j] = 0u;
        }
    }
}

// A lane's share of the warp's 32 raw keys: 8 codes of a row, D / 8 lanes to a row.
template <int D>
struct RawKeys {
    static constexpr int LT = D / 8, ROWS = 32 / LT, N = 32 / ROWS;     // lanes of a row; rows of an access; accesses
    uint2 k[N];
};

template <int D>
__device__ __forceinline__ void read_raw(RawKeys<D>& x, const unsigned char* raw, int warp, int lane) {
    using R = RawKeys<D>;
    raw += (warp * 32 + lane / R::LT) * D + lane % R::LT * 8;
#pragma unroll
    for (int i = 0; i < R::N; ++i) x.k[i] = *reinterpret_cast<const uint2*>(raw + i * R::ROWS * D);
}

// They as rows of the operand tile, times their blocks' factors (f16 pairs).
template <int D>
__device__ __forceinline__ void write_keys(unsigned char* dst, const RawKeys<D>& x, int warp, int lane, uint32_t f0, uint32_t f1) {
    using R = RawKeys<D>;
    const int piece = lane % R::LT, row = warp * 32 + lane / R::LT;
    dst += (piece >> 3) * (128 * 128) + row * 128;
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
        const uint32_t f = i < R::N / 2 ? f0 : f1;
        *reinterpret_cast<uint4*>(dst + i * R::ROWS * 128 + (((piece & 7) ^ ((row + i * R::ROWS) & 7)) << 4)) =
            make_uint4(mul_f16x2(e4m3x2_to_f16x2(x.k[i].x), f), mul_f16x2(e4m3x2_to_f16x2(x.k[i].x >> 16), f),
                       mul_f16x2(e4m3x2_to_f16x2(x.k[i].y), f), mul_f16x2(e4m3x2_to_f16x2(x.k[i].y >> 16), f));
    }
}

// V of the thread's 8 keys and D/8 dims, times their block's factor, as 16-byte
// pieces of V^T's rows.
template <int D>
__device__ __forceinline__ void write_values(unsigned char* dst, const RawValues<D>& x, int octet, int unit, uint32_t f) {
    unsigned char* base = dst + (octet >> 3) * (D * 128);
#pragma unroll
    for (int j = 0; j < RawValues<D>::VW; ++j) {
        uint32_t v[4][4];       // [pair of keys][dim]
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            pair_values(x.v[2 * p][j], x.v[2 * p + 1][j], v[p]);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[p][c] = mul_f16x2(v[p][c], f);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = unit * (D / 8) + 4 * j + c;
            *reinterpret_cast<uint4*>(base + row * 128 + (((octet & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0][c], v[1][c], v[2][c], v[3][c]);
        }
    }
}

// The f16 pair 2^-down, twice; down at most 15 (2^-15 is a subnormal number).
__device__ __forceinline__ uint32_t f16_factor(uint32_t down) { return (down < 15u ? (15u - down) << 10 : 0x200u) * 0x10001u; }

// How far apart the scales of a step's blocks may be.  Keys: for every code times its
// scale relative to the largest to be exact in f16, whose smallest number is 2^-9 times
// 2^-15.  Values: a row's reference takes the step's largest scale for its own key's,
// so that its weighted values may be held lower than it says by as much: 2^-1 at the
// largest, and weights that are subnormal in f16 off by 2^-24 of it in place of 2^-30.
constexpr uint32_t kNarrowKeys = 15, kNarrowValues = 7;

template <int D>
struct Fp8Prompt : Fp8Cache {
    static constexpr int ring = 2 * 128 * D;        // bytes of the raw keys

    // One warp; lane l cares for block l % 8 of a tile.  A tile's pages are loaded
    // two tiles before its copies, its scales one.  A tile is a step, unless its
    // blocks' scales are too far apart: then each step takes those of the blocks left
    // that are near the first of them.  `info` is eight steps deep: when a slot of the
    // ring is free again, the step four before has only been multiplied and may still
    // be in its softmax, the one five before is through.
    static __device__ __forceinline__ bool fetch(const AttnArgs& a, int req, int head, int key_begin, int last_pos, int tiles,
                                                 unsigned char* raw, uint64_t* full, uint64_t* empty, StepInfo* info) {
        constexpr int kBlock = kBlockTokens * D;
        const int lane = threadIdx.x & 31, block = lane & 7;
        const int* table = a.table + static_cast<int64_t>(req) * a.width;
        auto page_of = [&](int tile) {
            const int key = key_begin + tile * 128 + block * kBlockTokens;
            return key > last_pos ? -1 : __ldg(table + (key >> a.page_shift));
        };
        // (a page is compared with their number when it is used: next to its load
        // the warp would wait for it)
        auto checked = [&](int p) { return p < a.num_pages ? p : -1; };
        uint32_t kraw = 0u, vraw = 0u;
        auto load_scales = [&](int page, int tile) {
            if (page < 0) return;
            const int64_t at = static_cast<int64_t>(page) * 2 * a.kv_heads + head;
            const int in = (key_begin + tile * 128 + block * kBlockTokens) & ((1 << a.page_shift) - 1);
            const uint8_t* p = a.scales + (at << (a.page_shift - 4)) + (in >> 4);
            kraw = __ldg(p);
            vraw = __ldg(p + (static_cast<int64_t>(a.kv_heads) << (a.page_shift - 4)));
        };
        const uint64_t keep = l2_policy_evict_normal();
        int page = checked(page_of(0)), next = page_of(1), n = 0;
        bool ok = true;
        load_scales(page, 0);
#pragma unroll 1
        for (int tile = 0; tile < tiles && ok; ++tile) {
            uint32_t todo = __ballot_sync(kFull, page >= 0) & 0xffu;
#pragma unroll 1
            do {
                const int s = n & 1;
                ok = warp_wait(&empty[s], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                // The keys of all blocks left, before anything waits for their scales.
                if (lane == 0) mbar_expect_tx(&full[s], __popc(todo) * kBlock);
                __syncwarp();
                if (lane < 8 && (todo >> block & 1u))
                    bulk_g2s(raw + s * 128 * D + block * kBlock,
                             row_of<D>(a, page, 0, head, key_begin + tile * 128 + block * kBlockTokens), kBlock, &full[s], keep);
                const uint32_t kc = cache_scale_code(kraw), vc = cache_scale_code(vraw);
                bool take = todo >> block & 1u;
                uint32_t kmost = __reduce_max_sync(kFull, take ? kc : 0u), vmost = __reduce_max_sync(kFull, take ? vc : 0u);
                if (__any_sync(kFull, take && (kc + kNarrowKeys < kmost || vc + kNarrowValues < vmost))) {
                    const int first = __ffs(todo) - 1;
                    const uint32_t k0 = __shfl_sync(kFull, kc, first), v0 = __shfl_sync(kFull, vc, first);
                    // 7 below to 8 above, 3 below to 4 above
                    take = take && kc + 7u >= k0 && kc <= k0 + 8u && vc + 3u >= v0 && vc <= v0 + 4u;
                    kmost = __reduce_max_sync(kFull, take ? kc : 0u);
                    vmost = __reduce_max_sync(kFull, take ? vc : 0u);
                }
                const uint32_t taken = __ballot_sync(kFull, take) & 0xffu;
                todo &= ~taken;
                StepInfo& t = info[n & 7];
                if (lane < 4)
                    t.valid[lane] = (taken >> (2 * lane) & 1u) * 0xffffu | (taken >> (2 * lane + 1) & 1u) * 0xffff0000u;
                if (lane < 8) {
                    t.page[lane] = take ? page : -1;
                    t.fk[lane] = f16_factor(take ? kmost - kc : 0u);
                    t.fv[lane] = f16_factor(take ? vmost - vc : 0u);
                }
                if (lane == 0) {
                    t.k = cache_scale_value(max(kmost, 1u));
                    t.v = static_cast<float>(vmost);
                    t.key0 = key_begin + tile * 128;
                    t.last = tile + 1 == tiles && todo == 0u;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                ++n;
            } while (todo != 0u);
            page = checked(next);
            next = page_of(tile + 2);
            load_scales(page, tile + 1);
        }
        // its copies are through before it leaves
#pragma unroll 1
        for (int i = max(n - 2, 0); i < n; ++i) ok = warp_wait(&full[i & 1], (i >> 1) & 1) && ok;
        return ok;
    }

    // Four warps, keys and values in turn.  A step's raw keys are read, and its
    // values loaded, into the registers that the step before has just left: shared
    // memory is as busy with the matrix unit's operands that a read takes 400 clocks.
    static __device__ __forceinline__ bool convert(const AttnArgs& a, int head, const unsigned char* raw, unsigned char* ks,
                                                   unsigned char* vs, uint64_t* rawfull, uint64_t* rawempty, uint64_t* kfull,
                                                   uint64_t* kempty, uint64_t* vfull, uint64_t* vempty, const StepInfo* info) {
        constexpr int kTile = 128 * D * 2;      // bytes of an operand tile
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5 & 3;
        const int octet = (w & 1) * 8 + (lane & 7), unit = (w >> 1) * 4 + (lane >> 3), block = octet >> 1;
        RawKeys<D> keys;
        RawValues<D> values;
        if (!warp_wait(&rawfull[0], 0)) return false;
        read_raw<D>(keys, raw, w, lane);
        load_values<D>(values, a, info[0].key0 + octet * 8, info[0].page[block], head, unit);
#pragma unroll 1
        for (int n = 0;; ++n) {
            const int s = n & 1;
            const uint32_t parity = (n >> 1) & 1;
            const StepInfo& t = info[n & 7];
            const int last = t.last;
            if (!warp_wait(&kempty[s], parity ^ 1)) return false;
            write_keys<D>(ks + s * kTile, keys, w, lane, t.fk[2 * w], t.fk[2 * w + 1]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&kfull[s]);
                mbar_arrive(&rawempty[s]);
            }
            if (!last) {
                if (!warp_wait(&rawfull[s ^ 1], ((n + 1) >> 1) & 1)) return false;
                read_raw<D>(keys, raw + (s ^ 1) * 128 * D, w, lane);
            }
            if (!warp_wait(&vempty[s], parity ^ 1)) return false;
            const RawValues<D> now = values;
            const uint32_t fv = t.fv[block];
            if (!last) {
                const StepInfo& u = info[(n + 1) & 7];
                load_values<D>(values, a, u.key0 + octet * 8, u.page[block], head, unit);
            }
            write_values<D>(vs + s * kTile, now, octet, unit, fv);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&vfull[s]);
            if (last) return true;
        }
    }
};

}  // namespace rmsq
