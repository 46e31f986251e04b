// Attention over a paged cache, for few queries per request (decode): the
// kernels, with the NVFP4 cache's reader.  The FP8 cache's is in rmsq_attn8.cuh;
// a reader is a struct C with its step's layout, its copies and its loads.
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i.k_j) / sum_j' exp(scale q_i.k_j'),
//   keys j <= pos_i (and j > pos_i - window), pos_i = seq_len - query_len + i.
//
// The G query heads of a kv head read the same keys, so the rows of one
// matrix product are (query token, head of the group): row = i * G + g, taken
// ROWS = 8 * NB at a time.  One pass over the keys with a running maximum.
//
// Matrix instructions (m16n8k16, f16 operands, fp32 sums), transposed so that
// the 16-row operand is the cache and the rows are the 8 columns:
//   S^T[key, row] = K[key, :] . Q[row, :]      O^T[dim, row] += V[:, dim] . P[row, :]
// f16 holds the cached values exactly: an E2M1 code times its E4M3 scale has
// at most 6 significant bits and lies in [2^-10, 2688] (or is 0).  The global
// scales are factors of the logits and of the output.  bf16 queries are scaled
// by a power of two per row into f16's range, exact unless an element is
// 2^-28 of the row's largest (then off by 2^-39 of it).  Probabilities are
// rounded to f16 (11 bits; 8 would be as many as a bf16 output has), scaled by
// 2^9 so that those down to 2^-23 of the maximum keep all their bits (p_shift).  With
// 32-bit weights the relative error of fp16 outputs is 2.1e-4 and with these
// 2.9e-4 (3 requests of up to 131071 keys, against 64 bits); bf16 outputs hide it
// (1.7e-3 both ways).  The matrix unit's next wider type would halve its rate.
//
// Maxima are kept as logits and not as logits times f (the factor that turns
// them into powers of two): the product's rounding, half a unit of its last
// place, would be an error of the exponent, and from 2^24 on it takes weights
// out of f16's range.  A weight is 2^(f s + (9 - f t)) while the maximum f t is
// at most 2^10, where the bracket is off by 2^-14 at most, and 2^(f (s - t) + 9)
// beyond, exact where it matters: the largest logit's weight is 2^9 always.
//
// Layout: contractions may take their index in any order, so every lane loads
// the piece of the cache it needs in one access, with no shuffle.  Each warp
// keeps the next steps in flight as asynchronous copies into a ring of its own.
// Lane (g, t) = (lane / 4, lane % 4):
//   K: dims t * D/4 .. of keys kappa(g) and kappa(g) + 8;
//   V: dims g * D/8 .. of keys t, t + 4, t + 8, t + 12 (one scale block for
//      D = 128), whose nibbles are interleaved pairwise so that one
//      conversion yields the same dim of two keys, the pair a register of the
//      operand holds;
// kappa is the order of the keys that makes S^T's accumulator, transposed by
// movmatrix, the second product's operand.
//
// Bound by HBM and, nearly as much, by issue for long caches (9/16 byte per
// element, K and V): 128 requests of 2048 to 8192 keys, 8 heads on each of 4 kv
// heads of 128, take 81 us for 390 MB (4.8 TB/s; 71 with the arithmetic left out,
// 76 with the copies left out), 3 requests of up to 131071 keys on 8 kv heads 73
// us for 357 MB.  About 300 warp instructions per 16 keys and kv head are left, 64
// of them conversions of codes, 64 multiplications by scales, 16 products.
// Measured and not kept: the codes loaded straight into registers a step ahead
// (116 us), a ring of bulk copies on mbarriers (111), 16 keys per softmax step
// (111), a third stage (84), registers capped for five CTAs per SM (86).
//
// Work is split evenly over the CTAs whatever the lengths: the (request, row
// tile, kv head, 128-key tile) tiles form one sequence, cut into equal runs; a CTA
// writes the items its run holds whole, and leaves (O, m, l, f) in the workspace
// for the two that its ends may cut, which a second launch joins in order.  A
// reader with a `piece` counts that many tiles more for each item, places of the
// sequence without work: what a CTA does once per item it touches (queries, first
// copies, the warps' join) then counts like tiles, and a CTA of many short items
// gets fewer tiles.
#pragma once

#include "rmsq_device.cuh"
#include "rmsq_kv.cuh"

namespace rmsq {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnKeyTile = kAttnWarps * 32;   // keys per CTA step: 32 per warp
constexpr int kAttnMaxWorkers = 1216;           // CTAs of the split launch: 8 per SM of 152
constexpr int kPromptRows = 64;                 // see launch_attn
constexpr float kFar = 1024.0f;                 // maximum (in powers of two) from which it is subtracted first

// What the join has to know of an item that starts in a run and goes past its
// end: the runs it lies in, and its rows.
struct CutItem {
    int parts;      // 0: no such item
    int slot;       // of its first part
    int q0, qlen, qtile, head;
    int unused[2];
};

struct AttnArgs {
    const void* q;
    int64_t q_stride;       // elements between tokens
    const uint8_t* cache;
    const uint8_t* scales;  // of the FP8 cache's blocks
    const int* table;       // [requests, width]
    const int* q_start;     // [requests + 1]
    const int* seq_lens;    // [requests]
    const float* k_gs;      // global scales of the NVFP4 cache (null: 1)
    const float* v_gs;
    void* out;              // [tokens, heads, D]
    float* lse;             // [tokens, heads] or null
    CutItem* cut;           // [workers]
    float* part;            // [workers][2][ROWS][kPartRow<D>]
    int requests, width, tokens, heads, kv_heads, group;
    int page_shift, num_pages, window, workers;
    int most_rows;          // rows of a request above which it may be the prompt kernel's, see prompt_takes
    int half_items;         // prompt items of 128 rows per kv head up to which they have 128 and not 256
    int64_t share;          // 0, or what rows times requests have to reach for that
    float scale_log2;       // softmax scale * log2(e)
};

// A row of a part in the workspace: D sums, the maximum, the sum of the weights,
// the row's factor.
template <int D>
constexpr int kPartRow = D + 4;

// One request as the kernels see it: every value is clamped so that no
// length or offset in device memory can lead outside the buffers.
struct Req {
    int q0, qlen, seq, tile0, ktiles;
};

// Which kernel takes a request.  The prompt kernel walks all its keys in one
// CTA, the split kernel divides them over the card; the time of both is
// proportional to the length.  So a request of few rows is better with the split
// kernel unless there are enough others of its length beside it to fill the card
// with prompt CTAs: rows * n >= share, n the requests of more than most_rows rows
// whose keys are at least half as many (the same power of two and up).  Both
// kernels count n themselves, from the same lengths.  128 decodes of 8 x 8 heads
// on 2000 keys beside 9 queries on 100000: 1332 us with the prompt kernel for the
// 9, 234 with the split kernel for all.
__device__ __forceinline__ bool prompt_takes(const AttnArgs& a, int64_t rows, int ktiles, const int* longer) {
    return rows > a.most_rows && (a.share == 0 || rows * longer[31 - __clz(ktiles)] >= a.share);
}

__device__ __forceinline__ Req load_request(const AttnArgs& a, int r) {
    Req x;
    x.q0 = min(max(__ldg(a.q_start + r), 0), a.tokens);
    x.qlen = min(max(__ldg(a.q_start + r + 1), x.q0), a.tokens) - x.q0;
    x.seq = min(max(__ldg(a.seq_lens + r), 0), a.width << a.page_shift);
    const int first = a.window > 0 ? max(x.seq - x.qlen - a.window + 1, 0) : 0;
    x.tile0 = min(first, max(x.seq - 1, 0)) / kAttnKeyTile;
    x.ktiles = max((x.seq + kAttnKeyTile - 1) / kAttnKeyTile - x.tile0, 1);
    return x;
}

// prefix[r] = items(rows, the prompt kernel's or not) summed over the requests
// before r, prefix[requests] over all, in shared memory; with TILES their tiles, and
// where those of all kv heads are more than the workers, PIECE more for each item.
// Returns what was added to an item.  Ends with a barrier.  (Compact on purpose:
// it is cold code at the start of every CTA.)
template <int THREADS, bool TILES, int PIECE, class Items>
__device__ __forceinline__ int scan_requests(const AttnArgs& a, int64_t* prefix, Items items) {
    __shared__ int64_t wsum[THREADS / 32];
    __shared__ int witems[THREADS / 32];
    __shared__ int longer[32];      // candidates of 2^i key tiles and more
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.requests + THREADS - 1) / THREADS;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
    if (a.share != 0) {
        if (tid < 32) longer[tid] = 0;
        __syncthreads();
    }
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const Req x = load_request(a, r);
        const int rows = x.qlen * a.group;
        prefix[r + 1] = static_cast<int64_t>(rows) << 32 | x.ktiles;
        if (a.share != 0 && rows > a.most_rows)
#pragma unroll 1
            for (int i = 31 - __clz(x.ktiles); i >= 0; --i) atomicAdd(longer + i, 1);
    }
    if (a.share != 0) __syncthreads();
    int64_t sum = 0;
    int count = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int64_t rows = prefix[r + 1] >> 32;
        const int ktiles = static_cast<int>(prefix[r + 1]), length = TILES ? ktiles : 1;
        const int n = static_cast<int>(items(rows, prompt_takes(a, rows, ktiles, longer)));
        prefix[r + 1] = static_cast<int64_t>(n) << 32 | length;
        sum += static_cast<int64_t>(n) * length;
        count += n;
    }
    int64_t inc = sum;
    int inc_items = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
        if constexpr (PIECE != 0) {
            const int v = __shfl_up_sync(kFull, inc_items, o);
            if (lane >= o) inc_items += v;
        }
    }
    if (lane == 31) {
        wsum[warp] = inc;
        if constexpr (PIECE != 0) witems[warp] = inc_items;
    }
    __syncthreads();
    int64_t run = inc - sum;
    int more = 0;
    if constexpr (PIECE != 0) {
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) total += wsum[w];
        if (total * a.kv_heads > a.workers) more = PIECE;
        int before = inc_items - count;
#pragma unroll 1
        for (int w = 0; w < warp; ++w) before += witems[w];
        run += static_cast<int64_t>(before) * more;
    }
#pragma unroll 1
    for (int w = 0; w < warp; ++w) run += wsum[w];
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int64_t x = prefix[r + 1];
        run += (x >> 32) * (static_cast<int>(x) + more);
        prefix[r + 1] = run;
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
    return more;
}

// Where tile x of the whole sequence lies, whose items have `more` places behind
// their tiles.
struct Place {
    int r, head, qtile, tile;   // tile: index inside the item
    int64_t item0;              // first tile of the item in the sequence
};

__device__ __forceinline__ Place locate(const AttnArgs& a, const int64_t* prefix, int64_t x, int more, Req& req) {
    int lo = 0, hi = a.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] * a.kv_heads <= x) lo = mid;
        else hi = mid;
    }
    req = load_request(a, lo);
    const int64_t rest = x - prefix[lo] * a.kv_heads;
    const int length = req.ktiles + more;
    const int64_t item = rest / length;
    Place p;
    p.r = lo;
    p.tile = static_cast<int>(rest - item * length);
    p.qtile = static_cast<int>(item / a.kv_heads);
    p.head = static_cast<int>(item - static_cast<int64_t>(p.qtile) * a.kv_heads);
    p.item0 = x - p.tile;
    return p;
}

// Tiles per CTA of the even split.
__device__ __forceinline__ int64_t run_length(int64_t total, int workers) {
    return total <= workers ? 1 : (total + workers - 1) / workers;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes (low half of w) as an f16 pair; every E4M3 value is exact,
// and the minimum with 448 keeps a number where the code is NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "min.f16x2 %0, %0, %2;\n\t}" : "=r"(r) : "r"(w), "r"(0x5f005f00u));
    return r;
}

// A lane's share of 16 keys: codes and scale bytes.
template <int D>
struct KeyRegs {
    static constexpr int KW = D / 32;           // words of K codes per key (D/4 dims)
    static constexpr int VW = D / 64;           // words of V codes per key (D/8 dims)
    static constexpr int KS = D / 64;           // K scale bytes per key
    static constexpr int VS = D == 256 ? 2 : 1; // V scale bytes per key
    uint32_t k[2][KW], v[4][VW];
    uint32_t ks[2];     // KS bytes each
    uint32_t vs[4];     // VS bytes each
};

// A step of a warp: 32 keys, two halves of 16 that each lie on one page.
// Shared memory of a half: K codes, K scales, V codes, V scales.
template <int D>
struct Step {
    static constexpr int codes = 16 * D / 2, scales = D;      // bytes of a half, keys or values
    static constexpr int half = 2 * (codes + scales);
    static constexpr int stages = D == 64 ? 4 : 2;            // 9 or 18 KB in flight per warp
    static constexpr int ring = stages * 2 * half;            // per warp
};

// The reader of the NVFP4 cache.
struct Nvfp4Cache {
    static constexpr bool block_scales = false;     // its scales are multiplied into the elements
    static constexpr float p_shift = 9.0f;          // weights are scaled by 2^9 ...
    static constexpr float lazy = 6.0f;             // ... and by up to 2^6 more while the maximum lags: < 2^16 in f16
    static constexpr int piece = 0;                 // items are cut by their tiles alone
    template <int D> using Step = rmsq::Step<D>;
    template <int D> using Regs = KeyRegs<D>;
    // first of the lane's j-th eight dims
    template <int D>
    static __device__ __forceinline__ int q_dim(int t, int j) { return t * (D / 4) + 8 * j; }
    template <int D>
    static __device__ __forceinline__ void copy_half(unsigned char* dst, const AttnArgs& a, int in, int page, int head, int l);
};

// What a reader with block_scales has of a step's two halves: their scale
// bytes, 0 for a half that is not there.
struct HalfScales {
    uint32_t k[2], v[2];
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

// Starts the copies of a half from row `in` of a page: 16 lanes, lane l takes
// every 16th 16-byte chunk.
template <int D>
__device__ __forceinline__ void Nvfp4Cache::copy_half(unsigned char* dst, const AttnArgs& a, int in, int page, int head, int l) {
    using S = Step<D>;
    const uint32_t tile = static_cast<uint32_t>(D / 16 * 9) << a.page_shift;
    const uint8_t* kt = a.cache + (static_cast<int64_t>(page) * 2 * a.kv_heads + head) * tile;
    const uint8_t* vt = kt + static_cast<int64_t>(a.kv_heads) * tile;
    const uint32_t c = in * (D / 2) + l * 16, s = ((D / 2) << a.page_shift) + in * (D / 16);
    unsigned char* d = dst + l * 16;
#pragma unroll
    for (int i = 0; i < S::codes / 256; ++i) copy16(d + i * 256, kt + c + i * 256);
#pragma unroll
    for (int i = 0; i < S::codes / 256; ++i) copy16(d + S::codes + S::scales + i * 256, vt + c + i * 256);
    // the scales of both sides together: D / 16 chunks each
#pragma unroll
    for (int i = 0; i < (D + 127) / 128; ++i) {
        const int j = l + 16 * i, side = j >= D / 16, k = j - side * (D / 16);
        if (D >= 128 || l < D / 8)
            copy16(dst + S::codes + side * (S::codes + S::scales) + k * 16, (side ? vt : kt) + s + k * 16);
    }
}

// The lane's share of a half.  Rows of K at a 64-byte (D = 128) stride and 16
// bytes a lane, rows of V 4 at a time and 8 bytes a lane: contiguous over the
// warp, free of bank conflicts.
template <int D>
__device__ __forceinline__ void read_keys(KeyRegs<D>& x, const unsigned char* st, int g, int t) {
    using K = KeyRegs<D>;
    using S = Step<D>;
    const int kappa = (g >> 1) + ((g & 1) << 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned char* p = st + (kappa + 8 * i) * (D / 2) + t * (D / 8);
        if constexpr (D == 64) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            x.k[i][0] = u.x; x.k[i][1] = u.y;
        } else {
#pragma unroll
            for (int j = 0; j < K::KW; j += 4) {
                const uint4 u = reinterpret_cast<const uint4*>(p)[j / 4];
                x.k[i][j] = u.x; x.k[i][j + 1] = u.y; x.k[i][j + 2] = u.z; x.k[i][j + 3] = u.w;
            }
        }
        const unsigned char* s = st + S::codes + (kappa + 8 * i) * (D / 16) + t * K::KS;
        if constexpr (D == 64) x.ks[i] = *s;
        else if constexpr (D == 128) x.ks[i] = *reinterpret_cast<const uint16_t*>(s);
        else x.ks[i] = *reinterpret_cast<const uint32_t*>(s);
    }
}

template <int D>
__device__ __forceinline__ void read_values(KeyRegs<D>& x, const unsigned char* st, int g, int t) {
    using K = KeyRegs<D>;
    using S = Step<D>;
    const unsigned char* v = st + S::codes + S::scales;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned char* p = v + (t + 4 * i) * (D / 2) + g * (D / 16);
        if constexpr (D == 64) {
            x.v[i][0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            x.v[i][0] = u.x; x.v[i][1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            x.v[i][0] = u.x; x.v[i][1] = u.y; x.v[i][2] = u.z; x.v[i][3] = u.w;
        }
        const unsigned char* s = v + S::codes + (t + 4 * i) * (D / 16) + (D == 64 ? g / 2 : g * K::VS);
        if constexpr (D == 256) x.vs[i] = *reinterpret_cast<const uint16_t*>(s);
        else x.vs[i] = *s;
    }
}

// f16 pair (s, s) from half `hi` of an f16 pair.
__device__ __forceinline__ uint32_t dup_half(uint32_t pair, int hi) { return __byte_perm(pair, 0, hi ? 0x3232 : 0x1010); }

// The factor of a row's logits, kept within the normal numbers: zero or infinite,
// it would turn differences of logits into NaN.
__device__ __forceinline__ float clamp_factor(float f) { return fminf(fmaxf(f, 1.17549435e-38f), 3.40282347e38f); }

// The logit above which a maximum of t has to move.  Rounded down: half a unit of
// t's last place can be more than C::lazy.
template <class C>
__device__ __forceinline__ float lag_limit(float t, float f) { return t == -INFINITY ? t : __fadd_rd(t, C::lazy / f); }

// What the exponents of a row with maximum m are shifted by, and whether m is
// so far out that it is to be subtracted from the logits instead.
template <class C>
__device__ __forceinline__ float weight_shift(float m, float f) { return m == -INFINITY ? 0.0f : fmaf(-m, f, C::p_shift); }
__device__ __forceinline__ bool is_far(float shift) { return !(fabsf(shift) <= kFar); }

// 2^e, e from -126 to 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A warp's running state over its keys for one item.  The logits and their
// maximum m stay in the units of the product; f turns them into units of log2;
// limit is the logit above which the maximum has to move; far: some row's
// maximum is beyond kFar.
//
// With block_scales a half's keys share one power of two, a factor of its logits, and
// its values another, 2^v, a factor of its weights: neither is applied per element.
// What counts is then the weighted value, 2^(f s + v), so that the row's
// reference is the largest of those it has seen: m is the logit of that key and e
// the v of its block, and weights are 2^(f (s - m) + v - e + p_shift), whatever lies in
// places that the row does not see, or sees with a large scale and next to no weight.
// The sum l of the weights proper has v left out and would leave fp32's range if it
// were relative to the same key: it is in units of 2^(e - C::middle).  limit is e +
// lazy, shift what the exponent of a key with the reference's v is shifted by.
template <int D, int NB>
struct WarpState {
    float o[D / 16][NB][4];
    float m[NB][2], l[NB][2], limit[NB][2], shift[NB][2];
    bool far;
};

// A row's reference: a maximum, with block_scales its block's exponent beside it.
struct Peak {
    float m, e;
};
// log2 of what a is relative to b
template <class C>
__device__ __forceinline__ float above(Peak a, Peak b, float f) {
    return C::block_scales ? fmaf(a.m - b.m, f, a.e - b.e) : (a.m - b.m) * f;
}
// A sum of weights that is to be relative to a peak 2^x times as high.  (With
// block_scales x may be below the normal numbers' exponents where the result is not.)
template <class C>
__device__ __forceinline__ float lowered(float l, float x) {
    if constexpr (C::block_scales) {
        const float half = exp2_approx(0.5f * x);
        return l * half * half;
    } else {
        return l * exp2_approx(x);
    }
}
template <class C>
__device__ __forceinline__ Peak higher(Peak a, Peak b, float f) {
    if constexpr (C::block_scales) return above<C>(b, a, f) > 0.0f ? b : a;   // (-inf below -inf: NaN, a)
    else return {fmaxf(a.m, b.m), 0.0f};
}

// S^T of 16 keys: s[b][0..1] key kappa(g), rows 2t and 2t + 1; s[b][2..3] key + 8.
template <int D, int NB>
__device__ __forceinline__ void scores16(float (&s)[NB][4], const KeyRegs<D>& x, const uint32_t (&qf)[D / 16][NB][2]) {
    using K = KeyRegs<D>;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[b][j] = 0.0f;
    // duplicated f16 pair of each block's scale; D = 64: one block per key, 128: two, 256: four
    uint32_t sc[2][K::KS];
    if constexpr (D == 64) {
        const uint32_t p = e4m3x2_f16x2(x.ks[0] | (x.ks[1] << 8));
        sc[0][0] = dup_half(p, 0);
        sc[1][0] = dup_half(p, 1);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < K::KS; j += 2) {
                const uint32_t p = e4m3x2_f16x2(x.ks[i] >> (8 * j));
                sc[i][j] = dup_half(p, 0);
                sc[i][j + 1] = dup_half(p, 1);
            }
    }
#pragma unroll
    for (int j = 0; j < K::KW; ++j) {   // a word of codes: 8 dims, two k-steps
        uint32_t k0[4], k1[4];
        e2m1x8_f16x2(x.k[0][j], k0);
        e2m1x8_f16x2(x.k[1][j], k1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k0[i] = mul_f16x2(k0[i], sc[0][j / 2]);
            k1[i] = mul_f16x2(k1[i], sc[1][j / 2]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            mma_f16(s[b], k0[0], k1[0], k0[1], k1[1], qf[2 * j][b][0], qf[2 * j][b][1]);
            mma_f16(s[b], k0[2], k1[2], k0[3], k1[3], qf[2 * j + 1][b][0], qf[2 * j + 1][b][1]);
        }
    }
}

// O^T += V^T . P of 16 keys.
template <int D, int NB>
__device__ __forceinline__ void values16(WarpState<D, NB>& w, const KeyRegs<D>& x, const uint32_t (&pf)[NB][2]) {
    using K = KeyRegs<D>;
    // scales of the pairs (key t, key t + 4) and (t + 8, t + 12)
    uint32_t sc[2][K::VS];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t c = __byte_perm(x.vs[2 * i], x.vs[2 * i + 1], 0x5140);
        sc[i][0] = e4m3x2_f16x2(c);
        if constexpr (D == 256) sc[i][1] = e4m3x2_f16x2(c >> 16);
    }
#pragma unroll
    for (int j = 0; j < K::VW; ++j) {   // 8 dims: four m-tiles
        uint32_t even[2][4], odd[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t A = x.v[2 * i][j], B = x.v[2 * i + 1][j];
            e2m1x8_f16x2((A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u), even[i]);
            e2m1x8_f16x2(((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u), odd[i]);
            const uint32_t m = sc[i][K::VS == 2 ? j / 2 : 0];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                even[i][c] = mul_f16x2(even[i][c], m);
                odd[i][c] = mul_f16x2(odd[i][c], m);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                mma_f16(w.o[4 * j + c][b], even[0][c], odd[0][c], even[1][c], odd[1][c], pf[b][0], pf[b][1]);
    }
}

// One step: 32 keys from `base`.  pos / lo: last and first key each of the
// lane's columns may see; `full`: every key is inside for every row; bit i of
// `have`: half i is there.
template <class C, int D, int NB>
__device__ __forceinline__ void attend32(WarpState<D, NB>& w, const unsigned char* st, const uint32_t (&qf)[D / 16][NB][2],
                                         const float (&f)[NB][2], const int (&pos)[NB][2], const int (&lo)[NB][2],
                                         bool full, uint32_t have, int base, int g, int t, const HalfScales& sc) {
    using S = typename C::template Step<D>;
    float s[2][NB][4];
    typename C::template Regs<D> x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        read_keys<D>(x[h], st + h * S::half, g, t);
        scores16<D, NB>(s[h], x[h], qf);
        if constexpr (C::block_scales) {
            const float ks = __uint_as_float(sc.k[h] << 23);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[h][b][j] *= ks;
        }
    }
    if (!full) {
        const int key = base + (g >> 1) + ((g & 1) << 2);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = key + 16 * h + (j >> 1) * 8;
                    if (k > pos[b][j & 1] || k < lo[b][j & 1] || !(have >> h & 1u)) s[h][b][j] = -INFINITY;
                }
    }
    // The maximum is moved only when some logit (weighted value) passes it by more than
    // C::lazy.
    const float v[2] = {static_cast<float>(sc.v[0]), static_cast<float>(sc.v[1])}, larger = fmaxf(v[0], v[1]);
    float top[NB][2];
    bool grow = false;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            top[b][j] = fmaxf(fmaxf(s[0][b][j], s[0][b][j + 2]), fmaxf(s[1][b][j], s[1][b][j + 2]));
            // (as if both halves had the larger scale: which has it is looked at below;
            // nothing yet and nothing here is NaN)
            grow |= (C::block_scales ? fmaf(top[b][j] - w.m[b][j], f[b][j], larger) : top[b][j]) > w.limit[b][j];
        }
    if (__any_sync(kFull, grow)) {
        bool far = false;
        // Two scales that are near each other count as the larger one, which puts the
        // reference too high by 2^close at most: one maximum over the lanes instead of
        // two (for a block that is not there v is 0).
        const float smaller = fminf(v[0], v[1]);
        bool near = true;
        if constexpr (C::block_scales) near = smaller == 0.0f || larger - smaller <= C::close;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Peak was = {w.m[b][j], w.limit[b][j] - C::lazy};
                auto over_lanes = [](float x) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
                    return x;
                };
                const float first = near ? top[b][j] : fmaxf(s[0][b][j], s[0][b][j + 2]);
                Peak now = higher<C>(was, {over_lanes(first), near ? larger : v[0]}, f[b][j]);
                if (!near) now = higher<C>(now, {over_lanes(fmaxf(s[1][b][j], s[1][b][j + 2])), v[1]}, f[b][j]);
                const float x = now.m == -INFINITY ? 0.0f : above<C>(was, now, f[b][j]), r = exp2_approx(x);
                w.m[b][j] = now.m;
                w.limit[b][j] = C::block_scales ? now.e + C::lazy : lag_limit<C>(now.m, f[b][j]);
                const float shift = weight_shift<C>(now.m, f[b][j]);
                w.shift[b][j] = shift;
                far |= is_far(shift);
                w.l[b][j] = lowered<C>(w.l[b][j], x);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    w.o[i][b][j] *= r;
                    w.o[i][b][j + 2] *= r;
                }
            }
        w.far = __any_sync(kFull, far);
    }
    float shift[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) shift[b][j] = C::block_scales ? w.shift[b][j] : weight_shift<C>(w.m[b][j], f[b][j]);
    if (w.far) {    // the rows that are (the others as ever, whatever shares their warp)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool far = is_far(shift[b][j]);
                const float m = far ? w.m[b][j] : 0.0f;
                if (far) shift[b][j] = C::p_shift;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h][b][j] -= m;
                    s[h][b][j + 2] -= m;
                }
            }
    }
    uint32_t pf[2][NB][2];
    // block_scales: the weighted values, 2^(f (s - m) + v - e + p_shift), and from them the
    // weights in units of 2^(e - middle), by 2^(middle - v); where v is below middle the
    // other way round, so that neither underflows for the other.
    int over[2] = {0, 0};
    if constexpr (C::block_scales) {
#pragma unroll
        for (int h = 0; h < 2; ++h) over[h] = static_cast<int>(sc.v[h]) - C::middle;
    }
    const bool low = min(over[0], over[1]) < 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float p[4];
            if constexpr (C::block_scales) {
                // (v - e first, a whole number: shift keeps its bits)
                const float up = fmaxf(v[h], static_cast<float>(C::middle)) + C::lazy, weight = pow2(-max(over[h], 0));
                const float x[2] = {shift[b][0] + (up - w.limit[b][0]), shift[b][1] + (up - w.limit[b][1])};
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = exp2_approx(fmaf(s[h][b][j], f[b][j & 1], x[j & 1]));
                w.l[b][0] = fmaf(p[0] + p[2], weight, w.l[b][0]);
                w.l[b][1] = fmaf(p[1] + p[3], weight, w.l[b][1]);
                if (low) {
                    const float value = pow2(min(over[h], 0));
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] *= value;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = exp2_approx(fmaf(s[h][b][j], f[b][j & 1], shift[b][j & 1]));
                w.l[b][0] += p[0] + p[2];
                w.l[b][1] += p[1] + p[3];
            }
            pf[h][b][0] = transpose8x8(Fp16T::pack(p[0], p[1]));
            pf[h][b][1] = transpose8x8(Fp16T::pack(p[2], p[3]));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        read_values<D>(x[h], st + h * S::half, g, t);
        values16<D, NB>(w, x[h], pf[h]);
    }
}

// Where the warps' states meet; it takes the place of the copied steps.
template <int D, int NB>
struct AttnSmem {
    float o[kAttnWarps][8 * NB][D + 4];
    float m[kAttnWarps][8 * NB], l[kAttnWarps][8 * NB], e[kAttnWarps][8 * NB];
    float f[8 * NB];
};

// Bytes of the ring, or of the join if that is more.
template <class C, int D, int NB>
constexpr int kAttnMem = (kAttnWarps * C::template Step<D>::ring > static_cast<int>(sizeof(AttnSmem<D, NB>))
                              ? kAttnWarps * C::template Step<D>::ring : static_cast<int>(sizeof(AttnSmem<D, NB>)) + 127) / 128 * 128;

// Four dims of an output row, times the row's factor.
template <class E>
__device__ __forceinline__ void store_quad(void* out, int64_t at, float4 o, float inv) {
    reinterpret_cast<uint2*>(out)[at / 4] =
        make_uint2(E::pack(o.x * inv, o.y * inv), E::pack(o.z * inv, o.w * inv));
}

// ln of the sum of the weights: l of them relative to the maximum, times 2^p_shift, and
// with block_scales in units of 2^(e - middle).  (The exponents are added as whole
// numbers: log2f(l) alone may be large, and its rounding with it.)
template <class C>
__device__ __forceinline__ float row_lse(Peak top, float l, float f) {
    if (l == 0.0f) return -INFINITY;
    float log2_l = log2f(l);
    if constexpr (C::block_scales) {
        if (l > 0.0f && l < INFINITY) {
            const uint32_t u = __float_as_uint(l);
            const float whole = static_cast<float>(static_cast<int>(u >> 23) - 127 - C::middle) + top.e;
            log2_l = whole + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
        }
    }
    return fmaf(top.m, f, log2_l - C::p_shift) * 0.693147180559945309f;
}

template <class C, class E, int D, int NB>
__global__ void __launch_bounds__(kAttnThreads) attn_split_kernel(AttnArgs a) {
    constexpr int ROWS = 8 * NB;
    using S = typename C::template Step<D>;
    extern __shared__ __align__(128) unsigned char mem[];
    AttnSmem<D, NB>& sm = *reinterpret_cast<AttnSmem<D, NB>*>(mem);
    int64_t* prefix = reinterpret_cast<int64_t*>(mem + kAttnMem<C, D, NB>);
    allow_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int more = scan_requests<kAttnThreads, true, C::piece>(
        a, prefix, [](int64_t r, bool taken) { return taken ? 0 : (r + ROWS - 1) / ROWS; });
    const int64_t total = prefix[a.requests] * a.kv_heads;
    const int64_t run = run_length(total, a.workers);
    int64_t x = blockIdx.x * run;
    const int64_t end = x + run < total ? x + run : total;
    const float k_gs = C::block_scales ? 1.0f : __ldg(a.k_gs), v_gs = C::block_scales ? 1.0f : __ldg(a.v_gs);
    CutItem cut = {};
    unsigned char* ring = mem + warp * S::ring;

    while (x < end) {
        Req rq;
        const Place at = locate(a, prefix, x, more, rq);
        if (C::piece != 0 && at.tile >= rq.ktiles) {
            x = at.item0 + rq.ktiles + more;
            continue;
        }
        const int ntiles = static_cast<int>(min(static_cast<int64_t>(rq.ktiles - at.tile), end - x));
        const int rows = rq.qlen * a.group;      // of the request
        const int row0 = at.qtile * ROWS;

        // Range of the tile's rows: last key any row sees, and the keys every row sees.
        const int last_row = min(row0 + ROWS, rows) - 1;
        const int pos_min = rq.seq - rq.qlen + row0 / a.group, pos_max = rq.seq - rq.qlen + last_row / a.group;
        const int lo_min = a.window > 0 ? pos_min - a.window + 1 : 0, lo_max = a.window > 0 ? pos_max - a.window + 1 : 0;

        // The warp's steps, one per tile, copied S::stages - 1 steps ahead; the
        // page of a half is read one step before its copy.  Lanes 0-15 care
        // for the first half of a step, lanes 16-31 for the second.
        const int my_half = lane >> 4;
        const int first_key = (rq.tile0 + at.tile) * kAttnKeyTile + warp * 32;
        const int* row_table = a.table + static_cast<int64_t>(at.r) * a.width;
        auto page_of = [&](int j) {
            const int k = first_key + j * kAttnKeyTile + my_half * 16;
            if (j >= ntiles || k > pos_max || k + 15 < lo_min) return -1;
            return __ldg(row_table + (k >> a.page_shift));
        };
        // block_scales: bytes of the lane's half of the steps in flight, keys'
        // then values', loaded with the copies and not touched before their turn
        uint32_t raw[S::stages][2] = {};
        uint32_t have = 0;      // bits 2s, 2s + 1: halves of stage s
        // (a page is compared with their number here and not where it is
        // loaded: the warp would wait for the load there)
        auto issue = [&](int j, int s, int page) {
            if (page >= a.num_pages) page = -1;
            const uint32_t there = __ballot_sync(kFull, page >= 0);
            have = (have & ~(3u << (2 * s))) | (((there & 1u) | (there >> 16 & 1u) << 1) << (2 * s));
            if constexpr (C::block_scales) {
#pragma unroll
                for (int i = 0; i < S::stages - 1; ++i) {
                    raw[i][0] = raw[i + 1][0];
                    raw[i][1] = raw[i + 1][1];
                }
                raw[S::stages - 1][0] = raw[S::stages - 1][1] = 0u;
                if (page >= 0) {
                    const int in = (first_key + j * kAttnKeyTile + my_half * 16) & ((1 << a.page_shift) - 1);
                    const int64_t side = static_cast<int64_t>(a.kv_heads) << (a.page_shift - 4);
                    const uint8_t* p = a.scales + (static_cast<int64_t>(page) * 2 * a.kv_heads + at.head) *
                                                      (int64_t(1) << (a.page_shift - 4)) + (in >> 4);
                    raw[S::stages - 1][0] = __ldg(p);
                    raw[S::stages - 1][1] = __ldg(p + side);
                }
            }
            if (page >= 0)
                C::template copy_half<D>(ring + (s * 2 + my_half) * S::half, a,
                             (first_key + j * kAttnKeyTile + my_half * 16) & ((1 << a.page_shift) - 1), page, at.head,
                             lane & 15);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int j = 0; j < S::stages - 1; ++j) issue(j, j, page_of(j));
        int page = page_of(S::stages - 1);

        // Query fragments: column n = g of block b is row row0 + 8 b + g.
        uint32_t qf[D / 16][NB][2];
        float fs[NB][2];
        int pos[NB][2], lo[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int row = row0 + 8 * b + g;
            uint32_t w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = 0u;
            if (row < rows) {
                const int i = row / a.group, h = at.head * a.group + row % a.group;
                const uint16_t* p = static_cast<const uint16_t*>(a.q) + (rq.q0 + i) * a.q_stride + h * D;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + C::template q_dim<D>(t, j)));
                    w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
                }
            }
            float f = a.scale_log2 / k_gs;
            if constexpr (E::kBits87 == Bf16T::kBits87) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) top = max_abs3(top, E::lo(w[i]), E::hi(w[i]));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                // 2^e brings the row's largest magnitude into [2^14, 2^15)
                const int e = min(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                f *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) w[i] = Fp16T::pack(E::lo(w[i]) * up, E::hi(w[i]) * up);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                qf[i][b][0] = w[2 * i];
                qf[i][b][1] = w[2 * i + 1];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fs[b][j] = clamp_factor(__shfl_sync(kFull, f, (2 * t + j) * 4));
                const int col = row0 + 8 * b + 2 * t + j;
                pos[b][j] = col < rows ? rq.seq - rq.qlen + col / a.group : -1;
                lo[b][j] = a.window > 0 ? pos[b][j] - a.window + 1 : 0;
            }
        }
        WarpState<D, NB> w;
        w.far = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w.m[b][j] = -INFINITY;
                w.limit[b][j] = C::block_scales ? C::lazy : -INFINITY;
                w.shift[b][j] = 0.0f;
                w.l[b][j] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) w.o[i][b][j] = 0.0f;

        for (int j = 0; j < ntiles; ++j) {
            issue(j + S::stages - 1, (j + S::stages - 1) % S::stages, page);
            page = page_of(j + S::stages);
            asm volatile("cp.async.wait_group %0;" :: "n"(S::stages - 1) : "memory");
            __syncwarp();   // every lane's copies of this step are there
            const int s = j % S::stages;
            const uint32_t here = have >> (2 * s) & 3u;
            if (here) {
                const int base = first_key + j * kAttnKeyTile;
                HalfScales sc = {};
                if constexpr (C::block_scales) {
                    const uint32_t own = (here >> my_half & 1u) ? C::scale_codes(raw[0][0], raw[0][1]) : 0u;
                    const uint32_t first = __shfl_sync(kFull, own, 0), second = __shfl_sync(kFull, own, 16);
                    sc = {{first & 0xffu, second & 0xffu}, {first >> 8, second >> 8}};
                }
                attend32<C, D, NB>(w, ring + s * 2 * S::half, qf, fs, pos, lo,
                                   here == 3u && base + 31 <= pos_min && base >= lo_max, here, base, g, t, sc);
            }
            __syncwarp();   // every lane has read the stage that the next copy overwrites
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();

        // Join the warps.
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = w.l[b][j];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
                w.l[b][j] = l;
                if (g == 0) {
                    sm.m[warp][8 * b + 2 * t + j] = w.m[b][j];
                    if constexpr (C::block_scales) sm.e[warp][8 * b + 2 * t + j] = w.limit[b][j] - C::lazy;
                    if (warp == 0) sm.f[8 * b + 2 * t + j] = fs[b][j];
                }
            }
        __syncthreads();
        auto peak_of = [&](int k, int row) { return Peak{sm.m[k][row], C::block_scales ? sm.e[k][row] : 0.0f}; };
        auto top_of = [&](int row, float f) {
            Peak top = peak_of(0, row);
#pragma unroll
            for (int k = 1; k < kAttnWarps; ++k) top = higher<C>(top, peak_of(k, row), f);
            return top;
        };
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * b + 2 * t + j;
                const Peak top = top_of(row, fs[b][j]);
                const float x = above<C>({w.m[b][j], w.limit[b][j] - C::lazy}, top, fs[b][j]);
                float f = w.m[b][j] == -INFINITY ? 0.0f : exp2_approx(x);
                // (without a maximum the sum is 0, or NaN where the logits are)
                if (g == 0) sm.l[warp][row] = w.m[b][j] == -INFINITY ? w.l[b][j] : lowered<C>(w.l[b][j], x);
                // (sums of weighted values in units of 2^(e - 127), of weights in 2^(e -
                // middle): e drops out of their quotient)
                if constexpr (C::block_scales) f *= pow2(C::middle - 127);
                float* dst = &sm.o[warp][row][g * (D / 8)];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    dst[2 * i] = w.o[i][b][j] * f;
                    dst[2 * i + 1] = w.o[i][b][j + 2] * f;
                }
            }
        __syncthreads();
        const bool whole = at.tile == 0 && ntiles == rq.ktiles;
        float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (x == blockIdx.x * run ? 0 : 1)) * ROWS * kPartRow<D>;
        for (int i = tid; i < ROWS * (D / 4); i += kAttnThreads) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                const float4 u = *reinterpret_cast<const float4*>(&sm.o[k][row][d]);
                o.x += u.x; o.y += u.y; o.z += u.z; o.w += u.w;
                l += sm.l[k][row];
            }
            if (whole) {
                if (row0 + row < rows) {
                    const int64_t tok = rq.q0 + (row0 + row) / a.group;
                    const int64_t oh = tok * a.heads + at.head * a.group + (row0 + row) % a.group;
                    store_quad<E>(a.out, oh * D + d, o, l > 0.0f ? 1.0f / (l * v_gs) : (l == 0.0f ? 0.0f : l));
                    if (a.lse && d == 0) a.lse[oh] = row_lse<C>(top_of(row, sm.f[row]), l, sm.f[row]);
                }
            } else {
                *reinterpret_cast<float4*>(part + row * kPartRow<D> + d) = o;
                if (d == 0) {
                    const Peak top = top_of(row, sm.f[row]);
                    *reinterpret_cast<float4*>(part + row * kPartRow<D> + D) = make_float4(top.m, l, sm.f[row], top.e);
                }
            }
        }
        __syncthreads();
        if (at.tile == 0 && ntiles < rq.ktiles)
            cut = {static_cast<int>((at.item0 + rq.ktiles - 1) / run) - static_cast<int>(blockIdx.x) + 1,
                   x == blockIdx.x * run ? 0 : 1, rq.q0, rq.qlen, at.qtile, at.head, {0, 0}};
        x += ntiles;
    }
    if (tid == 0) a.cut[blockIdx.x] = cut;
}

// Joins the parts of the items that the runs cut: CTA (b, y) takes the y-th
// share of the rows of the item that starts in run b and goes past its end.
// Four dims per thread; the threads that a share leaves over split its parts
// and meet in shared memory (in order, so the result does not depend on
// timing).  The split has written down which items those are; a join that
// scanned the lengths again took 20 us for 3 long requests.  The loads of a
// round of four parts are independent: with one part after the other an item of
// 15 parts cost 15 memory latencies, 10 us of a 90 us launch.  One share (gridDim.y = 1) fits all the joins of a ragged batch on
// the card at once; eight shares serve few, long items of many parts.
constexpr int kJoinThreads = 256;
constexpr int kJoinShares = 8;

struct Partial {
    float4 o;
    Peak top;
    float l;
};

// The parts of a row have one factor, `factor`.
__device__ __forceinline__ Partial load_partial(const float* p, int d, int D, float& factor) {
    const float4 o = __ldcg(reinterpret_cast<const float4*>(p + d)), ml = __ldcg(reinterpret_cast<const float4*>(p + D));
    factor = ml.z;
    return {o, {ml.x, ml.w}, ml.y};
}

template <class C>
__device__ __forceinline__ void merge(Partial& a, const Partial& b, float factor) {
    const Peak top = higher<C>(a.top, b.top, factor);
    const float x = a.top.m == -INFINITY ? -INFINITY : above<C>(a.top, top, factor);
    const float y = b.top.m == -INFINITY ? -INFINITY : above<C>(b.top, top, factor);
    const float f = exp2_approx(x), h = exp2_approx(y);
    a.o.x = a.o.x * f + b.o.x * h;
    a.o.y = a.o.y * f + b.o.y * h;
    a.o.z = a.o.z * f + b.o.z * h;
    a.o.w = a.o.w * f + b.o.w * h;
    if constexpr (C::block_scales) a.l = lowered<C>(a.l, x) + lowered<C>(b.l, y);
    else a.l = a.l * f + b.l * h;
    a.top = top;
}

template <class C, class E, int D, int NB>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a) {
    constexpr int ROWS = 8 * NB;
    __shared__ __align__(16) Partial met[kJoinThreads];
    allow_dependents();
    grid_dependency_wait();
    const int4* c = reinterpret_cast<const int4*>(a.cut + blockIdx.x);
    const int4 c0 = __ldcg(c), c1 = __ldcg(c + 1);
    const int parts = c0.x, first_slot = c0.y, head = c1.y;
    if (parts == 0) return;
    const Req rq = {c0.z, c0.w, 0, 0, 0};
    const int w0 = blockIdx.x;
    const float v_gs = a.v_gs ? __ldg(a.v_gs) : 1.0f;
    const int rows = rq.qlen * a.group, row0 = c1.x * ROWS;
    const int64_t slot = ROWS * kPartRow<D>;
    const int quads = ROWS * (D / 4) / static_cast<int>(gridDim.y);      // of this share; a power of two
    const int across = min(quads, kJoinThreads), split = kJoinThreads / across;
    const int quad = threadIdx.x % across, group = threadIdx.x / across;
    for (int q0 = 0; q0 < quads; q0 += across) {
        const int at_quad = blockIdx.y * quads + q0 + quad, row = at_quad / (D / 4), d = at_quad % (D / 4) * 4;
        Partial acc = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), {-INFINITY, 0.0f}, 0.0f};
        auto part = [&](int w) {
            return a.part + (static_cast<int64_t>(w0 + w) * 2 + (w == 0 ? first_slot : 0)) * slot + row * kPartRow<D>;
        };
        float factor = 0.0f;
        for (int w = group; w < parts; w += 4 * split) {
            Partial p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), {-INFINITY, 0.0f}, 0.0f};
                if (w + i * split < parts) p[i] = load_partial(part(w + i * split), d, D, factor);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) merge<C>(acc, p[i], factor);
        }
        met[threadIdx.x] = acc;
        __syncthreads();
        if (group == 0 && row0 + row < rows) {
            for (int i = 1; i < split; ++i) merge<C>(acc, met[i * across + quad], factor);
            const int64_t tok = rq.q0 + (row0 + row) / a.group;
            const int64_t oh = tok * a.heads + head * a.group + (row0 + row) % a.group;
            const float l = acc.l;
            store_quad<E>(a.out, oh * D + d, acc.o, l > 0.0f ? 1.0f / (l * v_gs) : (l == 0.0f ? 0.0f : l));
            if (a.lse && d == 0) a.lse[oh] = row_lse<C>(acc.top, l, factor);
        }
        __syncthreads();
    }
}

}  // namespace rmsq
