// The FP8 cache's readers for the attention kernels (rmsq_attn.cuh,
// rmsq_attn_prompt.cuh).
//
// An E4M3 code is exact in f16, so that a code is converted and nothing else: the
// scale of a block of 16 tokens, which is a step's half and a chunk of a logit
// row in the two kernels, is a factor of the block's logits (keys) and of its
// weights (values), and costs nothing per element.  NaN codes of values read as
// 448: a masked place meets a weight of 0, which a NaN would survive (the store
// turns the token's keys to NaN as well, so that queries that see it are told).
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
    static constexpr int stages = D == 64 ? 4 : 2;            // 12, 8 or 16 KB in flight per warp
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

// A converting thread's share of a 128-key tile of the prompt kernel.
template <int D>
struct RawTile8 {
    uint32_t k[D / 4], v[8][D / 32];
    uint32_t ks, vs;        // scale bytes of the key's block, keys' and values'
};

template <int D>
struct Fp8Prompt : Fp8Cache {
    using Raw = RawTile8<D>;
};

template <int D>
__device__ __forceinline__ void load_keys(RawTile8<D>& x, const AttnArgs& a, int key, int kpage, int head) {
    if (kpage >= 0) {
        const int64_t at = static_cast<int64_t>(kpage) * 2 * a.kv_heads + head;
        const int in = key & ((1 << a.page_shift) - 1);
        const uint4* p = reinterpret_cast<const uint4*>(a.cache + ((at << a.page_shift) + in) * D);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) set4(&x.k[4 * j], __ldg(p + j));
        const uint8_t* s = a.scales + (at << (a.page_shift - 4)) + (in >> 4);
        x.ks = __ldg(s);
        x.vs = __ldg(s + (static_cast<int64_t>(a.kv_heads) << (a.page_shift - 4)));
    } else {
#pragma unroll
        for (int j = 0; j < D / 4; ++j) x.k[j] = 0u;
        x.ks = x.vs = 0u;
    }
}

template <int D>
__device__ __forceinline__ void load_values(RawTile8<D>& x, const AttnArgs& a, int key, int vpage, int head, int unit) {
    const int64_t at = (static_cast<int64_t>(max(vpage, 0)) * 2 + 1) * a.kv_heads + head;
    const int in = key & ((1 << a.page_shift) - 1);
    const uint8_t* p = a.cache + ((at << a.page_shift) + in) * D + unit * (D / 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (vpage >= 0) {
            if constexpr (D == 128) {
                set4(x.v[i], __ldg(reinterpret_cast<const uint4*>(p + i * D)));
            } else {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + i * D));
                x.v[i][0] = u.x; x.v[i][1] = u.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) x.v[i][j] = 0u;
        }
    }
}

// K of the thread's key as a row of the operand tile.
template <int D>
__device__ __forceinline__ void write_keys(unsigned char* dst, const RawTile8<D>& x, int row) {
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {       // 8 dims: a 16-byte chunk
        const uint32_t a = x.k[2 * j], b = x.k[2 * j + 1];
        *reinterpret_cast<uint4*>(dst + (j >> 3) * (128 * 128) + row * 128 + (((j & 7) ^ (row & 7)) << 4)) =
            make_uint4(e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b), e4m3x2_to_f16x2(b >> 16));
    }
}

// V of the thread's 8 keys and D/8 dims as 16-byte pieces of V^T's rows.
template <int D>
__device__ __forceinline__ void write_values(unsigned char* dst, const RawTile8<D>& x, int octet, int unit) {
    unsigned char* base = dst + (octet >> 3) * (D * 128);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        uint32_t v[4][4];       // [pair of keys][dim]
#pragma unroll
        for (int p = 0; p < 4; ++p) pair_values(x.v[2 * p][j], x.v[2 * p + 1][j], v[p]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = unit * (D / 8) + 4 * j + c;
            *reinterpret_cast<uint4*>(base + row * 128 + (((octet & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0][c], v[1][c], v[2][c], v[3][c]);
        }
    }
}

}  // namespace rmsq
