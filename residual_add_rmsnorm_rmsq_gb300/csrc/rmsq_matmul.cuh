// FP8 matrix product with block scales on the fifth-generation tensor cores.
//
//   out[m, n] = T( sum_kb sa[m, kb] * sb[n / 128, kb] * sum_{k in block kb} a[m, k] * b[n, k] )
//
// a: E4M3 codes [M, K] with one scale per row and 128 columns (what the
// FP8 group-128 modes of this library write), b: E4M3 codes [N, K] with one
// scale per 128 x 128 block.  The scales are general fp32 numbers, so they
// cannot be folded into the operands: the matrix unit sums one block of 128
// products (four K = 32 instructions, accumulator cleared by the first) into
// tensor memory, and the CTA's other warps read that block sum, multiply it by
// its scale and add it to the running sum in fp32 registers, while the matrix
// unit works on the next block in the other half of tensor memory.  That also
// keeps each chain of matrix-unit additions at 128 terms.
//
// Two kernels:
//  mm_rows_kernel    many rows.  Tile 256 rows x BN columns per pair of CTAs,
//                    accumulator lane = row of a, so a thread owns one row: its
//                    scale is one number per block.  Persistent, one CTA per SM.
//                    Each CTA holds 128 rows of a and half the tile's rows of b,
//                    and the matrix units of both read both halves, so that a
//                    CTA fills and reads 64 KB of shared memory per block of K
//                    instead of 96.  8192 x 4096 x 7168: 167 us, 2.88 PFLOP/s.
//                    Bound by the promotion: about 750 clocks per block of 256
//                    columns (465 to read them from tensor memory beside the
//                    products, 130 to add them, the rest hand-overs) where the
//                    products take 512.  What it took: 236 us with 16 columns
//                    read at a time, the scales multiplied next to their loads
//                    and an issuing thread with long waits; 209 with compact
//                    waits and descriptors; 206 with 64 columns at a time; 201 as
//                    a pair; 167 with the next scales loaded into the registers
//                    they are used from (a move of a loaded value waits for it).
//  mm_tokens_kernel  few rows (decode).  Bound by the bytes of b, so b's 128
//                    rows are the accumulator's lanes and the tokens its
//                    16 .. 128 columns, and the blocks of K are split over a
//                    cluster of up to eight CTAs to occupy the card; the
//                    partial sums are joined through distributed shared memory,
//                    in a fixed order.  33 x 4096 x 14336: 13.0 us, 4.6 TB/s of
//                    b; 1 x 4096 x 4096: 5.3 us, half of it launch and the filling
//                    of the ring.
//
// Both: one thread keeps a ring of operand tiles in flight (tensor-map copies,
// 128-byte swizzle), one thread issues the products, the other warps promote.
// Every wait is bounded; a role whose wait runs out records it in a flag the
// host can read, and the CTA drains what it has in flight, frees its tensor
// memory and returns with its output incomplete.
#pragma once

#include "rmsq_tc.cuh"

namespace rmsq {

static __device__ unsigned int g_mm_fault;

struct MmArgs {
    const void* sa;          // fp32 or UE8M0 bytes
    const float* sb;         // [ceil(N / 128), KB]
    void* out;               // T[M, N]
    int64_t sa_row, sa_kb;   // element strides of sa
    int m, n, kb;            // rows of a, rows of b, blocks of 128 along K
    bool ue8m0;
};

// Instruction descriptor: E4M3 x E4M3 -> fp32, both K-major, M x N.
template <int M, int N>
constexpr uint32_t kMmIdesc = (1u << 4) | (static_cast<uint32_t>(N / 8) << 17) | (static_cast<uint32_t>(M / 16) << 24);

// One block of 128 along K: D = A . B^T as four K = 32 products.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}"
                     :: "r"(d), "r"(a + 2 * i), "r"(b + 2 * i), "r"(idesc), "r"(i), "n"(kTileDescHigh) : "memory");
    }
}

// The same over a CTA pair: 128 rows of A in each, half the rows of B in each.
__device__ __forceinline__ void mma_block_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}"
                     :: "r"(d), "r"(a + 2 * i), "r"(b + 2 * i), "r"(idesc), "r"(i), "n"(kTileDescHigh) : "memory");
    }
}

// A scale of a as it lies in memory, and its value.  The kernels load a block's
// scales one block ahead and turn them into a factor only when it is their
// turn: arithmetic on the loaded value next to the load would make the warp,
// which issues in order, wait out the load's latency at every block.
__device__ __forceinline__ uint32_t load_sa(const MmArgs& a, int row, int kb) {
    const int64_t i = row * a.sa_row + kb * a.sa_kb;
    return a.ue8m0 ? __ldg(static_cast<const uint8_t*>(a.sa) + i) : __ldg(static_cast<const uint32_t*>(a.sa) + i);
}
__device__ __forceinline__ float sa_value(const MmArgs& a, uint32_t raw) {
    return __uint_as_float(!a.ue8m0 ? raw : raw ? raw << 23 : 0x00400000u);
}

constexpr int kMmTile = 128 * 128;   // bytes of a 128-row operand tile

// Waits (bounded) for the copies of the last `stages` of `issued` fills.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int issued) {
    for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
        mbar_wait(&full[i % stages], (i / stages) & 1);
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
template <int BN>
struct RowsTile {
    static constexpr int stage_bytes = kMmTile + BN / 2 * 128;      // of one CTA
    static constexpr int stages = 196608 / stage_bytes;     // 6 (BN = 256), 8 (BN = 128)
    static constexpr int buffers = 512 / BN;                // block sums in tensor memory
    static constexpr int staging = 128 * 128;               // 128 rows x 64 columns of T, per warpgroup
    static constexpr int smem = 1024 + stages * stage_bytes + 2 * staging;
};
// Three warpgroups: two promoting, one whose first warp copies and whose second
// issues.  Launched with 168 registers a thread, shared out as 224 + 224 + 56: a
// promoting thread holds up to 128 running sums and 64 block sums.
constexpr int kRowsThreads = 384;
constexpr int kPromoteRegs = 224, kOtherRegs = 56;
static_assert(2 * kPromoteRegs + kOtherRegs == 3 * 168, "the shares are the launch's registers");
constexpr int kRasterRows = 8;      // row tiles per raster group

// Tile `i` of the raster: groups of kRasterRows row tiles, columns outermost
// inside a group, so that the tiles in flight share rows and columns in L2.
__device__ __forceinline__ void raster(int i, int mt, int nt, int& tm, int& tn) {
    const int per = kRasterRows * nt, group = i / per, rest = i - group * per;
    const int rows = min(kRasterRows, mt - group * kRasterRows);
    tn = rest / rows;
    tm = group * kRasterRows + rest - tn * rows;
}

template <class E, int BN>
__global__ void __launch_bounds__(kRowsThreads, 1)
mm_rows_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_out, const MmArgs a) {
    using Tile = RowsTile<BN>;
    constexpr int S = Tile::stages, B = Tile::buffers, HALF = BN / 2;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t full[S], empty[S], tfull[B], tempty[B], drained;
    __shared__ uint32_t tmem_base;
    unsigned char* ring = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    unsigned char* staging = ring + S * Tile::stage_bytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < B; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 16);      // the promoting warps of both CTAs
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    const uint32_t rank = cluster_rank();
    // Tensor memory is taken only once the previous kernel of the stream has
    // ended, and the next one may start only after that: neither can hold
    // columns the other still waits for.
    grid_dependency_wait();
    if (warp == 9) tmem_alloc_pair(&tmem_base, 512);
    tc_fence_before();
    cluster_sync();     // barriers and tensor memory of both CTAs are ready
    tc_fence_after();
    allow_dependents();
    const uint32_t tmem = tmem_base;
    const int mt = (a.m + 255) / 256, nt = (a.n + BN - 1) / BN, tiles = mt * nt;
    const int first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    bool ok = true;

    if (warp == 8) {
        fewer_registers<kOtherRegs>();
        if (lane == 0) {
            int it = 0;
            for (int i = first; i < tiles && ok; i += pairs) {
                int tm, tn;
                raster(i, mt, nt, tm, tn);
                for (int kb = 0; kb < a.kb; ++kb, ++it) {
                    const int s = it % S;
                    ok = mbar_wait(&empty[s], ((it / S) & 1) ^ 1);
                    if (!ok) break;
                    // both CTAs' copies complete on the first one's barrier
                    unsigned char* st = ring + s * Tile::stage_bytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * Tile::stage_bytes);
                    const uint32_t bar = map_to_rank(&full[s], 0);
                    tma_load_2d_pair(st, &map_a, kb * 128, tm * 256 + rank * 128, bar);
                    tma_load_2d_pair(st + kMmTile, &map_b, kb * 128, tn * BN + rank * (BN / 2), bar);
                }
            }
            if (!ok && rank == 0) drain_copies(full, S, it);
        }
    } else if (warp == 9) {
        fewer_registers<kOtherRegs>();
        // The whole warp walks the loop, so that its addresses stay uniform;
        // one lane of the first CTA issues for both.
        if (rank == 0) {
            const bool issuer = elect_one();
            const uint32_t ring_desc = tile_desc(smem_u32(ring));
            int s = 0, b = 0;
            uint32_t phase = 0, tphase = 1;     // parities of full[s] and tempty[b]
            for (int i = first; i < tiles && ok; i += pairs) {
                for (int kb = 0; kb < a.kb; ++kb) {
                    ok = mbar_wait(&full[s], phase) && mbar_wait(&tempty[b], tphase);
                    if (!__all_sync(kFull, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (issuer) {
                        const uint32_t st = ring_desc + s * (Tile::stage_bytes >> 4);
                        mma_block_pair(tmem + b * BN, st, st + (kMmTile >> 4), kMmIdesc<256, BN>);
                        mma_commit_pair(&empty[s]);
                        mma_commit_pair(&tfull[b]);
                    }
                    if (++s == S) {
                        s = 0;
                        phase ^= 1u;
                    }
                    if (++b == B) {
                        b = 0;
                        tphase ^= 1u;
                    }
                }
            }
            if (!ok && issuer) {
                mma_commit_pair(&drained);
                mbar_wait(&drained, 0);
            }
        }
    } else if (warp > 9) {
        fewer_registers<kOtherRegs>();
    } else {
        more_registers<kPromoteRegs>();
        const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        unsigned char* stage = staging + wg * Tile::staging;
        const int64_t sa_bytes = a.ue8m0 ? 1 : 4, sa_step = a.sa_kb * sa_bytes;
        const uint32_t sa_shift = a.ue8m0 ? 23 : 0, sa_zero = a.ue8m0 ? 0x00400000u : 0u;
        const uint32_t tmem_at = tmem + wg * HALF + (static_cast<uint32_t>(quad * 32) << 16),
                       tempty_at = map_to_rank(tempty, 0);
        int b = 0;
        uint32_t tphase = 0;
        // A warp whose wait ran out keeps walking the loop (the warpgroup's
        // barriers need every warp) without waiting or reading any more.
        for (int i = first; i < tiles; i += pairs) {
            int tm, tn;
            raster(i, mt, nt, tm, tn);
            const int m_tile = tm * 256 + static_cast<int>(rank) * 128, m = m_tile + row, n0 = tn * BN + wg * HALF;
            const float* sb = a.sb + static_cast<int64_t>(min(n0, a.n - 1) / 128) * a.kb;
            float2 acc[HALF / 2];
#pragma unroll
            for (int j = 0; j < HALF / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            // The scales of the next block are on their way while this one is
            // promoted, into the registers that this one's have just left.
            // (Rows behind the last hold zeros and are not stored; they take the
            // first row's scales.)
            const unsigned char* sa = static_cast<const unsigned char*>(a.sa) +
                                      (m < a.m ? static_cast<int64_t>(m) * a.sa_row : 0) * sa_bytes;
            uint32_t raw = a.ue8m0 ? __ldg(sa) : __ldg(reinterpret_cast<const uint32_t*>(sa));
            float block = __ldg(sb);
#pragma unroll 1
            for (int kb = 0; kb < a.kb; ++kb) {
                ok = ok && warp_wait(&tfull[b], tphase);
                const uint32_t addr = tmem_at + b * BN, handed = tempty_at + b * 8;
                b = (b + 1) & (B - 1);
                tphase ^= b == 0 ? 1u : 0u;
                if (!ok) continue;
                tc_fence_after();
                // 64 block sums at a time: a load takes some 250 clocks to
                // arrive and the matrix unit waits for the buffer meanwhile
                float d[4][16];
                tmem_ld32(d[0], d[1], addr);
                tmem_ld32(d[2], d[3], addr + 32);
                // meanwhile the factor of this block, and the next one's loads
                // (the byte of a UE8M0 scale is the exponent, 0 standing for 2^-127)
                const float scale = __uint_as_float((raw << sa_shift) | (raw == 0u ? sa_zero : 0u)) * block;
                if (kb + 1 < a.kb) {
                    sa += sa_step;
                    ++sb;
                    raw = a.ue8m0 ? __ldg(sa) : __ldg(reinterpret_cast<const uint32_t*>(sa));
                    block = __ldg(sb);
                }
                const float2 s2 = make_float2(scale, scale);
#pragma unroll
                for (int h = 0; h < HALF / 64; ++h) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_wait(d[c]);
                    if (h + 1 == HALF / 64) {   // the block sums have been read: hand the buffer back
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(handed);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            acc[h * 32 + c * 8 + q] = fma2_rn(make_float2(d[c][2 * q], d[c][2 * q + 1]), s2, acc[h * 32 + c * 8 + q]);
                        if (h + 1 < HALF / 64 && (c & 1))
                            tmem_ld32(d[c - 1], d[c], addr + (h + 1) * 64 + (c - 1) * 16);
                    }
                }
            }
            // Round to T, through shared memory (swizzled as the tensor map
            // says) into 64-column stores; rows and columns beyond the matrix
            // are clipped by the copy.
#pragma unroll
            for (int h = 0; h < HALF / 64; ++h) {
                if (quad == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                named_sync(1 + wg, 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float2* v = &acc[h * 32 + c * 4];
                    *reinterpret_cast<uint4*>(stage + row * 128 + ((c ^ (row & 7)) << 4)) =
                        make_uint4(E::pack(v[0].x, v[0].y), E::pack(v[1].x, v[1].y), E::pack(v[2].x, v[2].y),
                                   E::pack(v[3].x, v[3].y));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                named_sync(1 + wg, 128);
                if (quad == 0 && lane == 0) {
                    if (ok && n0 + h * 64 < a.n && m_tile < a.m) tma_store_2d(&map_out, stage, n0 + h * 64, m_tile);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
        }
        if (quad == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (!ok) atomicOr(&g_mm_fault, 1u);
    __syncwarp();
    tc_fence_before();
    cluster_sync();     // nothing of either CTA reaches into the other any more
    tc_fence_after();
    if (warp == 9) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
constexpr int kTokThreads = 192;    // 4 promoting warps, the copying warp, the issuing warp
constexpr int kTokSmem = 110 * 1024;   // two CTAs per SM, never three: their tensor memory then always fits together

// Shared memory: the ring, then the scales [blocks of this CTA][NT].  The
// ring's space later holds the partial sums [NT][128].
template <int NT>
struct TokTile {
    static constexpr int stage_bytes = kMmTile + NT * 128;
    static constexpr int sums = NT * 128 * 4;
    static constexpr uint32_t cols = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr int max_stages = 8;
};

template <class E, int NT>
__global__ void __launch_bounds__(kTokThreads)
mm_tokens_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const MmArgs a,
                 const int splits, const int stages) {
    using Tile = TokTile<NT>;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t full[Tile::max_stages], empty[Tile::max_stages], tfull[2], tempty[2], drained;
    __shared__ uint32_t tmem_base;
    unsigned char* ring = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    float* scales = reinterpret_cast<float*>(ring + stages * Tile::stage_bytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The cluster spans blockIdx.x: its CTAs share a block of b's rows and
    // divide K.
    const int part = blockIdx.x % splits, tn = blockIdx.x / splits, m0 = blockIdx.y * NT;
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.kb) * part / splits);
    const int nkb = static_cast<int>(static_cast<int64_t>(a.kb) * (part + 1) / splits) - kb0;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    grid_dependency_wait();
    if (warp == 5) tmem_alloc(&tmem_base, Tile::cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    allow_dependents();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    if (warp == 4) {
        if (lane == 0) {
            int kb = 0;
            for (; kb < nkb; ++kb) {
                const int s = kb % stages;
                ok = mbar_wait(&empty[s], ((kb / stages) & 1) ^ 1);
                if (!ok) break;
                unsigned char* st = ring + s * Tile::stage_bytes;
                mbar_arrive_expect_tx(&full[s], Tile::stage_bytes);
                tma_load_2d(st, &map_b, (kb0 + kb) * 128, tn * 128, &full[s]);
                tma_load_2d(st + kMmTile, &map_a, (kb0 + kb) * 128, m0, &full[s]);
            }
            if (!ok) drain_copies(full, stages, kb);
        }
    } else if (warp == 5) {
        const bool issuer = elect_one();
        const uint32_t ring_desc = tile_desc(smem_u32(ring));
        int s = 0;
        uint32_t phase = 0;
        for (int kb = 0; kb < nkb; ++kb) {
            const int b = kb & 1;
            ok = mbar_wait(&tempty[b], ((kb >> 1) & 1) ^ 1) && mbar_wait(&full[s], phase);
            if (!__all_sync(kFull, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (issuer) {
                const uint32_t st = ring_desc + s * (Tile::stage_bytes >> 4);
                mma_block(tmem + b * NT, st, st + (kMmTile >> 4), kMmIdesc<128, NT>);
                mma_commit(&empty[s]);
                mma_commit(&tfull[b]);
            }
            if (++s == stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        if (!ok && issuer) {
            mma_commit(&drained);
            mbar_wait(&drained, 0);
        }
    } else {
        // sa * sb of the CTA's blocks, while the first tiles are on their way
        for (int i = tid; i < nkb * NT; i += 128) {
            const int kb = i / NT, m = m0 + i % NT;
            scales[i] = m < a.m ? sa_value(a, load_sa(a, m, kb0 + kb)) * __ldg(a.sb + static_cast<int64_t>(tn) * a.kb + kb0 + kb) : 0.0f;
        }
        named_sync(1, 128);
        float2 acc[NT / 2];
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
        for (int kb = 0; kb < nkb; ++kb) {
            const int b = kb & 1;
            ok = warp_wait(&tfull[b], (kb >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t addr = tmem + b * NT + (static_cast<uint32_t>(warp * 32) << 16);
            const float4* sc = reinterpret_cast<const float4*>(scales + kb * NT);
            float d[2][16];
            tmem_ld16(d[0], addr);
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                tmem_wait(d[c & 1]);
                if (c + 1 < NT / 16) {
                    tmem_ld16(d[(c + 1) & 1], addr + (c + 1) * 16);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[b]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 s = sc[c * 4 + j];
                    const float* v = &d[c & 1][4 * j];
                    acc[c * 8 + 2 * j] = fma2_rn(make_float2(v[0], v[1]), make_float2(s.x, s.y), acc[c * 8 + 2 * j]);
                    acc[c * 8 + 2 * j + 1] = fma2_rn(make_float2(v[2], v[3]), make_float2(s.z, s.w), acc[c * 8 + 2 * j + 1]);
                }
            }
        }
        if (ok) {   // every product has completed, so nothing reads the ring any more
            float* sums = reinterpret_cast<float*>(ring);
            const int row = warp * 32 + lane;
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                sums[(2 * j) * 128 + row] = acc[j].x;
                sums[(2 * j + 1) * 128 + row] = acc[j].y;
            }
        }
    }
    if (!ok) atomicOr(&g_mm_fault, 1u);
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 5) tmem_free(tmem, Tile::cols);
    // Join: CTA `part` sums its share of the columns over the cluster, in
    // order of K, two rows of b per thread.
    const int c0 = NT * part / splits, c1 = min(NT * (part + 1) / splits, a.m - m0);
    const uint32_t sums = smem_u32(ring);
    for (int i = tid; i < (c1 - c0) * 64; i += kTokThreads) {
        const int c = c0 + i / 64, r = i % 64 * 2, n = tn * 128 + r;
        if (n >= a.n) continue;
        float x = 0.0f, y = 0.0f;
        for (int p = 0; p < splits; ++p) {
            uint32_t at;
            float u, v;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sums + (c * 128 + r) * 4), "r"(p));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(u), "=f"(v) : "r"(at) : "memory");
            x += u;
            y += v;
        }
        static_cast<uint32_t*>(a.out)[(static_cast<int64_t>(m0 + c) * a.n + n) >> 1] = E::pack(x, y);
    }
    cluster_sync();   // the sums stay until every CTA has read them
}

}  // namespace rmsq
