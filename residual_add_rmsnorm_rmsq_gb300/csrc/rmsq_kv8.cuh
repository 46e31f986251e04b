// The FP8 cache format, shared by its store, load and attention.
//
// Codes: u8 [pages, 2 (keys, values), kv heads, P, D], E4M3; scales: u8
// [pages, 2, kv heads, P / 16], one power of two per block of 16 tokens: byte b
// stands for 2^(b - 127).  An element is code * scale.  A power of two costs
// E4M3 no precision but at its lower end, leaves every product with a scale
// exact, and lets a block whose scale has grown be rounded anew without loss
// (but for codes that become subnormal).
#pragma once

#include "rmsq_device.cuh"

namespace rmsq {

constexpr int kBlockTokens = 16;        // tokens that share a scale
// Scale bytes are 88 .. 187 (2^-39, the first power of two above the floor
// 1e-12, .. 2^60): with codes up to 448 and queries scaled into f16 no logit and
// no sum over values leaves fp32's range.
constexpr uint32_t kScaleMost = 187;

// A scale byte as it is read: what an unwritten block holds cannot become
// infinite or zero.
__device__ __forceinline__ uint32_t cache_scale_code(uint32_t byte) { return min(max(byte, 1u), kScaleMost); }
__device__ __forceinline__ float cache_scale_value(uint32_t code) { return __uint_as_float(code << 23); }

// Two E4M3 codes (low half of w) as an f16 pair; every value is exact, NaN
// codes give NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

}  // namespace rmsq
