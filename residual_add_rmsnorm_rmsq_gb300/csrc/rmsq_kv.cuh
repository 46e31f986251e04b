// The NVFP4 cache format, shared by its store, load and attention.
//
// A cache is u8 [pages, 2 (keys, values), kv heads, tile], one tile of
// P * D * 9 / 16 bytes per page (P tokens), side and head: first the codes,
// [P, D / 2] (element 2j in the low nibble of byte j), then the E4M3 block
// scales, [P, D / 16].  A tile is contiguous, so consecutive tokens of a head
// are read in one piece.
#pragma once

#include "rmsq_device.cuh"

namespace rmsq {

// The eight E2M1 codes of w as four f16 pairs: pair j holds byte j, its low
// nibble first (every E2M1 value is exact in f16).
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

// Value of a stored block scale.  The store writes codes 0x00 .. 0x7e; the
// NaN codes read as 448, so that a page nobody has written yet cannot put a
// NaN into a sum.
__device__ __forceinline__ float nvfp4_scale_value(uint32_t code) {
    const uint32_t c = code & 0x7fu;
    const float v = e4m3_value_nonneg(c);
    return c == 0x7fu ? 448.0f : (code & 0x80u) ? -v : v;
}

// Whether rows of `row` 16-byte chunks at a and b, both at the same stride,
// are separate column ranges of one buffer.
inline bool disjoint_columns(const void* a, const void* b, int64_t stride, int64_t row) {
    const int64_t d = (static_cast<const char*>(b) - static_cast<const char*>(a)) / 16;
    const int64_t m = ((d % stride) + stride) % stride;
    return m >= row && m + row <= stride;
}

}  // namespace rmsq
