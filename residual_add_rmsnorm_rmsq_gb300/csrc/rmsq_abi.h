// Status helpers shared by the C ABI's translation units (not part of the
// public interface).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace rmsq_abi {

// Records `e` for rmsq_last_cuda_error() on this thread, clears it if it is
// not sticky, and returns RMSQ_ERR_CUDA.
int fail_cuda(cudaError_t e);

// RMSQ_OK when the current device is a compute capability 10.3 part;
// RMSQ_ERR_NO_DEVICE without a CUDA device, RMSQ_ERR_UNSUPPORTED_DEVICE for
// another one, RMSQ_ERR_CUDA (recorded) when the query itself fails.
int check_device();

// Byte ranges of buffers, for the overlap checks.
struct Span {
    uintptr_t lo, hi;   // [lo, hi); empty when lo == hi
};

inline Span span(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + bytes : a};
}

inline bool overlaps(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace rmsq_abi
