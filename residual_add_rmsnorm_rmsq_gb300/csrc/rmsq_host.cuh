// Host-side launch helpers shared by the kernel units.
#pragma once

#include <atomic>
#include <mutex>
#include <cuda_runtime.h>

#include "rmsq_launch.h"

namespace rmsq {

// One kernel launch, with programmatic stream serialisation unless it is
// switched off: the kernel may then start while the previous kernel of the
// stream finishes; the kernels wait for it before any memory access.
inline cudaError_t launch_kernel(const void* fn, dim3 grid, dim3 block, void** params, size_t smem,
                                 cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic_launch() ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, params);
}

// SMs of the current device (cached per device).
inline int sm_count(cudaError_t* err) {
    static std::atomic<int> cached[128];
    int dev = 0;
    *err = cudaGetDevice(&dev);
    if (*err != cudaSuccess || dev < 0 || dev >= 128) return 0;
    int v = cached[dev].load(std::memory_order_acquire);
    if (v == 0) {
        *err = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (*err != cudaSuccess) return 0;
        cached[dev].store(v, std::memory_order_release);
    }
    return v;
}

// One cached occupancy.
struct OccEntry {
    int dev;
    const void* fn;
    int smem;
    int threads;
    int blocks;
};

// Resident CTAs per SM of `fn` at `threads` threads and `smem` dynamic
// shared-memory bytes (cached per device and launch shape).
inline int occupancy_blocks(const void* fn, int threads, int smem, cudaError_t* err) {
    static std::mutex mu;
    constexpr int kCache = 256;   // more than the launch shapes in use; beyond it, queried per call
    static OccEntry cache[kCache];
    static int used = 0;
    int dev = 0;
    *err = cudaGetDevice(&dev);
    if (*err != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].dev == dev && cache[i].fn == fn && cache[i].smem == smem && cache[i].threads == threads)
            return cache[i].blocks;
    int blocks = 0;
    *err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, fn, threads, smem);
    if (*err != cudaSuccess) return 0;
    if (used < kCache) cache[used++] = {dev, fn, smem, threads, blocks};
    return blocks;
}

}  // namespace rmsq
