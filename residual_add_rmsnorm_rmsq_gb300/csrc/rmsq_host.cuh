// Host-side launch helpers shared by the kernel units.
#pragma once

#include <atomic>
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

}  // namespace rmsq
