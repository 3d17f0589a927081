// Launches of the short kernels (8-bit cache, rotary positions): programmatic
// dependent launch.  Each of these kernels begins with grid_begin(): it waits for
// the kernels before it in the stream to complete, then lets the next such kernel
// be set up on the SMs meanwhile.  Launching one behind the other then costs the
// wait alone, not a launch's latency each (a step of single tokens is a chain of
// kernels of 2 to 10 us).  Such a kernel reads nothing through __ldg or restrict
// pointers: the compiler may move those loads in front of the wait.
#pragma once

#include <atomic>

#include "tq_internal.cuh"

namespace tq {

// Before the kernel's first access to global memory, by all threads.
__device__ __forceinline__ void grid_begin() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
int launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                  const A&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TQ_TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
    return TQ_OK;
}

// Lets a kernel have `bytes` of dynamic shared memory (always the same for one
// kernel): once a device.
template <auto Kernel>
int allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    TQ_TRY_CUDA(cudaGetDevice(&dev));
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return TQ_OK;
    TQ_TRY_CUDA(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done.fetch_or(bit, std::memory_order_relaxed);
    return TQ_OK;
}

}  // namespace tq
