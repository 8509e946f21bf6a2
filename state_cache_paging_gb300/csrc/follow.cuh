// follow.cuh -- launches of kernels that may start while the one before them
// in the stream still runs.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace lmc {

// A kernel launched by follow() waits with the first for the one before it in
// the stream to be done and its writes to be seen; it touches nothing in
// global memory before that (its own arguments are no part of it). It is there
// while the one before writes what it reads, so it reads nothing by the
// read-only path (__ldg, ld.global.nc), which is for memory that does not change
// in a kernel's lifetime, but by plain loads and __ldca. The second
// lets the next one be brought in. The short kernels do that at once, which
// hides its start-up; the attention kernel does not where its own joining (or
// weighing) blocks would be what waits beside it (two requests of 517 tokens
// 11.7 -> 14.3 us, four fp8 ones of 131072 161 -> 173).
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// cluster: 0 for none, else the blocks (along x) of one.
template <typename Plan>
bool follow(void (*kern)(Plan), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Plan &P,
            unsigned cluster = 0) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, P) == cudaSuccess)
        return true;
    cudaGetLastError();  // the caller reports it: not again at another call
    return false;
}

// Lets a kernel's launches take up to `bytes` of dynamic shared memory. The
// limit belongs to the kernel, for all host threads, and the call costs as much
// as a launch: so every caller gives a kernel's largest, and it is set once per
// device (`done`: a bit for each, of this kernel).
template <typename Plan>
bool allow_shared_memory(std::atomic<uint64_t> &done, void (*kern)(Plan), int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

}  // namespace lmc
