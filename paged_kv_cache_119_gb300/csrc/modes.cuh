// modes.cuh -- host launchers of the attention kernels in their other modes (modified
// scores, shared prefix, suffix; AttnMode in pa_internal.h).  Each modes_*.cu instantiates
// one kernel family.
#pragma once

#include <atomic>

#include "pa_internal.h"

namespace pa {

constexpr int kMaxCachedDevices = 64;

// Launches a kernel; with overlap it may start before the kernel in front of it has completed
// (as soon as all CTAs of that one have allowed it or left) and has to wait for what it needs.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, bool overlap,
                          cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (err != cudaSuccess)
        (void)cudaGetLastError();                // reported to the caller: not left for a later call
    return err;
}

// Whether the kernel may start while the one before it in the stream still runs.
inline bool may_overlap(const DecodeParams& p) { return p.overlap != 0; }
template <typename T>
bool may_overlap(const T&)
{
    return false;
}

// Launches one kernel variant V (kernel(), configure(), smem_bytes, threads) over
// (partitions, kv heads * chunks, sequences or groups).
template <typename V, typename... Args>
cudaError_t launch_mode_variant(dim3 grid, cudaStream_t stream, const Args&... args)
{
    cudaError_t err = V::configure();
    if (err != cudaSuccess)
        return err;
    return launch_behind(V::kernel(), grid, dim3(V::kThreads), V::kSmem, (may_overlap(args) || ...),
                         stream, args...);
}

// Resident CTAs per SM of variant V (0 if unknown).  Asked once per device: the query costs
// about a microsecond of host time, and a call asks for one or two kernels.
template <typename V>
int occupancy_mode_variant()
{
    static std::atomic<int> known[kMaxCachedDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    if (cached) {
        const int n = known[dev].load(std::memory_order_relaxed);
        if (n > 0)
            return n;
    }
    int n = 0;
    if (V::configure() != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, V::kernel(), V::kThreads, V::kSmem) !=
            cudaSuccess)
        return 0;
    if (cached)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace pa
