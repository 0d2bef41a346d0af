// qmv_launch.cuh -- launch helpers shared by every translation unit: the
// per-device dynamic shared-memory limit and the launch attributes.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

namespace qmv {

// Per (kernel, device): the dynamic shared-memory limit set so far.
using SmemCfg = std::atomic<int>[64];

// Raises kern's dynamic shared-memory limit on the current device to at least
// smem.  Host threads may race here: the fast path is one atomic load, and the
// raise itself runs under a lock so the limit only ever grows.
template <class Kern>
static cudaError_t ensure_smem(Kern kern, SmemCfg &configured, size_t smem)
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (configured[dev].load(std::memory_order_acquire) >= (int)smem) return cudaSuccess;
    std::lock_guard<std::mutex> lk(mu);
    if (configured[dev].load(std::memory_order_relaxed) >= (int)smem) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    configured[dev].store((int)smem, std::memory_order_release);
    return cudaSuccess;
}

// Launch `kern` with `arg`: raises the dynamic shared-memory limit once per
// (kernel, device) and adds the programmatic-serialization attribute when asked.
template <class Kern, class Arg>
static cudaError_t launch_with(Kern kern, SmemCfg &configured, const Arg &arg, dim3 grid, size_t smem,
                               cudaStream_t stream, bool pdl, bool cooperative = false, int threads = 256)
{
    cudaError_t e = ensure_smem(kern, configured, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    unsigned n_attr = 0;
    if (pdl) {
        attr[n_attr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n_attr].val.programmaticStreamSerializationAllowed = 1;
        ++n_attr;
    }
    if (cooperative) {      // all CTAs co-resident, or the launch fails (grid barriers)
        attr[n_attr].id = cudaLaunchAttributeCooperative;
        attr[n_attr].val.cooperative = 1;
        ++n_attr;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = n_attr ? attr : nullptr;
    cfg.numAttrs = n_attr;
    return cudaLaunchKernelEx(&cfg, kern, arg);
}

}  // namespace qmv
