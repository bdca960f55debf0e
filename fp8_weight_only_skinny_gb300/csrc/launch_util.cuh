// launch_util.cuh -- host-side launch helpers of the cache and log-probability
// kernels: programmatic dependent launch, clusters and the shared-memory limit.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "internal.h"

namespace sk {

// A scale of the cache: its steps (kv4_append) stay inside binary32's normal
// range for every FP16 input within these bounds.
inline bool kv4_scale_ok(float g) { return g >= 1e-20f && g <= 1e20f; }

// Head sizes the cache's kernels are built for, whole records per page, and
// slot numbers and record numbers (over all heads) that fit 31 bits: 2^31
// records are more than 2 TB.
inline bool kv4_shape_ok(int pages, int heads, int dim, int page) {
    return (dim == 64 || dim == 128 || dim == 256) && page % 16 == 0 &&
           (long long)pages * page <= 0x7FFFFFFFLL && heads <= 4096 &&
           (long long)pages * (page / 16) * heads <= 0x7FFFFFFFLL;
}

// Launch with programmatic dependent launch (while sk_set_pdl allows it) and,
// for cluster > 1, one-dimensional clusters of that many CTAs.  Every kernel
// launched this way waits for its predecessor (griddepcontrol.wait) before it
// touches memory the predecessor may write, in all of its CTAs.
template <typename P, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(P, Args...), int cluster, dim3 grid, dim3 block, size_t smem,
                               cudaStream_t stream, const P &p, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, args...);
}

template <typename P, typename... Args>
cudaError_t launch_pdl(void (*kernel)(P, Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       const P &p, Args... args) {
    return launch_pdl_cluster(kernel, 1, grid, block, smem, stream, p, args...);
}

// Once per kernel and device: allow `smem` bytes of dynamic shared memory
// (always the same number for one kernel) and, where asked, clusters of more
// than eight CTAs.
template <auto Kernel>
cudaError_t prepare_kernel(size_t smem, bool wide_clusters = false) {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess && wide_clusters)
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

// How many clusters of `cluster` CTAs (a power of two up to 16) of this kernel
// the current device runs at a time, after prepare_kernel.  Asked once.
template <auto Kernel>
long long resident_clusters(int cluster, int threads, size_t smem) {
    static std::atomic<int> known[64][5] = {};       // number + 1
    int dev = 0, log2 = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    while ((1 << log2) < cluster) ++log2;
    if (dev < 64) {
        const int v = known[dev][log2].load(std::memory_order_relaxed);
        if (v) return v - 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) return 0;
    if (dev < 64) known[dev][log2].store(n + 1, std::memory_order_relaxed);
    return n;
}

}  // namespace sk
