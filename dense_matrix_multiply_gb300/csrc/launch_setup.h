// What the launches of the 4-bit, gated, norm, head and update kernels look up once and keep (host code):
// the driver's encoder of TMA descriptors, and how many clusters of a kernel fit the
// device.  Only answers are kept: a look-up that failed is made again by the next call,
// and leaves nothing in the runtime's last error.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace gemm_gb300 {
namespace tc {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_fn() {
    static std::atomic<EncodeTiledFn> known{nullptr};
    EncodeTiledFn fn = known.load(std::memory_order_relaxed);
    if (fn) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    if (q != cudaDriverEntryPointSuccess) return nullptr;
    fn = reinterpret_cast<EncodeTiledFn>(p);
    known.store(fn, std::memory_order_relaxed);
    return fn;
}

// Largest number of co-resident clusters of `cs` CTAs of a kernel, after raising its
// shared-memory limit; -1 if that cannot be told.  known (0 at first): the answer + 1.
inline int cluster_limit(std::atomic<int> &known, const void *kern, int threads, int smem, int cs) {
    int n = known.load(std::memory_order_acquire);
    if (n > 0) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cs, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    known.store(n + 1, std::memory_order_release);
    return n;
}

}  // namespace tc
}  // namespace gemm_gb300
