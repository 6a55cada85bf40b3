// Stream-ordered scratch of the 4-bit and gated operators (host code).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "internal.h"

namespace gemm_gb300 {

// One memory pool a device, made at its first use and kept for the process; it holds
// up to kScratchKept bytes across synchronisations.  (The device's default pool
// gives everything back whenever the stream is waited for; mapping it anew cost a call
// that is waited for 200 us.)  A pool that could not be made is tried again by the
// next call.  Free with cudaFreeAsync on the same stream.
class ScratchPools {
  public:
    // *p is null, and the runtime's last error cleared, after a failure: the call that
    // asked reports it, and no later one finds it.
    cudaError_t alloc(void **p, size_t bytes, cudaStream_t s) {
        *p = nullptr;
        int dev = 0;
        cudaMemPool_t pool = nullptr;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = dev >= 0 && dev < kMaxDevices ? pool_of(dev, &pool) : cudaErrorInvalidDevice;
        if (e == cudaSuccess) e = cudaMallocFromPoolAsync(p, bytes, pool, s);
        if (e != cudaSuccess) {
            *p = nullptr;
            cudaGetLastError();
        }
        return e;
    }

  private:
    static constexpr unsigned long long kScratchKept = 1ull << 30;

    cudaError_t pool_of(int dev, cudaMemPool_t *out) {
        *out = pools_[dev].load(std::memory_order_acquire);
        if (*out) return cudaSuccess;
        std::lock_guard<std::mutex> lock(mutex_);
        *out = pools_[dev].load(std::memory_order_relaxed);
        if (*out) return cudaSuccess;
        // A thread that captures a stream may not make a pool in the default capture
        // mode, though the capture has no part in it.
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return e;
        cudaMemPoolProps props = {};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t pool = nullptr;
        e = cudaMemPoolCreate(&pool, &props);
        unsigned long long keep = kScratchKept;
        if (e == cudaSuccess) {
            e = cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
            if (e != cudaSuccess) cudaMemPoolDestroy(pool);
        }
        const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return e;
        *out = pool;
        pools_[dev].store(pool, std::memory_order_release);
        return back;
    }

    std::mutex mutex_;
    std::atomic<cudaMemPool_t> pools_[kMaxDevices] = {};
};

}  // namespace gemm_gb300
