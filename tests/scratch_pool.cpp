// ScratchPools against a CUDA runtime made here (no GPU, no CUDA library): what it
// does when a call of the runtime fails, is made by a capturing thread, by two
// threads at once, or on another device.
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include "scratch.h"

namespace {
std::atomic<int> creates{0}, destroys{0}, mallocs{0};
int fail_create = 0, fail_attr = 0, fail_malloc = 0, device = 0, bad_mode = 0;
unsigned long long kept = 0;
int made_on[64];
thread_local cudaStreamCaptureMode mode = cudaStreamCaptureModeGlobal;
thread_local cudaError_t last = cudaSuccess;
cudaError_t give(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
}
void check(bool ok, int line) {
    if (!ok) {
        std::printf("line %d\n", line);
        std::exit(1);
    }
}
#define CHECK(x) check((x), __LINE__)
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { const cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *m) {
    const cudaStreamCaptureMode was = mode;
    mode = *m;
    *m = was;
    return cudaSuccess;
}
cudaError_t cudaMemPoolCreate(cudaMemPool_t *p, const cudaMemPoolProps *props) {
    if (mode != cudaStreamCaptureModeRelaxed) ++bad_mode;
    if (fail_create-- > 0) return give(cudaErrorMemoryAllocation);
    std::this_thread::yield();
    const int n = ++creates;
    made_on[n] = props->location.id;
    *p = reinterpret_cast<cudaMemPool_t>((size_t)n * 16);
    return cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void *v) {
    if (fail_attr-- > 0) return give(cudaErrorInvalidValue);
    kept = *static_cast<unsigned long long *>(v);
    return cudaSuccess;
}
cudaError_t cudaMemPoolDestroy(cudaMemPool_t) { ++destroys; return cudaSuccess; }
cudaError_t cudaMallocFromPoolAsync(void **p, size_t, cudaMemPool_t pool, cudaStream_t) {
    ++mallocs;
    *p = reinterpret_cast<void *>(0x1000);
    if (fail_malloc-- > 0) return give(cudaErrorMemoryAllocation);
    *p = reinterpret_cast<void *>(made_on[reinterpret_cast<size_t>(pool) / 16] + 1);
    return cudaSuccess;
}
}

int main() {
    static gemm_gb300::ScratchPools s;
    void *p = &p;
    // the pool cannot be made: reported, not kept, nothing left behind
    fail_create = 1;
    CHECK(s.alloc(&p, 64, nullptr) == cudaErrorMemoryAllocation && !p && last == cudaSuccess && mallocs == 0);
    CHECK(mode == cudaStreamCaptureModeGlobal);
    // made, but not set up: given back
    fail_attr = 1;
    CHECK(s.alloc(&p, 64, nullptr) == cudaErrorInvalidValue && !p && destroys == 1 && last == cudaSuccess);
    // the next call has its pool
    CHECK(s.alloc(&p, 64, nullptr) == cudaSuccess && p && creates == 2 && kept == 1ull << 30);
    // an allocation fails: the pool stays
    fail_malloc = 1;
    CHECK(s.alloc(&p, 64, nullptr) == cudaErrorMemoryAllocation && !p && last == cudaSuccess);
    CHECK(s.alloc(&p, 64, nullptr) == cudaSuccess && creates == 2 && destroys == 1);
    CHECK(mode == cudaStreamCaptureModeGlobal && bad_mode == 0);
    // another device, first reached by eight threads at once: one pool, its own
    device = 5;
    std::vector<std::thread> t;
    std::atomic<int> good{0};
    for (int i = 0; i < 8; ++i)
        t.emplace_back([&] {
            void *q = nullptr;
            if (s.alloc(&q, 64, nullptr) == cudaSuccess && q == reinterpret_cast<void *>(6)) ++good;
        });
    for (auto &x : t) x.join();
    CHECK(good == 8 && creates == 3);
    device = 0;
    CHECK(s.alloc(&p, 64, nullptr) == cudaSuccess && p == reinterpret_cast<void *>(1) && creates == 3);
    device = gemm_gb300::kMaxDevices;
    CHECK(s.alloc(&p, 64, nullptr) == cudaErrorInvalidDevice && !p);
    std::puts("ok");
    return 0;
}
