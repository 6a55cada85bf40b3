// launch_setup.h's look-ups against a CUDA runtime made here (no GPU, no CUDA
// library): an answer is asked for once, a failure again.
#include <cstdio>
#include <cstdlib>

#include "launch_setup.h"

using namespace gemm_gb300::tc;

namespace {
int fail_attr = 0, fail_query = 0, fail_entry = 0, missing_entry = 0;
int attrs = 0, queries = 0, entries = 0, answer = 0, smem_set = 0, asked_cs = 0, asked_threads = 0;
cudaError_t last = cudaSuccess;
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
cudaError_t cudaGetLastError() { const cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) {
    ++attrs;
    smem_set = v;
    return fail_attr-- > 0 ? give(cudaErrorInvalidValue) : cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
    ++queries;
    asked_cs = (int)c->attrs[0].val.clusterDim.x;
    asked_threads = (int)c->blockDim.x;
    *n = 99;
    if (fail_query-- > 0) return give(cudaErrorMemoryAllocation);
    *n = answer;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    ++entries;
    *p = reinterpret_cast<void *>(0x40);
    *q = cudaDriverEntryPointSuccess;
    if (missing_entry-- > 0) { *q = cudaDriverEntryPointSymbolNotFound; *p = nullptr; }
    return fail_entry-- > 0 ? give(cudaErrorUnknown) : cudaSuccess;
}
}

int main() {
    std::atomic<int> known{0}, other{0};
    const int kernel = 0;
    answer = 76;
    fail_attr = 1;
    CHECK(cluster_limit(known, &kernel, 320, 1000, 2) == -1 && queries == 0 && last == cudaSuccess && known == 0);
    fail_attr = 0;
    fail_query = 1;
    CHECK(cluster_limit(known, &kernel, 320, 1000, 2) == -1 && last == cudaSuccess && known == 0);
    fail_query = 0;
    CHECK(cluster_limit(known, &kernel, 320, 1000, 2) == 76 && asked_cs == 2 && asked_threads == 320 && smem_set == 1000);
    const int n = queries;
    CHECK(cluster_limit(known, &kernel, 320, 1000, 2) == 76 && queries == n);
    answer = 0;  // "none" is an answer too
    CHECK(cluster_limit(other, &kernel, 192, 1000, 8) == 0 && cluster_limit(other, &kernel, 192, 1000, 8) == 0);
    CHECK(queries == n + 1);

    fail_entry = 1;
    CHECK(encode_fn() == nullptr && last == cudaSuccess);
    fail_entry = 0;
    missing_entry = 1;
    CHECK(encode_fn() == nullptr);
    missing_entry = 0;
    CHECK(encode_fn() == reinterpret_cast<EncodeTiledFn>(0x40) && encode_fn() == reinterpret_cast<EncodeTiledFn>(0x40));
    CHECK(entries == 3);
    std::puts("ok");
    return 0;
}
