// Product of two 4-bit block-scaled matrices on the CUDA cores: 64 x 64 tiles
// of C, both operands decoded to FP32 in shared memory 32 k at a time.
#include <cuda_runtime.h>

#include "fp4.h"

namespace gemm_gb300 {
namespace {

__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half *p, float x) { *p = __float2half_rn(x); }

template <typename T, bool NV>
__global__ void __launch_bounds__(256) fp4_simt_kernel(const Fp4Problem p)
{
    pdl_wait();
    __shared__ float a_s[32][65], b_s[32][65];
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3;  // row of the tile, group of 8 k
    const int atoms = fp4_atoms(NV, p.K);
    constexpr int B = fp4_block(NV);
    float acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 32) {
        const int k = k0 + c * 8;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int row = (side ? n0 : m0) + r;
            float v[8] = {};
            if (row < (side ? p.N : p.M)) {
                const uint8_t *q = static_cast<const uint8_t *>(side ? p.Qb : p.Qa);
                const uint8_t *s = static_cast<const uint8_t *>(side ? p.Sb : p.Sa);
                const uint32_t byte = s[fp4_scale_at(row, k / (4 * B), atoms) + (k / B & 3)];
                fp4_unpack8(*reinterpret_cast<const uint32_t *>(q + row * fp4_row_bytes(p.K) + k / 2),
                            fp4_scale_value<NV>(byte), v);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) (side ? b_s : a_s)[c * 8 + i][r] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 32; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a_s[kk][ty + 16 * i], b_s[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    const float f = NV ? (p.ga ? *p.ga : 1.0f) * (p.gb ? *p.gb : 1.0f) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) put(static_cast<T *>(p.C) + m * p.ldc + n, acc[i][j] * f);
        }
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Problem &p, int num_sms, int *status, cudaStream_t s) {
    (void)num_sms;
    (void)status;
    const dim3 grid((unsigned)((p.N + 63LL) / 64), (unsigned)((p.M + 63LL) / 64));
    if (grid.y > 65535) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(grid, dim3(256), 0, s, attr);
    if (p.elt == Elt::BF16)
        return p.nv ? launch_counted(&cfg, fp4_simt_kernel<__nv_bfloat16, true>, p)
                    : launch_counted(&cfg, fp4_simt_kernel<__nv_bfloat16, false>, p);
    return p.nv ? launch_counted(&cfg, fp4_simt_kernel<__half, true>, p)
                : launch_counted(&cfg, fp4_simt_kernel<__half, false>, p);
}

}  // namespace gemm_gb300
