// 4-bit block-scaled quantisation of 16-bit rows, and reading it back.
//
// Quantiser.  A lane holds 16 consecutive elements of a row (half an MX block
// or a whole NV block), a warp 512; the block's largest magnitude is an integer
// maximum over packed magnitude bits (a NaN is above an infinity is above every
// number), shared between two lanes for MX.  Rows past M and elements past K,
// up to the padded sizes, count as zeros: their scale bytes are written, so
// that no scale that a product reads is left undefined.
// Bound: HBM, 2 bytes read and 0.53 (MX) or 0.56 (NV) written an element.
#include <cuda_runtime.h>

#include "fp4.h"

namespace gemm_gb300 {
namespace {

constexpr int WARPS = 8;

template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(WARPS * 32)
fp4_quantize_kernel(const T *__restrict__ A, long long lda, const float *__restrict__ tensor_scale,
                    uint8_t *__restrict__ Q, uint8_t *__restrict__ S, int M, int K, int segs, long long units)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);  // one row's 512 elements
    if (unit >= units) return;
    const int row = (int)(unit / segs);
    const int k = (int)(unit - (long long)row * segs) * 512 + lane * 16;
    const float g = NV && tensor_scale ? *tensor_scale : 1.0f;
    uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (row < M && k < K) {
        const T *a = A + row * lda + k;
        if (VEC && k + 16 <= K) {
            const uint4 u0 = __ldg(reinterpret_cast<const uint4 *>(a)), u1 = __ldg(reinterpret_cast<const uint4 *>(a) + 1);
            v[0] = u0.x; v[1] = u0.y; v[2] = u0.z; v[3] = u0.w;
            v[4] = u1.x; v[5] = u1.y; v[6] = u1.z; v[7] = u1.w;
        } else {
            const unsigned short *h = reinterpret_cast<const unsigned short *>(a);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k + i < K) v[i >> 1] |= (uint32_t)__ldg(h + i) << (16 * (i & 1));
        }
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, abs2(v[i]));
    m = max(m & 0xFFFFu, m >> 16);
    if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const Fp4Scale sc = fp4_block_scale<NV>(bits16_to_f32<T>(m), 6.0f * g, g);
    const uint2 codes = fp4_codes16<T, NV>(v, sc);
    uint32_t byte = sc.byte;
    // four blocks' bytes to one word: lanes 4 i .. 4 i + 3 (NV), 8 i .. 8 i + 7 by twos (MX)
    constexpr int SPAN = NV ? 1 : 2;  // lanes to a block
    byte |= __shfl_down_sync(0xffffffffu, byte, SPAN) << 8;
    byte |= __shfl_down_sync(0xffffffffu, byte, 2 * SPAN) << 16;
    const int atoms = fp4_atoms(NV, K);
    const int a = k / (64 * SPAN);
    if (lane % (4 * SPAN) == 0 && a < atoms)
        *reinterpret_cast<uint32_t *>(S + fp4_scale_at(row, a, atoms)) = byte;
    const long long rb = fp4_row_bytes(K);
    if (row < M && k / 2 < rb) *reinterpret_cast<uint2 *>(Q + row * rb + k / 2) = codes;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// A lane reads eight codes (4 bytes) and their block's scale and writes eight
// values (16 bytes).  v s is exact in FP32 (6 significant bits at most); times
// g one rounding, and one to T.
template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(WARPS * 32)
fp4_dequantize_kernel(const uint8_t *__restrict__ Q, const uint8_t *__restrict__ S,
                      const float *__restrict__ tensor_scale, T *__restrict__ A, long long lda, int M, int K, int segs,
                      long long units)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);  // one row's 256 elements
    if (unit >= units) return;
    const int row = (int)(unit / segs);
    const int k = (int)(unit - (long long)row * segs) * 256 + lane * 8;
    if (k >= K) return;
    const float g = NV && tensor_scale ? *tensor_scale : 1.0f;
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(Q + row * fp4_row_bytes(K) + k / 2);
    constexpr int B = fp4_block(NV);
    const uint32_t byte = S[fp4_scale_at(row, k / (4 * B), fp4_atoms(NV, K)) + (k / B & 3)];
    float v[8];
    fp4_unpack8(codes, fp4_scale_value<NV>(byte), v);
    T *a = A + row * lda + k;
    T o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = from_f32<T>(NV ? v[i] * g : v[i]);
    if (VEC && k + 8 <= K) {
        uint4 w;
        memcpy(&w, o, 16);
        *reinterpret_cast<uint4 *>(a) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) a[i] = o[i];
    }
}

template <typename T, bool NV>
cudaError_t quantize(const void *A, long long lda, const float *g, void *Q, void *S, int M, int K, cudaStream_t s) {
    const int segs = (int)(((long long)K + 511) / 512);
    const long long units = fp4_row_tiles(M) * 128 * segs;
    const long long blocks = (units + WARPS - 1) / WARPS;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(WARPS * 32), 0, s, attr);
    const T *a = static_cast<const T *>(A);
    uint8_t *q = static_cast<uint8_t *>(Q), *sc = static_cast<uint8_t *>(S);
    if (((uintptr_t)A & 15u) == 0 && lda % 8 == 0)
        return launch_counted(&cfg, fp4_quantize_kernel<T, NV, true>, a, lda, g, q, sc, M, K, segs, units);
    return launch_counted(&cfg, fp4_quantize_kernel<T, NV, false>, a, lda, g, q, sc, M, K, segs, units);
}

template <typename T, bool NV>
cudaError_t dequantize(const void *Q, const void *S, const float *g, void *A, long long lda, int M, int K,
                       cudaStream_t s) {
    const int segs = (int)(((long long)K + 255) / 256);
    const long long units = (long long)M * segs;
    const long long blocks = (units + WARPS - 1) / WARPS;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(WARPS * 32), 0, s, attr);
    const uint8_t *q = static_cast<const uint8_t *>(Q), *sc = static_cast<const uint8_t *>(S);
    T *a = static_cast<T *>(A);
    if (((uintptr_t)A & 15u) == 0 && lda % 8 == 0)
        return launch_counted(&cfg, fp4_dequantize_kernel<T, NV, true>, q, sc, g, a, lda, M, K, segs, units);
    return launch_counted(&cfg, fp4_dequantize_kernel<T, NV, false>, q, sc, g, a, lda, M, K, segs, units);
}

}  // namespace

cudaError_t launch_fp4_quantize(Elt elt, bool nv, const void *A, long long lda, const float *g, void *Q, void *S,
                                int M, int K, cudaStream_t s) {
    if (elt == Elt::BF16)
        return nv ? quantize<__nv_bfloat16, true>(A, lda, g, Q, S, M, K, s)
                  : quantize<__nv_bfloat16, false>(A, lda, g, Q, S, M, K, s);
    return nv ? quantize<__half, true>(A, lda, g, Q, S, M, K, s) : quantize<__half, false>(A, lda, g, Q, S, M, K, s);
}

cudaError_t launch_fp4_dequantize(Elt elt, bool nv, const void *Q, const void *S, const float *g, void *A,
                                  long long lda, int M, int K, cudaStream_t s) {
    if (elt == Elt::BF16)
        return nv ? dequantize<__nv_bfloat16, true>(Q, S, g, A, lda, M, K, s)
                  : dequantize<__nv_bfloat16, false>(Q, S, g, A, lda, M, K, s);
    return nv ? dequantize<__half, true>(Q, S, g, A, lda, M, K, s)
              : dequantize<__half, false>(Q, S, g, A, lda, M, K, s);
}

}  // namespace gemm_gb300
