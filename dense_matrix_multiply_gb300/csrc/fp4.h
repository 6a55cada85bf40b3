// 4-bit block-scaled matrices: the formats' constants and where a scale byte
// lies.  Shared by the quantiser (fp4.cu) and the products (fp4_gemm.cu,
// fp4_skinny.cu); the formats are described in include/gemm.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"

namespace gemm_gb300 {

// Elements per scale: 32 (MX) or 16 (NV).
__host__ __device__ constexpr int fp4_block(bool nv) { return nv ? 16 : 32; }
// Bytes of one row's codes: two to a byte, rows padded to whole groups of 32
// elements, so that every row starts on 16 bytes.
__host__ __device__ constexpr long long fp4_row_bytes(int K) { return ((long long)K + 31) / 32 * 16; }
// Scale bytes are kept in atoms of 128 rows x 4 blocks, the order in which
// tcgen05.cp's 32x128b form takes them to tensor memory: byte (row % 32) * 16 +
// (row / 32) * 4 + block of 512.  Atoms per tile of 128 rows: K padded to 256.
__host__ __device__ constexpr int fp4_atoms(bool nv, int K) { return (int)(((long long)K + 255) / 256) * (nv ? 4 : 2); }
__host__ __device__ constexpr long long fp4_row_tiles(int rows) { return ((long long)rows + 127) / 128; }
__host__ __device__ constexpr long long fp4_scale_size(bool nv, int rows, int K) {
    return fp4_row_tiles(rows) * fp4_atoms(nv, K) * 512;
}

#ifdef __CUDACC__
// Offset of the four scale bytes of blocks 4 a .. 4 a + 3 of a row.
__device__ __forceinline__ long long fp4_scale_at(int row, int a, int atoms) {
    return ((long long)(row >> 7) * atoms + a) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Scale byte and step of a block from the bits of its largest magnitude
// (|a| as FP32 bits: their order is the values', infinities and NaN on top).
//   MX: e = clamp(floor(log2 amax) - 2, -127, 125), byte e + 127, so that the
//       largest magnitude lies in [4, 8) steps; the exponent field less 2.
//   NV: s = E4M3(amax / (6 g)), step s g.
// A NaN or an infinity makes the scale NaN and the codes 0.  *f is what the
// codes are formed with, 0 for codes of 0: the step (NV: a / step) or its
// reciprocal (MX: a power of two, so that the product is exact).
template <bool NV>
__device__ __forceinline__ uint32_t fp4_block_scale(uint32_t amax_bits, float g6, float g, float *f) {
    const bool bad = amax_bits >= 0x7F800000u;
    if constexpr (NV) {
        const uint32_t b = __nv_cvt_float_to_fp8(__uint_as_float(amax_bits) / g6, __NV_SATFINITE, __NV_E4M3);
        const __half s = __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3));
        *f = bad ? 0.0f : __half2float(s) * g;
        return bad ? 0x7Fu : b;
    } else {
        const int be = (int)(amax_bits >> 23);
        const int byte = be > 2 ? be - 2 : 0;
        *f = bad ? 0.0f : __uint_as_float((uint32_t)(254 - byte) << 23);
        return bad ? 0xFFu : (uint32_t)byte;
    }
}

// Two values in steps, as codes (the first in the low half): nearest, ties to
// the even code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

// Values of eight packed codes times a factor.
__device__ __forceinline__ void fp4_unpack8(uint32_t codes, float f, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * i)) & 255u), __NV_E2M1));
        const float2 p = __half22float2(h);
        v[2 * i] = p.x * f;
        v[2 * i + 1] = p.y * f;
    }
}
template <bool NV>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
    if constexpr (NV) return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// |x| of two packed 16-bit values as packed bits, and the FP32 bits of one.
__device__ __forceinline__ uint32_t abs2(uint32_t v) { return v & 0x7FFF7FFFu; }
template <typename T>
__device__ __forceinline__ uint32_t bits16_to_f32(uint32_t b) {
    if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) return b << 16;
    else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)b)));
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// Codes of the 16 values in v (eight packed pairs) of one block or half block.
template <typename T, bool NV>
__device__ __forceinline__ uint2 fp4_codes16(const uint32_t (&v)[8], float f) {
    uint32_t w[2] = {0u, 0u};
    if (f > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 x = unpack2<T>(v[i]);
            if constexpr (NV) {
                x.x = x.x / f;
                x.y = x.y / f;
            } else {
                x.x *= f;
                x.y *= f;
            }
            w[i >> 2] |= e2m1x2(x.x, x.y) << (8 * (i & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}
#endif

// fp4.cu
cudaError_t launch_fp4_quantize(Elt elt, bool nv, const void *A, long long lda, const float *g, void *Q, void *S,
                                int M, int K, cudaStream_t s);
cudaError_t launch_fp4_dequantize(Elt elt, bool nv, const void *Q, const void *S, const float *g, void *A,
                                  long long lda, int M, int K, cudaStream_t s);

// C [M,N] (leading dimension ldc) = ga gb (Qa Sa)(Qb Sb)^T, FP32 sums.
struct Fp4Problem {
    const void *Qa, *Sa, *Qb, *Sb;
    const float *ga, *gb;  // NV: the tensors' scales (null: 1)
    void *C;
    long long ldc;
    int M, N, K;
    Elt elt;   // of C
    bool nv;
};
// Any M (fp4_gemm.cu).
cudaError_t launch_fp4_gemm(const Fp4Problem &p, int *status, cudaStream_t s);
// M <= kFp4SkinnyMaxM (fp4_skinny.cu); X non-null: the first operand is X [M,K] in
// the element type of C, quantised as it is read (Qa, Sa unused).
constexpr int kFp4SkinnyMaxM = 64;
cudaError_t launch_fp4_skinny(const Fp4Problem &p, const void *X, long long ldx, int num_sms, int *status,
                              cudaStream_t s);

}  // namespace gemm_gb300
