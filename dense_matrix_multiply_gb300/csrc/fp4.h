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
// Rows of codes in scratch start on 128 bytes: a TMA load of 128 bytes a row then
// asks L2 for one line a row, not two (fp4_gemm.cu).
__host__ __device__ constexpr long long fp4_scratch_pitch(int K) { return (fp4_row_bytes(K) + 127) / 128 * 128; }
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

// A quotient rounded to nearest as IEEE division rounds it, from the correctly
// rounded reciprocal y of the divisor: with q = a y the remainder a - q b is exact
// in one FMA, and q + remainder * y is the correctly rounded quotient (Markstein,
// IBM J. Res. Dev. 34, 1990).  Three operations where a division takes about ten;
// valid away from the ends of FP32's range.
__device__ __forceinline__ float quotient(float a, float b, float y) {
    const float q = a * y;
    return fmaf(fmaf(-q, b, a), y, q);
}

// The tensor's scale and what blocks need of it.
struct Fp4Tensor {
    float g, g6, y6;  // g, 6 g, 1 / (6 g)
    bool mid;         // 6 g far from the ends of FP32's range: quotients by quotient()
};
template <bool NV>
__device__ __forceinline__ Fp4Tensor fp4_tensor(const float *tensor_scale) {
    Fp4Tensor t;
    t.g = NV && tensor_scale ? *tensor_scale : 1.0f;
    t.g6 = 6.0f * t.g;
    t.y6 = __frcp_rn(t.g6);
    t.mid = t.g6 >= 0x1p-60f && t.g6 <= 0x1p60f;
    return t;
}

// A block's scale byte, and what its codes are formed with.
struct Fp4Scale {
    uint32_t byte;
    float step;  // NV: the step.  0 (both): codes of 0
    float inv;   // 1 / step: MX a power of two, exact; NV correctly rounded
    bool near;   // NV: a / step by quotient()
};
// From the bits of the block's largest magnitude (|a| as FP32 bits: their order
// is the values', infinities and NaN on top).
//   MX: e = clamp(floor(log2 amax) - 2, -127, 125), byte e + 127, so that the
//       largest magnitude lies in [4, 8) steps; the exponent field less 2.
//   NV: s = E4M3(amax / (6 g)), step s g; a block of zeros has s = 0 whatever g is (a
//       tensor of zeros has g = 0, and 0 / 0 would make its scale NaN).
// A NaN or an infinity makes the scale NaN and the codes 0.
// (quotient() here: an amax below 2^-80, where the remainder could underflow, is
// under 2^-20 steps of s and rounds to 0 either way; of the codes, a value below
// 2^-4 steps likewise; a block far into saturation divides.)
template <bool NV>
__device__ __forceinline__ Fp4Scale fp4_block_scale(uint32_t amax_bits, const Fp4Tensor &t) {
    const bool bad = amax_bits >= 0x7F800000u;
    Fp4Scale r;
    if constexpr (NV) {
        const float amax = bad ? 0.0f : __uint_as_float(amax_bits);
        const float v = amax == 0.0f                  ? 0.0f
                        : t.mid && amax <= 0x1p60f ? quotient(amax, t.g6, t.y6)
                                                   : amax / t.g6;
        r.byte = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
        r.step = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)r.byte, __NV_E4M3))) * t.g;
        r.inv = __frcp_rn(r.step);
        r.near = t.mid && amax <= 1024.0f * r.step;
        if (bad) {
            r.byte = 0x7Fu;
            r.step = 0.0f;
        }
    } else {
        const int be = (int)(amax_bits >> 23);
        const int byte = be > 2 ? be - 2 : 0;
        r.byte = bad ? 0xFFu : (uint32_t)byte;
        r.inv = __uint_as_float((uint32_t)(254 - byte) << 23);
        r.step = bad ? 0.0f : 1.0f;
        r.near = true;
    }
    return r;
}

// What a product's FP32 sums are multiplied with, one factor after the other: ga gb and
// 1 where ga gb is a normal number, or one of them is 0; else (two small scales, or
// two large ones) the larger and then the smaller, since ga gb would lose bits, vanish
// or be infinite where the result need not.
struct Fp4Factors {
    float first, second;
};
template <bool NV>
__device__ __forceinline__ Fp4Factors fp4_factors(const float *ga, const float *gb) {
    if (!NV) return {1.0f, 1.0f};
    const float a = ga ? *ga : 1.0f, b = gb ? *gb : 1.0f, p = a * b;
    if ((p >= 0x1p-126f && p < __int_as_float(0x7F800000)) || a == 0.0f || b == 0.0f) return {p, 1.0f};
    return a >= b ? Fp4Factors{a, b} : Fp4Factors{b, a};
}

// Eight values in steps as codes, the first in the lowest four bits: nearest,
// ties to the even code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float2 &a, const float2 &b, const float2 &c, const float2 &d) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 mul2(const float2 &a, const float2 &b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(const float2 &a, const float2 &b, const float2 &c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Values of eight packed codes, in pairs.
__device__ __forceinline__ void fp4_unpack8(uint32_t codes, float2 (&v)[4]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
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

// The first `left` of 16 values (eight packed pairs), the others 0.
__device__ __forceinline__ void fp4_keep(int left, uint32_t (&v)[8]) {
    if (left >= 16) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 2 * i + 1 < left ? v[i] : 2 * i < left ? v[i] & 0xFFFFu : 0u;
}
// 16 consecutive values at a, of which `left` are in the row: a on VEC = 16 or 8
// bytes, or (2) value by value.
template <int VEC>
__device__ __forceinline__ void fp4_load16(const void *a, int left, uint32_t (&v)[8]) {
    if (VEC == 16 && left >= 16) {
        const uint4 u0 = __ldg(static_cast<const uint4 *>(a)), u1 = __ldg(static_cast<const uint4 *>(a) + 1);
        v[0] = u0.x; v[1] = u0.y; v[2] = u0.z; v[3] = u0.w;
        v[4] = u1.x; v[5] = u1.y; v[6] = u1.z; v[7] = u1.w;
        return;
    }
    if (VEC == 8 && left >= 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 u = __ldg(static_cast<const uint2 *>(a) + i);
            v[2 * i] = u.x;
            v[2 * i + 1] = u.y;
        }
        return;
    }
    const unsigned short *h = static_cast<const unsigned short *>(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 2 * i < left ? (uint32_t)__ldg(h + 2 * i) : 0u;
        if (2 * i + 1 < left) v[i] |= (uint32_t)__ldg(h + 2 * i + 1) << 16;
    }
}

// Rows that do not start on 16 bytes: a warp takes 16 values to a lane with loads
// of whole 16-byte pieces all the same, the pieces shifted by d bytes, the distance
// of a lane's first value from its piece (even, the same in all lanes), and each
// lane's last part from the lane after it.  The pieces' other bytes are of the same
// matrix (or are not read: load_piece).
// An aligned 16-byte piece of [lo, hi): whole, or its values one by one at the ends.
__device__ __forceinline__ uint4 load_piece(const uint8_t *p, const uint8_t *lo, const uint8_t *hi) {
    if (p >= lo && p + 16 <= hi) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint8_t *q = p + 2 * i;
        if (q >= lo && q < hi) w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(q)) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int WORDS>
__device__ __forceinline__ void fp4_shift_words(const uint32_t (&w)[12], int d, uint32_t (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __funnelshift_r(w[i + WORDS], w[i + WORDS + 1], 8 * (d & 2));
}
// The whole warp: the 16 values at a (lane l: base + 16 l values), of which `left`
// are in the row (K - k, so below 0 past its end; -32 or less in every lane for no
// row); [lo, hi): the matrix.
__device__ __forceinline__ void fp4_load16_any(const void *a, int left, const uint8_t *lo, const uint8_t *hi,
                                               uint32_t (&v)[8]) {
    const uint8_t *p = static_cast<const uint8_t *>(a);
    const int d = (int)((uintptr_t)p & 15);
    const uint8_t *q = p - d, *end = p + 2 * (long long)left;  // of the row, the same in all lanes
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 a0 = q < end ? load_piece(q, lo, hi) : zero;  // (may hold the last values of the lane before)
    const uint4 a1 = q + 16 < end ? load_piece(q + 16, lo, hi) : zero;
    uint32_t w[12] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    w[8] = __shfl_down_sync(0xffffffffu, a0.x, 1);
    w[9] = __shfl_down_sync(0xffffffffu, a0.y, 1);
    w[10] = __shfl_down_sync(0xffffffffu, a0.z, 1);
    w[11] = __shfl_down_sync(0xffffffffu, a0.w, 1);
    if ((threadIdx.x & 31) == 31 && d != 0 && q + 32 < end) {
        const uint4 a2 = load_piece(q + 32, lo, hi);
        w[8] = a2.x; w[9] = a2.y; w[10] = a2.z; w[11] = a2.w;
    }
    switch (d >> 2) {  // the same in all lanes
    case 0: fp4_shift_words<0>(w, d, v); break;
    case 1: fp4_shift_words<1>(w, d, v); break;
    case 2: fp4_shift_words<2>(w, d, v); break;
    default: fp4_shift_words<3>(w, d, v); break;
    }
    fp4_keep(left, v);
}

// Codes of the 16 values in v (eight packed pairs) of one block or half block.
template <typename T, bool NV>
__device__ __forceinline__ uint2 fp4_codes16(const uint32_t (&v)[8], const Fp4Scale &s) {
    if (!(s.step > 0.0f)) return make_uint2(0u, 0u);
    float2 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = unpack2<T>(v[i]);
    if (NV && !s.near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(x[i].x / s.step, x[i].y / s.step);
    } else {
        const float2 y = make_float2(s.inv, s.inv), b = make_float2(-s.step, -s.step);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 q = mul2(x[i], y);
            x[i] = NV ? fma2(fma2(q, b, x[i]), y, q) : q;  // quotient(), two at a time
        }
    }
    return make_uint2(e2m1x8(x[0], x[1], x[2], x[3]), e2m1x8(x[4], x[5], x[6], x[7]));
}
#endif

// fp4.cu; pitch: bytes from one row's codes to the next's.
cudaError_t launch_fp4_quantize(Elt elt, bool nv, const void *A, long long lda, const float *g, void *Q,
                                long long pitch, void *S, int M, int K, cudaStream_t s);
cudaError_t launch_fp4_dequantize(Elt elt, bool nv, const void *Q, const void *S, const float *g, void *A,
                                  long long lda, int M, int K, cudaStream_t s);

// C [M,N] (leading dimension ldc) = ga gb (Qa Sa)(Qb Sb)^T, FP32 sums.
struct Fp4Problem {
    const void *Qa, *Sa, *Qb, *Sb;
    long long pitch_a, pitch_b;  // bytes from one row's codes to the next's
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
