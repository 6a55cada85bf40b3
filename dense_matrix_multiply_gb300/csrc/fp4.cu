// 4-bit block-scaled quantisation of 16-bit rows, and reading it back.
//
// Quantiser.  A lane holds 16 consecutive elements of a row (half an MX block
// or a whole NV block), a warp 512 elements of each of ROWS rows, all of whose
// loads are in flight together; the block's largest magnitude is an integer
// maximum over packed magnitude bits (a NaN is above an infinity is above every
// number), shared between two lanes for MX.  Rows past M and elements past K,
// up to the padded sizes, count as zeros: their scale bytes are written, so
// that no scale that a product reads is left undefined.
// Read-back: a lane writes 16 bytes (eight values), a warp 512 elements of each
// of ROWS rows.
// Rows that do not start on 16 bytes (an odd K, a slice of a wider matrix) are
// loaded 8 bytes at a time, or in whole 16-byte pieces shifted between lanes
// (fp4.h), and stored in such pieces, each lane reading the codes of one.
//
// Bound: HBM, 2 bytes read and 0.53 (MX) or 0.56 (NV) written an element, or the
// other way round; NV's quantiser by its arithmetic nearly as much (a quotient of
// three operations an element, two elements to an instruction).  Measured back to
// back from DRAM: bf16 16384 x 8192 NV quantised in 60.6 us (5.67 TB/s, 0.85 of the
// copy bandwidth) and read back in 53.1 (6.47, 0.97); 4096 x 4096 MX 7.8 and 8.0 us,
// NV 9.7 and 8.2; f16 777 x 12300 NV (rows on 8 bytes) 7.6 and 6.6; 4096 x 4095 NV
// (rows on 2) 13.5 and 11.0, by the instructions of the shifts.  Two rows to a
// warp and four warps to a block: one row 75.9 and 66.1 us for the first, four rows
// 70.5 and 61.3, eight warps 68.4 and 63.7, against 63.3 and 59.4 (before row
// addresses were formed once a row, 12.9 instructions an element of the read-back).
#include <cuda_runtime.h>

#include "fp4.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

constexpr int WARPS = 4, ROWS = 2;

// Block (x, y): rows [8 x, 8 x + 8), elements [512 y, 512 y + 512) and, past
// 65535 x 512 elements, every gridDim.y-th such piece.
template <typename T, bool NV, int VEC>
__global__ void __launch_bounds__(WARPS * 32)
fp4_quantize_kernel(const T *__restrict__ A, long long lda, const float *__restrict__ tensor_scale,
                    uint8_t *__restrict__ Q, long long pitch, uint8_t *__restrict__ S, int M, int K)
{
    // The product that reads these codes may set up, and bring its first weights to
    // L2, meanwhile: linear layer of 32 x 4096 x 12288 (MX) 11.6 us from 12.9, 1024 x
    // 12288 x 4096 (NV) 27.3 from 28.9.
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int row0 = (int)blockIdx.x * (WARPS * ROWS) + (int)(threadIdx.x >> 5) * ROWS;
    const Fp4Tensor t = fp4_tensor<NV>(tensor_scale);
    const uint32_t atoms = (uint32_t)fp4_atoms(NV, K), rb = (uint32_t)fp4_row_bytes(K);
    constexpr uint32_t SPAN = NV ? 1 : 2;  // lanes to a block
    const T *a_row = A + row0 * lda;
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(A),
                  *hi = reinterpret_cast<const uint8_t *>(A + (M - 1) * lda + K);
    uint8_t *q_row = Q + row0 * pitch;
    uint8_t *s_row = S + fp4_scale_at(row0, 0, (int)atoms);  // ROWS divides 32: rows 16 bytes apart
    static_assert(32 % ROWS == 0, "rows of one group of 32");
    for (uint32_t k = blockIdx.y * 512 + lane * 16; k - lane * 16 < (uint32_t)K; k += gridDim.y * 512) {
        uint32_t v[ROWS][8];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int left = row0 + i < M ? (int)((uint32_t)K - k) : -512;
            if (VEC) fp4_load16<VEC>(a_row + i * lda + k, left, v[i]);
            else fp4_load16_any(a_row + i * lda + k, left, lo, hi, v[i]);
        }
        const uint32_t a = k / (64 * SPAN);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = __vmaxu2(m, abs2(v[i][j]));
            m = max(m & 0xFFFFu, m >> 16);
            if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const Fp4Scale sc = fp4_block_scale<NV>(bits16_to_f32<T>(m), t);
            const uint2 codes = fp4_codes16<T, NV>(v[i], sc);
            // four blocks' bytes to one word: lanes 4 j .. 4 j + 3 (NV), 8 j .. 8 j + 7 by twos (MX)
            uint32_t byte = sc.byte;
            byte |= __shfl_down_sync(0xffffffffu, byte, SPAN) << 8;
            byte |= __shfl_down_sync(0xffffffffu, byte, 2 * SPAN) << 16;
            if (lane % (4 * SPAN) == 0 && a < atoms)
                *reinterpret_cast<uint32_t *>(s_row + (size_t)a * 512 + i * 16) = byte;
            if (row0 + i < M && k / 2 < rb) *reinterpret_cast<uint2 *>(q_row + i * pitch + k / 2) = codes;
        }
    }
}

// v s is exact in FP32 (6 significant bits at most); times g one rounding, and one
// to T.
template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(WARPS * 32)
fp4_dequantize_kernel(const uint8_t *__restrict__ Q, const uint8_t *__restrict__ S,
                      const float *__restrict__ tensor_scale, T *__restrict__ A, long long lda, int M, int K)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int row0 = (int)blockIdx.x * (WARPS * ROWS) + (int)(threadIdx.x >> 5) * ROWS;
    const float g = NV && tensor_scale ? *tensor_scale : 1.0f;
    const uint32_t rb = (uint32_t)fp4_row_bytes(K);
    constexpr uint32_t B = fp4_block(NV);
    T *a_row = A + row0 * lda;
    const uint8_t *q_row = Q + (long long)row0 * rb;
    const uint8_t *s_row = S + fp4_scale_at(row0, 0, fp4_atoms(NV, K));  // rows 16 bytes apart, as above
    // VEC: a lane's eight values are k .. k + 7.  Else they are the ones that make up
    // an aligned 16-byte piece of the row: `off` before that, the row's distance from
    // 16 bytes, with the end of one code word and the start of the next, and the
    // scales of two blocks where they fall into two.  (A last piece past the
    // grid's 512 y + 511 is the first blocks' second.)
    for (uint32_t k0 = blockIdx.y * 512 + lane * 8; k0 - lane * 8 < (uint32_t)K + (VEC ? 0 : 7); k0 += gridDim.y * 512) {
        uint32_t codes[ROWS][2], byte[ROWS][2], before[VEC ? 1 : ROWS][2], byte1[VEC ? 1 : ROWS][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = k0 + h * 256;
            const size_t at = (size_t)(k / (4 * B)) * 512 + (k / B & 3);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                codes[i][h] = byte[i][h] = 0u;
                const bool here = row0 + i < M && k / 2 < rb;
                if (here) codes[i][h] = __ldg(reinterpret_cast<const uint32_t *>(q_row + (size_t)i * rb + k / 2));
                if (here) byte[i][h] = __ldg(s_row + at + i * 16);
                if constexpr (!VEC) {
                    before[i][h] = byte1[i][h] = 0u;
                    if (row0 + i < M && k >= 8 && (k - 8) / 2 < rb) {
                        const uint32_t p = k - 8;
                        before[i][h] = __ldg(reinterpret_cast<const uint32_t *>(q_row + (size_t)i * rb + p / 2));
                        byte1[i][h] = __ldg(s_row + (size_t)(p / (4 * B)) * 512 + (p / B & 3) + i * 16);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row0 + i >= M) break;  // warp-uniform
                const uint32_t k = k0 + h * 256;
                const float f = fp4_scale_value<NV>(byte[i][h]);
                T *a = a_row + i * lda + k;
                float2 v[4];
                uint32_t o[4];
                int first = 0, left = min((int)((uint32_t)K - k), 16);  // of the eight values, those in the row
                if constexpr (VEC) {
                    fp4_unpack8(codes[i][h], v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], make_float2(f, f));
                } else {
                    const int off = (int)(((uintptr_t)a & 15) >> 1);
                    // values 0 .. off - 1 are the last `off` of the word before (k - 8 .. k - 1)
                    const float f1 = fp4_scale_value<NV>(byte1[i][h]);
                    const uint32_t c = off ? __funnelshift_l(before[i][h], codes[i][h], 4 * off) : codes[i][h];
                    fp4_unpack8(c, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = mul2(v[j], make_float2(2 * j < off ? f1 : f, 2 * j + 1 < off ? f1 : f));
                    a -= off;
                    left += off;
                    first = k == 0 ? off : 0;  // (nothing lies before the row)
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (NV) v[j] = mul2(v[j], make_float2(g, g));
                    o[j] = tc::pack2(v[j].x, v[j].y, (T *)nullptr);
                }
                if (left >= 8 && first == 0) {
                    *reinterpret_cast<uint4 *>(a) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (2 * j < left && 2 * j >= first) tc::store1(a + 2 * j, v[j].x);
                        if (2 * j + 1 < left && 2 * j + 1 >= first) tc::store1(a + 2 * j + 1, v[j].y);
                    }
                }
            }
    }
}

// Whether every row of A starts on so many bytes.
bool rows_on(const void *A, long long lda, uintptr_t bytes) {
    return (((uintptr_t)A | (uintptr_t)(lda * 2)) & (bytes - 1)) == 0;
}
dim3 grid_of(long long rows, int K) {
    const long long pieces = ((long long)K + 511) / 512;
    return dim3((unsigned)((rows + WARPS * ROWS - 1) / (WARPS * ROWS)), (unsigned)(pieces < 65535 ? pieces : 65535));
}

template <typename T, bool NV>
cudaError_t quantize(const void *A, long long lda, const float *g, void *Q, long long pitch, void *S, int M, int K,
                     cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(grid_of(fp4_row_tiles(M) * 128, K), dim3(WARPS * 32), 0, s, attr);
    auto go = [&](auto kern) {
        return launch_counted(&cfg, kern, static_cast<const T *>(A), lda, g, static_cast<uint8_t *>(Q),
                              pitch, static_cast<uint8_t *>(S), M, K);
    };
    // Rows on 8 bytes: loads of 8 (f16 777 x 12300 NV 7.4 us, in shifted pieces 8.7).
    // On 4 or 2: in pieces (4096 x 4095 NV 13.2 us, value by value 18.9).
    return rows_on(A, lda, 16) ? go(fp4_quantize_kernel<T, NV, 16>)
           : rows_on(A, lda, 8) ? go(fp4_quantize_kernel<T, NV, 8>)
                                : go(fp4_quantize_kernel<T, NV, 0>);
}

template <typename T, bool NV>
cudaError_t dequantize(const void *Q, const void *S, const float *g, void *A, long long lda, int M, int K,
                       cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(grid_of(M, K), dim3(WARPS * 32), 0, s, attr);
    auto go = [&](auto kern) {
        return launch_counted(&cfg, kern, static_cast<const uint8_t *>(Q), static_cast<const uint8_t *>(S), g,
                              static_cast<T *>(A), lda, M, K);
    };
    return rows_on(A, lda, 16) ? go(fp4_dequantize_kernel<T, NV, true>) : go(fp4_dequantize_kernel<T, NV, false>);
}

}  // namespace

cudaError_t launch_fp4_quantize(Elt elt, bool nv, const void *A, long long lda, const float *g, void *Q,
                                long long pitch, void *S, int M, int K, cudaStream_t s) {
    if (elt == Elt::BF16)
        return nv ? quantize<__nv_bfloat16, true>(A, lda, g, Q, pitch, S, M, K, s)
                  : quantize<__nv_bfloat16, false>(A, lda, g, Q, pitch, S, M, K, s);
    return nv ? quantize<__half, true>(A, lda, g, Q, pitch, S, M, K, s)
              : quantize<__half, false>(A, lda, g, Q, pitch, S, M, K, s);
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
