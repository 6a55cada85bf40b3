/*
 * gemm.h -- C ABI of the GB300 (sm_103a) dense GEMM library.
 *
 * Every entry point computes C = A·B: C[i,j] = sum_k A[i,k]*B[k,j], 2*M*N*K
 * floating-point operations, with the sum accumulated in FP32 and rounded once
 * to the output type (round to nearest, ties to even).  Sources of the
 * operation:
 *   - the FP32 SGEMM and its FLOP convention: "SGEMM measured and the three
 *     ledgers" (section 2, the cuBLAS baseline in pure FP32 with TF32 off;
 *     K3 step 3, GFLOP/s = 2*M*N*K / t);
 *   - the half, column-major variant: "MTT S4000 FP16 GEMM", section 1 (the
 *     fixed contest signature gemm_optimized(d_A, d_B, d_C, M, N, K): A, B, C
 *     column-major, half in and out, FP32 accumulation);
 *   - the bf16, row-major projection: "Chapter 5 Operators and Runtime",
 *     section 5.2.1 (the FFN projection C = X·W, BF16 inputs, FP32 accumulator,
 *     the element loop over i, j, k) and figure 5-7.
 * alpha = 1 and beta = 0: C is write-only, never read.
 *
 * Pointers.  A, B and C are DEVICE pointers (cudaMalloc, torch CUDA tensors,
 * or any memory the current device can address), owned by the caller.  The
 * library keeps no reference to them after the call.  Half and bf16 elements
 * are passed as their 16-bit patterns.  Memory the library uses besides A, B,
 * C: one 4-byte status word per device (cudaMalloc on first use); and, only for
 * a 16-bit problem with M > 128, N >= 1024 whose A rows are not 16-byte
 * aligned (e.g. bf16 with K = 4100), an aligned copy of A taken from the
 * device's default stream-ordered pool (cudaMallocAsync / cudaFreeAsync on the
 * caller's stream); if that allocation fails the call uses a slower kernel
 * instead.  A 16-bit problem on the CTA-pair tensor-core kernel whose tiles
 * leave a nearly empty last wave (at most a quarter of the clusters busy, K of
 * at least 48 blocks of 64) takes FP32 partial tiles for its stream-K tail from
 * the same pool (512 KiB per participating CTA pair, at most ~39 MB), freed on
 * the stream after the call; without it the call runs whole tiles.  The other entry
 * points' scratch is named below, with them.  The allocation-free entry point
 * never allocates.
 *
 * Leading dimensions are tight:
 *   _rm (row-major):    A is [M,K] with lda = K, B is [K,N] with ldb = N,
 *                       C is [M,N] with ldc = N.
 *   _cm (column-major): A is [M,K] with lda = M, B is [K,N] with ldb = K,
 *                       C is [M,N] with ldc = M.
 * Any alignment is accepted.  Pointers or strides that are not 16-byte aligned
 * select slower kernels; they are never an error.
 *
 * Execution.  Calls are asynchronous and ordered on the calling host thread's
 * stream (gemm_set_stream; default: the legacy default stream).  A call returns
 * once its kernels are enqueued; gemm_synchronize() waits for them.  The kernels
 * are launched as programmatic dependents: one may start its set-up while the
 * kernel before it on the stream drains, but it touches global memory only once
 * that kernel has completed, so stream order holds for any producer of A or B
 * and any consumer of C, the library's or not.  (An FP32 call whose last round
 * of tiles is at most half full launches two grids; the second reads A and B
 * while the first still runs, and completes only after it; so do the two
 * products of gemm_gated_backward.)  A call launches one to five kernels, or
 * more for a general-form batch beyond 65535 matrices, for a gated block's
 * operands that are padded, for each piece of a head's vocabulary and each step of
 * gemm_orthogonalize (three);
 * gemm_kernel_launches() counts them.  Calls may be captured into CUDA
 * graphs.  Results are deterministic: the same inputs give bit-identical C on
 * every run (no atomics, fixed summation order per element; a head's dX grows by
 * one addition to an element a launch, in stream order).
 *
 * Errors.  Every entry point returns a status; nothing is thrown across the ABI.
 *   GEMM_ERR_INVALID_VALUE      a dimension < 0, or a null pointer needed by the
 *                               call (A and B when K > 0; C when M*N > 0), or a
 *                               forced kernel that cannot run this problem.
 *   GEMM_ERR_ALIAS              C overlaps A or B.
 *   GEMM_ERR_UNSUPPORTED_DEVICE the current device is not compute capability
 *                               10.3 (GB300).  There is no fallback to other
 *                               devices or to the CPU.
 *   GEMM_ERR_CUDA               a CUDA runtime call or kernel launch failed.
 *   GEMM_ERR_TIMEOUT            a kernel gave up waiting on one of its own
 *                               pipeline barriers (reported by gemm_synchronize).
 * M = 0 or N = 0 is a no-op returning GEMM_OK.  K = 0 fills C with zeros (the
 * empty sum).
 */
#ifndef GEMM_GB300_H
#define GEMM_GB300_H

#include <stdint.h>

#if defined(_WIN32)
#define GEMM_API __declspec(dllexport)
#else
#define GEMM_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm_status_t {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_VALUE = 1,
    GEMM_ERR_ALIAS = 2,
    GEMM_ERR_UNSUPPORTED_DEVICE = 3,
    GEMM_ERR_CUDA = 4,
    GEMM_ERR_TIMEOUT = 5
} gemm_status_t;

/* Pure FP32 row-major SGEMM on the CUDA cores: FP32 FFMA only, no TF32 and no
 * tensor cores ("SGEMM measured and the three ledgers", section 2).  A [M,K],
 * B [K,N], C [M,N], all row-major float. */
GEMM_API gemm_status_t gemm_f32_rm(const float *A, const float *B, float *C,
                                   int M, int N, int K);

/* Half column-major GEMM with FP32 accumulation ("MTT S4000 FP16 GEMM",
 * section 1).  A [M,K] (lda = M), B [K,N] (ldb = K), C [M,N] (ldc = M), all
 * column-major IEEE half bit patterns. */
GEMM_API gemm_status_t gemm_f16_cm(const uint16_t *A, const uint16_t *B, uint16_t *C,
                                   int M, int N, int K);

/* BF16 row-major projection GEMM with FP32 accumulation ("Chapter 5 Operators
 * and Runtime", section 5.2.1).  A [M,K], B [K,N], C [M,N], row-major bf16 bit
 * patterns. */
GEMM_API gemm_status_t gemm_bf16_rm(const uint16_t *A, const uint16_t *B, uint16_t *C,
                                    int M, int N, int K);

/* Fused FFN gate/up projection ("Chapter 5 Operators and Runtime", section 5.3.1
 * and example 5-4): Z = SiLU(X·W_g) ⊙ (X·W_u), with SiLU(x) = x / (1 + e^-x) and ⊙
 * the element-wise product.  All bf16 row-major with tight strides: X [M,K],
 * W_g [K,N], W_u [K,N], Z [M,N].  Both products accumulate in FP32 on the tensor
 * cores; the fused epilogue keeps the rounding points of the unfused chain
 * (section 5.3.1, figure 5-15): G and U rounded to bf16, T = bf16(SiLU(G)) with
 * SiLU evaluated in FP32, Z = bf16(T·U).  G, U and T are never written to
 * memory.  Needs X, W_g, W_u, Z 16-byte aligned and K, N multiples of 8
 * (GEMM_ERR_INVALID_VALUE otherwise); Z must not overlap an input
 * (GEMM_ERR_ALIAS).  K = 0 gives Z = 0. */
GEMM_API gemm_status_t gemm_bf16_rm_silu_mul(const uint16_t *X, const uint16_t *W_g, const uint16_t *W_u,
                                             uint16_t *Z, int M, int N, int K);

/* BF16 row-major GEMM that allocates no device memory.  The pages have no
 * counterpart to this entry point: it is an interface addition for callers that
 * cannot call cudaMalloc.  Some host applications own all device memory through
 * their own allocator (a framework's caching pool that has already reserved the
 * GPU's memory, or an embedding program with a fixed memory budget) and forbid
 * allocations made behind its back; others run on latency-critical paths where
 * cudaMalloc's implicit device-wide synchronisation is not acceptable.
 *
 * Same arguments, layout, rounding and error codes as gemm_bf16_rm, but always
 * on the tensor-core kernel, so it needs B and C 16-byte aligned with N a
 * multiple of 8, and A either 16-byte aligned with K a multiple of 8 or 8-byte
 * aligned with K a multiple of 4 (otherwise GEMM_ERR_INVALID_VALUE, with a
 * message in gemm_last_error).  The kernel's scratch -- its 4-byte pipeline-timeout status
 * word, the same for every M, N, K -- lives in a static device array of 256
 * bytes that every GPU loading this library holds until the process exits;
 * a problem needing more scratch than that would be refused with
 * GEMM_ERR_INVALID_VALUE.  No call makes cudaMalloc, cudaFree or any other
 * allocating call.
 *
 * The first call on a device does the set-up, once per device, with that device
 * current: it looks up the array's device address and zeroes the status word
 * (a synchronous cudaMemset, which allocates nothing); make that first call
 * before any stream capture.  A pipeline timeout sets the word, which stays set
 * until gemm_synchronize reads and clears it: gemm_synchronize returns
 * GEMM_ERR_TIMEOUT for it, as for the other entry points, and allocates nothing
 * itself.  All calls share the array, so calls that overlap on the GPU race on
 * it: a timeout of either is reported to whichever thread synchronises
 * first. */
GEMM_API gemm_status_t gemm_bf16_rm_noalloc(const uint16_t *A, const uint16_t *B, uint16_t *C,
                                            int M, int N, int K);

/* General form ("SGEMM measured and the three ledgers", section 2: the
 * library call with operation flags and leading dimensions, and the row- and
 * column-major readings of the same bytes; section 3, kernel K1:
 * alpha * acc + beta * C).  For b = 0 .. batch-1:
 *
 *     C_b <- alpha * op(A_b) * op(B_b) + beta * C_b
 *
 * op(X) is X (GEMM_OP_N) or its transpose (GEMM_OP_T); op(A) is M x K, op(B)
 * is K x N, C is M x N.  dtype gives the element type of A, B and C (float, or
 * IEEE half / bf16 bit patterns); alpha and beta are float.  The products are
 * accumulated in FP32; alpha * acc + beta * c is formed in FP32 and rounded
 * once to the output type.
 *
 * Storage.  A stored matrix of R x Cn elements with leading dimension ld holds
 * element (r, c) at r*ld + c (GEMM_ROW_MAJOR) or r + c*ld (GEMM_COL_MAJOR).
 * A is stored M x K for GEMM_OP_N and K x M for GEMM_OP_T; B is stored K x N or
 * N x K; C is stored M x N.  Each leading dimension must be at least the stored
 * matrix's contiguous extent (and at least 1).  Matrix b of A starts stride_a
 * elements after matrix b-1 (likewise B and C); stride_a or stride_b may be 0
 * (one matrix serves every b); stride_c must keep the C matrices apart when
 * batch > 1.  Leading dimensions and strides are in elements, int64.
 * All pointers are device pointers owned by the caller.
 *
 * Reads.  C is not read when beta == 0 (a NaN in C does not reach the result).
 * A and B are not read when alpha == 0 or K == 0; C is then scaled by beta
 * (or set to zero).
 *
 * Errors.  GEMM_ERR_INVALID_VALUE: an unknown enum value; a negative size or
 * stride; a leading dimension below the contiguous extent; overlapping C
 * matrices; a null pointer that would be read or written; sizes whose element
 * span overflows; a forced kernel family that cannot run the problem
 * ("simt" and "umma" are accepted here, the others are not).
 * GEMM_ERR_ALIAS: C's span overlaps A's or B's span.  Otherwise as the entry
 * points above.  M, N or batch == 0 is a no-op.
 *
 * Kernels.  16-bit problems whose A, B, C are 16-byte aligned and whose
 * leading dimensions (and, for batch > 1, nonzero batch strides) and stored
 * contiguous extents (K or M for A, N or K for B, N for C in row-major terms)
 * are multiples of 8 elements run on the tensor-core CTA pairs; everything
 * else, and every FP32 problem, on the SIMT kernel (float4 loads where
 * alignment allows). */
typedef enum gemm_dtype_t { GEMM_F32 = 0, GEMM_F16 = 1, GEMM_BF16 = 2 } gemm_dtype_t;
typedef enum gemm_layout_t { GEMM_ROW_MAJOR = 0, GEMM_COL_MAJOR = 1 } gemm_layout_t;
typedef enum gemm_op_t { GEMM_OP_N = 0, GEMM_OP_T = 1 } gemm_op_t;

GEMM_API gemm_status_t gemm_ex(gemm_dtype_t dtype, gemm_layout_t layout, gemm_op_t op_a, gemm_op_t op_b,
                               int M, int N, int K, float alpha,
                               const void *A, int64_t lda, int64_t stride_a,
                               const void *B, int64_t ldb, int64_t stride_b,
                               float beta, void *C, int64_t ldc, int64_t stride_c, int batch);

/* Row-wise FP8 quantisation ("Chapter 5 Operators and Runtime", section 5.4.3,
 * example 5-7).  A is [M,K] row-major IEEE half; for every row i:
 *     amax_i  = max_k |a_ik|
 *     Q[i,k]  = E4M3FN(a_ik * (448 / amax_i))   nearest, ties to even, clamped to +-448
 *     scale_i = amax_i / 448
 * with 448 / amax_i, the product and amax_i / 448 each one FP32 operation, so
 * a_ik ~ Q[i,k] * scale_i.  A row of zeros gives Q = 0 and scale 0.  The whole
 * row is read before any of its codes is written (the scale depends on it).
 * E4M3FN: 1 sign, 4 exponent (bias 7), 3 fraction bits, largest finite 448,
 * no infinities.  Q [M,K] row-major bytes, scale [M] float, device pointers
 * owned by the caller.  Any alignment (16-byte aligned A and 8-byte aligned Q
 * with K % 8 == 0 use vector loads).  NaN or infinite inputs are outside the
 * contract.  K = 0 sets every scale to 0.  Errors: GEMM_ERR_INVALID_VALUE for a
 * negative size or a null pointer; GEMM_ERR_ALIAS if Q, scale and A overlap. */
GEMM_API gemm_status_t gemm_quantize_rows_e4m3(const uint16_t *A, uint8_t *Q, float *scale, int M, int K);

/* Row-scaled FP8 projection ("Chapter 5 Operators and Runtime", section 5.4.4,
 * example 5-8: FP8 input times FP8 weights, FP16 output):
 *     C[i,j] = scale_i * sum_k Q[i,k] * W[k,j]
 * on the tensor cores (E4M3 x E4M3 products, FP32 accumulation), the row scale
 * applied to the FP32 sum, one rounding to half.  Q [M,K] row-major E4M3FN codes
 * and scale [M] as written by gemm_quantize_rows_e4m3; the weights W [K,N] are
 * given transposed, Wt [N,K] row-major (each output column's K codes
 * contiguous, the layout of a linear layer's weight); C [M,N] row-major half.
 * Needs Q, Wt, C 16-byte aligned, K % 16 == 0 and N % 8 == 0
 * (GEMM_ERR_INVALID_VALUE otherwise, with a message in gemm_last_error).
 * K = 0 gives C = 0.  GEMM_ERR_ALIAS if C overlaps Q, Wt or scale. */
GEMM_API gemm_status_t gemm_e4m3_rowscale(const uint8_t *Q, const float *scale, const uint8_t *Wt, uint16_t *C,
                                          int M, int N, int K);

/* Row-scaled FP8 projection with the quantisation fused into the product's
 * load path ("Chapter 5 Operators and Runtime", section 5.4.4, example 5-8, the
 * second scheme: the row scales from a first pass over the whole input, then
 * every column block of the product reads the half input and quantises it
 * locally):
 *     amax_i  = max_k |a_ik|
 *     C[i,j]  = (amax_i / 448) * sum_k E4M3(a_ik * (448 / amax_i)) * W[k,j]
 * -- the codes and the row scale of gemm_quantize_rows_e4m3 (the same FP32
 * steps), but never written to memory: the product's loader quantises each
 * tile of A as it stages it.  A [M,K] row-major IEEE half; the weights W [K,N]
 * given transposed, Wt [N,K] row-major E4M3FN codes; C [M,N] row-major half.
 * Results equal gemm_quantize_rows_e4m3 followed by gemm_e4m3_rowscale up to
 * the summation order of the FP32 accumulation.  The rows' amax (4 bytes per
 * row) are kept in the device's default stream-ordered pool for the duration
 * of the call (cudaMallocAsync / cudaFreeAsync on the caller's stream).  Needs
 * A, Wt, C 16-byte aligned, K % 16 == 0 and N % 8 == 0
 * (GEMM_ERR_INVALID_VALUE otherwise, with a message in gemm_last_error).
 * K = 0 gives C = 0.  GEMM_ERR_ALIAS if C overlaps A or Wt.  NaN or infinite
 * inputs are outside the contract. */
GEMM_API gemm_status_t gemm_e4m3_rowscale_fused(const uint16_t *A, const uint8_t *Wt, uint16_t *C,
                                                int M, int N, int K);

/* 4-bit block-scaled floating point.  A matrix [rows, K] is kept as codes and
 * scales; its rows are cut along K into blocks that share a scale.
 *
 *   GEMM_FP4_MX  blocks of 32, the scale a power of two (an E8M0 byte e + 127,
 *                255 = NaN): the OCP microscaling format MXFP4;
 *   GEMM_FP4_NV  blocks of 16, the scale an E4M3FN byte, and one FP32 scale g of
 *                the whole tensor (in device memory, so that it can be computed
 *                there; null: 1), which is not negative.
 *
 * Codes are E2M1 (a sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even
 * k in the low half.  A row takes 16 * ceil(K / 32) bytes; the codes past K are 0.
 * Scale bytes lie in atoms of 128 rows x 4 blocks, 512 bytes each, at
 *     atom (row / 128) * A + block / 4,  A = 2 (MX) or 4 (NV) * ceil(K / 256)
 *     byte (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4
 * -- the order in which the tensor cores take them.  gemm_fp4_code_bytes and
 * gemm_fp4_scale_bytes give the sizes (-1 for a negative size or an unknown
 * format).  Codes and scales need 16-byte alignment (GEMM_ERR_INVALID_VALUE
 * otherwise, with a message in gemm_last_error); everything else its elements'
 * alignment, and any K, M, N.
 *
 * For a block with the largest magnitude amax, a / step rounded to the nearest
 * code (ties to the even code, saturating at 6), in FP32 operations:
 *   MX  step = 2^e, e = clamp(floor(log2 amax) - 2, -127, 125);
 *   NV  s = E4M3(amax / (6 g)), nearest, saturating at 448; step = s g; codes of
 *       0 where the step is 0.  A block of zeros has s = 0 whatever g is, so that a
 *       tensor of zeros with the scale amax / 2688 = 0 stays one of zeros; with g = 0
 *       any other block has s = 448 and codes of 0: it reads back, and multiplies, as 0.
 * A NaN or an infinity in a block makes the block's scale NaN and its codes 0:
 * the block reads back as NaN, and products that use it are NaN. */
typedef enum gemm_fp4_format_t { GEMM_FP4_MX = 0, GEMM_FP4_NV = 1 } gemm_fp4_format_t;

GEMM_API int64_t gemm_fp4_code_bytes(int rows, int K);
GEMM_API int64_t gemm_fp4_scale_bytes(gemm_fp4_format_t format, int rows, int K);

/* Quantises A [M,K] (half or bf16 by dtype, row-major, leading dimension
 * lda >= K) to codes Q and scales S.  tensor_scale: NV's g; must be null for MX.
 * The scale bytes of rows past M and blocks past K, up to the padded sizes, are
 * written too (those of zeros).  GEMM_ERR_ALIAS if A, Q, S overlap. */
GEMM_API gemm_status_t gemm_fp4_quantize(gemm_dtype_t dtype, gemm_fp4_format_t format, const void *A, int64_t lda,
                                         const float *tensor_scale, uint8_t *Q, uint8_t *S, int M, int K);

/* Reads codes and scales back: A[i,k] = code * scale (* g), formed in FP32 and
 * rounded once to dtype. */
GEMM_API gemm_status_t gemm_fp4_dequantize(gemm_dtype_t dtype, gemm_fp4_format_t format, const uint8_t *Q,
                                           const uint8_t *S, const float *tensor_scale, void *A, int64_t lda, int M,
                                           int K);

/* Product of two quantised matrices of one format:
 *     C[i,j] = ga gb * sum_k a[i,k] b[j,k]
 * with a [M,K] and b [N,K] the values code * scale, summed in FP32 and rounded
 * once to dtype (half or bf16).  b is a linear layer's weight: every output
 * column's K codes contiguous.  C [M,N] row-major with ldc >= N.  K = 0 gives
 * C = 0.  GEMM_ERR_ALIAS if C overlaps an input. */
GEMM_API gemm_status_t gemm_fp4(gemm_dtype_t dtype, gemm_fp4_format_t format, const uint8_t *Qa, const uint8_t *Sa,
                                const float *ga, const uint8_t *Qb, const uint8_t *Sb, const float *gb, void *C,
                                int64_t ldc, int M, int N, int K);

/* A linear layer with 4-bit weights: X [M,K] (dtype, ldx >= K) quantised within
 * the call as gemm_fp4_quantize does with tensor scale gx, then the product
 * with the quantised weights [N,K].  For M > 8 (M > 1 where X's rows do not start
 * on 16 bytes) the codes and scales of X lie in stream-ordered scratch for the
 * duration of the call, from a pool of the library's own that keeps up to 1 GiB
 * on the device between calls; fewer rows are converted inside the product. */
GEMM_API gemm_status_t gemm_fp4_linear(gemm_dtype_t dtype, gemm_fp4_format_t format, const void *X, int64_t ldx,
                                       const float *gx, const uint8_t *Qw, const uint8_t *Sw, const float *gw,
                                       void *C, int64_t ldc, int M, int N, int K);

/* Gated feed-forward projections, for training and serving:
 *     G = X W_g,  U = X W_u,  Z = act(G) * U  (element by element)
 * X [M,K], W_g and W_u [K,N], Z [M,N] row-major half or bf16 (dtype) with tight
 * strides, both products and the activation in one kernel (a second one adds FP32
 * partials where the last wave of tiles is split along K, for M > 64); G, U and act in
 * FP32, Z rounded once.  act: SiLU, g / (1 + e^-g), or the tanh form of GELU,
 * g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2.  G and U (both or neither):
 * FP32 [M,N], stored for gemm_gated_backward.  (gemm_bf16_rm_silu_mul keeps the
 * rounding points of the unfused chain instead: G, U and act(G) rounded to bf16.)
 * Any M, N, K: one token to a long prompt.  Operands that are not 16-byte aligned,
 * or whose N or K is no multiple of 8, are copied to or from padded rows in scratch,
 * which costs a pass over each of them; so is X for a long product with neither N
 * nor K a multiple of 64.  N or K a multiple of 64 is fastest.  Scratch, for these
 * copies and the partials (256 KiB each, one at most for every two SMs), is
 * stream-ordered and lives for the duration of the call, from a pool of the
 * library's own that keeps up to 1 GiB on the device between calls; M <= 64 with
 * aligned operands takes none.  K = 0 gives zeros.  GEMM_ERR_ALIAS if an output
 * overlaps an input or another output. */
typedef enum gemm_act_t { GEMM_ACT_SILU = 0, GEMM_ACT_GELU_TANH = 1 } gemm_act_t;

GEMM_API gemm_status_t gemm_gated(gemm_dtype_t dtype, gemm_act_t act, const void *X, const void *W_g, const void *W_u,
                                  void *Z, float *G, float *U, int M, int N, int K);

/* Its gradients, from G and U as gemm_gated stored them and dZ [M,N] (dtype):
 *     dG = dZ * U * act'(G),  dU = dZ * act(G)
 *     dX = dG W_g^T + dU W_u^T,  dW_g = X^T dG,  dW_u = X^T dU
 * dX [M,K], dW_g and dW_u [K,N] (dtype), each overwritten; a null one is left out
 * (and X, W_g, W_u may be null where nothing that is asked for reads them).  dG
 * and dU are formed in FP32 and rounded to dtype, the operands of the products,
 * whose sums are FP32, rounded once.  dG, dU (rows of whole 128 bytes) and, where
 * the last wave of tiles of dX (M > 64) or of the weight gradients is split along its
 * sum, FP32 partials as in gemm_gated lie in the same scratch.  M = 0 or
 * N = 0 gives zeros.  Needs and errors as gemm_gated. */
GEMM_API gemm_status_t gemm_gated_backward(gemm_dtype_t dtype, gemm_act_t act, const void *X, const void *W_g,
                                           const void *W_u, const float *G, const float *U, const void *dZ, void *dX,
                                           void *dW_g, void *dW_u, int M, int N, int K);

/* Root-mean-square norm of rows with the residual's addition before it:
 *     H = X + R  (rounded to dtype),  rstd_i = 1 / sqrt(mean_k H[i,k]^2 + eps)
 *     Y[i,k] = w[k] H[i,k] rstd_i  (formed in FP32, rounded once)
 * X, R, H, Y [M,K] row-major half or bf16 (dtype) with tight strides, w [K] of dtype
 * (null: ones).  R null: no addition, H is X, and the argument H must be null.  H null
 * with R given: the sum is not stored.  H may be X or R itself (the residual stream
 * updated in place).  rstd (null: not stored): FP32 [M], for gemm_rms_norm_backward.
 * eps: a normal number below 2^30 (GEMM_ERR_INVALID_VALUE otherwise).  Any M and K: one
 * token to a long prompt.  Where the operands' bases lie alike to 16 bytes (any K), rows
 * of up to 16384 elements are read once, else twice.  Rows of bf16 whose squares overflow
 * FP32 are summed again, scaled down; a NaN or an infinity in a row reaches that row alone.
 * M = 0 or K = 0: nothing is written.  GEMM_ERR_ALIAS if any other output overlaps an
 * input or another output. */
GEMM_API gemm_status_t gemm_rms_norm(gemm_dtype_t dtype, const void *X, const void *R, const void *w, float eps, void *H,
                                     void *Y, float *rstd, int M, int K);

/* The same Y as row-scaled E4M3, the operand that gemm_e4m3_rowscale takes: of the
 * FP32 values, not rounded to dtype in between,
 *     scale_i = amax_k |Y[i,k]| / 448,  Q[i,k] = E4M3(Y[i,k] * (448 / amax_i))
 * nearest, ties to even, clamped to +-448 (as gemm_quantize_rows_e4m3).  Q [M,K] codes,
 * scale FP32 [M].  A row of zeros gives codes 0 and scale 0; a NaN or an infinity in a
 * row makes its scale NaN.  bf16 rows and gains at the ends of their range are gone over
 * twice or three times, so that no intermediate value leaves FP32; a scale below 2^-126 is
 * an FP32 subnormal and has fewer bits, a row whose largest |Y| is below 2^-150 gives 0. */
GEMM_API gemm_status_t gemm_rms_norm_e4m3(gemm_dtype_t dtype, const void *X, const void *R, const void *w, float eps,
                                          void *H, uint8_t *Q, float *scale, int M, int K);

/* Gradients of gemm_rms_norm from dY (of Y) and dH (of H from its other uses, the
 * residual's path; null: 0), with H (X where there was no residual) and rstd as the
 * forward call left them:
 *     dX = rstd (w dY - H rstd^2 mean_k(w dY H)) + dH   (of X and of R alike)
 *     dw = sum_i dY H rstd
 * dX [M,K] (dtype; may be dH itself), dw FP32 [K], each overwritten; a null one is left
 * out.  Sums in FP32, in a fixed order.  FP32 partials of dw (4 K bytes for each of up to
 * three CTAs an SM) lie in stream-ordered scratch for the duration of the call, from the
 * library's pool (see gemm_gated).  M = 0 gives dw = 0.  GEMM_ERR_ALIAS as above. */
GEMM_API gemm_status_t gemm_rms_norm_backward(gemm_dtype_t dtype, const void *H, const void *w, const float *rstd,
                                              const void *dY, const void *dH, void *dX, float *dw, int M, int K);

/* Softmax cross entropy of a linear head over a vocabulary of N, for training and for
 * scoring: of the logits Z = X W^T, which are never kept,
 *     lse_i = log sum_j exp(Z[i,j]),  loss_i = lse_i - Z[i,targets_i]
 * X [M,K] hidden states and W [N,K] (a row to each entry of the vocabulary: the layout of
 * an embedding, or of a linear layer's weight), row-major half or bf16 (dtype) with tight
 * strides; targets int64 [M]; loss and lse FP32 [M] (lse null: not stored).  A target
 * outside 0 .. N - 1 leaves its row out: loss 0 (lse is stored all the same), and no part
 * in the gradients, whatever the row of X holds.  Logits, largest value, sum and
 * logarithm in FP32; the loss is formed without lse's rounding.  N and K up to 2^31 - 256
 * (GEMM_ERR_INVALID_VALUE above); K and the bases multiples of 8 elements are fastest: of
 * other operands X is copied in scratch (up to eight times), W read in place where K is no
 * multiple of 8 and N large against M, else copied too, a piece at a time (up to 256 MiB, or
 * 256 rows where that is more).  Rows of the copies are padded to a multiple of 64 elements.
 * Scratch: 8 bytes for each row and 64 to 128 entries, for up to 16384 rows at once, and the
 * copies, in stream-ordered memory for the duration of the call from the library's pool (see
 * gemm_gated).  K = 0: logits of 0; N = 0: lse is -inf.  GEMM_ERR_ALIAS if an output
 * overlaps an input or the other output. */
GEMM_API gemm_status_t gemm_cross_entropy(gemm_dtype_t dtype, const void *X, const void *W, const int64_t *targets,
                                          float *loss, float *lse, int M, int N, int K);

/* Its gradients from dloss FP32 [M], the weight of each row's loss, and lse as
 * gemm_cross_entropy stored it:
 *     dZ[i,j] = (exp(Z[i,j] - lse_i) - [j = targets_i]) dloss_i  (0 in rows left out)
 *     dX = dZ W,  dW = dZ^T X
 * dX [M,K], dW [N,K] (dtype), each overwritten; a null one is left out.  The logits are
 * computed anew, a piece of the vocabulary at a time; exp(Z - lse) has lse's rounding, up to
 * 2^-24 |lse| of itself; dZ is formed in FP32 and rounded to
 * dtype, scaled by the largest |dloss| (so that neither small probabilities nor a weight
 * that dtype does not hold exactly are lost; any loss scale does), the operand of the
 * products, whose sums are FP32, in a fixed order, rounded once.  Scratch as above:
 * a piece of dZ (256 MiB, or 256 entries of every row where that is more), FP32 sums of
 * dX (rows padded to a multiple of 64; up to 256 MiB, or a single set where that is more) and
 * copies of X (one for dW, with zeros in the rows left out; up to sixteen where W is read in
 * place).  M too is at most 2^31 - 256.  M = 0 or N = 0 gives zeros.  GEMM_ERR_ALIAS as
 * above. */
GEMM_API gemm_status_t gemm_cross_entropy_backward(gemm_dtype_t dtype, const void *X, const void *W, const int64_t *targets,
                                                   const float *lse, const float *dloss, void *dX, void *dW, int M, int N,
                                                   int K);

/* Orthogonalised update of a weight matrix (the matrix that an optimiser such as Muon
 * applies in place of its momentum G): singular values driven towards 1 by products,
 *     X = G / |G|_F,  then `steps` times  X <- a X + (b A + c A^2) X,  A = X X^T
 * (from the right, with A = X^T X, where M > N: the same in exact arithmetic).  G and O
 * [M,N] row-major half or bf16 (dtype) with leading dimensions ldg, ldo >= N; O may be G
 * itself (with ldo = ldg).  The usual five steps with a = 3.4445, b = -4.7750, c = 2.0315
 * bring singular values from about 0.01 of |G|_F up to between 0.7 and 1.2.  steps >= 1;
 * a, b, c finite, and such that X and A stay within half's range: intermediate matrices
 * are half (X in two halves, 22 bits), sums and |G|_F^2 FP32 or more.  The relative error
 * of the usual five steps is 1e-3 to 2e-3 (Frobenius norm) before O's own rounding, up to
 * 1e-2 in matrices of a few rows or columns, whose few singular values it does not average
 * over.  A matrix of zeros gives zeros; a NaN or an infinity in G makes O NaN.  M, N up to
 * 2^31 - 256 (GEMM_ERR_INVALID_VALUE above), any alignment of elements.  Scratch: 8 bytes
 * for each element of G and 4 for each of A, rows of both padded to a multiple of 64
 * elements (a column of M elements takes 512 M bytes), in stream-ordered memory for the
 * duration of the call from the library's pool (see gemm_gated).  GEMM_ERR_ALIAS if O
 * overlaps G otherwise. */
GEMM_API gemm_status_t gemm_orthogonalize(gemm_dtype_t dtype, const void *G, int64_t ldg, void *O, int64_t ldo, int steps,
                                          float a, float b, float c, int M, int N);

/* Stream for the calling host thread's subsequent calls: a cudaStream_t passed
 * as void*.  NULL selects the legacy default stream.  The stream stays owned by
 * the caller and must outlive the calls issued on it. */
GEMM_API gemm_status_t gemm_set_stream(void *cuda_stream);

/* The calling host thread's current stream (NULL = legacy default stream). */
GEMM_API void *gemm_get_stream(void);

/* Waits for the calling thread's stream; returns GEMM_ERR_CUDA for an
 * asynchronous CUDA error and GEMM_ERR_TIMEOUT if a kernel of this library
 * recorded a pipeline timeout on the current device (the record is cleared).
 * It reads only status words that calls on this device have already set up,
 * so it allocates nothing. */
GEMM_API gemm_status_t gemm_synchronize(void);

/* Static, human-readable name of a status code. */
GEMM_API const char *gemm_status_string(gemm_status_t status);

/* Name of the kernel the calling thread's last call dispatched to, e.g.
 * "simt_f32_vec4", "umma_bf16", "gemv_bf16_vec", "zero_fill", "noop" (static
 * string; for tests and benchmarks). */
GEMM_API const char *gemm_last_kernel(void);

/* Number of CUDA kernels this library has launched in this process, on every
 * thread and device, since it was loaded (one count per launch call issued,
 * whether or not the kernel has run yet).  The difference over a span of calls
 * is the kernels those calls queued; for tests and benchmarks. */
GEMM_API unsigned long long gemm_kernel_launches(void);

/* Message of the last CUDA error seen by the calling thread ("" if none). */
GEMM_API const char *gemm_last_error(void);

/* Test and benchmark hook: forces the calling thread's later calls onto one
 * kernel family -- "simt", "simt_scalar", "gemv", "gemv_scalar", "umma",
 * "umma_skinny_wide" (16-bit, M <= 64: the skinny tensor-core kernel on
 * 256-column strips of B) -- or back to automatic dispatch with NULL or "".  A forced family that cannot run
 * a given problem makes that call return GEMM_ERR_INVALID_VALUE; an unknown
 * name is rejected here with GEMM_ERR_INVALID_VALUE.
 * "umma_stall" tests the tensor-core kernel's bounded waits: a 16-bit call whose
 * A, B and C suit the TMA kernel launches it with a producer that issues no
 * loads, every CTA gives up after about two seconds, C is left unwritten and
 * the next gemm_synchronize returns GEMM_ERR_TIMEOUT.  "umma_stall_pair" does the
 * same on the CTA-pair kernel (16-bit, M > 128, A 16-byte aligned with K a
 * multiple of 8), and "umma_stall_peer" makes the pair's second CTA give up
 * after loading one stage while the first has loaded further, so that the pair
 * ends with loads of only one CTA outstanding.  gemm_bf16_rm_noalloc
 * honours "umma_stall" (recording in its static status word) and ignores the
 * other families; the FP8, 4-bit, gated, norm, head and update entry points ignore
 * them all. */
GEMM_API gemm_status_t gemm_force_kernel(const char *family);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GB300_H */
