// C ABI of the library: argument checks, per-thread stream, device check,
// dispatch to the kernels.  See include/gemm.h for the contract.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <initializer_list>
#include <mutex>

#include "fp4.h"
#include "gated.h"
#include "gemm.h"
#include "internal.h"
#include "scratch.h"

using namespace gemm_gb300;

std::atomic<unsigned long long> gemm_gb300::g_launches{0};

namespace {
ScratchPools g_scratch;
}  // namespace

cudaError_t gemm_gb300::scratch_alloc(void **p, size_t bytes, cudaStream_t s) { return g_scratch.alloc(p, bytes, s); }

namespace {

enum class Family { Auto, Simt, SimtScalar, Gemv, GemvScalar, Umma, UmmaSkinnyWide, UmmaStall, UmmaStallPair, UmmaStallPeer };

thread_local cudaStream_t t_stream = nullptr;
thread_local const char *t_last_kernel = "none";
thread_local char t_last_error[256] = "";
thread_local Family t_force = Family::Auto;

struct DeviceInfo {
    std::mutex setup;
    std::atomic<bool> known{false};  // set once the device has been looked at
    std::atomic<bool> ready{false};  // set once the status word exists
    bool supported = false;
    int num_sms = 0;
    int *status = nullptr;  // device word the tensor-core kernel reports timeouts in
};
DeviceInfo g_devices[kMaxDevices];

__global__ void zero_fill_kernel(uint4 *p, size_t n16, uint8_t *tail, size_t ntail) {
    const size_t stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += stride)
        p[i] = make_uint4(0, 0, 0, 0);
    if (blockIdx.x == 0 && threadIdx.x < ntail) tail[threadIdx.x] = 0;
}

__global__ void zero_fill_bytes_kernel(uint8_t *p, size_t n) {
    const size_t stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) p[i] = 0;
}

// Zeros `bytes` bytes at p on stream s (16-byte stores when p is aligned).
cudaError_t zero_fill(void *p, size_t bytes, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)(num_sms * 4);
    note_launch();
    if (((uintptr_t)p & 15u) == 0) {
        zero_fill_kernel<<<grid, 256, 0, s>>>((uint4 *)p, bytes / 16, (uint8_t *)p + (bytes & ~(size_t)15),
                                              bytes & 15);
    } else {
        zero_fill_bytes_kernel<<<grid, 256, 0, s>>>((uint8_t *)p, bytes);
    }
    return cudaGetLastError();
}

__device__ __forceinline__ float elt_to_f32(float x) { return x; }
__device__ __forceinline__ float elt_to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float elt_to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void elt_from_f32(float *p, float x) { *p = x; }
__device__ __forceinline__ void elt_from_f32(__half *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void elt_from_f32(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The general form when the product term is absent (alpha == 0 or K == 0):
// C_b = beta * C_b over row-major [M, N] matrices with leading dimension ldc,
// and C_b = 0 without reading it when beta == 0.
template <typename T>
__global__ void scale_c_kernel(T *C, int M, int N, long long ldc, long long sc, long long batch, float beta) {
    const long long per = (long long)M * N, total = batch * per;
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const long long b = i / per, r = i - b * per;
        const long long row = r / N, col = r - row * N;
        T *p = C + b * sc + row * ldc + col;
        elt_from_f32(p, beta == 0.0f ? 0.0f : beta * elt_to_f32(*p));
    }
}

void record_cuda_error(cudaError_t e) {
    strncpy(t_last_error, cudaGetErrorString(e), sizeof(t_last_error) - 1);
    t_last_error[sizeof(t_last_error) - 1] = '\0';
}

// A zeroed device word.  The calling thread may be capturing a stream, which has no part
// in this: allocations are allowed meanwhile, and the word is zeroed on a stream that
// waits for no other.
cudaError_t make_status_word(int **out) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    int *word = nullptr;
    cudaStream_t s = nullptr;
    e = cudaMalloc(&word, sizeof(int));
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (s) cudaStreamDestroy(s);
    if (e != cudaSuccess && word) cudaFree(word);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) *out = word;
    return e != cudaSuccess ? e : back;
}

cudaError_t set_up(DeviceInfo &d, int dev) {
    int major = 0, minor = 0;
    cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && major == 10 && minor == 3) {
        d.supported = true;
        if (!d.status) e = make_status_word(&d.status);
        if (e == cudaSuccess) d.ready.store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) cudaGetLastError();  // reported by this call, found by no later one
    return e;
}

// Per-device set-up on first use: capability check, SM count, status word.  One that
// failed is tried again by the next call.
gemm_status_t device_info(DeviceInfo **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
    DeviceInfo &d = g_devices[dev];
    if (!d.known.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(d.setup);
        if (!d.known.load(std::memory_order_relaxed)) {
            e = set_up(d, dev);
            if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
            d.known.store(true, std::memory_order_release);
        }
    }
    if (!d.supported) return GEMM_ERR_UNSUPPORTED_DEVICE;
    *out = &d;
    return GEMM_OK;
}

bool overlaps(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return an && bn && a0 < b0 + bn && b0 < a0 + an;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

gemm_status_t finish(cudaError_t e, const char *name) {
    t_last_kernel = name;
    if (e == cudaSuccess) return GEMM_OK;
    record_cuda_error(e);
    return GEMM_ERR_CUDA;
}

const char *kernel_name(const char *fam, Elt elt) {
    // Static names: family x element type.
    static const char *names[5][3] = {
        {"simt_f32_vec4", "simt_f16_scalar", "simt_bf16_scalar"},
        {"simt_f32_scalar", "simt_f16_scalar", "simt_bf16_scalar"},
        {"gemv_f32_vec", "gemv_f16_vec", "gemv_bf16_vec"},
        {"gemv_f32_scalar", "gemv_f16_scalar", "gemv_bf16_scalar"},
        {"umma_f32", "umma_f16", "umma_bf16"},
    };
    int f = 0;
    if (!strcmp(fam, "simt")) f = 0;
    else if (!strcmp(fam, "simt_scalar")) f = 1;
    else if (!strcmp(fam, "gemv")) f = 2;
    else if (!strcmp(fam, "gemv_scalar")) f = 3;
    else f = 4;
    return names[f][(int)elt];
}

// Row-major problem C[M,N] = A[M,K] B[K,N] with tight strides.
gemm_status_t run(const void *A, const void *B, void *C, int M, int N, int K, Elt elt) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    const size_t es = elt == Elt::F32 ? 4 : 2;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!C || (K > 0 && (!A || !B))) return GEMM_ERR_INVALID_VALUE;
    const size_t c_bytes = (size_t)M * N * es;
    if (overlaps(C, c_bytes, A, (size_t)M * K * es) || overlaps(C, c_bytes, B, (size_t)K * N * es))
        return GEMM_ERR_ALIAS;

    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;

    if (K == 0) {
        if (t_force != Family::Auto) return GEMM_ERR_INVALID_VALUE;
        return finish(zero_fill(C, c_bytes, dev->num_sms, s), "zero_fill");
    }

    Problem p{A, B, C, M, N, K, elt};
    const int vw = elt == Elt::F32 ? 4 : 8;
    const bool gemv_vec_ok = (N % vw) == 0 && aligned16(B);
    const bool simt_vec_ok = elt == Elt::F32 && (K % 4) == 0 && (N % 4) == 0 && aligned16(A) &&
                             aligned16(B) && aligned16(C);

    switch (t_force) {
    case Family::Simt:
        if (elt == Elt::F32 && !simt_vec_ok) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_simt(p, elt == Elt::F32, dev->num_sms, s), kernel_name("simt", elt));
    case Family::SimtScalar:
        return finish(launch_simt(p, false, dev->num_sms, s), kernel_name("simt_scalar", elt));
    case Family::Gemv:
        if (M > kGemvMaxM || !gemv_vec_ok) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_gemv(p, true, dev->num_sms, s), kernel_name("gemv", elt));
    case Family::GemvScalar:
        if (M > kGemvMaxM) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_gemv(p, false, dev->num_sms, s), kernel_name("gemv_scalar", elt));
    case Family::Umma:
        if (!umma_supported(p)) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_umma(p, dev->num_sms, dev->status, s), kernel_name("umma", elt));
    case Family::UmmaSkinnyWide:
        if (!skinny_wide_supported(p)) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_skinny_wide(p, dev->num_sms, dev->status, s),
                      elt == Elt::BF16 ? "umma_skinny_wide_bf16" : "umma_skinny_wide_f16");
    case Family::UmmaStall:
        if (elt == Elt::F32) return GEMM_ERR_INVALID_VALUE;
        return finish(launch_umma_stall_test(p, dev->num_sms, dev->status, s), "umma_stall");
    case Family::UmmaStallPair:
    case Family::UmmaStallPeer: {
        if (elt == Elt::F32 || M <= 128) return GEMM_ERR_INVALID_VALUE;
        const bool peer = t_force == Family::UmmaStallPeer;
        return finish(launch_umma_pair_stall_test(p, peer ? 2 : 1, dev->status, s),
                      peer ? "umma_stall_peer" : "umma_stall_pair");
    }
    case Family::Auto:
        break;
    }

    // Skinny M: the streaming GEMV for FP32 and for 16-bit problems the
    // tensor-core kernels cannot take; other 16-bit problems with M <= 8 run on
    // the tensor cores (the skinny kernels, weights as the MMA's rows), which
    // stream B faster -- for M = 1 too whenever the X rows suit TMA and the
    // 256-column strips fit on the SMs at once.  Measured back to back (bf16, W
    // from DRAM), skinny against GEMV, M = 1: N = 12288, K = 4096 17.7 vs
    // 18.8 us; N = 4096, K = 12288 19.1 vs 22.2; N = 1024, K = 4096 5.5 vs 7.3;
    // N = 28672, K = 4096 38.1 vs 48.6.
    const bool m1_tensor = M == 1 && elt != Elt::F32 && umma_supported(p) && (K % 8) == 0 && aligned16(A) &&
                           (N + 255) / 256 <= dev->num_sms;
    if (M <= kGemvMaxM && (elt == Elt::F32 || (M == 1 && !m1_tensor) || !umma_supported(p)))
        return gemv_vec_ok ? finish(launch_gemv(p, true, dev->num_sms, s), kernel_name("gemv", elt))
                           : finish(launch_gemv(p, false, dev->num_sms, s), kernel_name("gemv_scalar", elt));
    if (elt == Elt::F32)
        return simt_vec_ok ? finish(launch_simt(p, true, dev->num_sms, s), kernel_name("simt", elt))
                           : finish(launch_simt(p, false, dev->num_sms, s), kernel_name("simt_scalar", elt));
    if (umma_supported(p)) return finish(launch_umma(p, dev->num_sms, dev->status, s), kernel_name("umma", elt));
    return finish(launch_simt(p, false, dev->num_sms, s), kernel_name("simt_scalar", elt));
}

// Capability and SM count of the current device, without allocating anything
// (used only by the allocation-free entry point).
struct PlainDeviceInfo {
    std::once_flag once;
    bool supported = false;
    int num_sms = 0;
    cudaError_t err = cudaSuccess;
};
PlainDeviceInfo g_plain_devices[kMaxDevices];

gemm_status_t plain_device_info(PlainDeviceInfo **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
    PlainDeviceInfo &d = g_plain_devices[dev];
    std::call_once(d.once, [&] {
        int major = 0, minor = 0;
        cudaError_t err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
        d.err = err;
        d.supported = err == cudaSuccess && major == 10 && minor == 3;
    });
    if (d.err != cudaSuccess) { record_cuda_error(d.err); return GEMM_ERR_CUDA; }
    if (!d.supported) return GEMM_ERR_UNSUPPORTED_DEVICE;
    *out = &d;
    return GEMM_OK;
}

void record_message(const char *msg) {
    strncpy(t_last_error, msg, sizeof(t_last_error) - 1);
    t_last_error[sizeof(t_last_error) - 1] = '\0';
}

// a * b + c for non-negative operands; false if it exceeds 2^62.
bool mul_add(long long a, long long b, long long c, long long *out) {
    const long long lim = 1LL << 62;
    if (a < 0 || b < 0 || c < 0) return false;
    if (a != 0 && b > (lim - c) / a) return false;
    *out = a * b + c;
    return true;
}

// Elements from the first to one past the last one that `batch` stored
// matrices of [outer, inner] (leading dimension ld, matrix stride `stride`)
// touch: (batch - 1) * stride + (outer - 1) * ld + inner.  false on overflow.
bool span_elems(long long batch, long long stride, long long outer, long long ld, long long inner, long long *out) {
    long long one = 0, all = 0;
    if (outer < 1 || inner < 1 || batch < 1) { *out = 0; return true; }
    if (!mul_add(outer - 1, ld, inner, &one)) return false;
    if (!mul_add(batch - 1, stride, one, &all)) return false;
    *out = all;
    return true;
}

gemm_status_t run_ex(int dtype, int layout, int op_a, int op_b, int M, int N, int K, float alpha, const void *A,
                     long long lda, long long sa, const void *B, long long ldb, long long sb, float beta, void *C,
                     long long ldc, long long sc, int batch) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16) return GEMM_ERR_INVALID_VALUE;
    if (layout != GEMM_ROW_MAJOR && layout != GEMM_COL_MAJOR) return GEMM_ERR_INVALID_VALUE;
    if ((op_a != GEMM_OP_N && op_a != GEMM_OP_T) || (op_b != GEMM_OP_N && op_b != GEMM_OP_T))
        return GEMM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || batch < 0 || sa < 0 || sb < 0 || sc < 0) return GEMM_ERR_INVALID_VALUE;
    const Elt elt = dtype == GEMM_F32 ? Elt::F32 : dtype == GEMM_F16 ? Elt::F16 : Elt::BF16;
    const long long es = elt == Elt::F32 ? 4 : 2;
    // Column-major C = op(A) op(B) is row-major C^T = op(B)^T op(A)^T on the
    // same buffers ("SGEMM measured and the three ledgers", section 2): swap the
    // operands, their flags, leading dimensions and strides, and M with N.
    if (layout == GEMM_COL_MAJOR) {
        const void *tp = A; A = B; B = tp;
        long long t = lda; lda = ldb; ldb = t;
        t = sa; sa = sb; sb = t;
        int ti = op_a; op_a = op_b; op_b = ti;
        ti = M; M = N; N = ti;
    }
    // Row-major from here on.  A is stored [M,K] ('N') or [K,M] ('T'); B is
    // stored [K,N] or [N,K]; C is [M,N].
    const bool a_t = op_a == GEMM_OP_T, b_t = op_b == GEMM_OP_T;
    const long long a_inner = a_t ? M : K, a_outer = a_t ? K : M;
    const long long b_inner = b_t ? K : N, b_outer = b_t ? N : K;
    const long long one = 1;
    if (ldc < (N > 1 ? N : one) || lda < (a_inner > 1 ? a_inner : one) || ldb < (b_inner > 1 ? b_inner : one))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0 || batch == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    const bool use_ab = alpha != 0.0f && K > 0;
    if (!C || (use_ab && (!A || !B))) return GEMM_ERR_INVALID_VALUE;
    long long c_one = 0, c_span = 0, a_span = 0, b_span = 0;
    if (!span_elems(1, 0, M, ldc, N, &c_one) || !span_elems(batch, sc, M, ldc, N, &c_span))
        return GEMM_ERR_INVALID_VALUE;
    if (batch > 1 && sc < c_one) return GEMM_ERR_INVALID_VALUE;  // the C matrices would overlap
    if (use_ab) {
        if (!span_elems(batch, sa, a_outer, lda, a_inner, &a_span) ||
            !span_elems(batch, sb, b_outer, ldb, b_inner, &b_span))
            return GEMM_ERR_INVALID_VALUE;
        if (c_span > (1LL << 62) / es || a_span > (1LL << 62) / es || b_span > (1LL << 62) / es)
            return GEMM_ERR_INVALID_VALUE;
        if (overlaps(C, (size_t)(c_span * es), A, (size_t)(a_span * es)) ||
            overlaps(C, (size_t)(c_span * es), B, (size_t)(b_span * es)))
            return GEMM_ERR_ALIAS;
    }

    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;

    if (!use_ab) {
        if (t_force != Family::Auto) return GEMM_ERR_INVALID_VALUE;
        const unsigned grid = (unsigned)(dev->num_sms * 8);
        note_launch();
        switch (elt) {
        case Elt::F32: scale_c_kernel<<<grid, 256, 0, s>>>((float *)C, M, N, ldc, sc, batch, beta); break;
        case Elt::F16: scale_c_kernel<<<grid, 256, 0, s>>>((__half *)C, M, N, ldc, sc, batch, beta); break;
        case Elt::BF16: scale_c_kernel<<<grid, 256, 0, s>>>((__nv_bfloat16 *)C, M, N, ldc, sc, batch, beta); break;
        }
        return finish(cudaGetLastError(), "scale_c");
    }

    ProblemEx p = {};
    p.A = A;
    p.B = B;
    p.C = C;
    p.M = M;
    p.N = N;
    p.K = K;
    p.batch = batch;
    p.a_t = a_t;
    p.b_t = b_t;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.sa = sa;
    p.sb = sb;
    p.sc = sc;
    p.alpha = alpha;
    p.beta = beta;
    p.elt = elt;
    static const char *simt_names[3] = {"simt_ex_f32", "simt_ex_f16", "simt_ex_bf16"};
    const char *simt_name = simt_ex_vec(p) ? "simt_ex_f32_vec4" : simt_names[(int)elt];
    const char *umma_name = elt == Elt::BF16 ? "umma_ex_bf16" : "umma_ex_f16";

    switch (t_force) {
    case Family::Simt:
        return finish(launch_simt_ex(p, s), simt_name);
    case Family::Umma: {
        if (!umma_ex_supported(p)) return GEMM_ERR_INVALID_VALUE;
        const cudaError_t e = launch_umma_ex(p, dev->status, s);
        if (e == cudaErrorNotSupported) return GEMM_ERR_INVALID_VALUE;
        return finish(e, umma_name);
    }
    case Family::Auto:
        break;
    default:
        return GEMM_ERR_INVALID_VALUE;
    }
    if (elt != Elt::F32 && umma_ex_supported(p)) {
        const cudaError_t e = launch_umma_ex(p, dev->status, s);
        if (e != cudaErrorNotSupported) return finish(e, umma_name);
    }
    return finish(launch_simt_ex(p, s), simt_name);
}

// 16-bit operands on 2 bytes, FP32 ones on 4: the kernels load whole elements.
bool elements_aligned(const char *who, std::initializer_list<const void *> halves,
                      std::initializer_list<const void *> floats) {
    uintptr_t h = 0, f = 0;
    for (const void *p : halves) h |= (uintptr_t)p;
    for (const void *p : floats) f |= (uintptr_t)p;
    if ((h & 1) == 0 && (f & 3) == 0) return true;
    snprintf(t_last_error, sizeof(t_last_error), "%s: needs 16-bit operands on 2 bytes and FP32 ones on 4", who);
    return false;
}

// ------------------------------------------------------------ 4-bit block scales
// What the four entry points share: types, format, and the codes' and scales'
// sizes of a [rows, K] matrix (0 where nothing is stored).
bool fp4_types_ok(int dtype, int format) {
    return (dtype == GEMM_F16 || dtype == GEMM_BF16) && (format == GEMM_FP4_MX || format == GEMM_FP4_NV);
}
Elt elt16(int dtype) { return dtype == GEMM_BF16 ? Elt::BF16 : Elt::F16; }
size_t fp4_code_size(int rows, int K) { return K > 0 ? (size_t)rows * fp4_row_bytes(K) : 0; }

// Checks of a quantised operand: codes and scales present and 16-byte aligned,
// a tensor scale only where the format has one.
bool fp4_operand_ok(const char *who, int format, const void *Q, const void *S, const float *g) {
    if (!Q || !S || !elements_aligned(who, {}, {g})) return false;
    if (!aligned16(Q) || !aligned16(S)) {
        snprintf(t_last_error, sizeof(t_last_error), "%s: codes and scales need 16-byte alignment", who);
        return false;
    }
    if (format == GEMM_FP4_MX && g) {
        snprintf(t_last_error, sizeof(t_last_error), "%s: the MX format has no tensor scale", who);
        return false;
    }
    return true;
}

// Quantise (to_codes) or read back: A [M,K] with leading dimension lda.
gemm_status_t run_fp4_convert(const char *who, bool to_codes, int dtype, int format, const void *A, int64_t lda,
                              const float *g, const void *Q, const void *S, int M, int K) {
    if (!fp4_types_ok(dtype, format) || M < 0 || K < 0 || lda < (K > 1 ? K : 1)) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!A || !fp4_operand_ok(who, format, Q, S, g) || !elements_aligned(who, {A}, {})) return GEMM_ERR_INVALID_VALUE;
    const bool nv = format == GEMM_FP4_NV;
    long long span = 0;
    if (!span_elems(1, 0, M, lda, K, &span) || span > (1LL << 61)) return GEMM_ERR_INVALID_VALUE;
    const size_t a = (size_t)span * 2, q = fp4_code_size(M, K), sc = (size_t)fp4_scale_size(nv, M, K), gs = g ? 4 : 0;
    if (overlaps(A, a, Q, q) || overlaps(A, a, S, sc) || overlaps(Q, q, S, sc)) return GEMM_ERR_ALIAS;
    if (to_codes ? overlaps(g, gs, Q, q) || overlaps(g, gs, S, sc) : overlaps(g, gs, A, a)) return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    if (to_codes)
        return finish(launch_fp4_quantize(elt16(dtype), nv, A, lda, g, const_cast<void *>(Q),
                                          fp4_row_bytes(K), const_cast<void *>(S), M, K, t_stream),
                      nv ? "fp4_quantize_nv" : "fp4_quantize_mx");
    return finish(launch_fp4_dequantize(elt16(dtype), nv, Q, S, g, const_cast<void *>(A), lda, M, K, t_stream),
                  nv ? "fp4_dequantize_nv" : "fp4_dequantize_mx");
}

// The product of two quantised matrices; X non-null: the first operand is
// X [M,K] in dtype, quantised within the call.
gemm_status_t run_fp4(const char *who, int dtype, int format, const void *X, int64_t ldx, const void *Qa,
                      const void *Sa, const float *ga, const void *Qb, const void *Sb, const float *gb, void *C,
                      int64_t ldc, int M, int N, int K, bool linear) {
    if (!fp4_types_ok(dtype, format) || M < 0 || N < 0 || K < 0 || ldc < (N > 1 ? N : 1)) return GEMM_ERR_INVALID_VALUE;
    if (linear && ldx < (K > 1 ? K : 1)) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!C || !elements_aligned(who, {C, X}, {ga})) return GEMM_ERR_INVALID_VALUE;
    const bool nv = format == GEMM_FP4_NV;
    const Elt elt = elt16(dtype);
    long long span = 0, x_span = 0;
    if (!span_elems(1, 0, M, ldc, N, &span) || span > (1LL << 61)) return GEMM_ERR_INVALID_VALUE;
    const size_t c = (size_t)span * 2;
    if (K > 0) {
        if (!fp4_operand_ok(who, format, Qb, Sb, gb)) return GEMM_ERR_INVALID_VALUE;
        if (linear) {
            if (!X || (format == GEMM_FP4_MX && ga)) return GEMM_ERR_INVALID_VALUE;
            if (!span_elems(1, 0, M, ldx, K, &x_span) || x_span > (1LL << 61)) return GEMM_ERR_INVALID_VALUE;
            if (overlaps(C, c, X, (size_t)x_span * 2)) return GEMM_ERR_ALIAS;
        } else {
            if (!fp4_operand_ok(who, format, Qa, Sa, ga)) return GEMM_ERR_INVALID_VALUE;
            if (overlaps(C, c, Qa, fp4_code_size(M, K)) || overlaps(C, c, Sa, (size_t)fp4_scale_size(nv, M, K)))
                return GEMM_ERR_ALIAS;
        }
        if (overlaps(C, c, Qb, fp4_code_size(N, K)) || overlaps(C, c, Sb, (size_t)fp4_scale_size(nv, N, K)) ||
            overlaps(C, c, ga, ga ? 4 : 0) || overlaps(C, c, gb, gb ? 4 : 0))
            return GEMM_ERR_ALIAS;
    }
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {  // the empty sum
        const unsigned grid = (unsigned)(dev->num_sms * 8);
        note_launch();
        scale_c_kernel<<<grid, 256, 0, s>>>((__half *)C, M, N, ldc, 0, 1, 0.0f);
        return finish(cudaGetLastError(), "zero_fill");
    }
    Fp4Problem p = {};
    p.Qa = Qa;
    p.Sa = Sa;
    p.Qb = Qb;
    p.Sb = Sb;
    p.pitch_a = p.pitch_b = fp4_row_bytes(K);
    p.ga = ga;
    p.gb = gb;
    p.C = C;
    p.ldc = ldc;
    p.M = M;
    p.N = N;
    p.K = K;
    p.elt = elt;
    p.nv = nv;
    // Few rows run on the weight stream.  A linear layer's X is quantised inside it
    // for M <= 8, by a launch of its own above: every strip of 128 outputs converts X
    // anew, which for M = 8 is hidden behind the stream (N = 12288, K = 4096, NV: 10.9
    // us against 11.1 in two launches; N = 4096, K = 12288, MX: 8.9 against 11.3) and
    // for M = 16 no longer is (15.6 against 11.2).  Rows of X that do not start on 16
    // bytes are read value by value there, and only for one row (N = 12288, K = 4095, NV:
    // M = 1 10.2 against 10.8 us, M = 8 20.8 against 11.8).
    const bool skinny = M <= kFp4SkinnyMaxM;
    const bool x16 = aligned16(X) && ldx % 8 == 0;
    if (linear && M <= (x16 ? 8 : 1))
        return finish(launch_fp4_skinny(p, X, ldx, dev->num_sms, dev->status, s),
                      nv ? "fp4_skinny_fused_nv" : "fp4_skinny_fused_mx");
    auto product = [&] { return skinny ? launch_fp4_skinny(p, nullptr, 0, dev->num_sms, dev->status, s) : launch_fp4_gemm(p, dev->status, s); };
    const char *name = skinny ? (nv ? "fp4_skinny_nv" : "fp4_skinny_mx") : (nv ? "fp4_gemm_nv" : "fp4_gemm_mx");
    if (!linear) return finish(product(), name);
    // X's codes and scales in stream-ordered scratch for the duration of the call
    p.pitch_a = fp4_scratch_pitch(K);
    const size_t q = ((size_t)M * p.pitch_a + 255) & ~(size_t)255;
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(&ws, q + (size_t)fp4_scale_size(nv, M, K), s);
    if (e != cudaSuccess) return finish(e, "fp4_linear");
    p.Qa = ws;
    p.Sa = static_cast<uint8_t *>(ws) + q;
    e = launch_fp4_quantize(elt, nv, X, ldx, ga, ws, p.pitch_a, static_cast<uint8_t *>(ws) + q, M, K, s);
    if (e == cudaSuccess) e = product();
    const cudaError_t f = cudaFreeAsync(ws, s);
    return finish(e != cudaSuccess ? e : f, name);
}

// ------------------------------------------------------------ gated block
bool gated_args_ok(const char *who, int dtype, int act, int M, int N, int K, std::initializer_list<const void *> halves,
                   std::initializer_list<const void *> floats) {
    if ((dtype != GEMM_F16 && dtype != GEMM_BF16) || (act != GEMM_ACT_SILU && act != GEMM_ACT_GELU_TANH)) return false;
    return M >= 0 && N >= 0 && K >= 0 && elements_aligned(who, halves, floats);
}
struct Span {
    const void *p;
    size_t bytes;
};
bool any_overlap(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    for (const Span *o = out.begin(); o != out.end(); ++o) {
        for (const Span &i : in)
            if (o->p && i.p && overlaps(o->p, o->bytes, i.p, i.bytes)) return true;
        for (const Span *q = o + 1; q != out.end(); ++q)
            if (o->p && q->p && overlaps(o->p, o->bytes, q->p, q->bytes)) return true;
    }
    return false;
}
cudaError_t zero(const Span &s, cudaStream_t st, cudaError_t e) {
    return e == cudaSuccess && s.p && s.bytes ? cudaMemsetAsync(const_cast<void *>(s.p), 0, s.bytes, st) : e;
}

gemm_status_t run_gated(int dtype, int act, const void *X, const void *Wg, const void *Wu, void *Z, float *G, float *U,
                        int M, int N, int K) {
    if (!gated_args_ok("gemm_gated", dtype, act, M, N, K, {X, Wg, Wu, Z}, {G, U})) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!Z || (K > 0 && (!X || !Wg || !Wu)) || !G != !U) return GEMM_ERR_INVALID_VALUE;
    const size_t mn = (size_t)M * N, x = (size_t)M * K * 2, w = (size_t)K * N * 2;
    const Span z{Z, mn * 2}, gs{G, mn * 4}, us{U, mn * 4};
    if (any_overlap({z, gs, us}, {{X, x}, {Wg, w}, {Wu, w}})) return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0)  // G = U = 0, and act(0) * 0 = 0
        return finish(zero(us, s, zero(gs, s, zero(z, s, cudaSuccess))), "zero_fill");
    const GatedProblem p{X, Wg, Wu, Z, G, U, M, N, K, elt16(dtype), act == GEMM_ACT_GELU_TANH, K};
    return finish(launch_gated_forward(p, dev->num_sms, dev->status, s), M <= kGatedSkinnyMaxM ? "gated_skinny" : "gated_pair");
}

gemm_status_t run_gated_backward(int dtype, int act, const void *X, const void *Wg, const void *Wu, const float *G,
                                 const float *U, const void *dZ, void *dX, void *dWg, void *dWu, int M, int N, int K) {
    if (!gated_args_ok("gemm_gated_backward", dtype, act, M, N, K, {X, Wg, Wu, dZ, dX, dWg, dWu}, {G, U}))
        return GEMM_ERR_INVALID_VALUE;
    if (K == 0 || (!dX && !dWg && !dWu)) { t_last_kernel = "noop"; return GEMM_OK; }
    const size_t mn = (size_t)M * N, x = (size_t)M * K * 2, w = (size_t)K * N * 2;
    const Span ox{dX, x}, og{dWg, w}, ou{dWu, w};
    const bool work = M > 0 && N > 0;
    if (work && (!G || !U || !dZ || (dX && (!Wg || !Wu)) || ((dWg || dWu) && !X))) return GEMM_ERR_INVALID_VALUE;
    if (any_overlap({ox, og, ou}, {{X, x}, {Wg, w}, {Wu, w}, {G, mn * 4}, {U, mn * 4}, {dZ, mn * 2}}))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (!work)  // empty sums: no rows (dW), no hidden units (dX)
        return finish(zero(ou, s, zero(og, s, zero(ox, s, cudaSuccess))), "zero_fill");
    const GatedBackward p{X, Wg, Wu, dZ, G, U, dX, dWg, dWu, M, N, K, elt16(dtype), act == GEMM_ACT_GELU_TANH};
    return finish(launch_gated_gradients(p, dev->num_sms, dev->status, s), "gated_backward");
}

}  // namespace

extern "C" {

GEMM_API gemm_status_t gemm_ex(gemm_dtype_t dtype, gemm_layout_t layout, gemm_op_t op_a, gemm_op_t op_b, int M,
                               int N, int K, float alpha, const void *A, int64_t lda, int64_t stride_a,
                               const void *B, int64_t ldb, int64_t stride_b, float beta, void *C, int64_t ldc,
                               int64_t stride_c, int batch) {
    return run_ex((int)dtype, (int)layout, (int)op_a, (int)op_b, M, N, K, alpha, A, lda, stride_a, B, ldb,
                  stride_b, beta, C, ldc, stride_c, batch);
}

GEMM_API gemm_status_t gemm_f32_rm(const float *A, const float *B, float *C, int M, int N, int K) {
    return run(A, B, C, M, N, K, Elt::F32);
}

// Column-major C = A·B is row-major C^T = B^T·A^T on the same buffers: the
// column-major B buffer read row-major is B^T [N,K], the column-major A buffer
// read row-major is A^T [K,M], and the row-major [N,M] result is the
// column-major [M,N] C ("SGEMM measured and the three ledgers", section 2).
GEMM_API gemm_status_t gemm_f16_cm(const uint16_t *A, const uint16_t *B, uint16_t *C, int M, int N, int K) {
    return run(B, A, C, N, M, K, Elt::F16);
}

GEMM_API gemm_status_t gemm_bf16_rm(const uint16_t *A, const uint16_t *B, uint16_t *C, int M, int N, int K) {
    return run(A, B, C, M, N, K, Elt::BF16);
}

// Allocation-free bf16 entry point: the tensor-core kernel with its status word
// in a static device array instead of library-allocated memory.
GEMM_API gemm_status_t gemm_bf16_rm_noalloc(const uint16_t *A, const uint16_t *B, uint16_t *C, int M, int N,
                                            int K) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!C || (K > 0 && (!A || !B))) return GEMM_ERR_INVALID_VALUE;
    const size_t c_bytes = (size_t)M * N * 2;
    if (overlaps(C, c_bytes, A, (size_t)M * K * 2) || overlaps(C, c_bytes, B, (size_t)K * N * 2))
        return GEMM_ERR_ALIAS;
    PlainDeviceInfo *dev = nullptr;
    gemm_status_t st = plain_device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {
        return finish(zero_fill(C, c_bytes, dev->num_sms, s), "zero_fill");
    }
    Problem p{A, B, C, M, N, K, Elt::BF16};
    const bool stall = t_force == Family::UmmaStall;
    if (stall && !umma_supported(p)) return GEMM_ERR_INVALID_VALUE;
    if (!umma_supported(p)) {
        record_message("gemm_bf16_rm_noalloc: needs B and C 16-byte aligned with N % 8 == 0, and A 16-byte "
                       "aligned with K % 8 == 0 or 8-byte aligned with K % 4 == 0");
        return GEMM_ERR_INVALID_VALUE;
    }
    if (umma_noalloc_scratch_need(p) > kNoallocScratchBytes) {
        record_message("gemm_bf16_rm_noalloc: problem needs more scratch than the static array holds");
        return GEMM_ERR_INVALID_VALUE;
    }
    if (stall) return finish(launch_umma_noalloc(p, dev->num_sms, s, true), "umma_stall");
    return finish(launch_umma_noalloc(p, dev->num_sms, s), "umma_bf16_noalloc");
}

GEMM_API gemm_status_t gemm_bf16_rm_silu_mul(const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu, uint16_t *Z,
                                             int M, int N, int K) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!Z || (K > 0 && (!X || !Wg || !Wu))) return GEMM_ERR_INVALID_VALUE;
    const size_t z_bytes = (size_t)M * N * 2, w_bytes = (size_t)K * N * 2;
    if (overlaps(Z, z_bytes, X, (size_t)M * K * 2) || overlaps(Z, z_bytes, Wg, w_bytes) ||
        overlaps(Z, z_bytes, Wu, w_bytes))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {  // G = U = 0, SiLU(0) * 0 = 0
        return finish(zero_fill(Z, z_bytes, dev->num_sms, s), "zero_fill");
    }
    Problem p{X, Wg, Z, M, N, K, Elt::BF16};
    if (!umma_silu_mul_supported(p, Wu)) {
        record_message("gemm_bf16_rm_silu_mul: needs X, W_g, W_u, Z 16-byte aligned and K, N multiples of 8");
        return GEMM_ERR_INVALID_VALUE;
    }
    return finish(launch_umma_silu_mul(p, Wu, dev->status, s), "umma_bf16_silu_mul");
}

GEMM_API gemm_status_t gemm_quantize_rows_e4m3(const uint16_t *A, uint8_t *Q, float *scale, int M, int K) {
    if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!scale || (K > 0 && (!A || !Q))) return GEMM_ERR_INVALID_VALUE;
    const size_t a_bytes = (size_t)M * K * 2, q_bytes = (size_t)M * K, s_bytes = (size_t)M * 4;
    if (overlaps(Q, q_bytes, A, a_bytes) || overlaps(scale, s_bytes, A, a_bytes) ||
        overlaps(scale, s_bytes, Q, q_bytes))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {  // every row is empty: amax = 0, scale 0
        const cudaError_t e = cudaMemsetAsync(scale, 0, s_bytes, s);
        return finish(e, "zero_fill");
    }
    return finish(launch_quantize_rows_e4m3(A, Q, scale, M, K, s),
                  quantize_rows_vec_ok(A, Q, K) ? "quantize_e4m3_vec" : "quantize_e4m3_scalar");
}

GEMM_API gemm_status_t gemm_e4m3_rowscale(const uint8_t *Q, const float *scale, const uint8_t *Wt, uint16_t *C,
                                          int M, int N, int K) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!C || (K > 0 && (!Q || !scale || !Wt))) return GEMM_ERR_INVALID_VALUE;
    const size_t c_bytes = (size_t)M * N * 2;
    if (overlaps(C, c_bytes, Q, (size_t)M * K) || overlaps(C, c_bytes, Wt, (size_t)N * K) ||
        overlaps(C, c_bytes, scale, (size_t)M * 4))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {
        return finish(zero_fill(C, c_bytes, dev->num_sms, s), "zero_fill");
    }
    if (!umma_e4m3_supported(Q, Wt, C, N, K)) {
        record_message("gemm_e4m3_rowscale: needs Q, Wt, C 16-byte aligned, K % 16 == 0 and N % 8 == 0");
        return GEMM_ERR_INVALID_VALUE;
    }
    const cudaError_t e = launch_umma_e4m3_rowscale(Q, scale, Wt, C, M, N, K, dev->status, s);
    if (e == cudaErrorNotSupported) {
        record_message("gemm_e4m3_rowscale: the tensor-core kernel cannot describe these operands");
        return GEMM_ERR_INVALID_VALUE;
    }
    return finish(e, "umma_e4m3_rowscale");
}

GEMM_API gemm_status_t gemm_e4m3_rowscale_fused(const uint16_t *A, const uint8_t *Wt, uint16_t *C, int M, int N,
                                                int K) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) { t_last_kernel = "noop"; return GEMM_OK; }
    if (!C || (K > 0 && (!A || !Wt))) return GEMM_ERR_INVALID_VALUE;
    const size_t c_bytes = (size_t)M * N * 2;
    if (overlaps(C, c_bytes, A, (size_t)M * K * 2) || overlaps(C, c_bytes, Wt, (size_t)N * K))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status_t st = device_info(&dev);
    if (st != GEMM_OK) return st;
    cudaStream_t s = t_stream;
    if (K == 0) {
        return finish(zero_fill(C, c_bytes, dev->num_sms, s), "zero_fill");
    }
    if (!umma_e4m3_fused_supported(A, Wt, C, N, K)) {
        record_message("gemm_e4m3_rowscale_fused: needs A, Wt, C 16-byte aligned, K % 16 == 0 and N % 8 == 0");
        return GEMM_ERR_INVALID_VALUE;
    }
    const cudaError_t e = launch_umma_e4m3_fused(A, Wt, C, M, N, K, dev->status, s);
    if (e == cudaErrorNotSupported) {
        record_message("gemm_e4m3_rowscale_fused: the tensor-core kernel cannot describe these operands");
        return GEMM_ERR_INVALID_VALUE;
    }
    return finish(e, "umma_e4m3_rowscale_fused");
}

GEMM_API int64_t gemm_fp4_code_bytes(int rows, int K) {
    if (rows < 0 || K < 0) return -1;
    return (int64_t)fp4_code_size(rows, K);
}

GEMM_API int64_t gemm_fp4_scale_bytes(gemm_fp4_format_t format, int rows, int K) {
    if (rows < 0 || K < 0 || ((int)format != GEMM_FP4_MX && (int)format != GEMM_FP4_NV)) return -1;
    return fp4_scale_size((int)format == GEMM_FP4_NV, rows, K);
}

GEMM_API gemm_status_t gemm_fp4_quantize(gemm_dtype_t dtype, gemm_fp4_format_t format, const void *A, int64_t lda,
                                         const float *tensor_scale, uint8_t *Q, uint8_t *S, int M, int K) {
    return run_fp4_convert("gemm_fp4_quantize", true, (int)dtype, (int)format, A, lda, tensor_scale, Q, S, M, K);
}

GEMM_API gemm_status_t gemm_fp4_dequantize(gemm_dtype_t dtype, gemm_fp4_format_t format, const uint8_t *Q,
                                           const uint8_t *S, const float *tensor_scale, void *A, int64_t lda, int M,
                                           int K) {
    return run_fp4_convert("gemm_fp4_dequantize", false, (int)dtype, (int)format, A, lda, tensor_scale, Q, S, M, K);
}

GEMM_API gemm_status_t gemm_fp4(gemm_dtype_t dtype, gemm_fp4_format_t format, const uint8_t *Qa, const uint8_t *Sa,
                                const float *ga, const uint8_t *Qb, const uint8_t *Sb, const float *gb, void *C,
                                int64_t ldc, int M, int N, int K) {
    return run_fp4("gemm_fp4", (int)dtype, (int)format, nullptr, 0, Qa, Sa, ga, Qb, Sb, gb, C, ldc, M, N, K, false);
}

GEMM_API gemm_status_t gemm_fp4_linear(gemm_dtype_t dtype, gemm_fp4_format_t format, const void *X, int64_t ldx,
                                       const float *gx, const uint8_t *Qw, const uint8_t *Sw, const float *gw,
                                       void *C, int64_t ldc, int M, int N, int K) {
    return run_fp4("gemm_fp4_linear", (int)dtype, (int)format, X, ldx, nullptr, nullptr, gx, Qw, Sw, gw, C, ldc, M, N,
                   K, true);
}

GEMM_API gemm_status_t gemm_gated(gemm_dtype_t dtype, gemm_act_t act, const void *X, const void *W_g, const void *W_u,
                                  void *Z, float *G, float *U, int M, int N, int K) {
    return run_gated((int)dtype, (int)act, X, W_g, W_u, Z, G, U, M, N, K);
}

GEMM_API gemm_status_t gemm_gated_backward(gemm_dtype_t dtype, gemm_act_t act, const void *X, const void *W_g,
                                           const void *W_u, const float *G, const float *U, const void *dZ, void *dX,
                                           void *dW_g, void *dW_u, int M, int N, int K) {
    return run_gated_backward((int)dtype, (int)act, X, W_g, W_u, G, U, dZ, dX, dW_g, dW_u, M, N, K);
}

GEMM_API gemm_status_t gemm_set_stream(void *cuda_stream) {
    t_stream = static_cast<cudaStream_t>(cuda_stream);
    return GEMM_OK;
}

GEMM_API void *gemm_get_stream(void) { return t_stream; }

GEMM_API gemm_status_t gemm_synchronize(void) {
    cudaError_t e = cudaStreamSynchronize(t_stream);
    if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
    // The status words that exist on this device: the allocating entry points'
    // (once one of them has run here) and the allocation-free entry point's
    // (once it has run here).  Reading them allocates nothing.
    int code = 0;
    DeviceInfo &d = g_devices[dev];
    if (d.ready.load(std::memory_order_acquire)) {
        e = cudaMemcpy(&code, d.status, sizeof(int), cudaMemcpyDeviceToHost);
        if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
        if (code != 0) {
            e = cudaMemset(d.status, 0, sizeof(int));
            if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
        }
    }
    int code_na = 0;
    e = take_noalloc_status(dev, &code_na);
    if (e != cudaSuccess) { record_cuda_error(e); return GEMM_ERR_CUDA; }
    return (code | code_na) != 0 ? GEMM_ERR_TIMEOUT : GEMM_OK;
}

GEMM_API const char *gemm_status_string(gemm_status_t s) {
    switch (s) {
    case GEMM_OK: return "GEMM_OK";
    case GEMM_ERR_INVALID_VALUE: return "GEMM_ERR_INVALID_VALUE";
    case GEMM_ERR_ALIAS: return "GEMM_ERR_ALIAS";
    case GEMM_ERR_UNSUPPORTED_DEVICE: return "GEMM_ERR_UNSUPPORTED_DEVICE";
    case GEMM_ERR_CUDA: return "GEMM_ERR_CUDA";
    case GEMM_ERR_TIMEOUT: return "GEMM_ERR_TIMEOUT";
    }
    return "GEMM_ERR_UNKNOWN";
}

GEMM_API const char *gemm_last_kernel(void) { return t_last_kernel; }

GEMM_API unsigned long long gemm_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

GEMM_API const char *gemm_last_error(void) { return t_last_error; }

GEMM_API gemm_status_t gemm_force_kernel(const char *family) {
    if (!family || !*family) { t_force = Family::Auto; return GEMM_OK; }
    if (!strcmp(family, "simt")) t_force = Family::Simt;
    else if (!strcmp(family, "simt_scalar")) t_force = Family::SimtScalar;
    else if (!strcmp(family, "gemv")) t_force = Family::Gemv;
    else if (!strcmp(family, "gemv_scalar")) t_force = Family::GemvScalar;
    else if (!strcmp(family, "umma")) t_force = Family::Umma;
    else if (!strcmp(family, "umma_skinny_wide")) t_force = Family::UmmaSkinnyWide;
    else if (!strcmp(family, "umma_stall")) t_force = Family::UmmaStall;
    else if (!strcmp(family, "umma_stall_pair")) t_force = Family::UmmaStallPair;
    else if (!strcmp(family, "umma_stall_peer")) t_force = Family::UmmaStallPeer;
    else return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

}  // extern "C"
