// Gated feed-forward block, any N, K and alignment.  TMA describes matrices that
// start, and whose rows start, on 16 bytes.  Operands that do not (N or K no
// multiple of 8, a base off 16 bytes) are copied to scratch with rows of whole 16
// bytes, zeros behind the row and below the matrix, the products run over the
// padded sizes, and results are copied back: the zeros add nothing to a sum, and a
// column past N or K is dropped.  (X alone goes to rows of 128 bytes for speed, below.)
//
// A copy is bound by memory, each byte read and written once, a call of few rows
// by it: bf16 SiLU forward 1 x 12289 x 4096 110 us (both weights copied at 5.1 TB/s),
// where 1 x 12288 x 4096 takes 30.7; 1024 x 12285 x 4095 201 us against 113.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.h"
#include "gated.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

constexpr int WARPS = 4;

// dst [dst_rows, dst_cols] = src [src_rows, src_cols], cut off or zeros behind and
// below; rows of 16-bit elements (FP32: two) without gaps, on any 2 bytes.  A lane
// stores two aligned 16-byte pieces of a dst row, a warp 512 elements, from
// 16-byte loads shifted to their place (fp4.h).
__global__ void __launch_bounds__(WARPS * 32)
gated_copy_kernel(const uint16_t *__restrict__ src, long long src_rows, long long src_cols, uint16_t *__restrict__ dst,
                  long long dst_rows, long long dst_cols)
{
    pdl_wait();
    const long long row = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (row >= dst_rows) return;  // warp-uniform
    const int lane = threadIdx.x & 31;
    uint16_t *d = dst + row * dst_cols;
    const int off = (int)(((uintptr_t)d & 15) >> 1);
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(src),
                  *hi = reinterpret_cast<const uint8_t *>(src + src_rows * src_cols);
    const long long width = row < src_rows ? min(src_cols, dst_cols) : -1024;
    for (long long k0 = blockIdx.y * 512LL; k0 < dst_cols + off; k0 += gridDim.y * 512LL) {
        const long long k = k0 + lane * 16 - off;
        uint32_t v[8];
        fp4_load16_any(src + row * src_cols + k, (int)max(min(width - k, 512LL), -512LL), lo, hi, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long at = k + 8 * h;
            if (at >= 0 && at + 8 <= dst_cols) {
                *reinterpret_cast<uint4 *>(d + at) = make_uint4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + j >= 0 && at + j < dst_cols) d[at + j] = (uint16_t)(v[4 * h + (j >> 1)] >> (16 * (j & 1)));
            }
        }
    }
}

cudaError_t copy(const void *src, long long src_rows, long long src_cols, void *dst, long long dst_rows,
                 long long dst_cols, cudaStream_t s) {
    const long long gx = (dst_rows + WARPS - 1) / WARPS, gy = std::min<long long>((dst_cols + 7 + 511) / 512, 65535);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)gx, (unsigned)gy), dim3(WARPS * 32), 0, s, attr);
    return launch_counted(&cfg, gated_copy_kernel, static_cast<const uint16_t *>(src), src_rows, src_cols,
                          static_cast<uint16_t *>(dst), dst_rows, dst_cols);
}

long long up8(long long n) { return (n + 7) & ~7LL; }
bool on16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// A call's operands and, for those that need one, their padded copies.
class Padded {
  public:
    // A matrix [rows, cols] of `words` 16-bit words an element (null: left out), which
    // the products see as [prows, pcols]; *at: the address for them, once begin() has
    // returned.
    void add(const void **at, const void *user, long long rows, long long prows, long long cols, long long pcols,
             int words, bool out) {
        *at = user;
        if (!user || (on16(user) && rows == prows && cols == pcols)) return;
        Operand &o = ops_[n_++];
        o = {at, const_cast<void *>(user), rows, prows, cols * words, pcols * words, out, bytes_};
        bytes_ += ((size_t)(o.prows * o.pcols) * 2 + 255) & ~(size_t)255;
    }
    cudaError_t begin(cudaStream_t s) {
        if (n_ == 0) return cudaSuccess;
        cudaError_t e = scratch_alloc(&ws_, bytes_, s);
        for (int i = 0; i < n_ && e == cudaSuccess; ++i) {
            Operand &o = ops_[i];
            o.pad = static_cast<uint8_t *>(ws_) + o.offset;
            *o.at = o.pad;
            if (!o.out) e = copy(o.user, o.rows, o.cols, o.pad, o.prows, o.pcols, s);
        }
        return e;
    }
    // After the products, which returned e.
    cudaError_t end(cudaError_t e, cudaStream_t s) {
        for (int i = 0; i < n_ && e == cudaSuccess; ++i) {
            const Operand &o = ops_[i];
            if (o.out) e = copy(o.pad, o.prows, o.pcols, o.user, o.rows, o.cols, s);
        }
        const cudaError_t f = ws_ ? cudaFreeAsync(ws_, s) : cudaSuccess;
        return e != cudaSuccess ? e : f;
    }

  private:
    struct Operand {
        const void **at;
        void *user;
        long long rows, prows, cols, pcols;  // columns in 16-bit words
        bool out;
        size_t offset;
        void *pad;
    };
    Operand ops_[9];
    int n_ = 0;
    size_t bytes_ = 0;
    void *ws_ = nullptr;
};

}  // namespace

cudaError_t launch_gated_forward(const GatedProblem &p, int num_sms, int *status, cudaStream_t s) {
    const long long n8 = up8(p.N), k8 = up8(p.K);
    if (n8 > 0x7FFFFFFFLL || k8 > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    GatedProblem q = p;
    const void *z, *g, *u;
    // X also goes to rows of 128 bytes where rows of neither it nor the weights start
    // on 128 and the products, some 1.3 times slower then (gated.cu), take long
    // enough: the copy's own time and about 10 us of allocation, launch and lost
    // overlap.  Forward of 1024 x 12280 x 4088 122 us, 153 as it lies.
    const bool odd = p.N % 64 != 0 && p.K % 64 != 0, large = p.M > kGatedSkinnyMaxM;
    const double ns = 4.0 * p.M * p.N * p.K / 1.7e6, copy_ns = 1e4 + 4.0 * p.M * p.K / 5e3;
    q.ldx = p.K % 8 != 0 || !on16(p.X) || (odd && large && 0.3 * ns > copy_ns) ? (p.K + 63LL) / 64 * 64 : p.K;
    Padded pad;
    pad.add(&q.X, p.X, p.M, p.M, p.K, q.ldx, 1, false);
    pad.add(&q.Wg, p.Wg, p.K, k8, p.N, n8, 1, false);
    pad.add(&q.Wu, p.Wu, p.K, k8, p.N, n8, 1, false);
    pad.add(&z, p.Z, p.M, p.M, p.N, n8, 1, true);
    pad.add(&g, p.G, p.M, p.M, p.N, n8, 2, true);
    pad.add(&u, p.U, p.M, p.M, p.N, n8, 2, true);
    cudaError_t e = pad.begin(s);
    q.Z = const_cast<void *>(z);
    q.G = static_cast<float *>(const_cast<void *>(g));
    q.U = static_cast<float *>(const_cast<void *>(u));
    q.N = (int)n8;
    q.K = (int)k8;
    if (e == cudaSuccess)
        e = q.M <= kGatedSkinnyMaxM ? launch_gated_skinny(q, num_sms, status, s) : launch_gated(q, status, s);
    return pad.end(e, s);
}

cudaError_t launch_gated_gradients(const GatedBackward &p, int num_sms, int *status, cudaStream_t s) {
    const long long n8 = up8(p.N), k8 = up8(p.K);
    if (n8 > 0x7FFFFFFFLL || k8 > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    GatedBackward q = p;
    const void *g, *u, *dx, *dwg, *dwu;
    Padded pad;
    const bool weights = p.dWg || p.dWu;
    if (weights) pad.add(&q.X, p.X, p.M, p.M, p.K, k8, 1, false);
    if (p.dX) {
        pad.add(&q.Wg, p.Wg, p.K, k8, p.N, n8, 1, false);
        pad.add(&q.Wu, p.Wu, p.K, k8, p.N, n8, 1, false);
    }
    pad.add(&q.dZ, p.dZ, p.M, p.M, p.N, n8, 1, false);
    pad.add(&g, p.G, p.M, p.M, p.N, n8, 2, false);
    pad.add(&u, p.U, p.M, p.M, p.N, n8, 2, false);
    pad.add(&dx, p.dX, p.M, p.M, p.K, k8, 1, true);
    pad.add(&dwg, p.dWg, p.K, k8, p.N, n8, 1, true);
    pad.add(&dwu, p.dWu, p.K, k8, p.N, n8, 1, true);
    cudaError_t e = pad.begin(s);
    q.G = static_cast<const float *>(g);
    q.U = static_cast<const float *>(u);
    q.dX = const_cast<void *>(dx);
    q.dWg = const_cast<void *>(dwg);
    q.dWu = const_cast<void *>(dwu);
    q.N = (int)n8;
    q.K = (int)k8;
    if (e == cudaSuccess) e = launch_gated_backward(q, num_sms, status, s);
    return pad.end(e, s);
}

}  // namespace gemm_gb300
