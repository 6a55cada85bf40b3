// Softmax cross entropy of a linear head, Z = X W^T over a large vocabulary, and its
// gradients, without the logits in memory.
//
// Forward: tiles of Z stay in tensor memory; the epilogue takes the largest logit m and
// s = sum exp(z - m) of each row's 64 to 128 columns (online, 32 at a time: s <- s e^(m - m')
// + sum e^(z - m')), and the row's own target's logit.  A second kernel joins the pairs
// of a row, in order: lse = m + log s.  All in FP32.
//
// Rows of W off 16 bytes (K no multiple of 8) are read in place by classes of their alignment
// where there are few rows of X against them (Classes; pair_pipe.cuh), else copied, padded.
//
// Backward, in pieces of the vocabulary: the piece's logits anew, dZ = (e^(z - lse) -
// [j = t]) dloss rounded to 16 bits (the operand of the products to come) in scratch,
// dW of the piece = dZ^T X, and dX += dZ W in FP32.  Where a piece of dX has few tiles
// its sum is cut into K ranges, a slab of FP32 each; the ranges' sums grow piece after
// piece (one addition to an element a launch, in stream order) and are added in order by
// the last kernel: deterministic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "cross_entropy.h"
#include "fp4.h"
#include "pair_pipe.cuh"

namespace gemm_gb300 {
namespace {

using namespace pair;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {  // 2^x, 2 units of 2^-23 off; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A partial sum s of e^z with the largest logit m is kept as the sum of 2^(z log2 e - base_of(m)),
// terms of one fused operation each.  base_of(m) is m log2 e rounded, everywhere: m log2 e left to
// a fused operation differs from it, so that a maximum that stayed took up to 2^-24 m with it
// from each sum to the next (loss of 131072 logits of 1000 3e-4 off), and from 2^31 on left no
// sum at all.  Logits beyond kFar are 32 and more apart, and m log2 e may overflow: 2^(z - m),
// which is 1 or as good as nothing; of infinite m 2^z.
constexpr float kFar = 0x1p29f;
__device__ __forceinline__ bool is_far(float m) { return !(fabsf(m) <= kFar); }
__device__ __forceinline__ float base_of(float m) { return __fmul_rn(m, kLog2e); }
// m log2 e - base_of(m)
__device__ __forceinline__ float left_of(float m) { return is_far(m) ? 0.0f : fmaf(m, kLog2e, -base_of(m)); }

// Of the columns [c0, c0 + 32) within a row's [0, N), c0 < N: the rest count as -inf.
struct LseArgs {
    float2 *part;             // (m, s) of a warp's columns of a tile, [slot][M], slots from slot0 on
    float *zt;                // Z_i,t_i
    const long long *target;
    int M, N, v0, total;      // rows; columns of this piece, and its first; of Z
    int slot0, classes;
};
template <bool JOINED, bool OF_CLASSES>
struct LseEpi : LseArgs {
    static constexpr bool LOWER = false, JOIN = JOINED, CLASSES = OF_CLASSES;
    static constexpr int BOXES = JOINED ? 2 : 1;

    struct Pre {};
    __device__ __forceinline__ void prefetch(const Part &, Pre &) const {}
    __device__ __forceinline__ void run(Part &p, const Pre &) const {
        const int row = p.row0 + p.lane, first = p.col0 + p.first;
        long long t = row < M ? target[row] : -1;
        t = t >= 0 && t < total ? t - v0 : -1;
        int cols = N;
        if (CLASSES) {  // columns cls, cls + classes, ... of N
            cols = (N - p.cls + classes - 1) / classes;
            t = t >= 0 && (int)t % classes == p.cls ? (int)t / classes : -1;
        }
        const int width = min(p.width, cols - first);
        float m = -INFINITY, s = 0.0f;
#pragma unroll 1
        for (int c = 0; c < width; c += 32) {
            uint32_t r[32];
            p.load<JOIN>(p.first + c, r);
            const int left = width - c;
            if (left < 32) {  // warp-uniform
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= left) r[j] = 0xFF800000u;
            }
            const long long at = t - (first + c);
            if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j == at) zt[row] = __uint_as_float(r[j]);
            }
            float top = __uint_as_float(r[0]);
#pragma unroll
            for (int j = 1; j < 32; ++j) top = fmaxf(top, __uint_as_float(r[j]));
            top = fmaxf(top, m);
            const bool far = is_far(top);
            const float base = far ? (isinf(top) ? 0.0f : top) : base_of(top), by = far ? 1.0f : kLog2e;
            float s0 = s * ex2(far ? (m == top ? 0.0f : -INFINITY) : base_of(m) - base), s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                s0 += ex2(fmaf(__uint_as_float(r[j]), by, -base));
                s1 += ex2(fmaf(__uint_as_float(r[j + 1]), by, -base));
                s2 += ex2(fmaf(__uint_as_float(r[j + 2]), by, -base));
                s3 += ex2(fmaf(__uint_as_float(r[j + 3]), by, -base));
            }
            s = (s0 + s1) + (s2 + s3);
            m = top;
        }
        if (row < M) part[(long long)(slot0 + p.tile_n * p.ranges + p.range) * M + row] = make_float2(m, s);
    }
};

// Scale factors of dZ: (up, down), whose product is 1 but for rounding.
struct DzArgs {
    CUtensorMap tm;  // dZ of the piece
    const float *lse, *dloss;
    const long long *target;
    const float2 *scale;
    int M, N, v0, total;  // total: columns of Z
    int classes;          // of columns (N: of the largest class): a matrix of dZ each
    bool bf16;
};
template <bool JOINED, bool OF_CLASSES>
struct DzEpi : DzArgs {
    static constexpr bool LOWER = false, JOIN = JOINED, CLASSES = OF_CLASSES;
    static constexpr int BOXES = JOINED ? 2 : 1;

    struct Pre {  // a row's
        long long t;
        bool counts;
        float base, by;  // p is 2^(z by - base) 2^-left, left the base's rounding: the latter goes with d
        float d, one;
    };
    __device__ __forceinline__ void prefetch(const Part &p, Pre &pre) const {
        const int row = p.row0 + p.lane;
        pre.t = row < M ? target[row] : -1;
        pre.counts = pre.t >= 0 && pre.t < total;
        const float l = pre.counts ? lse[row] : 0.0f, left = left_of(l);
        pre.base = is_far(l) ? l : base_of(l);
        pre.by = is_far(l) ? 1.0f : kLog2e;
        pre.d = pre.counts ? dloss[row] * scale->x * ex2(-left) : 0.0f;
        pre.one = ex2(left);
    }
    __device__ __forceinline__ void run(Part &p, const Pre &pre) const {
        const bool counts = pre.counts;
        const float d = pre.d, base = pre.base, by = pre.by, one = pre.one;
        long long t = pre.t;
        t = counts ? t - v0 : -1;
        int cols = N;
        if (CLASSES) {
            cols = (total - p.cls + classes - 1) / classes;
            t = t >= 0 && (int)t % classes == p.cls ? (int)t / classes : -1;
        }
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 64) {
            const int c0 = p.col0 + g;
            if (c0 >= N) return;  // warp-uniform
            uint32_t z[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                p.load<JOIN>(g + h * 32, r);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = ex2(fmaf(__uint_as_float(r[j]), by, -base));
                const long long at = t - (c0 + h * 32);
                if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == at) v[j] -= one;
                }
                if (CLASSES && c0 + h * 32 + 32 > cols) {  // (a class may be one column short)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c0 + h * 32 + j >= cols) v[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x = counts ? v[2 * j] * d : 0.0f, y = counts ? v[2 * j + 1] * d : 0.0f;
                    z[h * 16 + j] = bf16 ? pack2(x, y, (__nv_bfloat16 *)nullptr) : pack2(x, y, (__half *)nullptr);
                }
            }
            uint8_t *box = box_next<BOXES>(p);
            box_put(box, p.lane, z);
            box_store(&tm, box, p.lane, c0, p.row0, p.cls);
        }
    }
};

// FP32 sums to slab `split`, or added to it.
template <bool OF_CLASSES>
struct AccEpi {
    static constexpr bool LOWER = false, JOIN = false, CLASSES = OF_CLASSES;
    static constexpr int BOXES = 1;
    CUtensorMap tm;
    int N;
    bool add;

    struct Pre {};
    __device__ __forceinline__ void prefetch(const Part &, Pre &) const {}
    __device__ __forceinline__ void run(Part &p, const Pre &) const {
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 32) {
            if (p.col0 + g >= N) return;  // warp-uniform
            uint32_t r[32];
            p.load<false>(g, r);
            uint8_t *box = box_next<BOXES>(p);
            box_put(box, p.lane, r);
            if (add) {
                fence_async_shared();
                __syncwarp();
                if (p.lane == 0) tma_add_3d(&tm, box, p.col0 + g, p.row0, p.split);
            } else {
                box_store(&tm, box, p.lane, p.col0 + g, p.row0, p.split);
            }
        }
    }
};

// Columns g .. g + 63 of a tile times f, in 16 bits.
__device__ __forceinline__ void scaled(const Part &p, int g, float f, bool bf16, uint32_t (&z)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        p.load<false>(g + h * 32, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float x = __uint_as_float(r[2 * j]) * f, y = __uint_as_float(r[2 * j + 1]) * f;
            z[h * 16 + j] = bf16 ? pack2(x, y, (__nv_bfloat16 *)nullptr) : pack2(x, y, (__half *)nullptr);
        }
    }
}

// 16-bit results times scale->y.
struct OutEpi {
    static constexpr bool LOWER = false, JOIN = false, CLASSES = false;
    static constexpr int BOXES = 2;
    CUtensorMap tm;
    const float2 *scale;
    uint16_t *out;        // not null: by the element, rows ld apart
    long long ld;
    int M, N;
    bool bf16;

    struct Pre {};
    __device__ __forceinline__ void prefetch(const Part &, Pre &) const {}
    __device__ __forceinline__ void run(Part &p, const Pre &) const {
        const float f = scale->y;
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 64) {
            const int c0 = p.col0 + g;
            if (c0 >= N) return;  // warp-uniform
            uint32_t z[32];
            scaled(p, g, f, bf16, z);
            uint8_t *box = box_next<BOXES>(p);
            box_put(box, p.lane, z);
            if (out) box_scatter(box, p.lane, out, ld, p.row0, c0, M, N);
            else box_store(&tm, box, p.lane, c0, p.row0, 0);
        }
    }
};

// The same to rows off 16 bytes, of classes (pair_pipe.cuh): D has a class's rows after the
// other's, class_rows (whole tiles) each, and its columns are turned, from the first whole 16
// bytes of out's row, u_r elements behind its start, to its end and on from its start.  Whole
// pieces go by TMA, a matrix of every classes-th row each, the up to seven elements at each
// end of a row one by one (dW of 1 x 32000 x 4095 78 us, by
// the element 126).
struct TurnEpi {
    static constexpr bool LOWER = false, JOIN = false, CLASSES = false;
    static constexpr int BOXES = 2;
    BMaps<true> tm;
    const float2 *scale;
    uint16_t *out;
    int classes, class_rows;
    uint32_t turns;  // u_r, four bits each
    int M, N;        // of out
    bool bf16;

    struct Pre {};
    __device__ __forceinline__ void prefetch(const Part &, Pre &) const {}
    __device__ __forceinline__ void run(Part &p, const Pre &) const {
        const float f = scale->y;
        const int cls = p.row0 / class_rows, row0 = p.row0 - cls * class_rows, rows = (M - cls + classes - 1) / classes;
        if (row0 >= rows) return;
        const int u = turns >> (4 * cls) & 7, whole = (N - u) & ~7;
        uint16_t *const row = out + ((long long)(row0 + p.lane) * classes + cls) * N;
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 64) {
            const int c0 = p.col0 + g;
            if (c0 >= N) return;  // warp-uniform
            uint32_t z[32];
            scaled(p, g, f, bf16, z);
            uint8_t *box = box_next<BOXES>(p);
            box_put(box, p.lane, z);
            if (c0 < whole) box_store(&tm.m[cls], box, p.lane, c0, row0, 0);
            else box_unstored(p.lane);  // 64 columns of a row's tail alone: K of 64 i + 1 to 64 i + 14
            if (row0 + p.lane < rows) {
                for (int c = max(c0, whole); c < min(c0 + 64, N); ++c) {
                    const int e = c - c0;
                    row[c + u < N ? c + u : c + u - N] =
                        *reinterpret_cast<const uint16_t *>(box + p.lane * 128 + (((e >> 3) ^ (p.lane & 7)) << 4) + (e & 7) * 2);
                }
            }
        }
    }
};

// A row's (m, s), joined with another's.
struct MaxSum {
    float m = -INFINITY, s = 0.0f;

    __device__ __forceinline__ void join(float om, float os) {
        const float top = fmaxf(m, om), b = base_of(m), ob = base_of(om);
        float f = ex2(fminf(b, ob) - fmaxf(b, ob));
        if (is_far(top)) f = m == om ? 1.0f : 0.0f;
        s = m >= om ? fmaf(os, f, s) : fmaf(s, f, os);
        m = top;
    }
    // The loss without lse's rounding, which is of m's size.
    __device__ __forceinline__ void store(float zt, long long t, int N, float *loss, float *lse) const {
        const float o = isfinite(m) ? m : 0.0f, l = logf(s) - left_of(o) * kLn2;
        *loss = t >= 0 && t < N ? (o - zt) + l : 0.0f;
        if (lse) *lse = o + l;
    }
};
// Joins the slots.  ROWS to a CTA: 8 (of a slot 64 adjacent bytes, two whole sectors), slots
// dealt to 128 lanes of each, or, of few rows, 1 -- a row's joins are a chain of latencies
// (forward of 200 x 50257 x 64 12.5 us, against 14.9 with 256 threads to a row; 65 x 50257 x 64
// 11.0, against 12.3 with 8).
template <int ROWS>
__global__ void __launch_bounds__(1024)
head_join_kernel(const float2 *__restrict__ part, const float *__restrict__ zt, const long long *__restrict__ target,
                 float *__restrict__ loss, float *__restrict__ lse, int slots, int M, int N)
{
    __shared__ float2 mine[32][ROWS];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane % ROWS;
    const long long row = (long long)blockIdx.x * ROWS + r;
    MaxSum v;
    if (row < M) {
#pragma unroll 4
        for (int i = threadIdx.x / ROWS; i < slots; i += 1024 / ROWS) {
            const float2 p = __ldcg(part + (long long)i * M + row);
            v.join(p.x, p.y);
        }
    }
    auto fold = [&] {  // the lanes of a row
#pragma unroll
        for (int o = 16; o >= ROWS; o >>= 1) {
            const float om = __shfl_down_sync(0xffffffffu, v.m, o), os = __shfl_down_sync(0xffffffffu, v.s, o);
            v.join(om, os);
        }
    };
    fold();
    if (lane < ROWS) mine[warp][r] = make_float2(v.m, v.s);
    __syncthreads();
    if (warp != 0) return;
    const float z = lane < ROWS && row < M ? zt[row] : 0.0f;
    const long long t = lane < ROWS && row < M ? target[row] : -1;
    v = MaxSum{};
#pragma unroll
    for (int w = 0; w < ROWS; ++w) {
        const float2 p = mine[lane / ROWS * ROWS + w][r];
        v.join(p.x, p.y);
    }
    fold();
    if (lane < ROWS && row < M) v.store(z, t, N, loss + row, lse ? lse + row : nullptr);
}

__global__ void __launch_bounds__(256)
head_flat_kernel(const long long *__restrict__ target, float *__restrict__ loss, float *__restrict__ lse, int M, int N)
{
    pdl_wait();
    const long long row = blockIdx.x * 256LL + threadIdx.x;
    if (row >= M) return;
    const float l = logf((float)N);
    const long long t = target[row];
    loss[row] = t >= 0 && t < N ? l : 0.0f;
    if (lse) lse[row] = l;
}

// The factor that takes the largest |dloss| of a row with a target to `peak`, and its inverse.
// peak is a power of two, so that where all rows weigh alike a probable target's dZ, -peak
// (1 - p), is nearly representable: a weight of 1 / 777 in 16 bits is off by a relative 2^-9
// or less, but by the same in every row, and both gradients with it (bf16, 1100 x 5000 x 512,
// weights of 1 / 848: 0.0034 off against 0.0017).  Half: 2^14, so that dZ keeps half's full
// precision down to probabilities of 2^-28.  By a CTA.
struct ScaleArgs {
    const float *dloss;
    const long long *target;
    float2 *scale;
    float peak;
    int M, N;
};
template <int THREADS>
__device__ __forceinline__ void find_scale(const ScaleArgs &a) {
    __shared__ float tops[THREADS / 32];
    float top = 0.0f;
#pragma unroll 4
    for (long long i = threadIdx.x; i < a.M; i += THREADS) {
        const long long t = a.target[i];
        const float d = fabsf(a.dloss[i]);
        if (t >= 0 && t < a.N) top = fmaxf(top, d);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < THREADS / 32; ++w) top = fmaxf(top, tops[w]);
    // (no factor leaves the normal numbers)
    top = top > 0.0f && isfinite(top) ? fminf(fmaxf(top, 0x1p-110f), 0x1p110f) : a.peak;
    *a.scale = make_float2(a.peak / top, top / a.peak);
}
__global__ void __launch_bounds__(1024)
head_scale_kernel(const ScaleArgs a)
{
    pdl_wait();
    find_scale<1024>(a);
}

// dst [rows, dst_cols] (rows of whole 16 bytes) = src [rows, cols] (any 2 bytes), zeros
// behind the row and, where targets are given, in rows whose target is no column of N: a
// lane two 16-byte pieces (fp4.h).  A scale to find is one more CTA's.  Of classes: matrix z
// of dst has its rows behind as many zeros as the z-th four bits of `fronts` say, 7 at most,
// or turned left by as many elements as those of `turns` do.
constexpr int COPY_WARPS = 4;
__global__ void __launch_bounds__(COPY_WARPS * 32)
head_copy_kernel(const uint16_t *__restrict__ src, long long rows, long long cols, uint16_t *__restrict__ dst,
                 long long dst_cols, const long long *__restrict__ target, int N, unsigned long long fronts,
                 unsigned long long turns, const ScaleArgs a)
{
    pdl_wait();
    if (a.scale && blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0 && blockIdx.z == 0) find_scale<COPY_WARPS * 32>(a);
        return;
    }
    const long long row = (long long)blockIdx.x * COPY_WARPS + (threadIdx.x >> 5);
    if (row >= rows) return;  // warp-uniform
    const int lane = threadIdx.x & 31;
    const long long t = target ? target[row] : 0;
    const long long width = t >= 0 && t < N ? cols : -1024;
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(src), *hi = reinterpret_cast<const uint8_t *>(src + rows * cols);
    uint16_t *d = dst + (blockIdx.z * rows + row) * dst_cols;
    const int front = (int)(fronts >> (4 * blockIdx.z) & 7), turn = (int)(turns >> (4 * blockIdx.z) & 7);
    for (long long k0 = blockIdx.y * 512LL; k0 < dst_cols; k0 += gridDim.y * 512LL) {
        const long long k = k0 + lane * 16;
        uint32_t v[8];
        fp4_load16_any(src + row * cols + k - front + turn, (int)max(min(width + front - turn - k, 512LL), -512LL), lo, hi, v);
        if (turn && width > 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const long long at = k + j - (cols - turn);
                if (at >= 0 && at < turn) v[j >> 1] |= (uint32_t)src[row * cols + at] << (16 * (j & 1));
            }
        }
        if (k == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] &= (2 * j < front ? 0u : 0xFFFFu) | (2 * j + 1 < front ? 0u : 0xFFFF0000u);
        }
        if (k < dst_cols) *reinterpret_cast<uint4 *>(d + k) = make_uint4(v[0], v[1], v[2], v[3]);
        if (k + 8 < dst_cols) *reinterpret_cast<uint4 *>(d + k + 8) = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
cudaError_t copy(const void *src, long long rows, long long cols, void *dst, long long dst_cols, const long long *target,
                 int N, const ScaleArgs &scale, cudaStream_t s, int matrices = 1, unsigned long long fronts = 0,
                 unsigned long long turns = 0) {
    const long long gx = (rows + COPY_WARPS - 1) / COPY_WARPS + (scale.scale ? 1 : 0), gy = std::min<long long>((dst_cols + 511) / 512, 65535);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)gx, (unsigned)gy, (unsigned)matrices), dim3(COPY_WARPS * 32), 0, s, attr);
    return launch_counted(&cfg, head_copy_kernel, static_cast<const uint16_t *>(src), rows, cols, static_cast<uint16_t *>(dst),
                          dst_cols, target, N, fronts, turns, scale);
}

// dX = (sum of the slabs, in order) scale->y, four elements to a thread.  Of classes, `per`
// slabs each, a slab's columns lie as far right as the class's four bits of `shifts` say.
template <typename T>
__global__ void __launch_bounds__(256)
head_finish_kernel(const float *__restrict__ slab, int slabs, long long rows, int cols, long long ld, int per, uint32_t shifts,
                   const float2 *scale, T *__restrict__ out)
{
    pdl_wait();
    const long long quads = (cols + 3) / 4, i = blockIdx.x * 256LL + threadIdx.x;
    if (i >= rows * quads) return;
    const long long row = i / quads;
    const int c = (int)(i - row * quads) * 4;
    const float *p = slab + row * ld + c;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (per) {
#pragma unroll 4
        for (int j = 0; j < slabs; ++j) {
            const float *q = p + j * rows * ld + (shifts >> (4 * (j / per)) & 7);
            v.x += __ldcg(q); v.y += __ldcg(q + 1); v.z += __ldcg(q + 2); v.w += __ldcg(q + 3);
        }
    } else {
#pragma unroll 4
        for (int j = 0; j < slabs; ++j) {
            const float4 w = __ldcg(reinterpret_cast<const float4 *>(p + j * rows * ld));
            v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
        }
    }
    const float f = scale->y;
    T *o = out + row * cols + c;
    if (((uintptr_t)o & 7) == 0 && c + 4 <= cols) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack2(v.x * f, v.y * f, (T *)nullptr), pack2(v.z * f, v.w * f, (T *)nullptr));
    } else {
        const float e[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 4 && c + j < cols; ++j) store1(o + j, e[j] * f);
    }
}

long long up(long long n, long long to) { return (n + to - 1) / to * to; }
bool on16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// A piece's part of scratch, 256 bytes aligned.
struct Layout {
    size_t bytes = 0;
    size_t add(size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) & ~(size_t)255;
        return at;
    }
};

constexpr long long kPiece = 256LL << 20;  // bytes of a piece of dZ, or of a padded piece of W

// How the logits' tiles are cut: few go in 128 columns, and where one wave of them takes
// joined pairs, a half of K each, if they are done first (forward of 1 x 1000 x 4096 16.6 us
// against 26.8, 4 x 5000 x 4096 22.6 against 27.0, 1500 x 1500 x 4000 24.6 against 28.7; 1 x
// 12000 x 4096, three waves of joined pairs, 45.6 against 29.0).  Up to 128 rows in tiles of
// 128 x 256 (128 x 50257 x 1000: 28.7 us, backward 90, against 30.8 and 95; 64 x 32000 x 4096
// 51.5 and 154 against 53.4 and 158).  192 columns where that fills the waves (700 x 9000 x
// 2000 23.8 us, against 26.9 in 256 and 29.8 in 128; 1000 x 32000 x 512 29.5 against 27.0 in
// 256).  Times in 1/100 us: a block of 64 k of rows x bn, a join.
struct LogitPlan {
    int bn, joined, clusters, rows;
    long long tiles;

    int ranges() const { return rows == 128 ? 4 : 2; }  // of a tile's columns, a warp each
};
template <uint32_t FORMAT, template <bool, bool> class Epi, bool CLASSES>
LogitPlan logit_plan(int M, int N, long long kb, int classes, int dev) {
    LogitPlan best = {};
    long long least = 0;
    constexpr struct {
        int bn, joined, rows, block;
    } ways[5] = {{256, 1, 256, 28}, {256, 1, 128, 15}, {192, 1, 256, 24}, {128, 1, 256, 20}, {128, 2, 256, 20}};
    for (const auto &w : ways) {
        if (w.rows < 256 && M > w.rows) continue;
        const int c = w.joined == 1 ? clusters_max<FORMAT, Epi<false, CLASSES>>(dev) : joined_max<FORMAT, Epi<true, CLASSES>>(dev);
        const long long tiles = ceil_div(M, 256) * ceil_div(ceil_div(N, classes), w.bn) * classes;
        if (c <= 0 || tiles > 0x7FFFFFFFLL || (w.joined > 1 && (tiles > c || kb < 2))) continue;
        const long long time = ceil_div(tiles, c) * ceil_div(kb, w.joined) * w.block + (w.joined > 1 ? 80 : 0);
        if (!best.bn || time < least) {
            best = {w.bn, w.joined, c, w.rows, tiles};
            least = time;
        }
    }
    return best;
}

// W read in place where its rows lie off 16 bytes (pair_pipe.cuh), of K elements from w on: its
// classes and their shifts.
struct Classes {
    int n;
    uint32_t shifts;

    Classes(const void *w, int K) : n(1), shifts(0) {
        if (K < 8) return;  // a class's rows, up to seven elements in front, would overlap
        while (n * (K % 8) % 8) n *= 2;
        for (int r = 0; r < n; ++r) shifts |= (uint32_t)(((uintptr_t)w / 2 + (uintptr_t)r * (K % 8)) % 8) << (4 * r);
    }
    // W in place costs a copy of X for each class and a pause of the MMAs for the zeros in front
    // of each tile, W's copy twice its reading and writing (forward of 22 x 60179 x 951 36 us
    // against 71, 1000 x 50000 x 2001 148 against 188; 3000 x 60000 x 701 225 against 180, 1000
    // x 8000 x 2001 43 against 39).
    bool pay(long long M, int N) const { return n > 1 && N <= 1 << 30 && 4LL * n * M <= N; }
    int shift(int r) const { return (int)(shifts >> (4 * r) & 7); }
    // Class r of N rows, K-major.
    bool map(CUtensorMap *m, const void *w, uint32_t format, int N, long long K, int r, int box_rows) const {
        const int s = shift(r);
        return map16(m, static_cast<const uint16_t *>(w) + r * K - s, format, (N - r + n - 1) / n, K + s, n * K, box_rows, BK);
    }
};

// Rows of a class of N, whole tiles of them.
long long head_class_rows(long long N, int classes) { return up(ceil_div(N, classes), 256); }

template <uint32_t FORMAT, bool CLASSES>
cudaError_t launch_lse(const CUtensorMap &ta, const BMaps<CLASSES> &tb, const LseArgs &lse, const Args &a, int clusters, cudaStream_t s) {
    return a.joined > 1 ? launch<FORMAT>(ta, tb, LseEpi<true, CLASSES>{lse}, a, clusters, s)
                        : launch<FORMAT>(ta, tb, LseEpi<false, CLASSES>{lse}, a, clusters, s);
}

template <uint32_t FORMAT>
cudaError_t forward(const HeadProblem &p, int dev, int *status, cudaStream_t s) {
    const bool aligned = p.K % 8 == 0;
    const int rows_max = 16384;
    const int rows = std::min(p.M, rows_max);
    const bool off_w = !aligned || !on16(p.W);
    const Classes cl(p.W, p.K);
    const bool classes = cl.pay(rows, p.N) && 2LL * cl.n * rows * up(p.K + 7LL, 64) <= kPiece;
    const bool pad_w = off_w && !classes, pad_x = classes || !aligned || !on16(p.X);
    const long long kp = classes ? up(p.K + 7LL, 64) : aligned ? p.K : up(p.K, 64);
    const long long vp = pad_w ? std::min<long long>(up(p.N, 256), std::max<long long>(kPiece / (2 * kp) / 256 * 256, 256)) : p.N;
    const int vn = (int)std::min<long long>(vp, p.N), num_kb = (int)ceil_div(kp, BK);
    const LogitPlan pl = classes ? logit_plan<FORMAT, LseEpi, true>(rows, vn, num_kb, cl.n, dev)
                                 : logit_plan<FORMAT, LseEpi, false>(rows, vn, num_kb, 1, dev);
    if (!pl.bn) return cudaErrorNotSupported;
    const int bn = pl.bn, class_tiles = (int)ceil_div(ceil_div(vn, classes ? cl.n : 1), bn),
              piece_slots = class_tiles * (classes ? cl.n : 1) * pl.ranges();
    const long long last = (p.N - 1) / vp;  // piece
    const int slots = classes ? piece_slots : (int)(last * piece_slots + ceil_div(p.N - last * vp, bn) * pl.ranges());
    Layout l;
    const size_t at_x = l.add(pad_x ? (size_t)(classes ? cl.n : 1) * rows * kp * 2 : 0),
                 at_w = l.add(pad_w ? (size_t)vp * kp * 2 : 0), at_part = l.add((size_t)slots * rows * 8),
                 at_zt = l.add((size_t)rows * 4);
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(&ws, l.bytes, s);
    if (e != cudaSuccess) return e;
    uint8_t *base = static_cast<uint8_t *>(ws);
    for (long long r0 = 0; r0 < p.M && e == cudaSuccess; r0 += rows) {
        const int m = (int)std::min<long long>(rows, p.M - r0);
        const uint16_t *x = static_cast<const uint16_t *>(p.X) + r0 * p.K;
        if (pad_x) {
            e = copy(x, m, p.K, base + at_x, kp, nullptr, 1, {}, s, classes ? cl.n : 1, classes ? cl.shifts : 0);
            x = reinterpret_cast<const uint16_t *>(base + at_x);
        }
        LseArgs lse = {reinterpret_cast<float2 *>(base + at_part), reinterpret_cast<float *>(base + at_zt), p.target + r0, m, 0, 0, p.N, 0, cl.n};
        const int box = left_rows(m, pl.rows);
        for (long long v0 = 0; v0 < p.N && e == cudaSuccess; v0 += vp) {
            const int n = (int)std::min<long long>(vp, p.N - v0);
            const uint16_t *w = static_cast<const uint16_t *>(p.W) + v0 * p.K;
            if (pad_w) {
                e = copy(w, n, p.K, base + at_w, kp, nullptr, 1, {}, s);
                if (e != cudaSuccess) break;
                w = reinterpret_cast<const uint16_t *>(base + at_w);
            }
            lse.N = n;
            lse.v0 = (int)v0;
            lse.slot0 = (int)(v0 / vp) * piece_slots;
            const int n_tiles = classes ? class_tiles * cl.n : (int)ceil_div(n, bn);
            const long long tiles = ceil_div(m, 256) * n_tiles;
            const Args a = {m, classes ? n_tiles * bn : n, num_kb, bn, 0, 0, (int)tiles, 1, pl.joined, box, BK, pl.rows, class_tiles, 0,
                            cl.shifts, 0, status};
            CUtensorMap ta;
            bool ok = tiles <= 0x7FFFFFFFLL;
            if (classes) {
                BMaps<true> tb = {};
                ok = ok && make_map3(&ta, x, map_type(FORMAT), kp, m, cl.n, kp * 2, m * kp * 2, BK, box, 1, 128);
                for (int r = 0; r < cl.n; ++r) ok = ok && cl.map(&tb.m[r], w, FORMAT, n, p.K, r, bn / 2);
                e = ok ? launch_lse<FORMAT, true>(ta, tb, lse, a, pl.clusters, s) : cudaErrorInvalidValue;
            } else {
                BMaps<false> tb;
                ok = ok && map_operand(&ta, x, FORMAT, false, m, kp, kp, box) && map_operand(&tb.m[0], w, FORMAT, false, n, kp, kp, bn / 2);
                e = ok ? launch_lse<FORMAT, false>(ta, tb, lse, a, pl.clusters, s) : cudaErrorInvalidValue;
            }
        }
        if (e != cudaSuccess) break;
        cudaLaunchAttribute attr[1];
        const bool few = m <= 128;  // (one to an SM)
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(few ? m : ceil_div(m, 8))), dim3(1024), 0, s, attr);
        e = launch_counted(&cfg, few ? head_join_kernel<1> : head_join_kernel<8>, static_cast<const float2 *>(lse.part), static_cast<const float *>(lse.zt),
                           lse.target, p.loss + r0, p.lse ? p.lse + r0 : nullptr, slots, m, p.N);
    }
    const cudaError_t f = cudaFreeAsync(ws, s);
    return e != cudaSuccess ? e : f;
}

// K ranges of dX's tiles over a piece: as many as end first, a block of 64 in 0.3 us,
// writing a tile about 2 us, a slab's share of the last kernel.
int dx_splits(long long tiles, long long num_kb, int cmax, double slab_us) {
    int best = 1;
    double least = 0.0;
    for (int n = 1; n <= 16 && num_kb / n >= 8; ++n) {
        const double t = (double)ceil_div(tiles * n, cmax) * ((double)ceil_div(num_kb, n) * 0.3 + 2.0) + n * slab_us;
        if (n == 1 || t < least) { best = n; least = t; }
    }
    return best;
}

template <uint32_t FORMAT, bool CLASSES>
cudaError_t launch_dz(const CUtensorMap &ta, const BMaps<CLASSES> &tb, const DzArgs &dz, const Args &a, int clusters, cudaStream_t s) {
    if (a.joined > 1) {
        DzEpi<true, CLASSES> epi;
        static_cast<DzArgs &>(epi) = dz;
        return launch<FORMAT>(ta, tb, epi, a, clusters, s);
    }
    DzEpi<false, CLASSES> epi;
    static_cast<DzArgs &>(epi) = dz;
    return launch<FORMAT>(ta, tb, epi, a, clusters, s);
}

// CLASSES: of the vocabulary's rows (Classes), all in one piece; dZ a matrix [M, class_rows]
// to a class, side by side.
template <typename T, uint32_t FORMAT, bool CLASSES>
cudaError_t backward(const HeadBackward &p, const Classes &cl, int dev, int *status, cudaStream_t s) {
    const int cx = clusters_max<FORMAT, AccEpi<CLASSES>>(dev),
              cw = CLASSES ? clusters_max<FORMAT, TurnEpi>(dev) : clusters_max<FORMAT, OutEpi>(dev);
    if (cx <= 0 || cw <= 0) return cudaErrorNotSupported;
    const int G = CLASSES ? cl.n : 1, front = CLASSES ? 7 : 0;  // elements in front of a row, at most
    const bool aligned = p.K % 8 == 0;
    const long long kp = aligned ? p.K : up(p.K + front, 64);
    // X: rows without a target are zeros in dW's product, whatever they hold (0 times an
    // infinity is a NaN).  Of classes a copy with each front, and for dW one turned for each
    const bool copy_x = p.dW || !aligned || !on16(p.X), pad_w = !CLASSES && (!aligned || !on16(p.W));
    const int copies = CLASSES && p.dW ? 2 * G : G;
    unsigned long long turns = 0;
    if (CLASSES) {
        const Classes out(p.dW, p.K);
        for (int r = 0; r < G; ++r) turns |= (unsigned long long)(-out.shift(r) & 7) << (4 * r);
    }
    long long vp;
    if (CLASSES) {
        vp = head_class_rows(p.N, G) * G;
    } else {
        vp = std::max<long long>(kPiece / (2LL * p.M) / 256 * 256, 256);
        if (pad_w) vp = std::min(vp, std::max<long long>(kPiece / (2 * kp) / 256 * 256, 256));
        const long long pieces = ceil_div(p.N, vp);
        vp = up(ceil_div(p.N, pieces), 256);
    }
    // dX
    const long long x_cols = p.K + front, x_tiles = ceil_div(p.M, 256) * ceil_div(x_cols, 256), ldx = up(x_cols + (CLASSES ? 3 : 0), 64);
    const double slab_us = (double)p.M * ldx * 4 * 2 / 5e6;
    int splits = dx_splits(x_tiles * G, vp / G / BK, cx, G * slab_us);  // of a class
    splits = (int)std::max<long long>(1, std::min<long long>(splits, kPiece / ((long long)p.M * ldx * 4 * G)));
    Layout l;
    const size_t at_z = l.add((size_t)p.M * vp * 2), at_x = l.add(copy_x ? (size_t)copies * p.M * kp * 2 : 0),
                 at_w = l.add(pad_w ? (size_t)vp * kp * 2 : 0),
                 at_slab = l.add(p.dX ? (size_t)splits * G * p.M * ldx * 4 : 0), at_scale = l.add(8);
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(&ws, l.bytes, s);
    if (e != cudaSuccess) return e;
    uint8_t *base = static_cast<uint8_t *>(ws);
    cudaLaunchAttribute attr[1];
    const bool bf16 = FORMAT == 1;
    ScaleArgs find = {p.dloss, p.target, reinterpret_cast<float2 *>(base + at_scale), bf16 ? 1.0f : 16384.0f, p.M, p.N};
    const float2 *const scale = find.scale;
    // X's copy finds the scale of few rows (1100 x 5000 x 512 39.2 us, in a launch of its own
    // 41.0; 2000 x 5000 x 512 50.2 and 49.7)
    if (!copy_x || p.M > 1536) {
        const cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(1024), 0, s, attr);
        e = launch_counted(&cfg, head_scale_kernel, find);
        find = {};
    }
    const uint16_t *x = static_cast<const uint16_t *>(p.X);
    if (e == cudaSuccess && copy_x) {
        e = copy(p.X, p.M, p.K, base + at_x, kp, p.dW ? p.target : nullptr, p.dW ? p.N : 1, find, s, copies, CLASSES ? cl.shifts : 0, p.dW ? turns << (4 * G) : 0);
        x = reinterpret_cast<const uint16_t *>(base + at_x);
    }
    for (long long v0 = 0; v0 < p.N && e == cudaSuccess; v0 += vp) {
        const int n = (int)std::min<long long>(vp, p.N - v0), cn = (int)ceil_div(n, G);  // of the (largest) class
        const uint16_t *w = static_cast<const uint16_t *>(p.W) + v0 * p.K;
        if (pad_w) {
            e = copy(w, n, p.K, base + at_w, kp, nullptr, 1, {}, s);
            if (e != cudaSuccess) break;
            w = reinterpret_cast<const uint16_t *>(base + at_w);
        }
        const uint8_t *z = base + at_z;
        const int num_kb = (int)ceil_div(kp, BK);
        const LogitPlan pl = logit_plan<FORMAT, DzEpi, CLASSES>(p.M, n, num_kb, G, dev);
        // dZ's columns as rows of dW: all that there are, of classes the gaps behind them too
        const int z_rows = CLASSES ? (int)vp : n;
        const long long w_tiles = ceil_div(z_rows, 256) * ceil_div(p.K, 256);
        if (!pl.bn || w_tiles > 0x7FFFFFFFLL || x_tiles * splits * G > 0x7FFFFFFFLL) {
            e = cudaErrorInvalidValue;
            break;
        }
        CUtensorMap ta;
        BMaps<CLASSES> tb = {};
        // dZ in boxes of rows x 64
        auto map_z = [&](CUtensorMap *m, int rows) {
            return make_map3(m, z, map_type(FORMAT), cn, p.M, G, vp * 2, CLASSES ? vp / G * 2 : p.M * vp * 2, 64, rows, 1, 128);
        };
        {
            DzArgs epi;
            const int box = left_rows(p.M, pl.rows), class_tiles = (int)ceil_div(cn, pl.bn);
            bool ok = make_map3(&ta, x, map_type(FORMAT), kp, p.M, G, kp * 2, p.M * kp * 2, BK, box, 1, 128) && map_z(&epi.tm, 32);
            for (int r = 0; r < G && ok; ++r)
                ok = CLASSES ? cl.map(&tb.m[r], w, FORMAT, n, p.K, r, pl.bn / 2)
                             : map_operand(&tb.m[0], w, FORMAT, false, n, kp, kp, pl.bn / 2);
            if (!ok) {
                e = cudaErrorInvalidValue;
                break;
            }
            epi.lse = p.lse;
            epi.dloss = p.dloss;
            epi.target = p.target;
            epi.scale = scale;
            epi.M = p.M;
            epi.N = cn;
            epi.v0 = (int)v0;
            epi.total = p.N;
            epi.classes = G;
            epi.bf16 = bf16;
            const Args a = {p.M, CLASSES ? class_tiles * G * pl.bn : n, num_kb, pl.bn, 0, 0, (int)pl.tiles, 1, pl.joined, box, BK, pl.rows,
                            class_tiles, 0, cl.shifts, 0, status};
            e = launch_dz<FORMAT, CLASSES>(ta, tb, epi, a, pl.clusters, s);
        }
        if (e == cudaSuccess && p.dW) {
            CUtensorMap tx;
            uint16_t *out = static_cast<uint16_t *>(p.dW) + v0 * p.K;
            const int k_rows = p.M <= 48 ? (p.M + 15) / 16 * 16 : BK, class_rows = (int)(vp / G);
            const Args a = {z_rows, p.K, (int)ceil_div(p.M, BK), 256, 1, 1, (int)w_tiles, 1, 1, 128, k_rows, 256, 0, 0, 0,
                            CLASSES ? class_rows : 0, status};
            bool ok = map_operand(&ta, z, FORMAT, true, z_rows, p.M, vp, 0, k_rows) &&
                      make_map3(&tx, x + (CLASSES ? G * (long long)p.M * kp : 0), map_type(FORMAT), kp, p.M, G, kp * 2, p.M * kp * 2, 64,
                                k_rows, 1, 128);
            if constexpr (CLASSES) {
                TurnEpi epi;
                epi.tm = {};
                for (int r = 0; r < G && ok; ++r) {
                    const int u = (int)(turns >> (4 * r) & 7);
                    ok = map16(&epi.tm.m[r], out + (long long)r * p.K + u, FORMAT, (n - r + G - 1) / G, (p.K - u) / 8 * 8, (long long)G * p.K, 32, 64);
                }
                epi.scale = scale;
                epi.out = out;
                epi.classes = G;
                epi.class_rows = class_rows;
                epi.turns = (uint32_t)turns;
                epi.M = n;
                epi.N = p.K;
                epi.bf16 = bf16;
                e = ok ? launch<FORMAT>(ta, tx, epi, a, cw, s) : cudaErrorInvalidValue;
            } else {
                OutEpi epi;
                const bool tma = aligned && on16(p.dW);
                ok = ok && map16(&epi.tm, tma ? (const void *)out : z, FORMAT, n, tma ? p.K : 64, tma ? p.K : 64, 32, 64);
                epi.scale = scale;
                epi.out = tma ? nullptr : out;
                epi.ld = p.K;
                epi.M = n;
                epi.N = p.K;
                epi.bf16 = bf16;
                e = ok ? launch<FORMAT>(ta, tx, epi, a, cw, s) : cudaErrorInvalidValue;
            }
        }
        if (e == cudaSuccess && p.dX) {
            AccEpi<CLASSES> epi;
            const int box = left_rows(p.M, tile_rows(p.M));
            bool ok = map_z(&ta, box) && make_map3(&epi.tm, base + at_slab, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, x_cols, p.M, splits * G,
                                                   ldx * 4, p.M * ldx * 4, 32, 32, 1, 128);
            for (int r = 0; r < G && ok; ++r)
                ok = CLASSES ? cl.map(&tb.m[r], w, FORMAT, n, p.K, r, BK) : map_operand(&tb.m[0], w, FORMAT, true, kp, n, kp, 0);
            if (!ok) {
                e = cudaErrorInvalidValue;
                break;
            }
            epi.N = (int)x_cols;
            epi.add = v0 > 0;
            // (a short last piece: fewer ranges, each of one block at least)
            const int kb = (int)ceil_div(cn, BK), ranges = std::min(splits, kb);
            const Args a = {p.M, (int)x_cols, kb, 256, 0, 1, (int)x_tiles, ranges * G, 1, box, BK, tile_rows(p.M), 0, CLASSES ? ranges : 0,
                            cl.shifts, 0, status};
            e = launch<FORMAT>(ta, tb, epi, a, cx, s);
        }
    }
    if (e == cudaSuccess && p.dX) {
        const long long blocks = ceil_div((long long)p.M * ((p.K + 3) / 4), 256);
        const int used = (int)std::min<long long>(splits, ceil_div(ceil_div(std::min<long long>(vp, p.N), G), BK));
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(256), 0, s, attr);
        e = blocks > 0x7FFFFFFFLL ? cudaErrorInvalidValue
                                  : launch_counted(&cfg, head_finish_kernel<T>, reinterpret_cast<const float *>(base + at_slab),
                                                   used * G, (long long)p.M, p.K, ldx, CLASSES ? used : 0, cl.shifts, scale,
                                                   static_cast<T *>(p.dX));
    }
    const cudaError_t f = cudaFreeAsync(ws, s);
    return e != cudaSuccess ? e : f;
}
template <typename T, uint32_t FORMAT>
cudaError_t backward(const HeadBackward &p, int dev, int *status, cudaStream_t s) {
    const Classes cl(p.W, p.K);
    const long long z = 2LL * p.M * head_class_rows(p.N, cl.n) * cl.n, slabs = 4LL * cl.n * p.M * up(p.K + 10LL, 64);
    // a slab of dX for each class: for fewer rows yet, and a W of 4 MB or more (22 x 60179 x 951
    // 101 us against 151, 1 x 32000 x 4095 180 against 293, 300 x 40000 x 1500 152 against 193;
    // 300 x 12000 x 2001 98 both ways, 1000 x 50000 x 2001 480 against 447, 30 x 3000 x 701 32
    // against 29)
    const bool classes = cl.pay(8LL * p.M, p.N) && p.K >= 64 && (long long)p.N * p.K >= 2 << 20;
    return classes && z <= kPiece && slabs <= kPiece ? backward<T, FORMAT, true>(p, cl, dev, status, s)
                                                     : backward<T, FORMAT, false>(p, cl, dev, status, s);
}

cudaError_t device(int *dev) {
    const cudaError_t e = cudaGetDevice(dev);
    return e != cudaSuccess ? e : *dev < 0 || *dev >= kMaxDevices ? cudaErrorInvalidDevice : cudaSuccess;
}

}  // namespace

cudaError_t launch_cross_entropy(const HeadProblem &p, int *status, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = device(&dev);
    if (e != cudaSuccess) return e;
    return p.elt == Elt::BF16 ? forward<1>(p, dev, status, s) : forward<0>(p, dev, status, s);
}

cudaError_t launch_cross_entropy_backward(const HeadBackward &p, int *status, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = device(&dev);
    if (e != cudaSuccess) return e;
    return p.elt == Elt::BF16 ? backward<__nv_bfloat16, 1>(p, dev, status, s) : backward<__half, 0>(p, dev, status, s);
}

cudaError_t launch_cross_entropy_flat(const HeadProblem &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)ceil_div(p.M, 256)), dim3(256), 0, s, attr);
    return launch_counted(&cfg, head_flat_kernel, p.target, p.loss, p.lse, p.M, p.N);
}

}  // namespace gemm_gb300
