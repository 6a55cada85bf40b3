// Root-mean-square norm with the residual's addition, and its gradients.
//     H = X + R,  rstd = 1 / sqrt(mean(H^2) + eps),  Y = w H rstd
// (16 bits, or E4M3 with a scale a row), and, with g = w dY,
//     dX = rstd g - H rstd^3 mean(g H) + dH,  dw = sum over rows of dY H rstd
//
// Bound: memory, every operand once.  A row stays in the registers of one to sixteen
// warps between its sums and its result: pieces of eight elements (16 bytes), NV to
// a lane.  The E4M3 form needs one reduction too: |Y| = |w H| rstd rises with |w H|,
// so the largest |w H| is found with the sum of squares.
//
// Pieces lie on 16 bytes of memory.  Where K is no multiple of 8 a row starts inside a
// piece, `off` elements behind its start; whole pieces are still loaded and stored as
// such (every operand's row lies alike, if the bases do), the row's two ends by the
// element.  An operand whose base lies otherwise is read and written by the element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "norm.h"

namespace gemm_gb300 {
namespace {

constexpr int NV = 4;                 // pieces a lane
constexpr int WARP_ELEMS = NV * 256;  // elements of a row a warp holds
constexpr int MAX_WPR = 16;

__device__ __forceinline__ float2 to_f2(uint32_t v, const __nv_bfloat16 *) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 to_f2(uint32_t v, const __half *) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }
__device__ __forceinline__ uint32_t to_u32(float2 v, const __nv_bfloat16 *) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t to_u32(float2 v, const __half *) {
    __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = to_f2(w[j], (const T *)nullptr);
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = to_u32(make_float2(f[2 * j], f[2 * j + 1]), (const T *)nullptr);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements k .. k + 7 of a row of K, 0 outside it.  ODD: some may lie outside, or the
// row is not `wide` (its pieces off 16 bytes); else all lie inside or none.
template <bool ODD>
__device__ __forceinline__ uint4 load8(const uint16_t *row, long long k, int K, bool wide) {
    if (!ODD) return k < K ? *reinterpret_cast<const uint4 *>(row + k) : make_uint4(0u, 0u, 0u, 0u);
    if (wide && k >= 0 && k + 8 <= K) return *reinterpret_cast<const uint4 *>(row + k);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) w[j >> 1] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool ODD>
__device__ __forceinline__ void store8(uint16_t *row, long long k, int K, bool wide, const uint4 &v) {
    if (!ODD) {
        if (k < K) *reinterpret_cast<uint4 *>(row + k) = v;
        return;
    }
    if (wide && k >= 0 && k + 8 <= K) {
        *reinterpret_cast<uint4 *>(row + k) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) row[k + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}
// Eight E4M3 codes of v scale, clamped at +-448; a NaN gives the NaN code.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2 * j] * inv, v[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
template <bool ODD>
__device__ __forceinline__ void store8_codes(uint8_t *row, long long k, int K, bool wide, const uint2 &v) {
    if (!ODD) {
        if (k < K) *reinterpret_cast<uint2 *>(row + k) = v;
        return;
    }
    if (wide && k >= 0 && k + 8 <= K) {
        *reinterpret_cast<uint2 *>(row + k) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) row[k + j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
}
__host__ __device__ __forceinline__ bool on(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Sum and maximum over the WPR warps of a row; every thread of the CTA calls it.
// `red`: two floats a warp, free on entry and again once every warp has passed the
// next barrier of the CTA (`flip` alternates between two sets).
template <int WPR>
__device__ __forceinline__ void reduce_row(float &sum, float &top, float2 *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if constexpr (WPR > 1) {
        const int warp = threadIdx.x >> 5, first = warp / WPR * WPR;
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(sum, top);
        __syncthreads();
        float2 v = red[first];
        sum = v.x;
        top = v.y;
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
            v = red[first + w];
            sum += v.x;
            top = fmaxf(top, v.y);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 add8(const uint4 &a, const uint4 &b) {
    float x[8], y[8];
    unpack8<T>(a, x);
    unpack8<T>(b, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += y[j];
    return pack8<T>(x);
}
// The gains of elements k .. k + 7 (w null: ones).
template <typename T, bool ODD>
__device__ __forceinline__ void weight8(const uint16_t *w, long long k, int K, bool wide, float (&f)[8]) {
    if (w) {
        unpack8<T>(load8<ODD>(w, k, K, wide), f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.0f;
    }
}

struct FwdArgs {
    const uint16_t *X, *R, *w;
    uint16_t *H, *Y;
    uint8_t *Q;
    float *scale, *rstd;
    float eps;
    int M, K;
};
__host__ __device__ constexpr int row_warps(int wpr) { return wpr < 4 ? 4 : wpr; }

// Squares of bf16 overflow from 2^64 on: a row whose sum does is summed again of values
// taken down by 2^70 (half's squares stay within FP32).
constexpr float kDown = 8.470329472543003e-22f;  // 2^-70
template <typename T>
constexpr bool kMayOverflow = std::is_same<T, __nv_bfloat16>::value;
// 1 / sqrt(mean + eps) of values times `by`
__device__ __forceinline__ float rstd_of(float sum, int K, float eps, float by) {
    return 1.0f / sqrtf(sum / (float)K + eps * by * by);
}

// Rows held in registers, WPR warps to a row, four warps at least to a CTA.
template <typename T, int WPR, bool ODD, bool E4M3>
__global__ void __launch_bounds__(row_warps(WPR) * 32)
rms_norm_kernel(const FwdArgs a)
{
    __shared__ float2 red[2][row_warps(WPR)];
    pdl_wait();  // dependents launch as this grid's CTAs exit (several CTAs per SM: no early trigger)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = a.K;
    constexpr int ROWS = row_warps(WPR) / WPR;
    const long long row = (long long)blockIdx.x * ROWS + warp / WPR;
    const bool valid = row < a.M, first = valid && lane == 0 && warp % WPR == 0;
    if (WPR == 1 && !valid) return;
    const long long at = valid ? row * K : 0;
    const int n = valid ? K : 0;
    const int off = ODD ? (int)(((uintptr_t)(a.X + at) & 15) >> 1) : 0;
    const long long k0 = (long long)(warp % WPR * 32 + lane) * 8 - off;
    constexpr long long STEP = WPR * 256;

    uint4 h[NV];
    const bool wx = on(a.X + at - off, 16), wr = on(a.R + at - off, 16), ww = on(a.w - off, 16);
#pragma unroll
    for (int i = 0; i < NV; ++i) h[i] = load8<ODD>(a.X + at, k0 + i * STEP, n, wx);
    if (a.R) {
        uint4 r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i] = load8<ODD>(a.R + at, k0 + i * STEP, n, wr);
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = add8<T>(h[i], r[i]);
        if (a.H) {
            const bool wh = on(a.H + at - off, 16);
#pragma unroll
            for (int i = 0; i < NV; ++i) store8<ODD>(a.H + at, k0 + i * STEP, n, wh, h[i]);
        }
    }
    float by = 1.0f, sum, top;
    auto sums = [&] {
        sum = top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8], g[8];
            unpack8<T>(h[i], f);
            if (E4M3) weight8<T, ODD>(a.w, k0 + i * STEP, n, ww, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = f[j] * by;
                sum = fmaf(v, v, sum);
                if (E4M3) top = fmaxf(top, fabsf(v * g[j]));
            }
        }
    };
    sums();
    reduce_row<WPR>(sum, top, red[0]);
    if (kMayOverflow<T>) {
        const bool over = sum == INFINITY;
        if (over) by = kDown;
        if (WPR > 1 ? __syncthreads_or(over) : over) {
            sums();
            reduce_row<WPR>(sum, top, red[1]);
        }
    }
    const float r = rstd_of(sum, K, a.eps, by);
    if (first && a.rstd) a.rstd[row] = r * by;
    float inv = 0.0f;
    if (E4M3) {
        const float amax = isfinite(sum) ? top * r : NAN;
        inv = amax == 0.0f ? 0.0f : 448.0f / amax;
        if (first) a.scale[row] = amax / 448.0f;
    }
    const bool wy = E4M3 ? on(a.Q + at - off, 8) : on(a.Y + at - off, 16);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8], g[8];
        unpack8<T>(h[i], f);
        weight8<T, ODD>(a.w, k0 + i * STEP, n, ww, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * by * r * g[j];
        if (E4M3) store8_codes<ODD>(a.Q + at, k0 + i * STEP, n, wy, codes8(f, inv));
        else store8<ODD>(a.Y + at, k0 + i * STEP, n, wy, pack8<T>(f));
    }
}

// Longer rows: a CTA to a row, which is read twice (three times where its squares
// overflow), the second time mostly from L2.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(MAX_WPR * 32)
rms_norm_long_kernel(const FwdArgs a)
{
    __shared__ float2 red[2][MAX_WPR];
    pdl_wait();
    const long long row = blockIdx.x;
    const int K = a.K;
    const long long at = row * K;
    const int off = (int)(((uintptr_t)(a.X + at) & 15) >> 1);
    const long long k0 = (long long)threadIdx.x * 8 - off;
    constexpr long long STEP = MAX_WPR * 256;
    const bool wx = on(a.X + at - off, 16), wr = on(a.R + at - off, 16), ww = on(a.w - off, 16), wh = on(a.H + at - off, 16);
    auto value = [&](long long k) {
        const uint4 x = load8<true>(a.X + at, k, K, wx);
        return a.R ? add8<T>(x, load8<true>(a.R + at, k, K, wr)) : x;
    };
    float by = 1.0f, sum, top;
    auto sums = [&] {
        sum = top = 0.0f;
        for (long long k = k0; k < K; k += STEP) {
            float f[8], g[8];
            unpack8<T>(value(k), f);
            if (E4M3) weight8<T, true>(a.w, k, K, ww, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = f[j] * by;
                sum = fmaf(v, v, sum);
                if (E4M3) top = fmaxf(top, fabsf(v * g[j]));
            }
        }
    };
    sums();
    reduce_row<MAX_WPR>(sum, top, red[0]);
    if (kMayOverflow<T> && sum == INFINITY) {  // the same in every thread
        by = kDown;
        sums();
        reduce_row<MAX_WPR>(sum, top, red[1]);
    }
    const float r = rstd_of(sum, K, a.eps, by);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r * by;
    float inv = 0.0f;
    if (E4M3) {
        const float amax = isfinite(sum) ? top * r : NAN;
        inv = amax == 0.0f ? 0.0f : 448.0f / amax;
        if (threadIdx.x == 0) a.scale[row] = amax / 448.0f;
    }
    const bool wy = E4M3 ? on(a.Q + at - off, 8) : on(a.Y + at - off, 16);
    for (long long k = k0; k < K; k += STEP) {
        const uint4 h = value(k);
        if (a.H) store8<true>(a.H + at, k, K, wh, h);
        float f[8], g[8];
        unpack8<T>(h, f);
        weight8<T, true>(a.w, k, K, ww, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * by * r * g[j];
        if (E4M3) store8_codes<true>(a.Q + at, k, K, wy, codes8(f, inv));
        else store8<true>(a.Y + at, k, K, wy, pack8<T>(f));
    }
}

struct BwdArgs {
    const uint16_t *H, *w;
    const float *rstd;
    const uint16_t *dY, *dH;
    uint16_t *dX;
    float *part;  // dw of each CTA's rows [CTA][K], or null
    int M, K;
};

// CTAs walk over the rows; dw's sums stay with them, in registers (every row of a
// thread has the same columns) or, ODD, in shared memory, element k of a group of
// warps at (k % 8) WPR 128 + k / 8 (a warp's threads on different banks).
template <typename T, int WPR, bool ODD>
__global__ void __launch_bounds__(row_warps(WPR) * 32)
rms_norm_backward_kernel(const BwdArgs a)
{
    extern __shared__ float acc_s[];
    constexpr int WARPS = row_warps(WPR), ROWS = WARPS / WPR, PLANE = WPR * 128;
    __shared__ float2 red[2][WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = a.K, group = warp / WPR;
    constexpr long long STEP = WPR * 256;
    float *mine = acc_s + group * 8 * PLANE;
    if (ODD && a.part) {
        for (int i = threadIdx.x; i < ROWS * 8 * PLANE; i += WARPS * 32) acc_s[i] = 0.0f;
        __syncthreads();
    }
    pdl_wait();
    float acc[ODD ? 1 : NV][8] = {};
    int flip = 0;
    for (long long row0 = (long long)blockIdx.x * ROWS; row0 < a.M; row0 += (long long)gridDim.x * ROWS, flip ^= 1) {
        const long long row = row0 + group;
        const bool valid = row < a.M;
        const long long at = valid ? row * K : 0;
        const int n = valid ? K : 0;
        const int off = ODD ? (int)(((uintptr_t)(a.H + at) & 15) >> 1) : 0;
        const long long k0 = (long long)(warp % WPR * 32 + lane) * 8 - off;
        const bool wh = on(a.H + at - off, 16), wy = on(a.dY + at - off, 16), wd = on(a.dH + at - off, 16),
                   wx = on(a.dX + at - off, 16), ww = on(a.w - off, 16);
        uint4 h[NV], dy[NV], dh[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = load8<ODD>(a.H + at, k0 + i * STEP, n, wh);
#pragma unroll
        for (int i = 0; i < NV; ++i) dy[i] = load8<ODD>(a.dY + at, k0 + i * STEP, n, wy);
        if (a.dH && a.dX) {
#pragma unroll
            for (int i = 0; i < NV; ++i) dh[i] = load8<ODD>(a.dH + at, k0 + i * STEP, n, wd);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) dh[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        const float r = valid ? a.rstd[row] : 0.0f;
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8], d[8], g[8];
            unpack8<T>(h[i], f);
            unpack8<T>(dy[i], d);
            weight8<T, ODD>(a.w, k0 + i * STEP, n, ww, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xhat = f[j] * r, k = d[j] * xhat;
                sum = fmaf(k, g[j], sum);
                if constexpr (ODD) {
                    const long long at_k = k0 + i * STEP + j;
                    if (a.part && at_k >= 0 && at_k < n) mine[(int)(at_k & 7) * PLANE + (int)(at_k >> 3)] += k;
                } else {
                    acc[i][j] += k;
                }
            }
        }
        reduce_row<WPR>(sum, top, red[flip]);
        const float mean = sum / (float)K;
        if (a.dX) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8], d[8], g[8], e[8];
                unpack8<T>(h[i], f);
                unpack8<T>(dy[i], d);
                unpack8<T>(dh[i], e);
                weight8<T, ODD>(a.w, k0 + i * STEP, n, ww, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-f[j] * r, mean, d[j] * g[j]), e[j]);
                store8<ODD>(a.dX + at, k0 + i * STEP, n, wx, pack8<T>(d));
            }
        }
    }
    if (!a.part) return;
    float *part = a.part + (long long)blockIdx.x * K;
    if constexpr (!ODD && ROWS == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const long long k = (long long)(warp * 32 + lane) * 8 + i * STEP;
            if (k < K) {
                *reinterpret_cast<float4 *>(part + k) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                *reinterpret_cast<float4 *>(part + k + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
    } else {
        if constexpr (!ODD) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) mine[j * PLANE + (warp % WPR * 32 + lane) + i * WPR * 32] = acc[i][j];
        }
        __syncthreads();
        for (int k = threadIdx.x; k < K; k += WARPS * 32) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < ROWS; ++g) s += acc_s[g * 8 * PLANE + (k & 7) * PLANE + (k >> 3)];
            part[k] = s;
        }
    }
}

// dX of longer rows, a CTA to a row.
template <typename T>
__global__ void __launch_bounds__(MAX_WPR * 32)
rms_norm_long_dx_kernel(const BwdArgs a)
{
    __shared__ float2 red[MAX_WPR];
    pdl_wait();
    const long long row = blockIdx.x;
    const int K = a.K;
    const long long at = row * K;
    const int off = (int)(((uintptr_t)(a.H + at) & 15) >> 1);
    constexpr long long STEP = MAX_WPR * 256;
    const long long k0 = (long long)threadIdx.x * 8 - off;
    const bool wh = on(a.H + at - off, 16), wy = on(a.dY + at - off, 16), wd = on(a.dH + at - off, 16),
               wx = on(a.dX + at - off, 16), ww = on(a.w - off, 16);
    const float r = a.rstd[row];
    float sum = 0.0f, top = 0.0f;
    for (long long k = k0; k < K; k += STEP) {
        float f[8], d[8], g[8];
        unpack8<T>(load8<true>(a.H + at, k, K, wh), f);
        unpack8<T>(load8<true>(a.dY + at, k, K, wy), d);
        weight8<T, true>(a.w, k, K, ww, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(d[j] * (f[j] * r), g[j], sum);
    }
    reduce_row<MAX_WPR>(sum, top, red);
    const float mean = sum / (float)K;
    for (long long k = k0; k < K; k += STEP) {
        float f[8], d[8], g[8], e[8];
        unpack8<T>(load8<true>(a.H + at, k, K, wh), f);
        unpack8<T>(load8<true>(a.dY + at, k, K, wy), d);
        unpack8<T>(a.dH ? load8<true>(a.dH + at, k, K, wd) : make_uint4(0u, 0u, 0u, 0u), e);
        weight8<T, true>(a.w, k, K, ww, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-f[j] * r, mean, d[j] * g[j]), e[j]);
        store8<true>(a.dX + at, k, K, wx, pack8<T>(d));
    }
}
// Their dw: a thread to a column, block y a range of the rows.
template <typename T>
__global__ void __launch_bounds__(256)
rms_norm_long_dw_kernel(const BwdArgs a)
{
    pdl_wait();
    const long long k = blockIdx.x * 256LL + threadIdx.x;
    if (k >= a.K) return;
    const int lo = (int)((long long)a.M * blockIdx.y / gridDim.y), hi = (int)((long long)a.M * (blockIdx.y + 1) / gridDim.y);
    const T *H = reinterpret_cast<const T *>(a.H), *dY = reinterpret_cast<const T *>(a.dY);
    float s = 0.0f;
#pragma unroll 8
    for (long long row = lo; row < hi; ++row)
        s = fmaf((float)dY[row * a.K + k], (float)H[row * a.K + k] * a.rstd[row], s);
    a.part[blockIdx.y * (long long)a.K + k] = s;
}

// dw[k] = sum over n partials, each warp its share of them in order, then the warps' sums in order.
__global__ void __launch_bounds__(256)
rms_norm_dw_kernel(const float *__restrict__ part, float *__restrict__ dw, int n, int K)
{
    __shared__ float sums[8][32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long k = blockIdx.x * 32LL + lane;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int g = warp; g < n; g += 8) s += __ldcg(part + (long long)g * K + k);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && k < K) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sums[w][lane];
        dw[k] = s;
    }
}

// Warps to a row of K elements (of so many pieces, if its rows start inside one); 0: a long row.
int row_split(int K, bool odd) {
    const long long n = (long long)K + (odd ? 14 : 0);
    for (int w = 1; w <= MAX_WPR; w *= 2)
        if (n <= (long long)w * WARP_ELEMS) return w;
    return 0;
}
bool all_on16(std::initializer_list<const void *> ps, int K) {
    uintptr_t a = 0;
    for (const void *p : ps) a |= (uintptr_t)p;
    return (a & 15) == 0 && K % 8 == 0;
}

template <typename F>
cudaError_t with_split(int wpr, F f) {
    switch (wpr) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return f(std::integral_constant<int, 16>());
    }
}

template <typename T, bool E4M3>
cudaError_t forward(const NormProblem &p, cudaStream_t s) {
    FwdArgs a = {};
    a.X = static_cast<const uint16_t *>(p.X);
    a.R = static_cast<const uint16_t *>(p.R);
    a.w = static_cast<const uint16_t *>(p.w);
    a.H = static_cast<uint16_t *>(p.H);
    a.Y = static_cast<uint16_t *>(p.Y);
    a.Q = static_cast<uint8_t *>(p.Q);
    a.scale = p.scale;
    a.rstd = p.rstd;
    a.eps = p.eps;
    a.M = p.M;
    a.K = p.K;
    const bool odd = !all_on16({p.X, p.R, p.w, p.H, p.Y}, p.K) || !on(p.Q, 8);
    const int wpr = row_split(p.K, odd);
    cudaLaunchAttribute attr[1];
    if (wpr == 0) {
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.M), dim3(MAX_WPR * 32), 0, s, attr);
        return launch_counted(&cfg, rms_norm_long_kernel<T, E4M3>, a);
    }
    return with_split(wpr, [&](auto w) {
        constexpr int W = decltype(w)::value, ROWS = row_warps(W) / W;
        const cudaLaunchConfig_t cfg =
            pdl_config(dim3((unsigned)(((long long)p.M + ROWS - 1) / ROWS)), dim3(row_warps(W) * 32), 0, s, attr);
        return odd ? launch_counted(&cfg, rms_norm_kernel<T, W, true, E4M3>, a)
                   : launch_counted(&cfg, rms_norm_kernel<T, W, false, E4M3>, a);
    });
}

template <typename T, int W, bool ODD>
cudaError_t launch_backward(const BwdArgs &a, unsigned grid, size_t smem, cudaStream_t s) {
    auto kern = rms_norm_backward_kernel<T, W, ODD>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
    }
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(row_warps(W) * 32), smem, s, attr);
    return launch_counted(&cfg, kern, a);
}

template <typename T>
cudaError_t backward(const NormBackward &p, int num_sms, cudaStream_t s) {
    BwdArgs a = {};
    a.H = static_cast<const uint16_t *>(p.H);
    a.w = static_cast<const uint16_t *>(p.w);
    a.rstd = p.rstd;
    a.dY = static_cast<const uint16_t *>(p.dY);
    a.dH = static_cast<const uint16_t *>(p.dH);
    a.dX = static_cast<uint16_t *>(p.dX);
    a.M = p.M;
    a.K = p.K;
    const bool odd = !all_on16({p.H, p.w, p.dY, p.dH, p.dX}, p.K);
    const int wpr = row_split(p.K, odd);
    const int rows = wpr ? row_warps(wpr) / wpr : 1;
    // as many CTAs as stay resident, and partial sums of dw
    const int per_sm = wpr <= 4 ? 4 : wpr == 8 ? 2 : 1;
    const long long ctas = std::min<long long>(((long long)p.M + rows - 1) / rows, (long long)num_sms * per_sm);
    const int n = wpr ? (int)ctas : std::min(p.M, 256);
    void *ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (p.dw) {
        a.part = p.dw;  // a single partial is dw (written 16 bytes at a time)
        if (n > 1 || !on(p.dw, 16)) {
            e = scratch_alloc(&ws, (size_t)n * p.K * 4, s);
            if (e != cudaSuccess) return e;
            a.part = static_cast<float *>(ws);
        }
    }
    cudaLaunchAttribute attr[1];
    if (wpr == 0) {
        if (p.dw) {
            const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((p.K + 255LL) / 256), (unsigned)n), dim3(256), 0, s, attr);
            e = launch_counted(&cfg, rms_norm_long_dw_kernel<T>, a);
        }
        if (e == cudaSuccess && p.dX) {
            const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.M), dim3(MAX_WPR * 32), 0, s, attr);
            e = launch_counted(&cfg, rms_norm_long_dx_kernel<T>, a);
        }
    } else {
        e = with_split(wpr, [&](auto w) {
            constexpr int W = decltype(w)::value;
            const size_t smem = p.dw && (odd || rows > 1) ? (size_t)row_warps(W) * WARP_ELEMS * 4 : 0;
            return odd ? launch_backward<T, W, true>(a, (unsigned)ctas, smem, s)
                       : launch_backward<T, W, false>(a, (unsigned)ctas, smem, s);
        });
    }
    if (e == cudaSuccess && ws) {
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((p.K + 31LL) / 32)), dim3(256), 0, s, attr);
        e = launch_counted(&cfg, rms_norm_dw_kernel, static_cast<const float *>(ws), p.dw, n, p.K);
    }
    const cudaError_t f = ws ? cudaFreeAsync(ws, s) : cudaSuccess;
    return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_rms_norm(const NormProblem &p, cudaStream_t s) {
    if (p.elt == Elt::BF16) return p.Y ? forward<__nv_bfloat16, false>(p, s) : forward<__nv_bfloat16, true>(p, s);
    return p.Y ? forward<__half, false>(p, s) : forward<__half, true>(p, s);
}

cudaError_t launch_rms_norm_backward(const NormBackward &p, int num_sms, cudaStream_t s) {
    return p.elt == Elt::BF16 ? backward<__nv_bfloat16>(p, num_sms, s) : backward<__half>(p, num_sms, s);
}

}  // namespace gemm_gb300
