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
// Pieces lie on 16 bytes of memory.  Where K is no multiple of 8, a row is whole pieces
// between a head and a tail of up to seven elements, which one thread each takes; every
// operand's row lies alike, if the bases do.  (Pieces that reach over the row's ends,
// masked there, took 8192 x 4095 from 42 to 123 us: masks and elements cost more
// instructions than the row.)  Rows longer than 16384, and operands whose bases lie
// otherwise to 16 bytes, are read twice, piece by piece, by the element where need be.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "norm.h"
#include "tc_ptx.cuh"

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

// Bytes of an address behind 16.
__device__ __forceinline__ int behind16(const void *p) { return (int)((uintptr_t)p & 15); }

// Elements k .. k + 7 of a row of K by the element, 0 outside it; the same stored, in 16 or
// 8 bits.  For rows' ends and what lies off 16 bytes; not inlined, so that the code of the
// whole pieces around them stays small (8192 x 4095 with these inlined: 2500 instructions a
// warp, 123 us).
__device__ __noinline__ uint4 elements8(const uint16_t *row, long long k, int K) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) w[j >> 1] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __noinline__ void put8(uint16_t *row, long long k, int K, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) row[k + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}
__device__ __noinline__ void put8_codes(uint8_t *row, long long k, int K, uint2 v) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j >= 0 && k + j < K) row[k + j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
}
// Bytes d .. d + 15 of two pieces, d even and below 16.
__device__ __forceinline__ uint4 shift16(const uint4 &a, const uint4 &b, int d) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t[5];
#pragma unroll
    for (int j = 0; j < 5; ++j)  // d / 4 whole words: 0, 1, 2 or 3
        t[j] = d < 8 ? (d < 4 ? w[j] : w[j + 1]) : (d < 12 ? w[j + 2] : w[j + 3]);
    const uint32_t sh = (d & 2) * 8;
    return make_uint4(__funnelshift_r(t[0], t[1], sh), __funnelshift_r(t[1], t[2], sh), __funnelshift_r(t[2], t[3], sh),
                      __funnelshift_r(t[3], t[4], sh));
}
__device__ __forceinline__ uint4 ld16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
constexpr uint4 kZero = {0u, 0u, 0u, 0u};

// One piece of a row, anywhere.
__device__ __forceinline__ uint4 load8(const uint16_t *row, long long k, int K) {
    const int d = behind16(row + k), e = d >> 1;
    if (d == 0 && k >= 0 && k + 8 <= K) return ld16(row + k);
    if (d != 0 && k >= e && k - e + 16 <= K) return shift16(ld16(row + k - e), ld16(row + k - e + 8), d);
    return elements8(row, k, K);
}
// The same stored; wide: the row's pieces lie on 16 bytes (codes: 8).
__device__ __forceinline__ void store8(uint16_t *row, long long k, int K, bool wide, const uint4 &v) {
    if (wide && k >= 0 && k + 8 <= K) *reinterpret_cast<uint4 *>(row + k) = v;
    else put8(row, k, K, v);
}
__device__ __forceinline__ void store8_codes(uint8_t *row, long long k, int K, bool wide, const uint2 &v) {
    if (wide && k >= 0 && k + 8 <= K) *reinterpret_cast<uint2 *>(row + k) = v;
    else put8_codes(row, k, K, v);
}
// Eight E4M3 codes of v scale, clamped at +-448; a NaN gives the NaN code.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2 * j] * inv, v[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
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
// Eight gains (none: ones).
template <typename T>
__device__ __forceinline__ void gains8(bool some, const uint4 &w, float (&f)[8]) {
    if (some) {
        unpack8<T>(w, f);
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

// A row's scales, from its sum of squares and, for E4M3, the largest |w H|, top: |Y| rises with
// it.  They come from one pass over the row; of bf16, at the ends of its range, from two or
// three, each with H times another power of two:
//   squares overflow from 2^64 on: a row whose sum does is taken down by 2^80, its squares
//     below 2^96, the sum of 2^31 of them below 2^127;
//   a top below 2^-100 (448 / amax overflows from 2^-119 on): up by 2^100, or by 2^60 where
//     elements may be above 1 (below 2^64: the sum is finite);
//   a top past FP32's largest, where Y need not be: by rstd's power of two, H rstd being
//     below sqrt(K).
// (Half's squares, and w H between 2^-48 and 2^32, stay within FP32.)
constexpr float kDown = 0x1p-80f, kLeast = 0x1p-100f;
template <typename T>
constexpr bool kMayOverflow = std::is_same<T, __nv_bfloat16>::value;
template <typename T, bool E4M3>
struct RowScales {
    float by = 1.0f;     // what H is to be multiplied by, all passes' together, and the last one's
    float last = 1.0f;
    float r, rstd;       // 1 / sqrt(mean + eps) of the values summed; of H
    float q, amax;       // E4M3: codes are of H by w q = Y / down, whose largest is amax
    float down = 1.0f;
    bool summed = false;

    // A pass's sums; true: one more is needed.  (Again of a row that needed none: nothing changes.)
    __device__ __forceinline__ bool take(float sum, float top, int K, float eps) {
        last = 1.0f;
        if (!summed) {
            if (kMayOverflow<T> && __builtin_expect(sum == INFINITY && by == 1.0f, 0)) {
                by = last = kDown;
                return true;
            }
            summed = true;
            r = 1.0f / sqrtf(sum / (float)K + eps * by * by);
            rstd = r * by;
            q = isfinite(sum) ? r : NAN;
            if (E4M3 && kMayOverflow<T> && __builtin_expect(isfinite(sum) && !(top >= kLeast && top < INFINITY), 0)) {
                if (top < kLeast) {
                    last = sum < 1.0f ? 0x1p100f : 0x1p60f;
                    down = sum < 1.0f ? 0x1p-100f : 0x1p-60f;
                } else {
                    last = __uint_as_float(__float_as_uint(r) & 0x7F800000u);
                    q = __uint_as_float((__float_as_uint(r) & 0x007FFFFFu) | 0x3F800000u);
                }
                by *= last;
                return true;
            }
        }
        if (E4M3) {
            if (down == 1.0f && top * q < kLeast) {
                down = 0x1p-50f;
                q *= 0x1p50f;
            }
            amax = top * q;
            if (amax * 0x1p50f * down < kLeast) amax = 0.0f;  // Y below 2^-150: 0 in FP32
        }
        return false;
    }
    __device__ __forceinline__ float inverse() const { return amax == 0.0f ? 0.0f : 448.0f / amax; }
    __device__ __forceinline__ float scale() const { return amax / 448.0f * down; }
};

// How a thread of a row's warps takes the row: pieces k0 + i STEP below `body` from element
// `head` on, and, where they are not whole pieces, one element `one` of the head or the tail.
struct Share {
    int head, body, k0, one;  // one: -1 for none
};
template <int WPR, bool ODD>
__device__ __forceinline__ Share share_of(const uint16_t *row, int K) {
    Share s;
    const int t = (int)(threadIdx.x & (WPR * 32 - 1));
    s.k0 = t * 8;
    if (!ODD) {
        s.head = 0;
        s.body = K;
        s.one = -1;
        return s;
    }
    s.head = min((8 - (behind16(row) >> 1)) & 7, K);
    s.body = (K - s.head) & ~7;
    s.one = t < s.head ? t : t < K - s.body ? s.body + t : -1;
    return s;
}
// The gains in shared memory (ODD: pieces start at any element of theirs), w null: ones.
__device__ __forceinline__ int gains_bytes(int K) { return ((K + 15) & ~7) * 2; }
template <typename T>
__device__ __forceinline__ void stage_gains(const uint16_t *w, int K, uint16_t *to) {
    const bool wide = w && behind16(w) == 0;
    const int whole = wide ? K >> 3 : 0;
    for (int i = threadIdx.x; i < whole; i += blockDim.x) reinterpret_cast<uint4 *>(to)[i] = ld16(w + 8 * i);
    const T unit = T(1.0f);
    for (int k = whole * 8 + threadIdx.x; k < ((K + 15) & ~7); k += blockDim.x)
        to[k] = k >= K ? (uint16_t)0 : w ? w[k] : *reinterpret_cast<const uint16_t *>(&unit);
}
// Gains of the piece k of a row with this head.
__device__ __forceinline__ uint4 staged8(const uint16_t *w, int head, int k) {
    return shift16(ld16(w + k), ld16(w + k + 8), head * 2);
}
template <typename T>
__device__ __forceinline__ float value(const uint16_t *p) { return (float)*reinterpret_cast<const T *>(p); }
template <typename T>
__device__ __forceinline__ uint16_t bits(float f) {
    const T t = T(f);
    return *reinterpret_cast<const uint16_t *>(&t);
}

// Rows held in registers, WPR warps to a row, four warps at least to a CTA.  ODD: K is no
// multiple of 8, or the bases lie off 16 bytes, all alike.  CTAs an SM: registers for eight of
// 128 threads, but for odd rows' (E4M3 of 8192 x 4096 39.5 us against 39.8 with seven, of 10000
// x 2047 29.6 against 30.5 with eight).
__host__ __device__ constexpr int fwd_ctas(int wpr, bool odd) { return wpr == 16 ? 2 : wpr == 8 ? 4 : odd ? 7 : 8; }
template <typename T, int WPR, bool ODD, bool E4M3>
__global__ void __launch_bounds__(row_warps(WPR) * 32, fwd_ctas(WPR, ODD))
rms_norm_kernel(const FwdArgs a)
{
    extern __shared__ __align__(16) uint16_t gains_s[];  // ODD
    __shared__ float2 red[3][row_warps(WPR)];
    pdl_wait();  // dependents launch as this grid's CTAs exit (several CTAs per SM: no early trigger)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = a.K;
    constexpr int ROWS = row_warps(WPR) / WPR, STEP = WPR * 256;
    const long long row = (long long)blockIdx.x * ROWS + warp / WPR;
    const bool valid = row < a.M, first = valid && lane == 0 && warp % WPR == 0;
    if (WPR == 1 && !ODD && !valid) return;
    const long long at = valid ? row * K : 0;
    const Share me = share_of<WPR, ODD>(a.X + at, valid ? K : 0);

    uint4 h[NV];
    const long long body = at + me.head;
#pragma unroll
    for (int i = 0; i < NV; ++i) h[i] = me.k0 + i * STEP < me.body ? ld16(a.X + body + me.k0 + i * STEP) : kZero;
    float one = ODD && me.one >= 0 ? value<T>(a.X + at + me.one) : 0.0f;
    if (a.R) {
        uint4 r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i] = me.k0 + i * STEP < me.body ? ld16(a.R + body + me.k0 + i * STEP) : kZero;
        if (ODD && me.one >= 0) one = (float)T(one + value<T>(a.R + at + me.one));
        if (ODD) stage_gains<T>(a.w, K, gains_s);
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = add8<T>(h[i], r[i]);
        if (a.H) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (me.k0 + i * STEP < me.body) *reinterpret_cast<uint4 *>(a.H + body + me.k0 + i * STEP) = h[i];
            if (ODD && me.one >= 0) a.H[at + me.one] = bits<T>(one);
        }
    } else if (ODD) {
        stage_gains<T>(a.w, K, gains_s);
    }
    if (ODD) __syncthreads();
    // the gains of piece i: from shared memory, or from L1
    auto gains = [&](int i, float(&g)[8]) {
        const int k = me.k0 + i * STEP;
        if (ODD) unpack8<T>(k < me.body ? staged8(gains_s, me.head, k) : kZero, g);
        else gains8<T>(a.w != nullptr, a.w && k < me.body ? ld16(a.w + k) : kZero, g);
    };
    const float one_gain = ODD && me.one >= 0 ? value<T>(gains_s + me.one) : 0.0f;
    auto sums = [&](float by, float &sum, float &top) {
        sum = ODD ? (one * by) * (one * by) : 0.0f;
        top = ODD && E4M3 ? fabsf(one * one_gain) : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8], g[8];
            unpack8<T>(h[i], f);
            if (E4M3) gains(i, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = f[j] * by;
                sum = fmaf(v, v, sum);
                if (E4M3) top = fmaxf(top, fabsf(f[j] * g[j]));
            }
        }
    };
    RowScales<T, E4M3> c;
    float sum, top;
    sums(1.0f, sum, top);
    reduce_row<WPR>(sum, top, red[0]);
    bool more = c.take(sum, top, K, a.eps);
    if (kMayOverflow<T>) {
#pragma unroll 1
        for (int t = 1; t < (E4M3 ? 3 : 2) && __builtin_expect(WPR > 1 ? __syncthreads_or(more) : more, 0); ++t) {
            if (E4M3) {  // of codes H itself is multiplied (the ordinary row then needs no factor); elements
                         // that leave bf16's range are nothing beside the largest
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float f[8];
                    unpack8<T>(h[i], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= c.last;
                    h[i] = pack8<T>(f);
                }
                one *= c.last;
            }
            sums(E4M3 ? 1.0f : c.by, sum, top);
            reduce_row<WPR>(sum, top, red[t]);
            more = c.take(sum, top, K, a.eps);
        }
    }
    if (first && a.rstd) a.rstd[row] = c.rstd;
    const float inv = E4M3 ? c.inverse() : 0.0f;
    if (E4M3 && first) a.scale[row] = c.scale();
    auto y = [&](float v, float w) { return E4M3 ? v * w * c.q : v * c.by * c.r * w; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (me.k0 + i * STEP >= me.body) break;
        float f[8], g[8];
        unpack8<T>(h[i], f);
        gains(i, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = y(f[j], g[j]);
        if (E4M3) *reinterpret_cast<uint2 *>(a.Q + body + me.k0 + i * STEP) = codes8(f, inv);
        else *reinterpret_cast<uint4 *>(a.Y + body + me.k0 + i * STEP) = pack8<T>(f);
    }
    if (ODD && me.one >= 0) {
        const float v = y(one, one_gain);
        if (E4M3) a.Q[at + me.one] = (uint8_t)__nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
        else a.Y[at + me.one] = bits<T>(v);
    }
}

// Any rows: a CTA to a row, which is read twice (three times where its squares
// overflow), the second time mostly from L2.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(MAX_WPR * 32)
rms_norm_long_kernel(const FwdArgs a)
{
    __shared__ float2 red[3][MAX_WPR];
    pdl_wait();
    const long long row = blockIdx.x;
    const int K = a.K;
    const long long at = row * K;
    const int off = behind16(a.X + at) >> 1;
    const long long k0 = (long long)threadIdx.x * 8 - off;
    constexpr long long STEP = MAX_WPR * 256;
    const bool wh = on(a.H + at - off, 16);
    auto value = [&](long long k) {
        const uint4 x = load8(a.X + at, k, K);
        return a.R ? add8<T>(x, load8(a.R + at, k, K)) : x;
    };
    auto gain = [&](long long k, float(&g)[8]) { gains8<T>(a.w != nullptr, a.w ? load8(a.w, k, K) : kZero, g); };
    auto sums = [&](float by, float &sum, float &top) {
        sum = top = 0.0f;
        for (long long k = k0; k < K; k += STEP) {
            float f[8], g[8];
            unpack8<T>(value(k), f);
            if (E4M3) gain(k, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = f[j] * by;
                sum = fmaf(v, v, sum);
                if (E4M3) top = fmaxf(top, fabsf(v * g[j]));
            }
        }
    };
    RowScales<T, E4M3> c;
    float sum, top;
    sums(1.0f, sum, top);
    reduce_row<MAX_WPR>(sum, top, red[0]);
    bool more = c.take(sum, top, K, a.eps);  // the same in every thread
    if (kMayOverflow<T>) {
#pragma unroll 1
        for (int t = 1; more; ++t) {  // (twice at most)
            sums(c.by, sum, top);
            reduce_row<MAX_WPR>(sum, top, red[t]);
            more = c.take(sum, top, K, a.eps);
        }
    }
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = c.rstd;
    const float inv = E4M3 ? c.inverse() : 0.0f;
    if (E4M3 && threadIdx.x == 0) a.scale[row] = c.scale();
    const bool wy = E4M3 ? on(a.Q + at - off, 8) : on(a.Y + at - off, 16);
    for (long long k = k0; k < K; k += STEP) {
        const uint4 h = value(k);
        if (a.H) store8(a.H + at, k, K, wh, h);
        float f[8], g[8];
        unpack8<T>(h, f);
        gain(k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = E4M3 ? f[j] * c.by * g[j] * c.q : f[j] * c.by * c.r * g[j];
        if (E4M3) store8_codes(a.Q + at, k, K, wy, codes8(f, inv));
        else store8(a.Y + at, k, K, wy, pack8<T>(f));
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

// Rows on 16 bytes: CTAs walk over the rows, ROWS at a time, which come to shared memory
// by bulk copies a few turns ahead (adjacent rows are adjacent in memory), so that enough
// bytes are under way at all times; loads to registers, waited for row by row, reached
// half of the rate (8192 x 4096: 72 us against 39).  dw's sums stay in registers: a thread
// has the same columns of every row.
// After a wait that gave up: no copy is left in flight when the CTA ends.
__device__ __noinline__ void drain_copies(uint64_t *full, int stages, int turns, volatile int *abort) {
    for (int i = max(turns - stages, 0); i < turns; ++i) tc::mbar_wait(&full[i % stages], (uint32_t)((i / stages) & 1), abort, false);
}
constexpr int bulk_ctas(int wpr) { return wpr <= 8 ? 2 : 1; }  // an SM
template <typename T, int WPR>
__global__ void __launch_bounds__(row_warps(WPR) * 32, bulk_ctas(WPR))
rms_norm_backward_bulk_kernel(const BwdArgs a, const int stages, int *status)
{
    constexpr int WARPS = row_warps(WPR), ROWS = WARPS / WPR, MAX_STAGES = 8;
    extern __shared__ __align__(16) uint8_t ring[];  // stage: H, dY and dH, ROWS rows each
    __shared__ uint64_t full[MAX_STAGES];
    __shared__ float2 red[2][WARPS];
    __shared__ int abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = a.K, group = warp / WPR;
    const uint32_t plane = (uint32_t)(ROWS * K * 2), stage_bytes = 3 * plane;
    const bool has_dh = a.dH && a.dX;
    const uint32_t step = gridDim.x * ROWS, row00 = blockIdx.x * ROWS, M = (uint32_t)a.M;  // (M + 8 steps < 2^32)
    if (threadIdx.x == 0) {
        abort = 0;
        for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
        tc::mbar_init_fence();
    }
    __syncthreads();
    pdl_wait();
    auto fetch = [&](uint32_t row0, int stage) {  // one thread
        if (row0 >= M) return;
        const uint32_t bytes = min((uint32_t)ROWS, M - row0) * (uint32_t)(K * 2);
        uint8_t *to = ring + stage * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], bytes * (has_dh ? 3u : 2u));
        tc::bulk_load(to, a.H + (long long)row0 * K, bytes, &full[stage]);
        tc::bulk_load(to + plane, a.dY + (long long)row0 * K, bytes, &full[stage]);
        if (has_dh) tc::bulk_load(to + 2 * plane, a.dH + (long long)row0 * K, bytes, &full[stage]);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < stages; ++i) fetch(row00 + i * step, i);
    constexpr int STEP = WPR * 256;
    const int k0 = (warp % WPR * 32 + lane) * 8;
    constexpr bool KEEP = WPR <= 4;  // the gains, in registers; else from L1
    uint4 w[NV];
    auto gain = [&](int i) { return a.w && k0 + i * STEP < K ? ld16(a.w + k0 + i * STEP) : kZero; };
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) w[i] = gain(i);
    }
    float acc[NV][8] = {};
    int stage = 0, flip = 0;
    uint32_t phase = 0;
    for (uint32_t row0 = row00; row0 < M; row0 += step, flip ^= 1) {
        const uint32_t row = row0 + group;
        const bool valid = row < M;
        const float r = valid ? a.rstd[row] : 0.0f;
        if (!tc::mbar_wait(&full[stage], phase, &abort, true)) {  // (the results are then undefined)
            abort = 1;
            if (lane == 0) atomicOr(status, tc::ST_PRODUCER);
        }
        const uint8_t *at = ring + stage * stage_bytes + group * K * 2;
        uint4 h[NV], dy[NV], dh[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = k0 + i * STEP;
            const bool in = valid && k < K;
            h[i] = in ? *reinterpret_cast<const uint4 *>(at + k * 2) : kZero;
            dy[i] = in ? *reinterpret_cast<const uint4 *>(at + plane + k * 2) : kZero;
            dh[i] = in && has_dh ? *reinterpret_cast<const uint4 *>(at + 2 * plane + k * 2) : kZero;
        }
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8], d[8], g[8];
            unpack8<T>(h[i], f);
            unpack8<T>(dy[i], d);
            gains8<T>(a.w != nullptr, KEEP ? w[i] : gain(i), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float k = d[j] * (f[j] * r);
                sum = fmaf(k, g[j], sum);
                acc[i][j] += k;
            }
        }
        if (WPR == 1) __syncthreads();
        reduce_row<WPR>(sum, top, red[flip]);
        // every thread has its part of the stage
        if (threadIdx.x == 0) fetch(row0 + stages * step, stage);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
        if (a.dX) {
            const float mean = sum / (float)K;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8], d[8], g[8], e[8];
                unpack8<T>(h[i], f);
                unpack8<T>(dy[i], d);
                unpack8<T>(dh[i], e);
                gains8<T>(a.w != nullptr, KEEP ? w[i] : gain(i), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-f[j] * r, mean, d[j] * g[j]), e[j]);
                if (valid && k0 + i * STEP < K) *reinterpret_cast<uint4 *>(a.dX + (long long)row * K + k0 + i * STEP) = pack8<T>(d);
            }
        }
    }
    if (abort && threadIdx.x == 0)
        drain_copies(full, stages, (int)((a.M - blockIdx.x * ROWS + gridDim.x * ROWS - 1) / (gridDim.x * ROWS)), &abort);
    if (!a.part) return;
    float *part = a.part + (long long)blockIdx.x * K;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = k0 + i * STEP;
            if (k < K) {
                *reinterpret_cast<float4 *>(part + k) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                *reinterpret_cast<float4 *>(part + k + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
    } else {
        // the groups' sums meet in the ring, [group][K], every copy into which has been read
        __syncthreads();
        float *sums = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = k0 + i * STEP;
            if (k < K) {
                *reinterpret_cast<float4 *>(sums + group * K + k) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                *reinterpret_cast<float4 *>(sums + group * K + k + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < K; k += WARPS * 32) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < ROWS; ++g) s += sums[g * K + k];
            part[k] = s;
        }
    }
}

// Rows that are no whole pieces (as in rms_norm_kernel), through registers.  dw's sums lie
// in shared memory behind the gains, element k of a group of warps at (k % 8) PLANE + k / 8
// (a warp's threads on different banks): a thread's columns are others in every row.
template <typename T, int WPR>
__global__ void __launch_bounds__(row_warps(WPR) * 32)
rms_norm_backward_odd_kernel(const BwdArgs a)
{
    extern __shared__ __align__(16) uint16_t gains_s[];
    constexpr int WARPS = row_warps(WPR), ROWS = WARPS / WPR, PLANE = WPR * 128 + 1, STEP = WPR * 256;
    __shared__ float2 red[2][WARPS];
    const int warp = threadIdx.x >> 5, K = a.K, group = warp / WPR;
    float *sums = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(gains_s) + gains_bytes(K));
    float *mine = sums + group * 8 * PLANE;
    if (a.part)
        for (int i = threadIdx.x; i < ROWS * 8 * PLANE; i += WARPS * 32) sums[i] = 0.0f;
    pdl_wait();
    stage_gains<T>(a.w, K, gains_s);
    __syncthreads();
    int flip = 0;
    for (long long row0 = (long long)blockIdx.x * ROWS; row0 < a.M; row0 += (long long)gridDim.x * ROWS, flip ^= 1) {
        const long long row = row0 + group;
        const bool valid = row < a.M;
        const long long at = valid ? row * K : 0;
        const Share me = share_of<WPR, true>(a.H + at, valid ? K : 0);
        const long long body = at + me.head;
        const bool has_dh = a.dH && a.dX, some = me.one >= 0;
        uint4 h[NV], dy[NV], dh[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = me.k0 + i * STEP;
            h[i] = k < me.body ? ld16(a.H + body + k) : kZero;
            dy[i] = k < me.body ? ld16(a.dY + body + k) : kZero;
            dh[i] = k < me.body && has_dh ? ld16(a.dH + body + k) : kZero;
        }
        const float h1 = some ? value<T>(a.H + at + me.one) : 0.0f, y1 = some ? value<T>(a.dY + at + me.one) : 0.0f,
                    d1 = some && has_dh ? value<T>(a.dH + at + me.one) : 0.0f, g1 = some ? value<T>(gains_s + me.one) : 0.0f;
        const float r = valid ? a.rstd[row] : 0.0f;
        float sum = y1 * (h1 * r) * g1, top = 0.0f;
        if (a.part && some) mine[(me.one & 7) * PLANE + (me.one >> 3)] += y1 * (h1 * r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = me.k0 + i * STEP;
            if (k >= me.body) break;
            float f[8], d[8], g[8];
            unpack8<T>(h[i], f);
            unpack8<T>(dy[i], d);
            unpack8<T>(staged8(gains_s, me.head, k), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = d[j] * (f[j] * r);
                sum = fmaf(t, g[j], sum);
                if (a.part) mine[((me.head + j) & 7) * PLANE + ((me.head + k + j) >> 3)] += t;
            }
        }
        reduce_row<WPR>(sum, top, red[flip]);
        if (WPR == 1) __syncwarp();  // the group's sums: the next row's columns are other threads'
        const float mean = sum / (float)K;
        if (a.dX) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int k = me.k0 + i * STEP;
                if (k >= me.body) break;
                float f[8], d[8], g[8], e[8];
                unpack8<T>(h[i], f);
                unpack8<T>(dy[i], d);
                unpack8<T>(dh[i], e);
                unpack8<T>(staged8(gains_s, me.head, k), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-f[j] * r, mean, d[j] * g[j]), e[j]);
                *reinterpret_cast<uint4 *>(a.dX + body + k) = pack8<T>(d);
            }
            if (some) a.dX[at + me.one] = bits<T>(fmaf(r, fmaf(-h1 * r, mean, y1 * g1), d1));
        }
    }
    if (!a.part) return;
    float *part = a.part + (long long)blockIdx.x * K;
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += WARPS * 32) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < ROWS; ++g) s += sums[g * 8 * PLANE + (k & 7) * PLANE + (k >> 3)];
        part[k] = s;
    }
}

// dX of any rows, a CTA to a row.
template <typename T>
__global__ void __launch_bounds__(MAX_WPR * 32)
rms_norm_long_dx_kernel(const BwdArgs a)
{
    __shared__ float2 red[MAX_WPR];
    pdl_wait();
    const long long row = blockIdx.x;
    const int K = a.K;
    const long long at = row * K;
    const int off = behind16(a.H + at) >> 1;
    constexpr long long STEP = MAX_WPR * 256;
    const long long k0 = (long long)threadIdx.x * 8 - off;
    const bool wx = on(a.dX + at - off, 16);
    auto gain = [&](long long k, float(&g)[8]) { gains8<T>(a.w != nullptr, a.w ? load8(a.w, k, K) : kZero, g); };
    const float r = a.rstd[row];
    float sum = 0.0f, top = 0.0f;
    for (long long k = k0; k < K; k += STEP) {
        float f[8], d[8], g[8];
        unpack8<T>(load8(a.H + at, k, K), f);
        unpack8<T>(load8(a.dY + at, k, K), d);
        gain(k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(d[j] * (f[j] * r), g[j], sum);
    }
    reduce_row<MAX_WPR>(sum, top, red);
    const float mean = sum / (float)K;
    for (long long k = k0; k < K; k += STEP) {
        float f[8], d[8], g[8], e[8];
        unpack8<T>(load8(a.H + at, k, K), f);
        unpack8<T>(load8(a.dY + at, k, K), d);
        unpack8<T>(a.dH ? load8(a.dH + at, k, K) : kZero, e);
        gain(k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-f[j] * r, mean, d[j] * g[j]), e[j]);
        store8(a.dX + at, k, K, wx, pack8<T>(d));
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

// dw[k] = sum over n partials, each of 32 warps its share of them in order, then the
// warps' sums in order.
__global__ void __launch_bounds__(1024)
rms_norm_dw_kernel(const float *__restrict__ part, float *__restrict__ dw, int n, int K)
{
    __shared__ float sums[32][32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long k = blockIdx.x * 32LL + lane;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int g = warp; g < n; g += 32) s += __ldcg(part + (long long)g * K + k);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && k < K) {
#pragma unroll
        for (int w = 1; w < 32; ++w) s += sums[w][lane];
        dw[k] = s;
    }
}

// Warps to a row of K elements that lies as kind_of says; 0: for the kernels of any rows.
int row_split(int K, int kind) {
    if (kind == 2) return 0;
    for (int w = 1; w <= MAX_WPR; w *= 2)
        if (K <= w * WARP_ELEMS) return w;
    return 0;
}
// How the rows of operands lie: 0 all on 16 bytes, 1 alike, 2 otherwise (null ones lie anywhere).
int kind_of(const void *first, std::initializer_list<const void *> others, const void *w, int K) {
    uintptr_t a = (uintptr_t)first & 15, any = a | ((uintptr_t)w & 15);
    bool alike = true;
    for (const void *p : others)
        if (p) {
            alike = alike && ((uintptr_t)p & 15) == a;
            any |= (uintptr_t)p & 15;
        }
    return any == 0 && K % 8 == 0 ? 0 : alike ? 1 : 2;
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

template <typename... KArgs, typename... Args>
cudaError_t launch_smem(void (*kern)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    // Above 48 KB, a kernel's own few hundred bytes included, a launch needs leave: for as much
    // as any takes, so that no call takes back what another, on another thread, is about to use.
    constexpr size_t kFree = 47 * 1024, kMost = 224 * 1024;
    if (smem > kFree) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
    }
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3((unsigned)threads), smem, s, attr);
    return launch_counted(&cfg, kern, args...);
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
    int kind = kind_of(p.X, {p.R, p.H, p.Y}, p.w, p.K);
    if (p.Q && ((uintptr_t)p.Q & 7) != ((uintptr_t)p.X & 15) >> 1) kind = 2;  // codes on 8 bytes where X is on 16
    const int wpr = row_split(p.K, kind);
    cudaLaunchAttribute attr[1];
    if (wpr == 0) {
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.M), dim3(MAX_WPR * 32), 0, s, attr);
        return launch_counted(&cfg, rms_norm_long_kernel<T, E4M3>, a);
    }
    return with_split(wpr, [&](auto w) {
        constexpr int W = decltype(w)::value, ROWS = row_warps(W) / W;
        const unsigned grid = (unsigned)(((long long)p.M + ROWS - 1) / ROWS);
        const size_t gains = kind ? (size_t)((p.K + 15) & ~7) * 2 : 0;
        return launch_smem(kind ? rms_norm_kernel<T, W, true, E4M3> : rms_norm_kernel<T, W, false, E4M3>, grid,
                           row_warps(W) * 32, gains, s, a);
    });
}

template <typename T>
cudaError_t backward(const NormBackward &p, int num_sms, int *status, cudaStream_t s) {
    BwdArgs a = {};
    a.H = static_cast<const uint16_t *>(p.H);
    a.w = static_cast<const uint16_t *>(p.w);
    a.rstd = p.rstd;
    a.dY = static_cast<const uint16_t *>(p.dY);
    a.dH = static_cast<const uint16_t *>(p.dH);
    a.dX = static_cast<uint16_t *>(p.dX);
    a.M = p.M;
    a.K = p.K;
    const int kind = kind_of(p.H, {p.dY, p.dH, p.dX}, p.w, p.K);
    const int wpr = row_split(p.K, kind);
    const int rows = wpr ? row_warps(wpr) / wpr : 1;
    // as many CTAs as stay resident, and partial sums of dw
    const int per_sm = kind == 0 ? bulk_ctas(wpr ? wpr : MAX_WPR) : wpr <= 4 ? 3 : wpr == 8 ? 2 : 1;
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
            constexpr int THREADS = row_warps(W) * 32;
            if (kind != 0) {
                const size_t gains = (size_t)((p.K + 15) & ~7) * 2, sums = (size_t)rows * 8 * (W * 128 + 1) * 4;
                return launch_smem(rms_norm_backward_odd_kernel<T, W>, (unsigned)ctas, THREADS, gains + (p.dw ? sums : 0), s, a);
            }
            // stages: those that per_sm CTAs find room for, at most eight
            const size_t stage = (size_t)3 * rows * p.K * 2;
            const int stages = (int)std::max<size_t>(2, std::min<size_t>(8, 220 * 1024 / per_sm / stage));
            return launch_smem(rms_norm_backward_bulk_kernel<T, W>, (unsigned)ctas, THREADS, stages * stage, s, a, stages, status);
        });
    }
    if (e == cudaSuccess && ws) {
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((p.K + 31LL) / 32)), dim3(1024), 0, s, attr);
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

cudaError_t launch_rms_norm_backward(const NormBackward &p, int num_sms, int *status, cudaStream_t s) {
    return p.elt == Elt::BF16 ? backward<__nv_bfloat16>(p, num_sms, status, s) : backward<__half>(p, num_sms, status, s);
}

}  // namespace gemm_gb300
