// Orthogonalised update: the singular values of G / |G|_F driven towards 1 by steps of an
// odd quintic polynomial, products only (Newton-Schulz):
//     A = X X^T,  B = b A + c A^2,  X <- a X + B X
// for M <= N; for M > N from the right, A = X^T X and X <- a X + X B, so that A is the
// smaller square, m = min(M, N), without a transposed copy.
//
// Bound: the tensor cores, m^2 n + m^3 + 2 m^2 n operations a step: A and B are
// symmetric, and only the tiles on and below the diagonal blocks of 256 are computed and
// written twice, the second time transposed.
//
// Precision.  Operands are half: iterates and A are bounded by about 1.2 in norm, so
// that half's 11 bits serve where bf16 has 8.  What the rounding of X loses in
// directions of small singular values the coming steps magnify, up to 3.4 times each; so
// X is kept as hi + lo, two halves (22 bits): the products take hi, the epilogue adds
// a (hi + lo) in FP32 -- lo left out of B X costs lo times B, which is small in just those
// directions.  Relative error (2-norm) of the five usual steps, in simulation against 64
// bits, 512 x 1024: singular values from 1 down to 1e-4 7.5e-4 (hi alone 5.4e-3, bf16
// 3e-2), Gaussian 1.6e-3, 16 strong directions in noise 1.5e-4 (4.0e-3).  G goes in
// unrounded, times a power of two that takes |G|_F to [2^14, 2^15), and its norm is
// applied to the sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "fp4.h"
#include "orthogonalize.h"
#include "pair_pipe.cuh"

namespace gemm_gb300 {
namespace {

using namespace pair;

constexpr float kLo = 2048.0f;  // lo is stored times 2^11, within half's normal range

__device__ __forceinline__ float2 half2_at(uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }

// A 32 x 64 block of half from memory, a row to eight lanes and four rows to a load (a row
// to a lane costs a load 32 cycles), and each lane's row of it, through the warp's box.
struct Block {
    uint4 v[8];
    // rows left, 1 or more: those from row0 on that exist
    __device__ __forceinline__ void fetch(const uint16_t *at, long long ld, int lane, int rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            if (r < rows) v[i] = *reinterpret_cast<const uint4 *>(at + r * ld + (lane & 7) * 8);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void to_box(uint8_t *box, int lane) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            *reinterpret_cast<uint4 *>(box + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = v[i];
        }
    }
};
// Half h of a lane's row: 32 values.
__device__ __forceinline__ void row_half(const uint8_t *box, int lane, int h, uint32_t (&w)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(box + lane * 128 + (((h * 4 + c) ^ (lane & 7)) << 4));
        w[4 * c] = v.x;
        w[4 * c + 1] = v.y;
        w[4 * c + 2] = v.z;
        w[4 * c + 3] = v.w;
    }
}

// A [m, m] = f X X^T, or B = b A + c A A^T: both triangles.
struct SymEpi {
    static constexpr bool LOWER = true, JOIN = true, CLASSES = false;
    static constexpr int BOXES = 2;
    CUtensorMap tm, tmT;    // the output, and in boxes of 64 rows x 32 columns
    const uint16_t *old;    // A, or null
    long long ld;
    const float *scale;     // null: 1; its square is a factor of the sums
    float f, b;             // f the sums' other factor, b A's
    int m;

    struct Pre {
        Block old;
    };
    // The tile's columns c .. c + 63 of A.
    __device__ __forceinline__ void fetch(const Part &p, int c, Pre &pre) const {
        if (old && p.col0 + c < m) pre.old.fetch(old + p.row0 * ld + p.col0 + c, ld, p.lane, m - p.row0);
    }
    __device__ __forceinline__ void prefetch(const Part &p, Pre &pre) const {
        pre.old.clear();
        fetch(p, p.first, pre);
    }
    __device__ __forceinline__ void run(Part &p, Pre &pre) const {
        const float s = scale ? *scale : 1.0f, by = f * s * s;
        const bool mirror = p.col0 + p.bn <= p.row0 / 256 * 256;
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 64) {
            const int c0 = p.col0 + g;
            if (c0 >= m) return;  // warp-uniform
            box_begin(p.lane);
            if (old) {
                pre.old.to_box(p.box, p.lane);
                __syncwarp();
                if (g + 64 < p.first + p.width) fetch(p, g + 64, pre);
            }
            uint32_t z[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                p.load<true>(g + h * 32, r);
                uint32_t w[16] = {};
                if (old) row_half(p.box, p.lane, h, w);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 e = half2_at(w[j]);
                    z[h * 16 + j] = pack2(fmaf(b, e.x, __uint_as_float(r[2 * j]) * by),
                                          fmaf(b, e.y, __uint_as_float(r[2 * j + 1]) * by), (__half *)nullptr);
                }
            }
            box_put(p.box, p.lane, z);  // (each lane its own row, which it alone has read)
            box_store(&tm, p.box, p.lane, c0, p.row0, 0);
            if (mirror) {
                uint8_t *box = p.box + STG_BOX;
#pragma unroll
                for (int j = 0; j < 32; ++j) {  // columns 2 j and 2 j + 1 are rows of 64 bytes, 64-byte swizzle
                    const int r0 = 2 * j, at = (((p.lane >> 3) ^ (j & 3)) << 4) + (p.lane & 7) * 2;
                    *reinterpret_cast<uint16_t *>(box + r0 * 64 + at) = (uint16_t)z[j];
                    *reinterpret_cast<uint16_t *>(box + (r0 + 1) * 64 + at) = (uint16_t)(z[j] >> 16);
                }
                box_store(&tmT, box, p.lane, p.row0, c0, 0);
            }
        }
    }
};

// X' = s (a (hi + lo) + sums): hi and lo, or (LAST) the result in its own type.  LO: X has a
// lo, and s is 1 (the first step's X has none).
struct MulArgs {
    CUtensorMap tm, tmLo;         // hi or the result; lo
    const uint16_t *hi, *lo;      // X
    long long ld;
    const float *scale;           // s
    float a;
    int M, N;
    bool bf16;                    // the result's type, or half
    uint16_t *out;                // not null: the result by the element
    long long ldo;
};
template <bool LO, bool LAST>
struct MulEpi : MulArgs {
    static constexpr bool LOWER = false, JOIN = true, CLASSES = false;
    static constexpr int BOXES = 2;

    struct Pre {
        Block hi, lo;
    };
    __device__ __forceinline__ void fetch(const Part &p, int c, Pre &pre) const {
        if (p.col0 + c >= N) return;
        const long long at = p.row0 * ld + p.col0 + c;
        pre.hi.fetch(hi + at, ld, p.lane, M - p.row0);
        if (LO) pre.lo.fetch(lo + at, ld, p.lane, M - p.row0);
    }
    __device__ __forceinline__ void prefetch(const Part &p, Pre &pre) const {
        pre.hi.clear();
        if (LO) pre.lo.clear();
        fetch(p, p.first, pre);
    }
    // Two lanes of FP32 at a time: the conversions and these, ten instructions for two
    // elements, bound a tile's writing.
    __device__ __forceinline__ void run(Part &p, Pre &pre) const {
        const float s = LO ? 1.0f : *scale, sa = s * a;
        const float2 s2 = make_float2(s, s), a2 = make_float2(sa, sa), lo2 = make_float2(sa / kLo, sa / kLo),
                     up2 = make_float2(kLo, kLo), down2 = make_float2(-kLo, -kLo), zero2 = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int g = p.first; g < p.first + p.width; g += 64) {
            const int c0 = p.col0 + g;
            if (c0 >= N) return;  // warp-uniform
            uint8_t *box_lo = p.box + STG_BOX;
            box_begin(p.lane);
            pre.hi.to_box(p.box, p.lane);
            if (LO) pre.lo.to_box(box_lo, p.lane);
            __syncwarp();
            if (g + 64 < p.first + p.width) fetch(p, g + 64, pre);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32], z[16], w[16], e[16];
                p.load<true>(g + h * 32, r);
                row_half(p.box, p.lane, h, w);
                if (LO) row_half(box_lo, p.lane, h, e);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float2 x = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    if (LO) x = __ffma2_rn(half2_at(e[j]), lo2, x);
                    else x = __ffma2_rn(x, s2, zero2);
                    x = __ffma2_rn(half2_at(w[j]), a2, x);
                    if (LAST) {
                        z[j] = bf16 ? pack2(x.x, x.y, (__nv_bfloat16 *)nullptr) : pack2(x.x, x.y, (__half *)nullptr);
                    } else {
                        z[j] = pack2(x.x, x.y, (__half *)nullptr);
                        x = __ffma2_rn(half2_at(z[j]), down2, __ffma2_rn(x, up2, zero2));
                        e[j] = pack2(x.x, x.y, (__half *)nullptr);
                    }
                }
                // (each lane its own row, which it alone has read)
                box_put_half(p.box, p.lane, h, z);
                if (!LAST) box_put_half(box_lo, p.lane, h, e);
            }
            if (LAST && out) {
                box_scatter(p.box, p.lane, out, ldo, p.row0, c0, M, N);
                continue;
            }
            box_store(&tm, p.box, p.lane, c0, p.row0, 0);
            if (!LAST) box_store(&tmLo, box_lo, p.lane, c0, p.row0, 0);
        }
    }
};

// Sixteen packed 16-bit values in FP32.
template <bool BF16>
__device__ __forceinline__ void widen16(const uint32_t (&v)[8], float (&f)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 t = BF16 ? make_float2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xFFFF0000u)) : half2_at(v[j]);
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}
// The row pieces of 512 elements of G, dealt to the grid's warps: f(row, first element of
// the lane's sixteen, its values; zeros past N).
constexpr int SCAN_WARPS = 8;
template <bool BF16, typename F>
__device__ __forceinline__ void scan(const uint16_t *G, long long ldg, int M, int N, F f) {
    const long long per = (N + 511LL) / 512, total = M * per;
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(G),
                  *hi = reinterpret_cast<const uint8_t *>(G + (M - 1) * ldg + N);
    for (long long i = (long long)blockIdx.x * SCAN_WARPS + (threadIdx.x >> 5); i < total;
         i += (long long)gridDim.x * SCAN_WARPS) {
        const long long row = i / per;
        const long long k = (i - row * per) * 512 + (threadIdx.x & 31) * 16;
        uint32_t v[8];
        fp4_load16_any(G + row * ldg + k, (int)max(min(N - k, 512LL), -512LL), lo, hi, v);
        float x[16];
        widen16<BF16>(v, x);
        f(row, k, x);
    }
}

// Sums of squares, one to a CTA, in 64 bits: sixteen values at a time in FP32, taken by a
// power of two so that the largest is in [1, 2) -- no square overflows or is lost.
template <bool BF16>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
orth_norm_kernel(const uint16_t *G, long long ldg, int M, int N, double *part)
{
    __shared__ double sums[SCAN_WARPS];
    pdl_wait();
    double sum = 0.0;
    scan<BF16>(G, ldg, M, N, [&](long long, long long, const float(&x)[16]) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
        const int e = max(min((int)(__float_as_uint(top) >> 23), 253), 1) - 127;
        const float by = __uint_as_float((uint32_t)(127 - e) << 23);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(x[j] * by, x[j] * by, s);
        sum += (double)s * __longlong_as_double((long long)(1023 + 2 * e) << 52);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < SCAN_WARPS; ++w) sum += sums[w];
    part[blockIdx.x] = sum;
}

// X = G 2^k in half, and s = 2^-k / |G|; every CTA adds the partial sums alike.  A matrix
// of zeros has s = 0 (and stays zero), one with a NaN or an infinity s = NaN.
template <bool BF16>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
orth_start_kernel(const uint16_t *G, long long ldg, int M, int N, const double *part, int parts, float *scale, uint16_t *X,
                  long long ldx)
{
    __shared__ double sums[SCAN_WARPS];
    __shared__ float by_s;
    pdl_wait();
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += SCAN_WARPS * 32) sum += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    {
        if (threadIdx.x == 0) {
            for (int w = 1; w < SCAN_WARPS; ++w) sum += sums[w];
            const double norm = sqrt(sum);
            double by = 0.0, s = 0.0;
            if (!isfinite(norm)) {
                s = NAN;
            } else if (norm > 0.0) {
                int e;
                frexp(norm, &e);
                by = ldexp(1.0, max(min(15 - e, 126), -126));
                s = 1.0 / (norm * by);
            }
            by_s = (float)by;
            if (blockIdx.x == 0) *scale = (float)s;
        }
    }
    __syncthreads();
    const float by = by_s;
    scan<BF16>(G, ldg, M, N, [&](long long row, long long k, const float(&x)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack2(x[2 * j] * by, x[2 * j + 1] * by, (__half *)nullptr);
        uint4 *o = reinterpret_cast<uint4 *>(X + row * ldx + k);
        if (k < ldx) o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (k + 8 < ldx) o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    });
}

long long up64(long long n) { return (n + 63) / 64 * 64; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// A product's tiles: their width, and, where one wave of them takes it, pairs joined on a
// tile, as are done first (five steps of 512 x 512 98 us with joined pairs, 115 without, 1024
// x 1024 119 and 196, 1000 x 3001 165 and 221; three waves of joined pairs for X of 1000 x
// 3001 220).  Times in 1/100 us: a block of 64 k of 256 x bn, a tile's writing and join.
struct Plan {
    int bn, joined, clusters;
    long long tiles;
};
// Clusters of every kernel of X's product (all of one size and shared memory).
template <bool LO, bool LAST>
int mul_clusters_of(int dev, int joined) {
    return joined == 1 ? clusters_max<0, MulEpi<LO, LAST>>(dev) : joined_max<0, MulEpi<LO, LAST>>(dev);
}
int mul_clusters(int dev, int joined) {
    return std::min({mul_clusters_of<false, false>(dev, joined), mul_clusters_of<true, false>(dev, joined),
                     mul_clusters_of<false, true>(dev, joined), mul_clusters_of<true, true>(dev, joined)});
}
template <bool LO, bool LAST>
cudaError_t launch_mul(const CUtensorMap &ta, const CUtensorMap &tb, const MulArgs &m, const Args &args, int clusters,
                       cudaStream_t s) {
    MulEpi<LO, LAST> e;
    static_cast<MulArgs &>(e) = m;
    return launch<0>(ta, tb, e, args, clusters, s);
}
Plan plan(bool lower, int rows, int cols, int k, int dev) {
    const long long kb = ceil_div(k, BK);
    Plan best = {};
    long long least = 0;
    for (int bn = 256; bn >= 128; bn /= 2) {
        const long long tiles = lower ? lower_tiles(rows, bn) : ceil_div(rows, 256) * ceil_div(cols, bn);
        if (tiles > 0x7FFFFFFFLL) continue;
        for (int joined = 1; joined <= (bn == 128 ? 2 : 1); ++joined) {
            const int c = !lower        ? mul_clusters(dev, joined)
                          : joined == 1 ? clusters_max<0, SymEpi>(dev)
                                        : joined_max<0, SymEpi>(dev);
            if (c <= 0 || (joined > 1 && (tiles > c || kb < 2))) continue;
            const long long block = bn == 256 ? 30 : 20, write = bn == 256 ? 250 : joined == 1 ? 150 : 200;
            const long long time = ceil_div(tiles, c) * ceil_div(kb, joined) * block + write;
            if (!best.bn || time < least) {
                best = {bn, joined, c, tiles};
                least = time;
            }
        }
    }
    return best;
}

cudaError_t run(const OrthProblem &p, int dev, int num_sms, int *status, cudaStream_t s) {
    if (clusters_max<0, SymEpi>(dev) <= 0 || mul_clusters(dev, 1) <= 0) return cudaErrorNotSupported;
    const bool tall = p.M > p.N, bf16 = p.elt == Elt::BF16;
    const int m = std::min(p.M, p.N), n = std::max(p.M, p.N);
    const long long ldx = up64(p.N), lda = up64(m);
    const size_t x_bytes = (size_t)p.M * ldx * 2, a_bytes = (size_t)m * lda * 2;
    const int parts = (int)std::min<long long>(8LL * num_sms, ceil_div(p.M * ceil_div(p.N, 512), SCAN_WARPS));
    auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
    const size_t need = 4 * al(x_bytes) + 2 * al(a_bytes) + al((size_t)parts * 8) + 256;
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(&ws, need, s);
    if (e != cudaSuccess) return e;
    uint8_t *at = static_cast<uint8_t *>(ws);
    auto take = [&](size_t b) {
        uint8_t *q = at;
        at += al(b);
        return q;
    };
    uint16_t *hi[2], *lo[2];
    for (int i = 0; i < 2; ++i) {
        hi[i] = reinterpret_cast<uint16_t *>(take(x_bytes));
        lo[i] = reinterpret_cast<uint16_t *>(take(x_bytes));
    }
    uint16_t *A = reinterpret_cast<uint16_t *>(take(a_bytes)), *B = reinterpret_cast<uint16_t *>(take(a_bytes));
    double *part = reinterpret_cast<double *>(take((size_t)parts * 8));
    float *scale = reinterpret_cast<float *>(take(4));

    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)parts), dim3(SCAN_WARPS * 32), 0, s, attr);
    const uint16_t *G = static_cast<const uint16_t *>(p.G);
    e = bf16 ? launch_counted(&cfg, orth_norm_kernel<true>, G, p.ldg, p.M, p.N, part)
             : launch_counted(&cfg, orth_norm_kernel<false>, G, p.ldg, p.M, p.N, part);
    if (e == cudaSuccess)
        e = bf16 ? launch_counted(&cfg, orth_start_kernel<true>, G, p.ldg, p.M, p.N, static_cast<const double *>(part), parts,
                                  scale, hi[0], ldx)
                 : launch_counted(&cfg, orth_start_kernel<false>, G, p.ldg, p.M, p.N, static_cast<const double *>(part), parts,
                                  scale, hi[0], ldx);
    // A over n, B over m, X over m
    const Plan pa = plan(true, m, m, n, dev), pb = plan(true, m, m, m, dev), px = plan(false, p.M, p.N, m, dev);
    if (e == cudaSuccess && (!pa.bn || !pb.bn || !px.bn)) e = cudaErrorInvalidValue;
    SymEpi sy;
    MulArgs mu;
    CUtensorMap aL, aR, aM, outA, outAT, outB, outBT, hiM[2], loM[2], sym[2][2], mul[2];
    // operands: A's rows as the left one, and as the right one of B's product and of X's
    bool ok = map16(&outA, A, 0, m, m, lda, 32, 64) && map16(&outB, B, 0, m, m, lda, 32, 64) &&
              make_map3(&outAT, A, map_type(0), m, m, 1, lda * 2, m * lda * 2, 32, 64, 1, 64) &&
              make_map3(&outBT, B, map_type(0), m, m, 1, lda * 2, m * lda * 2, 32, 64, 1, 64) &&
              map_operand(&aL, A, 0, false, m, m, lda, 128) && map_operand(&aR, A, 0, false, m, m, lda, pb.bn / 2) &&
              map_operand(&aM, B, 0, false, m, m, lda, tall ? px.bn / 2 : 128);
    for (int i = 0; i < 2; ++i)
        ok = ok && map16(&hiM[i], hi[i], 0, p.M, p.N, ldx, 32, 64) && map16(&loM[i], lo[i], 0, p.M, p.N, ldx, 32, 64) &&
             map_operand(&sym[i][0], hi[i], 0, tall, m, n, ldx, 128) &&
             map_operand(&sym[i][1], hi[i], 0, tall, m, n, ldx, pa.bn / 2) &&
             map_operand(&mul[i], hi[i], 0, !tall, n, m, ldx, 128);
    // (TMA writes whole 16-byte pieces, past a row's last element too)
    const bool tma_out = ((uintptr_t)p.O & 15) == 0 && p.ldo % 8 == 0 && p.N % 8 == 0;
    CUtensorMap res = hiM[0];
    if (tma_out) ok = ok && map16(&res, p.O, bf16 ? 1 : 0, p.M, p.N, p.ldo, 32, 64);
    if (!ok && e == cudaSuccess) e = cudaErrorInvalidValue;
    auto args = [&](int rows, int cols, int k, const Plan &q, bool a_mn, bool b_mn) {
        return Args{rows, cols, (int)ceil_div(k, BK), q.bn, a_mn, b_mn, (int)q.tiles, 1, q.joined, 128, BK, 256, 0, 0, 0, 0, status};
    };
    for (int i = 0; i < p.steps && e == cudaSuccess; ++i) {
        const int in = i & 1, out = in ^ 1;
        const bool last = i == p.steps - 1;
        // A = X X^T, or X^T X
        sy.tm = outA;
        sy.tmT = outAT;
        sy.old = nullptr;
        sy.ld = lda;
        sy.scale = i == 0 ? scale : nullptr;
        sy.f = 1.0f;
        sy.b = 0.0f;
        sy.m = m;
        e = launch<0>(sym[in][0], sym[in][1], sy, args(m, m, n, pa, tall, tall), pa.clusters, s);
        if (e != cudaSuccess) break;
        sy.tm = outB;
        sy.tmT = outBT;
        sy.old = A;
        sy.scale = nullptr;
        sy.f = p.c;
        sy.b = p.b;
        e = launch<0>(aL, aR, sy, args(m, m, m, pb, false, false), pb.clusters, s);
        if (e != cudaSuccess) break;
        mu.tm = last ? res : hiM[out];
        mu.tmLo = loM[out];
        mu.hi = hi[in];
        mu.lo = lo[in];
        mu.ld = ldx;
        mu.scale = scale;
        mu.a = p.a;
        mu.M = p.M;
        mu.N = p.N;
        mu.bf16 = bf16;
        mu.out = last && !tma_out ? static_cast<uint16_t *>(p.O) : nullptr;
        mu.ldo = p.ldo;
        // B X: B's rows and X, [m, N], N-major; X B: X's rows and B's
        const auto f = i == 0 ? (last ? launch_mul<false, true> : launch_mul<false, false>)
                              : (last ? launch_mul<true, true> : launch_mul<true, false>);
        e = tall ? f(mul[in], aM, mu, args(p.M, p.N, m, px, false, false), px.clusters, s)
                 : f(aM, mul[in], mu, args(p.M, p.N, m, px, false, true), px.clusters, s);
    }
    const cudaError_t f = cudaFreeAsync(ws, s);
    return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_orthogonalize(const OrthProblem &p, int num_sms, int *status, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    return run(p, dev, num_sms, status, s);
}

}  // namespace gemm_gb300
