// 4-bit block-scaled product for few rows (M <= 64: single tokens, decode
// batches), bound by reading the weights [N, K] once: 0.53 (MX) or 0.56 (NV)
// bytes an element.
//
// The operands swap roles: 128 weight rows are the MMA's M, the M rows of X its
// N = nb (M rounded up to 16), D[n, m] in nb tensor-memory columns.  A CTA takes
// a strip of 128 weight rows; the CS CTAs of a cluster share a strip's K and add
// their FP32 partials through distributed shared memory in rank order
// (deterministic, one launch, no workspace).  CS is the largest for which every
// CTA is resident at once, two to an SM, so that all SMs stream: N = 12288 gives
// 96 strips, 288 CTAs.  A stage is 256 k: 16 KiB of codes and 2 (NV) or 1 (MX) KiB
// of scales, loaded by TMA; scales go to tensor memory with tcgen05.cp (fp4_gemm.cu
// describes the scales' order).
//
// FUSED: X is in 16 bits and is quantised by the four epilogue warps while the
// weights stream, each CTA its own K range: the codes and scale bytes of
// fp4.cu's quantiser, written to shared memory as TMA would have.  Otherwise X
// is codes and scales, loaded by TMA.
//
// Every wait is bounded; on expiry a code goes to the status word, the CTA's own
// loads and MMAs are waited for, and its tensor memory is released.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "fp4.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

using namespace tc;

constexpr int THREADS = 192;
constexpr int KB = 256;
constexpr int MAX_STAGES = 6;
constexpr int RING = 108 * 1024;             // two CTAs to an SM
constexpr int SMEM = 1024 + RING + 256;
constexpr int W_STAGE = 128 * KB / 2;        // 16 KiB
constexpr uint32_t TMEM_COLS = 128, SF_COL = 64;  // D: 64 columns at most
constexpr int LD = 128 + 4;                  // floats per row of a partial [nb][128]
static_assert(64 * LD * 4 <= RING, "a partial fits the drained ring");

__host__ __device__ constexpr int sf_stage(bool nv) { return nv ? 2048 : 1024; }
__host__ __device__ constexpr int nb_of(int M) { return (M + 15) / 16 * 16; }
__host__ __device__ constexpr int stage_bytes(bool nv, int nb) { return W_STAGE + nb * 128 + 2 * sf_stage(nv); }
__host__ __device__ constexpr int stages_of(bool nv, int nb) {
    return RING / stage_bytes(nv, nb) < MAX_STAGES ? RING / stage_bytes(nv, nb) : MAX_STAGES;
}

// FUSED: converting warp j mod 4 at use j of the ring has seen every use up to j - 4 -
// stages done, and its wait on one bit of phase needs j - 2 stages.
static_assert(RING / stage_bytes(true, 16) >= 4 && RING / stage_bytes(false, 16) >= 4, "stages of the fused form");

struct Bars {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full;
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Args {
    const void *X;  // FUSED: [M,K], leading dimension ldx
    long long ldx;
    void *C;
    long long ldc;
    const float *ga, *gb;
    int M, N, K, cs;
    int x_vec;  // X's rows suit 16-byte loads
    int c_vec;  // C's rows suit 8-byte stores
    int *status;
};

template <bool NV>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t acc) {
    if constexpr (NV)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
}
__device__ __forceinline__ void cp_scales_one(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <bool NV>
__device__ __forceinline__ uint32_t make_idesc(uint32_t nb, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((nb >> 3) << 17) | ((NV ? 0u : 1u) << 23) | ((128u >> 4) << 24) |
           (id << 29);
}

template <typename T, bool NV, bool FUSED>
__global__ void __launch_bounds__(THREADS, 2)
fp4_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSw,
                  const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSx, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int SF = sf_stage(NV), ATOMS = SF / 512;
    const int M = args.M, N = args.N, K = args.K, cs = args.cs;
    const int nb = nb_of(M), stages = stages_of(NV, nb), x_stage = nb * 128;
    uint8_t *w_tiles = smem;
    uint8_t *x_tiles = w_tiles + stages * W_STAGE;
    uint8_t *sf_tiles = x_tiles + stages * x_stage;  // per stage: W's 128 rows, then X's
    float *part = reinterpret_cast<float *>(smem);   // [nb][LD] once the ring is drained
    Bars *bars = reinterpret_cast<Bars *>(smem + RING);
    volatile int *abort_flag = &bars->abort;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int strip = (int)(cs > 1 ? cluster_id_x() : blockIdx.x);
    const int num_kb = (K + KB - 1) / KB;
    const int kb0 = (int)((long long)num_kb * rank / cs), kb1 = (int)((long long)num_kb * (rank + 1) / cs);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&bars->full[s], FUSED ? 2 : 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        mbar_init_fence();
        prefetch_desc(&tmW);
        prefetch_desc(&tmSw);
    }
    if (warp == 1) tmem_alloc<1>(&bars->tmem_base, TMEM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    if (warp == 0 && lane == 0 && g_pdl) {
        // The strip's first weights to L2 while the previous kernel drains: a hint,
        // which changes no value that a later load returns.
        for (int kb = kb0; kb < min(kb1, kb0 + stages); ++kb) {
            tma_prefetch_l2_3d(&tmW, kb * (KB / 2), strip * 128, 0);
            tma_prefetch_l2_3d(&tmSw, 0, kb * (SF / 1024), strip);
        }
    }
    pdl_wait();

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        const uint32_t tx = (uint32_t)(W_STAGE + SF + (FUSED ? 0 : x_stage + SF));
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag, true)) {
                atomicOr(args.status, ST_PRODUCER);
                *abort_flag = 1;
                break;
            }
            mbar_arrive_expect_tx(&bars->full[stage], tx);
            uint8_t *sf = sf_tiles + stage * 2 * SF;
            tma_load_3d(w_tiles + stage * W_STAGE, &tmW, &bars->full[stage], kb * (KB / 2), strip * 128, 0);
            tma_load_3d(sf, &tmSw, &bars->full[stage], 0, kb * (SF / 1024), strip);
            if (!FUSED) {
                tma_load_3d(x_tiles + stage * x_stage, &tmX, &bars->full[stage], kb * (KB / 2), 0, 0);
                tma_load_3d(sf + SF, &tmSx, &bars->full[stage], 0, kb * (SF / 1024), 0);
            }
            ++issued;
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        pdl_launch_dependents();
        // Every load of this thread lands before the ring is reused or the CTA
        // ends.  (FUSED, after an abort: a phase whose converter gave up never
        // completes, so the wait runs out; its loads have landed long since.)
        for (long long i = (issued > stages ? issued - stages : 0); i < issued; ++i)
            if (!mbar_wait(&bars->full[i % stages], (uint32_t)((i / stages) & 1), abort_flag, false)) {
                atomicOr(args.status, ST_DRAIN);
                break;
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const bool issuer = elect_one();
        const uint64_t w_desc0 = desc_sw128(smem_u32(w_tiles), 16, 1024);
        const uint64_t x_desc0 = desc_sw128(smem_u32(x_tiles), 16, 1024);
        const uint64_t sf_desc0 = desc_plain(smem_u32(sf_tiles), 128);
        const uint32_t sfw = tmem_base + SF_COL, sfx = sfw + 4 * ATOMS;
        const uint32_t idesc0 = make_idesc<NV>((uint32_t)nb, 0), idesc1 = make_idesc<NV>((uint32_t)nb, 2);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&bars->full[stage], phase, abort_flag, true)) { ok = false; break; }
            fence_after();
            const uint64_t wd = w_desc0 + (uint64_t)((stage * W_STAGE) >> 4);
            const uint64_t xd = x_desc0 + (uint64_t)((stage * x_stage) >> 4);
            const uint64_t sd = sf_desc0 + (uint64_t)((stage * 2 * SF) >> 4);
            if (issuer) {
#pragma unroll
                for (int a = 0; a < ATOMS; ++a) {
                    cp_scales_one(sfw + 4 * a, sd + a * 32);
                    cp_scales_one(sfx + 4 * a, sd + (ATOMS + a) * 32);
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const int a = NV ? ks : ks >> 1;
                    mma_one<NV>(tmem_base, wd + ks * 2, xd + ks * 2, NV || (ks & 1) == 0 ? idesc0 : idesc1, sfw + 4 * a,
                                sfx + 4 * a, (uint32_t)(kb != kb0 || ks != 0));
                }
                commit<1>(&bars->empty[stage]);
            }
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (issuer) {
            if (ok) {
                commit<1>(&bars->acc_full);
            } else {
                atomicOr(args.status, ST_MMA);
                *abort_flag = 1;
            }
            commit<1>(&bars->drain);
            if (!mbar_wait(&bars->drain, 0, abort_flag, false)) atomicOr(args.status, ST_DRAIN);
        }
    } else if (warp >= 2) {
        bool ok = true;
        if constexpr (FUSED) {
            // ------------------------------------------------------------ X quantised, a stage to a warp
            // Warp w takes stages w, w + 4, ...: a stage's conversion is a chain of
            // dependent steps, so four stages are under way at once.  A unit is 16
            // consecutive k of a row (half an MX block, an NV block); lanes 0-15
            // hold one row's 256 k, 16-31 the next row's.
            const int half = lane >> 4, u = lane & 15;
            const T *X = static_cast<const T *>(args.X);
            auto load = [&](int kb, int r, uint32_t (&v)[8]) {
                const long long k = (long long)kb * KB + u * 16;
                if (r >= M || k >= K) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0u;
                    return;
                }
                const T *x = X + (long long)r * args.ldx + k;
                if (args.x_vec) fp4_load16<16>(x, (int)(K - k), v);
                else fp4_load16<2>(x, (int)(K - k), v);
            };
            int slot = warp - 2;
            uint32_t phase = 0;
            while (slot >= stages) { slot -= stages; phase ^= 1u; }
            // UNITS row pairs at a time, the next ones' values in flight meanwhile
            constexpr int UNITS = 2;
            uint32_t next[UNITS][8];
#pragma unroll
            for (int i = 0; i < UNITS; ++i) load(kb0 + warp - 2, half + 2 * i, next[i]);
            const Fp4Tensor ts = fp4_tensor<NV>(args.ga);
            for (int kb = kb0 + warp - 2; kb < kb1; kb += 4) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->empty[slot], phase ^ 1u, abort_flag, true))) {
                    ok = false;
                    break;
                }
                uint8_t *xs = x_tiles + slot * x_stage, *sx = sf_tiles + slot * 2 * SF + SF;
                for (int r0 = 0; r0 < M; r0 += 2 * UNITS) {
                    uint32_t v[UNITS][8];
                    const bool more = r0 + 2 * UNITS < M;
#pragma unroll
                    for (int i = 0; i < UNITS; ++i) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] = next[i][j];
                        load(more ? kb : kb + 4, (more ? r0 + 2 * UNITS : 0) + half + 2 * i, next[i]);
                    }
#pragma unroll
                    for (int i = 0; i < UNITS; ++i) {
                        const int r = r0 + 2 * i + half;
                        if (r0 + 2 * i >= M) break;  // warp-uniform
                        uint32_t m = 0u;
#pragma unroll
                        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, abs2(v[i][j]));
                        m = max(m & 0xFFFFu, m >> 16);
                        if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        const Fp4Scale sc = fp4_block_scale<NV>(bits16_to_f32<T>(m), ts);
                        const uint2 codes = fp4_codes16<T, NV>(v[i], sc);
                        if (r < M) {
                            *reinterpret_cast<uint2 *>(xs + r * 128 + (((u >> 1) ^ (r & 7)) << 4) + ((u & 1) << 3)) = codes;
                            const int b = NV ? u : u >> 1;  // block of the stage
                            if (NV || (u & 1) == 0) sx[(b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)] = (uint8_t)sc.byte;
                        }
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->full[slot]);
                slot += 4;
                while (slot >= stages) { slot -= stages; phase ^= 1u; }
            }
            if (!ok && lane == 0) {
                atomicOr(args.status, ST_PRODUCER);
                *abort_flag = 1;
            }
        }
        // ------------------------------------------------------------ epilogue
        // lane = weight row of the strip, column = row of X
        const int quarter = warp & 3, nl = quarter * 32 + lane, n = strip * 128 + nl;
        if (ok && kb1 > kb0 && !__all_sync(0xffffffffu, mbar_wait(&bars->acc_full, 0, abort_flag, true))) {
            ok = false;
            if (lane == 0) {
                atomicOr(args.status, ST_EPILOGUE);
                *abort_flag = 1;
            }
        }
        fence_after();
        __syncwarp();
        const Fp4Factors f = fp4_factors<NV>(args.ga, args.gb);
#pragma unroll 1
        for (int c = 0; c < M; c += 32) {
            uint32_t r[32];
            if (ok && kb1 > kb0) {
                tmem_ld32(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = 0u;
            }
            if (cs == 1) {
                T *col = static_cast<T *>(args.C) + n;
                if (n < N) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < M) store1(col + (long long)(c + j) * args.ldc, __uint_as_float(r[j]) * f.first * f.second);
                }
            } else {
                // (the ring is drained: every MMA that read it has completed)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j < M) part[(c + j) * LD + nl] = __uint_as_float(r[j]) * f.first * f.second;
            }
        }
    }

    fence_before();
    __syncwarp();
    if (cs > 1) {
        cluster_sync();
        // (row, four columns) pairs dealt out to the CTAs in equal ranges; partials added in rank order
        const int cols = min(128, N - strip * 128), groups = (cols + 3) / 4;
        const int total = M * groups;
        const int e1 = (int)((long long)total * (rank + 1) / cs);
        for (int e = (int)((long long)total * rank / cs) + (int)threadIdx.x; e < e1; e += THREADS) {
            const int m = e / groups, c4 = (e - m * groups) * 4;
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cs) v[j] = ld_cluster_f4(map_to_rank(part + m * LD + c4, (uint32_t)j));
            float4 a = v[0];
#pragma unroll
            for (int j = 1; j < 8; ++j)
                if (j < cs) {
                    a.x += v[j].x; a.y += v[j].y; a.z += v[j].z; a.w += v[j].w;
                }
            T *dst = static_cast<T *>(args.C) + (long long)m * args.ldc + strip * 128 + c4;
            if (args.c_vec && c4 + 4 <= cols) {
                uint2 w;
                w.x = pack2(a.x, a.y, (T *)nullptr);
                w.y = pack2(a.z, a.w, (T *)nullptr);
                *reinterpret_cast<uint2 *>(dst) = w;
            } else {
                const float o[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c4 + i < cols) store1(dst + i, o[i]);
            }
        }
        __syncwarp();
        cluster_sync();  // every CTA keeps its shared memory until the others have read it
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem_base, TMEM_COLS);
    }
}

template <typename T, bool NV, bool FUSED>
int clusters_max(int dev, int cs) {
    static std::atomic<int> known[kMaxDevices][9];
    return cluster_limit(known[dev][cs], reinterpret_cast<const void *>(fp4_skinny_kernel<T, NV, FUSED>),
                         THREADS, SMEM, cs);
}

template <typename T, bool NV, bool FUSED>
cudaError_t launch(const Fp4Problem &p, const void *X, long long ldx, int num_sms, int *status, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const long long strips = fp4_row_tiles(p.N), num_kb = (p.K + KB - 1LL) / KB;
    int cs = 1;
    if (clusters_max<T, NV, FUSED>(dev, 1) <= 0) return cudaErrorNotSupported;
    for (int c = 2; c <= 8 && c <= num_kb && strips * c <= 2LL * num_sms; ++c) {
        const int n = clusters_max<T, NV, FUSED>(dev, c);
        if (n < 0) return cudaErrorNotSupported;  // not another split, whose sums would differ
        if (n >= strips) cs = c;
    }
    const long long rb = fp4_row_bytes(p.K), chunks = (long long)fp4_atoms(NV, p.K) / 2;
    constexpr int SFC = sf_stage(NV) / 1024;
    const int nb = nb_of(p.M);
    CUtensorMap tw, tsw, tx, tsx;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    if (!make_map3(&tw, p.Qb, u8, rb, p.N, 1, p.pitch_b, p.pitch_b * p.N, 128, 128, 1, 128) ||
        !make_map3(&tsw, p.Sb, u32, 256, chunks, strips, 1024, chunks * 1024, 256, SFC, 1, 0))
        return cudaErrorInvalidValue;
    if (FUSED) {
        tx = tw;
        tsx = tsw;
    } else if (!make_map3(&tx, p.Qa, u8, rb, p.M, 1, p.pitch_a, p.pitch_a * p.M, 128, nb, 1, 128) ||
               !make_map3(&tsx, p.Sa, u32, 256, chunks, 1, 1024, chunks * 1024, 256, SFC, 1, 0)) {
        return cudaErrorInvalidValue;
    }
    Args a = {};
    a.X = X;
    a.ldx = ldx;
    a.C = p.C;
    a.ldc = p.ldc;
    a.ga = p.ga;
    a.gb = p.gb;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.cs = cs;
    a.x_vec = ((uintptr_t)X & 15u) == 0 && ldx % 8 == 0;
    a.c_vec = ((uintptr_t)p.C & 7u) == 0 && p.ldc % 4 == 0;
    a.status = status;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(strips * cs), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    pdl_attr(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = g_pdl ? attr : attr + 1;
    cfg.numAttrs = (g_pdl ? 1 : 0) + (cs > 1 ? 1 : 0);
    return launch_counted(&cfg, fp4_skinny_kernel<T, NV, FUSED>, tw, tsw, tx, tsx, a);
}

template <bool FUSED>
cudaError_t launch_any(const Fp4Problem &p, const void *X, long long ldx, int num_sms, int *status, cudaStream_t s) {
    if (p.elt == Elt::BF16)
        return p.nv ? launch<__nv_bfloat16, true, FUSED>(p, X, ldx, num_sms, status, s)
                    : launch<__nv_bfloat16, false, FUSED>(p, X, ldx, num_sms, status, s);
    return p.nv ? launch<__half, true, FUSED>(p, X, ldx, num_sms, status, s)
                : launch<__half, false, FUSED>(p, X, ldx, num_sms, status, s);
}

}  // namespace

cudaError_t launch_fp4_skinny(const Fp4Problem &p, const void *X, long long ldx, int num_sms, int *status,
                              cudaStream_t s) {
    if (p.M < 1 || p.M > kFp4SkinnyMaxM) return cudaErrorInvalidValue;
    return X ? launch_any<true>(p, X, ldx, num_sms, status, s) : launch_any<false>(p, nullptr, 0, num_sms, status, s);
}

}  // namespace gemm_gb300
