// Gated block for few rows (M <= 64: single tokens, decode batches): the forward
// projections and dX, bound by reading Wg and Wu [K, N] once.
//
// The operands swap roles: 128 rows of the weights' side are the MMA's M, the M
// rows of X (or of dG and dU) its N = nb (M rounded up to 16; K-major, two boxes of
// 64 k a stage), D[row, m] in nb tensor-memory columns.
//   Forward: a CTA's strip is 64 columns of Z, and the 128 rows are those columns
//   of Wg and the same of Wu (MN-major in shared memory: one 64-column x 128-k box
//   of each per stage).  So tensor-memory lanes 0-63 hold G and 64-127 U of the
//   strip, and both meet in shared memory, where Z is formed.
//   dX = [dG dU] [Wg Wu]^T: a strip is 128 columns of dX, that is 128 rows of Wg
//   and Wu, with the joined index (2N long, two boxes of 64 a stage, K-major) as
//   the reduction.
// The CS CTAs of a cluster share a strip's reduction and add their FP32 partials
// through distributed shared memory in rank order; CS is the largest for which
// every CTA is resident at once, two to an SM.  Deterministic, one launch, no
// workspace.
//
// Every wait is bounded; on expiry a code goes to the status word, the CTA's own
// loads and MMAs are waited for, and its tensor memory is released.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "gated.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

using namespace tc;

constexpr int THREADS = 192;
constexpr int KB = 128;                // k per stage
constexpr int MAX_STAGES = 3;
constexpr int W_BOX = 64 * KB * 2;     // 64 columns x 128 k, or 128 rows x 64: 16 KiB
constexpr int W_STAGE = 2 * W_BOX;
constexpr int RING = 108 * 1024;       // two CTAs to an SM: 3 stages (M <= 16), 2 above
constexpr int SMEM = 1024 + RING + 256;
constexpr uint32_t TMEM_COLS = 64;
constexpr int LD = 128 + 4;            // floats per row of a partial [M][64 G, 64 U]
static_assert(64 * LD * 4 <= RING, "a partial fits the drained ring");

__host__ __device__ constexpr int nb_of(int M) { return (M + 15) / 16 * 16; }
__host__ __device__ constexpr int stages_of(int nb) {
    return RING / (W_STAGE + 2 * nb * 128) < MAX_STAGES ? RING / (W_STAGE + 2 * nb * 128) : MAX_STAGES;
}

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
    void *out;     // Z [M,N], or dX [M,N]
    float *G, *U;  // forward: stored when not null
    int M, N;      // of the output
    int num_kb;    // stages of the reduction (dX: of both halves)
    int kb_half;   // dX: stages of the first half
    int cs;
    // dX: runs beside the dW kernel before it, as in gated.cu (backward of 64 x 1000 x
    // 504 9.8 us from 12.5, 1 x 12288 x 4096 90 from 93)
    int beside;
    int *status;
};

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Forward: tmX = X, tmG = Wg, tmU = Wu.  DX: tmX = {dG, dU} (third coordinate).
template <typename T, uint32_t FORMAT, bool DX, bool GELU>
__global__ void __launch_bounds__(THREADS, 2)
gated_skinny_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ CUtensorMap tmU, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int M = args.M, N = args.N, cs = args.cs;
    const int nb = nb_of(M), stages = stages_of(nb), x_box = nb * 128, x_stage = 2 * x_box;
    uint8_t *w_tiles = smem;
    uint8_t *x_tiles = w_tiles + stages * W_STAGE;
    float *part = reinterpret_cast<float *>(smem);  // [M][LD] once the ring is drained
    Bars *bars = reinterpret_cast<Bars *>(smem + RING);
    volatile int *abort_flag = &bars->abort;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = cs > 1 ? (int)cluster_ctarank() : 0;
    constexpr int STRIP = DX ? 128 : 64;
    const int n0 = (int)(cs > 1 ? cluster_id_x() : blockIdx.x) * STRIP;
    const int num_kb = args.num_kb;
    const int kb0 = (int)((long long)num_kb * rank / cs), kb1 = (int)((long long)num_kb * (rank + 1) / cs);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        mbar_init_fence();
        prefetch_desc(&tmX);
        prefetch_desc(&tmG);
        prefetch_desc(&tmU);
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
            if (DX) {
                const bool second = kb >= args.kb_half;
                const int k0 = (kb - (second ? args.kb_half : 0)) * KB;
                tma_prefetch_l2_3d(second ? &tmU : &tmG, k0, n0, 0);
                tma_prefetch_l2_3d(second ? &tmU : &tmG, k0 + 64, n0, 0);
            } else {
                tma_prefetch_l2_3d(&tmG, n0, kb * KB, 0);
                tma_prefetch_l2_3d(&tmU, n0, kb * KB, 0);
            }
        }
    }
    if (!(DX && args.beside)) pdl_wait();

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        const uint32_t tx = (uint32_t)(W_STAGE + x_stage);
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
            uint8_t *w = w_tiles + stage * W_STAGE, *x = x_tiles + stage * x_stage;
            const int z = DX && kb >= args.kb_half ? 1 : 0, k0 = (kb - (z ? args.kb_half : 0)) * KB;
            if (DX) {
                tma_load_3d(w, z ? &tmU : &tmG, &bars->full[stage], k0, n0, 0);
                tma_load_3d(w + W_BOX, z ? &tmU : &tmG, &bars->full[stage], k0 + 64, n0, 0);
            } else {
                tma_load_3d(w, &tmG, &bars->full[stage], n0, k0, 0);
                tma_load_3d(w + W_BOX, &tmU, &bars->full[stage], n0, k0, 0);
            }
            tma_load_3d(x, &tmX, &bars->full[stage], k0, 0, z);
            tma_load_3d(x + x_box, &tmX, &bars->full[stage], k0 + 64, 0, z);
            ++issued;
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        pdl_launch_dependents();
        for (long long i = (issued > stages ? issued - stages : 0); i < issued; ++i)
            if (!mbar_wait(&bars->full[i % stages], (uint32_t)((i / stages) & 1), abort_flag, false)) {
                atomicOr(args.status, ST_DRAIN);
                break;
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // A = the weights, MN-major: 64-column boxes W_BOX bytes apart, a K step of
        // 16 rows is 2048 bytes (DX: K-major, as B).  B = X, K-major: a K step is 32
        // bytes of a row, the second 64 k in the next box.
        const bool issuer = elect_one();
        const uint32_t idesc = (1u << 4) | (FORMAT << 7) | (FORMAT << 10) | ((DX ? 0u : 1u) << 15) | (((uint32_t)nb >> 3) << 17) |
                               ((128u >> 4) << 24);
        const uint64_t w_desc0 = desc_sw128(smem_u32(w_tiles), DX ? 16 : W_BOX, 1024);
        const uint64_t x_desc0 = desc_sw128(smem_u32(x_tiles), 16, 1024);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&bars->full[stage], phase, abort_flag, true)) { ok = false; break; }
            fence_after();
            const uint64_t wd = w_desc0 + (uint64_t)((stage * W_STAGE) >> 4);
            const uint64_t xd = x_desc0 + (uint64_t)((stage * x_stage) >> 4);
            const uint64_t xd1 = xd + (uint64_t)(x_box >> 4);
            if (issuer) {
#pragma unroll
                for (int ks = 0; ks < KB / 16; ++ks)
                    mma_f16(tmem_base, wd + (DX ? (ks >> 2) * (W_BOX >> 4) + (ks & 3) * 2 : ks * (2048 >> 4)), (ks < 4 ? xd : xd1) + (ks & 3) * 2, idesc,
                            (uint32_t)(kb != kb0 || ks != 0));
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
        // ------------------------------------------------------------ partial to shared memory
        const int quarter = warp & 3, nl = quarter * 32 + lane;
        const bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full, 0, abort_flag, true));
        if (!ok && lane == 0) {
            atomicOr(args.status, ST_EPILOGUE);
            *abort_flag = 1;
        }
        fence_after();
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < M; c += 32) {
            uint32_t r[32];
            if (ok) {
                tmem_ld32(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = 0u;
            }
            // (the ring is drained: every MMA that read it has completed)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j < M) part[(c + j) * LD + nl] = __uint_as_float(r[j]);
        }
    }

    fence_before();
    __syncwarp();
    if (cs > 1) cluster_sync();
    else __syncthreads();
    {
        // (row, four columns) pairs dealt out to the CTAs in equal ranges; partials added in rank order
        const int groups = min(STRIP, N - n0) / 4;  // N % 8 == 0
        const int total = M * groups;
        const int e1 = (int)((long long)total * (rank + 1) / cs);
        for (int e = (int)((long long)total * rank / cs) + (int)threadIdx.x; e < e1; e += THREADS) {
            const int m = e / groups, c4 = (e - m * groups) * 4;
            const float *at = part + m * LD + c4;
            constexpr int NV = DX ? 1 : 2;  // a sum, or G and U 64 floats apart
            float4 v[NV];
            if (cs == 1) {
#pragma unroll
                for (int q = 0; q < NV; ++q) v[q] = *reinterpret_cast<const float4 *>(at + 64 * q);
            } else {
                float4 p[8][NV];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < cs) {
                        const uint32_t a = map_to_rank(at, (uint32_t)j);
#pragma unroll
                        for (int q = 0; q < NV; ++q) p[j][q] = ld_cluster_f4(a + 256 * q);
                    }
#pragma unroll
                for (int q = 0; q < NV; ++q) v[q] = p[0][q];
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    if (j < cs) {
#pragma unroll
                        for (int q = 0; q < NV; ++q) {
                            v[q].x += p[j][q].x; v[q].y += p[j][q].y; v[q].z += p[j][q].z; v[q].w += p[j][q].w;
                        }
                    }
            }
            const size_t o = (size_t)m * N + n0 + c4;
            const float4 g = v[0];
            uint2 w;
            if constexpr (DX) {
                w.x = pack2(g.x, g.y, (T *)nullptr);
                w.y = pack2(g.z, g.w, (T *)nullptr);
            } else {
                const float4 u = v[NV - 1];
                if (args.G) {
                    *reinterpret_cast<float4 *>(args.G + o) = g;
                    *reinterpret_cast<float4 *>(args.U + o) = u;
                }
                w.x = pack2(gate_act<GELU>(g.x) * u.x, gate_act<GELU>(g.y) * u.y, (T *)nullptr);
                w.y = pack2(gate_act<GELU>(g.z) * u.z, gate_act<GELU>(g.w) * u.w, (T *)nullptr);
            }
            *reinterpret_cast<uint2 *>(static_cast<T *>(args.out) + o) = w;
        }
    }
    __syncwarp();
    if (cs > 1) cluster_sync();  // every CTA keeps its shared memory until the others have read it
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem_base, TMEM_COLS);
    }
    if (DX && args.beside) pdl_wait();
}

template <typename T, uint32_t FORMAT, bool DX, bool GELU>
int clusters_max(int dev, int cs) {
    static std::atomic<int> known[kMaxDevices][9];
    return cluster_limit(known[dev][cs], reinterpret_cast<const void *>(gated_skinny_kernel<T, FORMAT, DX, GELU>),
                         THREADS, SMEM, cs);
}

constexpr CUtensorMapDataType map_type(uint32_t format) {
    return format == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

template <typename T, uint32_t FORMAT, bool DX, bool GELU>
cudaError_t launch(const CUtensorMap &tx, const CUtensorMap &tg, const CUtensorMap &tu, Args a, int num_sms,
                   cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    constexpr int STRIP = DX ? 128 : 64;
    const long long strips = (a.N + STRIP - 1LL) / STRIP;
    if (clusters_max<T, FORMAT, DX, GELU>(dev, 1) <= 0) return cudaErrorNotSupported;
    int cs = 1;
    for (int c = 2; c <= 8 && c <= a.num_kb && strips * c <= 2LL * num_sms; ++c) {
        const int n = clusters_max<T, FORMAT, DX, GELU>(dev, c);
        if (n < 0) return cudaErrorNotSupported;  // not another split, whose sums would differ
        if (n >= strips) cs = c;
    }
    a.cs = cs;
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
    return launch_counted(&cfg, gated_skinny_kernel<T, FORMAT, DX, GELU>, tx, tg, tu, a);
}

template <typename T, uint32_t FORMAT>
cudaError_t forward(const GatedProblem &p, int num_sms, int *status, cudaStream_t s) {
    constexpr auto dt = map_type(FORMAT);
    const long long xr = 2 * p.ldx, wr = 2LL * p.N;
    CUtensorMap tx, tg, tu;
    if (!make_map3(&tx, p.X, dt, p.K, p.M, 1, xr, xr * p.M, 64, nb_of(p.M), 1, 128) ||
        !make_map3(&tg, p.Wg, dt, p.N, p.K, 1, wr, wr * p.K, 64, KB, 1, 128) ||
        !make_map3(&tu, p.Wu, dt, p.N, p.K, 1, wr, wr * p.K, 64, KB, 1, 128))
        return cudaErrorInvalidValue;
    Args a = {};
    a.out = p.Z;
    a.G = p.G;
    a.U = p.U;
    a.M = p.M;
    a.N = p.N;
    a.num_kb = (p.K + KB - 1) / KB;
    a.status = status;
    return p.gelu ? launch<T, FORMAT, false, true>(tx, tg, tu, a, num_sms, s)
                  : launch<T, FORMAT, false, false>(tx, tg, tu, a, num_sms, s);
}

template <typename T, uint32_t FORMAT>
cudaError_t grad_x(const GatedBackward &p, const void *dGU, bool beside, int num_sms, int *status, cudaStream_t s) {
    constexpr auto dt = map_type(FORMAT);
    const long long wr = 2LL * p.N, gr = 2 * gated_ldg(p.N);
    CUtensorMap tx, tg, tu;
    if (!make_map3(&tx, dGU, dt, p.N, p.M, 2, gr, gr * p.M, 64, nb_of(p.M), 1, 128) ||
        !make_map3(&tg, p.Wg, dt, p.N, p.K, 1, wr, wr * p.K, 64, 128, 1, 128) ||
        !make_map3(&tu, p.Wu, dt, p.N, p.K, 1, wr, wr * p.K, 64, 128, 1, 128))
        return cudaErrorInvalidValue;
    Args a = {};
    a.out = p.dX;
    a.M = p.M;
    a.N = p.K;
    a.kb_half = (p.N + KB - 1) / KB;
    a.num_kb = 2 * a.kb_half;
    a.beside = beside;
    a.status = status;
    return launch<T, FORMAT, true, false>(tx, tg, tu, a, num_sms, s);
}

}  // namespace

cudaError_t launch_gated_skinny(const GatedProblem &p, int num_sms, int *status, cudaStream_t s) {
    if (p.M < 1 || p.M > kGatedSkinnyMaxM) return cudaErrorInvalidValue;
    return p.elt == Elt::BF16 ? forward<__nv_bfloat16, 1>(p, num_sms, status, s)
                              : forward<__half, 0>(p, num_sms, status, s);
}

cudaError_t launch_gated_skinny_dx(const GatedBackward &p, const void *dGU, bool beside, int num_sms, int *status,
                                   cudaStream_t s) {
    if (p.M < 1 || p.M > kGatedSkinnyMaxM) return cudaErrorInvalidValue;
    return p.elt == Elt::BF16 ? grad_x<__nv_bfloat16, 1>(p, dGU, beside, num_sms, status, s)
                              : grad_x<__half, 0>(p, dGU, beside, num_sms, status, s);
}

}  // namespace gemm_gb300
