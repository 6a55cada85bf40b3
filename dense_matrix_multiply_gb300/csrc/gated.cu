// Gated feed-forward block on the tensor cores, forward and backward:
//     G = X Wg, U = X Wu, Z = act(G) * U
//     dU = dZ * act(G), dG = dZ * U * act'(G)
//     dX = dG Wg^T + dU Wu^T, dWg = X^T dG, dWu = X^T dU
//
// Forward: one kernel.  A 256 x 128 tile of Z belongs to a cluster of two CTAs
// (tcgen05 cta_group::2); per K step of 64 CTA r loads 64 columns of Wg and the
// same 64 of Wu side by side, so that one N = 256 MMA gives G and U for the same
// columns of Z in one accumulator, and the epilogue forms Z from the FP32 sums,
// rounded once.  (Few tiles: 256 x 64 ones, for which CTA 0 loads Wg's columns and
// CTA 1 Wu's, N = 128.)  For training it also stores G and U, in FP32: a 16-bit copy would
// put a third rounding beside those of dG and dU and of the result on every
// gradient (1.7 times the error of the result's rounding, against 1.4).
//
// Backward: dG and dU (16 bits, the operands of the products to come) from G, U
// and dZ in one pass over memory; dX as one product over the joined reduction
// index of dG Wg^T and dU Wu^T (2N long), 256 x bn tiles on the same pair
// pipeline, FP32 sums of both in one accumulator; dWg and dWu in one launch over
// the tiles of both, 256 x 256, X and the gradients as they are stored (both
// operands MN-major).
//
// A last wave of tiles that would leave at least half of the clusters idle is split
// along K (plan()): FP32 partials go to scratch and are added, in order, by
// gated_fix_kernel.  The clusters of one split walk the same K range together, so
// that operands are still read from memory once (shares cut tile after tile, each
// cluster at a K of its own, took dX of 1024 x 12288 x 4096 from 145 us to 214).
//
// Warps: 0 loads (TMA), 1 issues the MMAs (leader) -- both converged, with one
// elected lane for the instructions, so that operands stay in uniform registers --
// and 2-9 write out, half of the tile's columns to each four.  Two accumulators,
// so that a tile is written while the next one is computed.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "gated.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

using namespace tc;

constexpr int THREADS = 320, EPI_WARPS = 8;
constexpr int BK = 64;                 // 16-bit k per stage: 128 bytes a row
constexpr int A_STAGE = 128 * BK * 2;  // 16 KiB per CTA
constexpr int B_STAGE = 128 * BK * 2;
constexpr int BOX64 = 64 * BK * 2;     // 64 columns x 64 k of an MN-major tile
constexpr int STG_BOX = 4096;          // 32 rows x 128 bytes of output
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP_M = 8;

// Two staging boxes per epilogue warp and five stages where a tile's output is
// much against its stages (Z, G and U; dW over few rows), one and six for dX.
enum Mode { FWD = 0, DX = 1, DW = 2 };
__host__ __device__ constexpr int n_boxes(int mode) { return mode == DX ? 1 : 2; }
__host__ __device__ constexpr int n_stages(int mode) { return mode == DX ? 6 : 5; }
__host__ __device__ constexpr int staging_bytes(int mode) { return EPI_WARPS * n_boxes(mode) * STG_BOX; }
__host__ __device__ constexpr int smem_bytes(int mode) {
    return 1024 + n_stages(mode) * (A_STAGE + B_STAGE) + staging_bytes(mode) + 256;
}
static_assert(smem_bytes(FWD) <= 232448 && smem_bytes(DX) <= 232448, "shared memory budget");

struct Bars {
    uint64_t full[6];
    uint64_t empty[6];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint64_t peer_done;
    long long peer_issued;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Args {
    int M, N;     // of the output: Z, dX or a dW
    int num_kb;   // K blocks of 64 (DX: of both halves together)
    int kb_half;  // DX: blocks of the first half
    int bn;       // the tile's N extent: FWD 128 or 64; DX 64, 128, 192 or 256; DW 256
    int batch;    // DW: outputs, 1 or 2; else 1
    int save;     // FWD: store G and U
    int whole;    // tiles computed whole; the rest are split
    int splits;   // in so many K ranges, one to a cluster
    int beside;   // DX: runs beside the dW kernel before it (below)
    int *status;
};

__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// FP32 accumulator, A and B of one 16-bit type (0 f16, 1 bf16), M = 256.
__device__ __forceinline__ uint32_t make_idesc(uint32_t format, uint32_t n, bool a_mn, bool b_mn) {
    return (1u << 4) | (format << 7) | (format << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((256u >> 4) << 24);
}

// A tile of the output: which output (DW), row and column of tiles.
struct Tile {
    int z, m, n;
};
__device__ __forceinline__ Tile tile_at(int t, int tiles_m, int tiles_n) {
    Tile r;
    r.z = t / (tiles_m * tiles_n);
    t -= r.z * tiles_m * tiles_n;
    const int per_group = GROUP_M * tiles_n;
    const int group = t / per_group;
    const int first_m = group * GROUP_M;
    const int gsize = min(tiles_m - first_m, GROUP_M);
    const int q = t - group * per_group;
    r.m = first_m + q % gsize;
    r.n = q / gsize;
    return r;
}
// Unit u of cluster c of G: the whole tiles c, c + G, ... first (slab -1), then,
// for c < (tiles - whole) * splits, K range c / (tiles - whole) of split tile
// c % (tiles - whole), whose partial is slab c.  Every warp walks the same sequence.
struct Unit {
    int t, kb0, kb1, slab;
};
__device__ __forceinline__ bool unit_at(int u, int c, int G, int tiles, const Args &a, Unit &r) {
    const int n = c < a.whole ? (a.whole - 1 - c) / G + 1 : 0, rest = tiles - a.whole;
    if (u < n) {
        r = {c + u * G, 0, a.num_kb, -1};
        return true;
    }
    if (u > n || c >= rest * a.splits) return false;
    const int j = c / rest;
    r.t = a.whole + c - j * rest;
    r.kb0 = (int)((long long)a.num_kb * j / a.splits);
    r.kb1 = (int)((long long)a.num_kb * (j + 1) / a.splits);
    r.slab = c;
    return true;
}

// 32 FP32 columns of this lane's row to a box, 128-byte swizzle.
__device__ __forceinline__ void box_put_f32(uint8_t *box, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
}

// FWD: tmA = X, tmB = Wg, tmB2 = Wu, tmC = Z, tmG, tmU (when saved).
// DX: tmA = {dG, dU} (third coordinate), tmB = Wg, tmB2 = Wu, tmC = dX.
// DW: tmA = X, tmB = {dG, dU}, tmC and tmG the outputs of its two matrices.
// tmP: the partials, slabs of 256 x 256 accumulators.
template <typename T, uint32_t FORMAT, int MODE, bool GELU>
__global__ void __launch_bounds__(THREADS, 1)
gated_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tmC,
                  const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
                  const __grid_constant__ CUtensorMap tmP, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int STAGES = n_stages(MODE), BOXES = n_boxes(MODE);
    uint8_t *a_tiles = smem;
    uint8_t *b_tiles = a_tiles + STAGES * A_STAGE;
    uint8_t *staging = b_tiles + STAGES * B_STAGE;
    Bars *bars = reinterpret_cast<Bars *>(staging + staging_bytes(MODE));
    volatile int *abort_flag = &bars->abort;

    const int M = args.M, N = args.N, bn = args.bn;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = (int)cluster_id_x(), nclusters = (int)cluster_count_x();
    const int tiles_m = (M + 255) / 256, tiles_n = (N + bn - 1) / bn;
    const int tiles = tiles_m * tiles_n * args.batch;
    const bool thin = MODE == FWD && bn == 64;
    const uint32_t stage_tx = 2u * (uint32_t)(A_STAGE + (MODE == DX ? (bn >> 1) * 128 : thin ? BOX64 : 2 * BOX64));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 2 * EPI_WARPS);
        }
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->peer_done, 1);
        bars->abort = 0;
        mbar_init_fence();
        prefetch_desc(&tmA);
        prefetch_desc(&tmB);
        prefetch_desc(&tmB2);
        prefetch_desc(&tmC);
    }
    if (warp == 1) tmem_alloc<2>(&bars->tmem_base, TMEM_COLS);
    fence_before();
    cluster_sync();  // barriers of both CTAs initialised before any cross-CTA use
    fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    // The backward pass launches dW, then dX, which reads nothing that dW writes: dW
    // lets its dependent start only after its own wait, so that dG and dU, written by the
    // grid before dW, are complete by then, and dX (args.beside; gated_skinny.cu's too)
    // begins at once, on the SMs that dW leaves, without a wait of its own (internal.h),
    // and waits for dW before it ends, so that whatever follows finds both.
    // Backward of 1024 x 12288 x 4096 270 us against 282 one after the other, 128 x
    // 12288 x 4096 108 against 114.
    if (MODE == DW) {
        pdl_wait();
        pdl_launch_dependents();
    } else {
        pdl_launch_dependents();
        if (!(MODE == DX && args.beside)) pdl_wait();
    }

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        // The whole warp runs the loop (operands in uniform registers), one lane issues.
        const bool issuer = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        Unit w;
        for (int u = 0; ok && unit_at(u, cluster, nclusters, tiles, args, w); ++u) {
            const Tile t = tile_at(w.t, tiles_m, tiles_n);
            const int row0 = t.m * 256 + (int)rank * 128, col0 = t.n * bn + (int)rank * (bn >> 1);
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag, true)) { ok = false; break; }
                const uint32_t full = map_to_rank(&bars->full[stage], 0);
                uint8_t *a = a_tiles + stage * A_STAGE, *b = b_tiles + stage * B_STAGE;
                if (issuer) {
                    if (leader) mbar_arrive_expect_tx(&bars->full[stage], stage_tx);
                    if (MODE == FWD) {
                        tma_load_3d_pair(a, &tmA, full, kb * BK, row0, 0);
                        if (thin) {
                            tma_load_3d_pair(b, leader ? &tmB : &tmB2, full, t.n * 64, kb * BK, 0);
                        } else {
                            tma_load_3d_pair(b, &tmB, full, col0, kb * BK, 0);
                            tma_load_3d_pair(b + BOX64, &tmB2, full, col0, kb * BK, 0);
                        }
                    } else if (MODE == DW) {
                        tma_load_3d_pair(a, &tmA, full, row0, kb * BK, 0);
                        tma_load_3d_pair(a + BOX64, &tmA, full, row0 + 64, kb * BK, 0);
                        tma_load_3d_pair(b, &tmB, full, col0, kb * BK, t.z);
                        tma_load_3d_pair(b + BOX64, &tmB, full, col0 + 64, kb * BK, t.z);
                    } else {
                        const int z = kb >= args.kb_half ? 1 : 0, k0 = (kb - z * args.kb_half) * BK;
                        tma_load_3d_pair(a, &tmA, full, k0, row0, z);
                        tma_load_3d_pair(b, z ? &tmB2 : &tmB, full, k0, col0, 0);
                    }
                }
                ++issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        if (!ok && issuer) {
            atomicOr(args.status, ST_PRODUCER);
            raise_abort_pair(abort_flag, rank);
        }
        // No load is left in flight into either CTA when the pair ends: the peer
        // tells the leader how many stages it loaded, and the leader waits until
        // every stage that either loaded has landed (the half that a side which
        // gave up never loaded is counted as done, or never armed).
        if (!issuer) {
        } else if (!leader) {
            st_cluster_s64(map_to_rank(&bars->peer_issued, 0), issued);
            mbar_arrive_cluster(map_to_rank(&bars->peer_done, 0));  // release: the count is visible first
        } else {
            long long ip = issued;
            if (mbar_wait(&bars->peer_done, 0, abort_flag, false))
                ip = *reinterpret_cast<volatile long long *>(&bars->peer_issued);
            else
                atomicOr(args.status, ST_DRAIN);
            const long long hi = issued > ip ? issued : ip;
            for (long long i = (hi > STAGES ? hi - STAGES : 0); i < hi; ++i) {
                const int s = (int)(i % STAGES);
                if (i >= issued) mbar_arrive_expect_tx(&bars->full[s], stage_tx / 2);
                else if (i >= ip) mbar_complete_tx(&bars->full[s], stage_tx / 2);
                if (!mbar_wait(&bars->full[s], (uint32_t)((i / STAGES) & 1), abort_flag, false)) {
                    atomicOr(args.status, ST_DRAIN);
                    break;
                }
            }
        }
    } else if (warp == 1 && leader) {
        // ------------------------------------------------------------ MMA issuer (leader)
        // The whole warp runs the loop (descriptors in uniform registers), one lane issues.
        const bool issuer = elect_one();
        // K-major: a K step of 16 is 32 bytes of a 128-byte row.  MN-major: 16 rows of
        // 128 bytes, 64-element boxes BOX64 bytes apart.
        constexpr bool a_mn = MODE == DW, b_mn = MODE != DX;
        const uint32_t idesc = make_idesc(FORMAT, MODE == DX ? (uint32_t)bn : thin ? 128u : 256u, a_mn, b_mn);
        const uint64_t a_desc0 = desc_sw128(smem_u32(a_tiles), a_mn ? BOX64 : 16, 1024);
        const uint64_t b_desc0 = desc_sw128(smem_u32(b_tiles), b_mn ? BOX64 : 16, 1024);
        constexpr uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        int stage = 0;
        uint32_t phase = 0;
        int it = 0;
        bool ok = true;
        Unit w;
        for (int u = 0; ok && unit_at(u, cluster, nclusters, tiles, args, w); ++u, ++it) {
            const int buf = it & 1;
            if (!mbar_wait(&bars->acc_empty[buf], (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag, true)) { ok = false; break; }
            fence_after();
            const uint32_t d = tmem_base + (uint32_t)(buf * 256);
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!mbar_wait(&bars->full[stage], phase, abort_flag, true)) { ok = false; break; }
                fence_after();
                const uint64_t ad = a_desc0 + (uint64_t)((stage * A_STAGE) >> 4);
                const uint64_t bd = b_desc0 + (uint64_t)((stage * B_STAGE) >> 4);
                if (issuer) {
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ++ks)
                        mma_f16_pair(d, ad + ks * a_step, bd + ks * b_step, idesc, (uint32_t)(kb != w.kb0 || ks != 0));
                    commit_pair_multicast(&bars->empty[stage]);
                }
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (issuer) commit_pair_multicast(&bars->acc_full[buf]);
        }
        if (issuer) {
            if (!ok) {
                atomicOr(args.status, ST_MMA);
                raise_abort_pair(abort_flag, rank);
            }
            commit<2>(&bars->drain);
            if (!mbar_wait(&bars->drain, 0, abort_flag, false)) atomicOr(args.status, ST_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t *my_stg = staging + (warp - 2) * BOXES * STG_BOX;
        int sb = 0, it = 0;
        bool ok = true;
        // The next staging box, once the store that last read it has done so.
        auto box_begin = [&]() {
            if (lane == 0) {
                if constexpr (BOXES == 2) tma_stores_read_wait1();
                else tma_stores_read_wait0();
            }
            __syncwarp();
            uint8_t *b = my_stg + sb * STG_BOX;
            if (BOXES == 2) sb ^= 1;
            return b;
        };
        auto box_end = [&](const CUtensorMap *map, uint8_t *b, int x, int y, int z) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && y < M) tma_store_3d(map, b, x, y, z);
        };
        Unit w;
        for (int u = 0; unit_at(u, cluster, nclusters, tiles, args, w); ++u, ++it) {
            const Tile t = tile_at(w.t, tiles_m, tiles_n);
            const int buf = it & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->acc_full[buf], (uint32_t)((it >> 1) & 1), abort_flag, true))) {
                ok = false;
                break;
            }
            fence_after();
            __syncwarp();
            const int row0 = t.m * 256 + (int)rank * 128 + quarter * 32;
            const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * 256);
            if (w.slab >= 0) {
                // a partial: the accumulators as they are
                const int chunks = (MODE == FWD ? 2 * bn : bn) / 32, mid = (chunks + 1) >> 1;
#pragma unroll 1
                for (int c = half ? mid : 0; c < (half ? chunks : mid); ++c) {
                    uint32_t r[32];
                    tmem_ld32(t_row + (uint32_t)(c * 32), r);
                    tmem_ld_wait();
                    uint8_t *b = box_begin();
                    box_put_f32(b, lane, r);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && row0 < M) tma_store_3d(&tmP, b, c * 32, (int)rank * 128 + quarter * 32, w.slab);
                }
            } else if (thin) {
                // columns 0-63: G, 64-127: U; 32 of them to each half
                const int c0 = t.n * 64 + half * 32;
                if (c0 < N) {  // warp-uniform
                    uint32_t rg[32], ru[32];
                    tmem_ld32(t_row + (uint32_t)(half * 32), rg);
                    tmem_ld32(t_row + (uint32_t)(64 + half * 32), ru);
                    tmem_ld_wait();
                    if (args.save) {
                        uint8_t *b = box_begin();
                        box_put_f32(b, lane, rg);
                        box_end(&tmG, b, c0, row0, 0);
                        b = box_begin();
                        box_put_f32(b, lane, ru);
                        box_end(&tmU, b, c0, row0, 0);
                    }
                    uint32_t z[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        z[j] = pack2(gate_act<GELU>(__uint_as_float(rg[2 * j])) * __uint_as_float(ru[2 * j]),
                                     gate_act<GELU>(__uint_as_float(rg[2 * j + 1])) * __uint_as_float(ru[2 * j + 1]),
                                     (T *)nullptr);
                    uint8_t *b = box_begin();
#pragma unroll
                    for (int c = 0; c < 4; ++c)  // 64 bytes a row, the 64-byte swizzle
                        *reinterpret_cast<uint4 *>(b + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(z[4 * c], z[4 * c + 1], z[4 * c + 2], z[4 * c + 3]);
                    box_end(&tmC, b, c0, row0, 0);
                }
            } else if constexpr (MODE == FWD) {
                // accumulator columns 128 g + j: G, 128 g + 64 + j: U of Z's column 64 g + j
                const int g = half, c0 = t.n * 128 + g * 64;
                if (c0 < N) {  // warp-uniform
                    uint32_t z[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t rg[32], ru[32];
                        tmem_ld32(t_row + (uint32_t)(g * 128 + h * 32), rg);
                        tmem_ld32(t_row + (uint32_t)(g * 128 + 64 + h * 32), ru);
                        tmem_ld_wait();
                        if (args.save && c0 + h * 32 < N) {
                            uint8_t *b = box_begin();
                            box_put_f32(b, lane, rg);
                            box_end(&tmG, b, c0 + h * 32, row0, 0);
                            b = box_begin();
                            box_put_f32(b, lane, ru);
                            box_end(&tmU, b, c0 + h * 32, row0, 0);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            z[h * 16 + j] = pack2(gate_act<GELU>(__uint_as_float(rg[2 * j])) * __uint_as_float(ru[2 * j]),
                                                  gate_act<GELU>(__uint_as_float(rg[2 * j + 1])) * __uint_as_float(ru[2 * j + 1]),
                                                  (T *)nullptr);
                    }
                    uint8_t *b = box_begin();
                    box_put_f32(b, lane, z);
                    box_end(&tmC, b, c0, row0, 0);
                }
            } else {
                const int groups = bn >> 6, mid = (groups + 1) >> 1;  // of 64 columns; this half's first or last
#pragma unroll 1
                for (int g = half ? mid : 0; g < (half ? groups : mid); ++g) {
                    const int c0 = t.n * bn + g * 64;
                    if (c0 >= N) break;  // warp-uniform
                    uint32_t r0[32], r1[32];
                    tmem_ld32(t_row + (uint32_t)(g * 64), r0);
                    tmem_ld32(t_row + (uint32_t)(g * 64 + 32), r1);
                    tmem_ld_wait();
                    uint32_t z[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        z[j] = pack2(__uint_as_float(r0[2 * j]), __uint_as_float(r0[2 * j + 1]), (T *)nullptr);
                        z[16 + j] = pack2(__uint_as_float(r1[2 * j]), __uint_as_float(r1[2 * j + 1]), (T *)nullptr);
                    }
                    uint8_t *b = box_begin();
                    box_put_f32(b, lane, z);
                    box_end(MODE == DW && t.z ? &tmG : &tmC, b, c0, row0, 0);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(&bars->acc_empty[buf], 0));
        }
        if (lane == 0) tma_stores_wait0();
        if (!ok && lane == 0) {
            atomicOr(args.status, ST_EPILOGUE);
            raise_abort_pair(abort_flag, rank);
        }
    }

    __syncwarp();
    fence_before();
    cluster_sync();  // no CTA leaves while its peer may still touch its memory
    if (warp == 1) {
        fence_after();
        tmem_dealloc<2>(tmem_base, TMEM_COLS);
    }
    if (MODE == DX && args.beside) pdl_wait();
}

__device__ __forceinline__ float2 unpack(uint32_t v, const __nv_bfloat16 *) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t v, const __half *) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }

// dG and dU from G, U and dZ, four times four elements to a thread (every load and
// store a full line across the warp): 10 bytes read and 4 written an element.  G, U
// and dZ lie without gaps, dG's and dU's rows are `pad` units further apart.
constexpr int GRAD_UNITS = 4;
template <typename T, bool GELU>
__global__ void __launch_bounds__(256)
gated_grad_kernel(const float4 *__restrict__ G, const float4 *__restrict__ U, const uint2 *__restrict__ dZ,
                  uint2 *__restrict__ dG, uint2 *__restrict__ dU, long long n4, uint32_t n4_row, uint32_t pad)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long i0 = (long long)blockIdx.x * (256 * GRAD_UNITS) + threadIdx.x;
    float4 g[GRAD_UNITS], u[GRAD_UNITS];
    uint2 z[GRAD_UNITS];
#pragma unroll
    for (int j = 0; j < GRAD_UNITS; ++j) {
        const long long i = i0 + j * 256;
        if (i < n4) {
            g[j] = __ldcs(G + i);
            u[j] = __ldcs(U + i);
            z[j] = __ldcs(dZ + i);
        }
    }
#pragma unroll
    for (int j = 0; j < GRAD_UNITS; ++j) {
        const long long i = i0 + j * 256;
        if (i >= n4) break;
        const float2 d0 = unpack(z[j].x, (const T *)nullptr), d1 = unpack(z[j].y, (const T *)nullptr);
        float a[4], da[4];
        gate_act_grad<GELU>(g[j].x, a[0], da[0]);
        gate_act_grad<GELU>(g[j].y, a[1], da[1]);
        gate_act_grad<GELU>(g[j].z, a[2], da[2]);
        gate_act_grad<GELU>(g[j].w, a[3], da[3]);
        const long long row = pad == 0 ? 0 : n4 <= 0xFFFFFFFFLL ? (uint32_t)i / n4_row : i / n4_row;
        const long long o = i + row * pad;
        dU[o] = make_uint2(pack2(d0.x * a[0], d0.y * a[1], (T *)nullptr), pack2(d1.x * a[2], d1.y * a[3], (T *)nullptr));
        dG[o] = make_uint2(pack2(d0.x * u[j].x * da[0], d0.y * u[j].y * da[1], (T *)nullptr),
                           pack2(d1.x * u[j].z * da[2], d1.y * u[j].w * da[3], (T *)nullptr));
    }
}

// The split tiles: each is the sum of its partials, in K order, through the
// epilogue of its mode.  Block (x, y, z): rows 8 x .. 8 x + 7 and columns 128 z ..
// 128 z + 127 of split tile y, four columns to a lane (FWD: G and U lie 64
// accumulators apart).
template <typename T, int MODE, bool GELU>
__global__ void __launch_bounds__(256)
gated_fix_kernel(const float *__restrict__ part, T *out0, T *out1, float *G, float *U, const Args a)
{
    pdl_wait();
    const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + a.bn - 1) / a.bn;
    const int k = (int)blockIdx.y;
    const Tile t = tile_at(a.whole + k, tiles_m, tiles_n);
    const int r = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int row = t.m * 256 + r;
    if (row >= a.M) return;
    const size_t next = (size_t)gridDim.y * 256 * 256;  // the next split's partial of this tile
    const int j = (int)blockIdx.z * 128 + lane * 4, col = t.n * a.bn + j;
    if (j >= a.bn || col >= a.N) return;
    const int acc = MODE == FWD ? (j >> 6) * 128 + (j & 63) : j;
    const float *p = part + ((size_t)k * 256 + r) * 256 + acc;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f), u = s;
#pragma unroll 8
    for (int c = 0; c < a.splits; ++c) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + c * next));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        if (MODE == FWD) {
            const float4 w = __ldcg(reinterpret_cast<const float4 *>(p + c * next + 64));
            u.x += w.x; u.y += w.y; u.z += w.z; u.w += w.w;
        }
    }
    const size_t o = (size_t)row * a.N + col;
    if (MODE == FWD) {
        if (a.save) {
            *reinterpret_cast<float4 *>(G + o) = s;
            *reinterpret_cast<float4 *>(U + o) = u;
        }
        s.x = gate_act<GELU>(s.x) * u.x;
        s.y = gate_act<GELU>(s.y) * u.y;
        s.z = gate_act<GELU>(s.z) * u.z;
        s.w = gate_act<GELU>(s.w) * u.w;
    }
    *reinterpret_cast<uint2 *>((t.z ? out1 : out0) + o) =
        make_uint2(pack2(s.x, s.y, (T *)nullptr), pack2(s.z, s.w, (T *)nullptr));
}

template <typename T, uint32_t FORMAT, int MODE, bool GELU>
int clusters_max(int dev) {
    static std::atomic<int> known[kMaxDevices];
    return cluster_limit(known[dev], reinterpret_cast<const void *>(gated_pair_kernel<T, FORMAT, MODE, GELU>), THREADS,
                         smem_bytes(MODE), 2);
}

constexpr CUtensorMapDataType map_type(uint32_t format) {
    return format == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
// A row-major 16-bit matrix [rows, cols], rows ld elements apart; z of them, one after the other.
bool map16(CUtensorMap *m, const void *p, uint32_t format, long long rows, long long cols, int box_cols, int box_rows,
           long long ld, int z) {
    return make_map3(m, p, map_type(format), cols, rows, z, ld * 2, rows * ld * 2, box_cols, box_rows, 1, 128);
}
bool map16(CUtensorMap *m, const void *p, uint32_t format, long long rows, long long cols, int box_cols, int box_rows) {
    return map16(m, p, format, rows, cols, box_cols, box_rows, cols, 1);
}

// How the tiles go to the clusters.  Whole waves of tiles first; the rest is split
// when that saves more than the partials and the second kernel cost; a split is
// eight blocks at least.  Times are in 256ths of a K block of a 256 x 256
// accumulator, 0.3 us.  Measured, forward: 1024 x 12288 x
// 4096 (384 tiles on 76 clusters) 112 us against 120 with whole tiles, 128 x 12288 x
// 4096 (96 tiles) 46.8 against 51.8; dX of 777 x 11008 x 4096 in 64 whole tiles
// 113 us, in 76 of 192 columns and 12 split in six 120.
// Partials and the second kernel: 4.2 us, and 0.06 a partial of 256 columns.
constexpr long long fix_time(long long slabs, int columns) { return 14 * 256 + slabs * columns / 5; }
// Blocks of narrower accumulators: dX of 128 x 12288 x 4096 in one wave takes 0.27 us
// a block at 256 columns, 0.22 at 192 and 0.205 at 128, forward 1024 x 12160 x 4096
// 0.33 at 256 and 0.23 at 128; at 64 (dX of 333 x 1000 x 1000 10.8 us, at 128 11.9;
// 700 x 2816 x 1024 takes wider ones) by what is loaded.  Where rows of neither
// operand start on 128 bytes, TMA asks L2 for two lines for most of a box's rows, and
// that bounds the blocks: forward of 1024 x 12280 x 4088 165 us, where 1024 x 12288 x
// 4088 and 1024 x 12280 x 4096, with one such operand, take 122 and 1024 x 12288 x 4096
// 114.
constexpr int block_time(int columns, bool rows_on_128) {
    return (columns == 256 ? 256 : columns == 192 ? 208 : columns == 128 ? 180 : 150) * (rows_on_128 ? 5 : 8) / 5;
}
struct Plan {
    long long tiles, time;
    int clusters, whole, splits;
};
// `columns`: of a tile's accumulator; rows_on_128: of one operand at least.
Plan plan(long long tiles, int cmax, long long num_kb, int columns, bool rows_on_128) {
    const int block = block_time(columns, rows_on_128);
    const long long waves = tiles / cmax, rem = tiles - waves * cmax;
    Plan p = {tiles, (waves + (rem > 0)) * num_kb * block, (int)std::min<long long>(tiles, cmax), (int)tiles, 1};
    if (rem == 0) return p;
    const long long splits = std::min<long long>({cmax / rem, num_kb / 8, 16});
    const long long fix = fix_time(rem * splits, columns);
    if (splits < 2 || (num_kb - num_kb / splits) * block < fix) return p;
    p.time = (waves * num_kb + num_kb / splits) * block + fix;
    p.whole = (int)(waves * cmax);
    p.splits = (int)splits;
    p.clusters = waves > 0 ? cmax : (int)(rem * splits);
    return p;
}
// A plan's partials: 256 x 256 FP32 slabs.
long long plan_slabs(const Plan &p) { return p.splits > 1 ? (p.tiles - p.whole) * p.splits : 0; }
size_t plan_scratch(const Plan &p) { return (size_t)plan_slabs(p) * 256 * 256 * 4; }

// Launches the pair kernel and, where tiles were split, the one that adds
// their partials (in `part`).
template <typename T, uint32_t FORMAT, int MODE, bool GELU>
cudaError_t launch_pair(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &tb2, const CUtensorMap &tc,
                        const CUtensorMap &tg, const CUtensorMap &tu, Args args, const Plan &p, void *part, T *out0,
                        T *out1, float *G, float *U, cudaStream_t s) {
    args.whole = p.whole;
    args.splits = p.splits;
    CUtensorMap tp = tc;
    if (p.splits > 1 && !make_map3(&tp, part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 256, 256, plan_slabs(p), 1024, 256 * 1024,
                                   32, 32, 1, 128))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.clusters), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(MODE);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    pdl_attr(attr[1]);
    cfg.attrs = attr;
    cfg.numAttrs = g_pdl ? 2 : 1;
    const cudaError_t e = launch_counted(&cfg, gated_pair_kernel<T, FORMAT, MODE, GELU>, ta, tb, tb2, tc, tg, tu, tp, args);
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchAttribute fa[1];
    const cudaLaunchConfig_t fc = pdl_config(dim3(32, (unsigned)(p.tiles - p.whole), (unsigned)((args.bn + 127) / 128)),
                                             dim3(256), 0, s, fa);
    return launch_counted(&fc, gated_fix_kernel<T, MODE, GELU>, static_cast<const float *>(part), out0, out1, G, U, args);
}

template <typename T, uint32_t FORMAT, bool GELU>
cudaError_t forward(const GatedProblem &p, int dev, int *status, cudaStream_t s) {
    const int cmax = clusters_max<T, FORMAT, FWD, GELU>(dev);
    if (cmax <= 0) return cudaErrorNotSupported;
    const long long tiles_m = (p.M + 255LL) / 256;
    const int num_kb = (p.K + BK - 1) / BK;
    // 64-wide tiles where they are done first, as they are where 128-wide ones leave
    // clusters idle (forward of 333 x 1000 x 1000 9.1 us against 12.4, 300 x 512 x 2048
    // 8.4 against 11.8; 128 x 12288 x 4096 55 against 45, 1024 x 12160 x 4096 149
    // against 107).
    const bool on128 = p.N % 64 == 0 || p.ldx % 64 == 0;
    Plan pl = plan(tiles_m * ((p.N + 127LL) / 128), cmax, num_kb, 256, on128);
    const Plan thin = plan(tiles_m * ((p.N + 63LL) / 64), cmax, num_kb, 128, on128);
    const int bn = thin.time < pl.time ? 64 : 128;
    if (bn == 64) pl = thin;
    if (pl.tiles > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    CUtensorMap tx, tg, tu, tz, tsg, tsu;
    const long long zr = 2LL * p.N;
    if (!map16(&tx, p.X, FORMAT, p.M, p.K, BK, 128, p.ldx, 1) || !map16(&tg, p.Wg, FORMAT, p.K, p.N, 64, BK) ||
        !map16(&tu, p.Wu, FORMAT, p.K, p.N, 64, BK) ||
        !make_map3(&tz, p.Z, map_type(FORMAT), p.N, p.M, 1, zr, zr * p.M, bn / 2, 32, 1, /*swizzle: a row's bytes*/ bn))
        return cudaErrorInvalidValue;
    tsg = tsu = tz;
    const long long row = 4LL * p.N;
    if (p.G && (!make_map3(&tsg, p.G, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.N, p.M, 1, row, row * p.M, 32, 32, 1, 128) ||
                !make_map3(&tsu, p.U, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.N, p.M, 1, row, row * p.M, 32, 32, 1, 128)))
        return cudaErrorInvalidValue;
    Args a = {};
    a.M = p.M;
    a.N = p.N;
    a.num_kb = num_kb;
    a.bn = bn;
    a.batch = 1;
    a.save = p.G != nullptr;
    a.status = status;
    void *ws = nullptr;
    cudaError_t e = pl.splits > 1 ? scratch_alloc(&ws, plan_scratch(pl), s) : cudaSuccess;
    if (e != cudaSuccess) return e;
    e = launch_pair<T, FORMAT, FWD, GELU>(tx, tg, tu, tz, tsg, tsu, a, pl, ws, static_cast<T *>(p.Z),
                                          static_cast<T *>(p.Z), p.G, p.U, s);
    const cudaError_t f = ws ? cudaFreeAsync(ws, s) : cudaSuccess;
    return e != cudaSuccess ? e : f;
}

template <typename T, uint32_t FORMAT, bool GELU>
cudaError_t backward(const GatedBackward &p, int dev, int num_sms, int *status, cudaStream_t s) {
    const int cmax = clusters_max<T, FORMAT, DX, false>(dev), wmax = clusters_max<T, FORMAT, DW, false>(dev);
    if (cmax <= 0 || wmax <= 0) return cudaErrorNotSupported;
    const long long mn = (long long)p.M * p.N;
    // dG and dU on rows of 128 bytes, whatever N: of a product's two operands one may
    // lie otherwise at little cost (block_time)
    const long long ldg = gated_ldg(p.N);
    const bool pair_dx = p.dX && p.M > kGatedSkinnyMaxM, both = p.dWg && p.dWu;
    const Plan pw = plan((p.K + 255LL) / 256 * ((p.N + 255LL) / 256) * (both ? 2 : 1), wmax, (p.M + BK - 1LL) / BK,
                         256, true);
    // (where dW's tiles are split, a kernel that adds them lies between, and the
    // partials' scratch is shared)
    const bool beside = p.dX && g_pdl && (p.dWg || p.dWu) && pw.splits == 1;
    // dX: the tile width and plan that are done first, widest on ties.  Beside dW, a
    // plan may keep to the clusters that dW leaves; one that needs more waits for dW,
    // its blocks and about 12 blocks' time of set-up and writing (backward of 500 x 1504
    // x 704 16.1 us, with dX's plan for all clusters 20.3; 333 x 1000 x 1000 13.7).
    const long long tiles_m = (p.M + 255LL) / 256;
    const int half = (p.N + BK - 1) / BK, left = beside ? std::max(cmax - pw.clusters, 0) : cmax;
    int bn = 0;
    Plan px = {};
    long long best = 0;
    for (int c = 256; c >= 64; c -= 64) {
        const long long tiles = tiles_m * ((p.K + c - 1LL) / c);
        for (int clusters : {cmax, left}) {
            if (clusters == 0) continue;
            const Plan q = plan(tiles, clusters, 2LL * half, c, true);
            const long long time = q.time + (q.clusters > left ? pw.time + 12 * 256 : 0);
            if (bn == 0 || time < best) { bn = c; px = q; best = time; }
        }
    }
    if (px.tiles > 0x7FFFFFFFLL || pw.tiles > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    // scratch: dG and dU, and the partials of the two products, one after the other
    const size_t off = ((size_t)(p.M * ldg) * 4 + 1023) & ~(size_t)1023;
    const size_t parts = std::max(pair_dx ? plan_scratch(px) : 0, p.dWg || p.dWu ? plan_scratch(pw) : 0);
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(&ws, off + parts, s);
    if (e != cudaSuccess) return e;
    void *part = static_cast<uint8_t *>(ws) + off;
    T *dG = static_cast<T *>(ws), *dU = dG + p.M * ldg;
    {
        const long long n4 = mn / 4, blocks = (n4 + 256 * GRAD_UNITS - 1) / (256 * GRAD_UNITS);
        cudaLaunchAttribute attr[1];
        const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(256), 0, s, attr);
        e = blocks > 0x7FFFFFFFLL
                ? cudaErrorInvalidValue
                : launch_counted(&cfg, gated_grad_kernel<T, GELU>, reinterpret_cast<const float4 *>(p.G),
                                 reinterpret_cast<const float4 *>(p.U), static_cast<const uint2 *>(p.dZ),
                                 reinterpret_cast<uint2 *>(dG), reinterpret_cast<uint2 *>(dU), n4, (uint32_t)(p.N / 4),
                                 (uint32_t)((ldg - p.N) / 4));
    }
    if (e == cudaSuccess && (p.dWg || p.dWu)) {
        T *w0 = static_cast<T *>(p.dWg ? p.dWg : p.dWu), *w1 = static_cast<T *>(p.dWu ? p.dWu : p.dWg);
        CUtensorMap ta, tb, tc, tc2;
        if (!map16(&ta, p.X, FORMAT, p.M, p.K, 64, BK) ||
            !map16(&tb, p.dWg ? dG : dU, FORMAT, p.M, p.N, 64, BK, ldg, both ? 2 : 1) ||
            !map16(&tc, w0, FORMAT, p.K, p.N, 64, 32) || !map16(&tc2, w1, FORMAT, p.K, p.N, 64, 32)) {
            e = cudaErrorInvalidValue;
        } else {
            Args a = {};
            a.M = p.K;
            a.N = p.N;
            a.num_kb = (p.M + BK - 1) / BK;
            a.bn = 256;
            a.batch = both ? 2 : 1;
            a.status = status;
            e = launch_pair<T, FORMAT, DW, false>(ta, tb, tb, tc, tc2, tc2, a, pw, part, w0, w1, nullptr, nullptr, s);
        }
    }
    if (e == cudaSuccess && p.dX && !pair_dx) {
        e = launch_gated_skinny_dx(p, dG, beside, num_sms, status, s);
    } else if (e == cudaSuccess && p.dX) {
        CUtensorMap ta, tb, tb2, tc;
        if (!map16(&ta, dG, FORMAT, p.M, p.N, BK, 128, ldg, 2) || !map16(&tb, p.Wg, FORMAT, p.K, p.N, BK, bn / 2) ||
            !map16(&tb2, p.Wu, FORMAT, p.K, p.N, BK, bn / 2) || !map16(&tc, p.dX, FORMAT, p.M, p.K, 64, 32)) {
            e = cudaErrorInvalidValue;
        } else {
            Args a = {};
            a.M = p.M;
            a.N = p.K;
            a.num_kb = 2 * half;
            a.kb_half = half;
            a.bn = bn;
            a.batch = 1;
            a.beside = beside;
            a.status = status;
            T *out = static_cast<T *>(p.dX);
            e = launch_pair<T, FORMAT, DX, false>(ta, tb, tb2, tc, tc, tc, a, px, part, out, out, nullptr, nullptr, s);
        }
    }
    const cudaError_t f = cudaFreeAsync(ws, s);
    return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_gated(const GatedProblem &p, int *status, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (p.elt == Elt::BF16)
        return p.gelu ? forward<__nv_bfloat16, 1, true>(p, dev, status, s) : forward<__nv_bfloat16, 1, false>(p, dev, status, s);
    return p.gelu ? forward<__half, 0, true>(p, dev, status, s) : forward<__half, 0, false>(p, dev, status, s);
}

cudaError_t launch_gated_backward(const GatedBackward &p, int num_sms, int *status, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (p.elt == Elt::BF16)
        return p.gelu ? backward<__nv_bfloat16, 1, true>(p, dev, num_sms, status, s)
                      : backward<__nv_bfloat16, 1, false>(p, dev, num_sms, status, s);
    return p.gelu ? backward<__half, 0, true>(p, dev, num_sms, status, s)
                  : backward<__half, 0, false>(p, dev, num_sms, status, s);
}

}  // namespace gemm_gb300
