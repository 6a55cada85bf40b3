// Product of two 4-bit block-scaled matrices on the tensor cores:
//     C[i,j] = ga gb sum_k (qa sa)[i,k] (qb sb)[j,k]
// tcgen05 kind::mxf4nvf4 with block scales: the MMA multiplies E2M1 codes,
// applies both blocks' scales to each partial sum and accumulates in FP32
// tensor memory; the tensors' FP32 scales are applied in the epilogue, before the
// rounding to the output type.
//
// A 256 x bn tile of C belongs to a cluster of two CTAs (cta_group::2): CTA r
// holds rows [128 r, 128 r + 128) of A's tile and its half of B's, and both
// hold the scales of their own 128 rows of A and of all of B's rows.  A stage is
// 256 k: 128 bytes a row, the 128-byte swizzle of 8- and 16-bit operands; four
// MMAs of K = 64.  The scales' atoms of 128 rows x 4 blocks (512 bytes) go to
// tensor memory with tcgen05.cp 32x128b.warpx4, in the order in which they are
// stored: row % 32 is the lane, row / 32 the column, and the four bytes of a
// column four blocks.  NV (16 k a block): an atom is one MMA's K.  MX (32 k): an
// atom serves two MMAs, which read bytes 0-1 and 2-3 (the descriptor's scale id).
// A tile of B that starts 64 rows into a 128-row tile of scales reads them from
// the third column on (tile widths are multiples of 64, because an MMA's scales
// must start on an even column).  cp and mma of one thread execute in order, so
// the scales need no second copy.
//
// Tile widths, by tensor memory (512 columns, 64 of them scales): 192 leaves two
// whole accumulators, so that a tile is written while the next is computed; 256
// two that share 64 columns, which the epilogue reads first before it lets the
// next tile's MMAs start (1.2 us a tile in which the tensor cores wait); 128 and 64
// for few tiles.  launch_pair says which runs when.
//
// The loading and issuing warps stay converged and elect a lane for the TMA and
// tcgen05 instructions only: with loops run by one lane alone, operands are moved
// to uniform registers anew for every instruction, 23-25 ns a copy of an atom, and
// the tensor cores wait for the issue (8192^3 in 256-wide tiles, NV 312 us, MX
// 236; so 162 and 164).
//
// Warps: 0 loads (TMA; every load of the pair counts on the leader's full[s]), 1
// issues the MMAs (leader), 2-9 write C, half of the tile's columns to each four.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "fp4.h"
#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace {

using namespace tc;

constexpr int THREADS = 320;
constexpr int KB = 256;                  // k per stage
constexpr int A_STAGE = 128 * KB / 2;    // 16 KiB per CTA
constexpr int ROW_STG = 80;              // a row of 32 outputs at its distance from 16 bytes
constexpr int STG_BOX = 32 * ROW_STG;    // one 32-row x 32-column output box (TMA: its first 2 KiB)
constexpr int EPI_WARPS = 8;
constexpr int SMEM_STAGING = EPI_WARPS * STG_BOX;
constexpr uint32_t TMEM_COLS = 512, SF_COL = 448;
constexpr int GROUP_M = 8;

__host__ __device__ constexpr int sf_stage(bool nv) { return nv ? 2048 : 1024; }  // of 128 rows
// A's codes, B's codes, the scales of A's 128 rows and of the one or two 128-row
// tiles that B's tile meets.
__host__ __device__ constexpr int stage_bytes(bool nv, int bn) {
    return A_STAGE + bn / 2 * (KB / 2) + (bn <= 128 ? 2 : 3) * sf_stage(nv);
}
constexpr int MAX_STAGES = 6;
__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 5 : 6; }
__host__ __device__ constexpr int ring_bytes(bool nv) {
    return stages_of(192) * stage_bytes(nv, 192) > stages_of(256) * stage_bytes(nv, 256)
               ? stages_of(192) * stage_bytes(nv, 192) : stages_of(256) * stage_bytes(nv, 256);
}
__host__ __device__ constexpr int smem_bytes(bool nv) { return 1024 + ring_bytes(nv) + SMEM_STAGING + 256; }
static_assert(smem_bytes(true) <= 232448, "shared memory budget");
static_assert(ring_bytes(true) % 1024 == 0 && ring_bytes(false) % 1024 == 0, "staging boxes on 1024 bytes");

struct Bars {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
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
    void *C;
    long long ldc;
    const float *ga, *gb;
    int M, N, K;
    int bn;         // 64, 128, 192 or 256
    int tma_store;  // C's rows suit TMA stores
    int *status;
};

// D[tmem of both CTAs] (+)= A B^T over one K step of 64, scales in tensor memory.
template <bool NV>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t acc) {
    if constexpr (NV)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
}
// One atom of scales (512 bytes) from shared memory to four columns, in both CTAs.
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Instruction descriptor: E2M1 x E2M1, both K-major, scale type E8M0 (MX) or
// E4M3 (NV), M = 256, N = bn, scale ids `id` in A and B.
template <bool NV>
__device__ __forceinline__ uint32_t make_idesc(uint32_t bn, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((bn >> 3) << 17) | ((NV ? 0u : 1u) << 23) | ((256u >> 4) << 24) |
           (id << 29);
}

__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int per_group = GROUP_M * tiles_n;
    const int group = t / per_group;
    const int first_m = group * GROUP_M;
    const int gsize = min(tiles_m - first_m, GROUP_M);
    const int r = t - group * per_group;
    tm = first_m + r % gsize;
    tn = r / gsize;
}

// Rows that TMA cannot write: a warp's 32 rows, on any 2 bytes, 64 bytes of each at
// a time.  A lane lays its row's 64 bytes out in shared memory (`box`) at the row's
// distance d from 16 bytes, behind the d bytes that the 64 before left over, and
// four lanes write a row's four 16-byte pieces; the d bytes after them wait for the
// next 64, or for flush().  Only a run's first 16 - d and last d bytes are written 2, 4
// and 8 at a time.  Measured, NV, against one column a lane, row after row: 3000 x 5001 x
// 1000 24.1 and 36.9 us, 4096 x 4095 x 4096 35.5 and 42.9, 8192 x 8191 x 8192 175
// and 179.
struct RowStore {
    uint8_t *box;
    long long row_bytes;
    int rows;          // of the 32, how many there are
    uint8_t *next;     // row 0's address after the last 64 bytes; null: nothing waits
    uint32_t carry;    // this lane's row: the last two values

    __device__ __forceinline__ void flush() {
        const int lane = threadIdx.x & 31;
        if (next != nullptr && lane < rows) {
            uint8_t *row = next + lane * row_bytes;
            const int d = (int)((uintptr_t)row & 15);
            uint8_t *g = row - d;
            const uint8_t *stg = box + lane * ROW_STG + 64;
            if (d & 8) *reinterpret_cast<uint2 *>(g) = *reinterpret_cast<const uint2 *>(stg);
            if (d & 4) *reinterpret_cast<uint32_t *>(g + (d & 8)) = *reinterpret_cast<const uint32_t *>(stg + (d & 8));
            if (d & 2) *reinterpret_cast<uint16_t *>(g + (d & 12)) = *reinterpret_cast<const uint16_t *>(stg + (d & 12));
        }
        next = nullptr;
        __syncwarp();
    }
    // Row 0's 64 bytes at dst, this lane's row in w.
    __device__ __forceinline__ void put(uint8_t *dst, const uint32_t (&w)[16]) {
        const int lane = threadIdx.x & 31;
        if (dst != next) flush();
        const bool cont = next != nullptr;
        {
            const int d = (int)((uintptr_t)(dst + lane * row_bytes) & 15);
            uint8_t *stg = box + lane * ROW_STG;
            if (cont) *reinterpret_cast<uint4 *>(stg) = *reinterpret_cast<const uint4 *>(stg + 64);
            uint32_t *at = reinterpret_cast<uint32_t *>(stg + (d & 12));
            uint32_t before = carry;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                at[i] = __funnelshift_l(before, w[i], 8 * (d & 2));
                before = w[i];
            }
            if (d & 2) at[16] = before >> 16;
            carry = before;
        }
        __syncwarp();
#pragma unroll 1
        for (int r = lane >> 2; r < min(rows, 32); r += 8) {
            uint8_t *row = dst + r * row_bytes;
            const int d = (int)((uintptr_t)row & 15), p = 16 * (lane & 3);
            uint8_t *g = row - d;
            const uint8_t *stg = box + r * ROW_STG;
            if (p > 0 || cont || d == 0) {
                *reinterpret_cast<uint4 *>(g + p) = *reinterpret_cast<const uint4 *>(stg + p);
            } else {
                int h = d;
                if (h & 2) {
                    *reinterpret_cast<uint16_t *>(g + h) = *reinterpret_cast<const uint16_t *>(stg + h);
                    h += 2;
                }
                if (h & 4) {
                    *reinterpret_cast<uint32_t *>(g + h) = *reinterpret_cast<const uint32_t *>(stg + h);
                    h += 4;
                }
                if (h == 8) *reinterpret_cast<uint2 *>(g + 8) = *reinterpret_cast<const uint2 *>(stg + 8);
            }
        }
        __syncwarp();
        next = dst + 64;
    }
};

template <typename T, bool NV>
__global__ void __launch_bounds__(THREADS, 1)
fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSa,
                const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSb,
                const __grid_constant__ CUtensorMap tmC, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int SF = sf_stage(NV);
    const int M = args.M, N = args.N, bn = args.bn;
    const int STAGES = stages_of(bn), B_STAGE = (bn >> 1) * (KB / 2);
    const int sf_tiles_b = bn <= 128 ? 1 : 2;  // 128-row tiles of scales that a tile of B meets
    const int SF_STAGE = (1 + sf_tiles_b) * SF;
    uint8_t *a_tiles = smem;
    uint8_t *b_tiles = a_tiles + STAGES * A_STAGE;
    uint8_t *sf_tiles = b_tiles + STAGES * B_STAGE;  // per stage: A's 128 rows, then B's row tiles
    uint8_t *staging = smem + ring_bytes(NV);
    Bars *bars = reinterpret_cast<Bars *>(staging + SMEM_STAGING);
    volatile int *abort_flag = &bars->abort;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = (int)cluster_id_x(), nclusters = (int)cluster_count_x();
    const int tiles_m = (M + 255) / 256, tiles_n = (N + bn - 1) / bn;
    const int num_tiles = tiles_m * tiles_n;
    const int num_kb = (args.K + KB - 1) / KB;
    const bool wide = bn == 256;
    constexpr uint32_t acc_off = 192;  // of the second accumulator
    // both CTAs' loads of a stage, all counted on the leader's barrier
    const uint32_t stage_tx = 2u * (uint32_t)(A_STAGE + B_STAGE + SF_STAGE);

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
        prefetch_desc(&tmSa);
        prefetch_desc(&tmSb);
        prefetch_desc(&tmC);
    }
    if (warp == 1) tmem_alloc<2>(&bars->tmem_base, TMEM_COLS);
    fence_before();
    cluster_sync();  // barriers of both CTAs initialised before any cross-CTA use
    fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    pdl_launch_dependents();
    pdl_wait();

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        const bool issuer = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        for (int t = cluster; t < num_tiles && ok; t += nclusters) {
            int tm, tn;
            tile_coords(t, tiles_m, tiles_n, tm, tn);
            const int row0 = tm * 256 + (int)rank * 128, col0 = tn * bn + (int)rank * (bn >> 1);
            const int sf_b = tn * bn / 128;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag, true)) { ok = false; break; }
                const uint32_t full = map_to_rank(&bars->full[stage], 0);
                uint8_t *sf = sf_tiles + stage * SF_STAGE;
                if (issuer) {
                    if (leader) mbar_arrive_expect_tx(&bars->full[stage], stage_tx);
                    tma_load_3d_pair(a_tiles + stage * A_STAGE, &tmA, full, kb * (KB / 2), row0, 0);
                    tma_load_3d_pair(b_tiles + stage * B_STAGE, &tmB, full, kb * (KB / 2), col0, 0);
                    tma_load_3d_pair(sf, &tmSa, full, 0, kb * (SF / 1024), row0 / 128);
                    tma_load_3d_pair(sf + SF, &tmSb, full, 0, kb * (SF / 1024), sf_b);
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
        // The whole warp runs the loop, so that descriptors stay in uniform
        // registers; one elected lane issues.
        const bool issuer = elect_one();
        const uint64_t a_desc0 = desc_sw128(smem_u32(a_tiles), 16, 1024);
        const uint64_t b_desc0 = desc_sw128(smem_u32(b_tiles), 16, 1024);
        const uint64_t sf_desc0 = desc_plain(smem_u32(sf_tiles), 128);
        constexpr int ATOMS = SF / 512;  // of a stage: 4 (NV) or 2 (MX)
        const uint32_t sfa = tmem_base + SF_COL, sfb = sfa + 4 * ATOMS;
        const uint32_t sfb_atom = 4u * (uint32_t)sf_tiles_b;
        const uint32_t idesc0 = make_idesc<NV>((uint32_t)bn, 0), idesc1 = make_idesc<NV>((uint32_t)bn, 2);
        int stage = 0;
        uint32_t phase = 0;
        int it = 0;
        bool ok = true;
        for (int t = cluster; t < num_tiles; t += nclusters, ++it) {
            int tm, tn;
            tile_coords(t, tiles_m, tiles_n, tm, tn);
            const int buf = it & 1;
            // 256: tile it - 1's shared columns have been read (and so all of it - 2)
            if (wide) {
                if (it > 0 && !mbar_wait(&bars->acc_empty[buf ^ 1], (uint32_t)(((it - 1) >> 1) & 1), abort_flag, true))
                    ok = false;
            } else if (!mbar_wait(&bars->acc_empty[buf], (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag, true)) {
                ok = false;
            }
            if (!ok) break;
            fence_after();
            const uint32_t d = tmem_base + (uint32_t)buf * acc_off;
            const uint32_t sfb_first = ((uint32_t)(tn * bn) & 64u) >> 5;  // column of the tile's first row
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!mbar_wait(&bars->full[stage], phase, abort_flag, true)) { ok = false; break; }
                fence_after();
                const uint64_t ad = a_desc0 + (uint64_t)((stage * A_STAGE) >> 4);
                const uint64_t bd = b_desc0 + (uint64_t)((stage * B_STAGE) >> 4);
                const uint64_t sd = sf_desc0 + (uint64_t)((stage * SF_STAGE) >> 4);
                if (issuer) {
#pragma unroll
                    for (int a = 0; a < ATOMS; ++a) {
                        cp_scales_pair(sfa + 4 * a, sd + a * 32);
                        cp_scales_pair(sfb + sfb_atom * a, sd + (ATOMS + a) * 32);
                        if (bn > 128) cp_scales_pair(sfb + sfb_atom * a + 4, sd + (2 * ATOMS + a) * 32);
                    }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const int a = NV ? ks : ks >> 1;
                        mma_pair<NV>(d, ad + ks * 2, bd + ks * 2, NV || (ks & 1) == 0 ? idesc0 : idesc1, sfa + 4 * a,
                                     sfb + sfb_first + sfb_atom * a, (uint32_t)((kb | ks) != 0));
                    }
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
        uint8_t *box = staging + (warp - 2) * STG_BOX;
        uint8_t *rowp = box + lane * 64;
        const Fp4Factors f = fp4_factors<NV>(args.ga, args.gb);
        const float2 first = make_float2(f.first, f.first), second = make_float2(f.second, f.second);
        const int groups = bn >> 6, group0 = half * groups;  // this half's groups of 32 columns
        int it = 0;
        bool ok = true;
        for (int t = cluster; t < num_tiles; t += nclusters, ++it) {
            int tm, tn;
            tile_coords(t, tiles_m, tiles_n, tm, tn);
            const int buf = it & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->acc_full[buf], (uint32_t)((it >> 1) & 1), abort_flag, true))) {
                ok = false;
                break;
            }
            fence_after();
            __syncwarp();
            const int row0 = tm * 256 + (int)rank * 128 + quarter * 32;
            const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)buf * acc_off;
            const uint32_t empty = map_to_rank(&bars->acc_empty[buf], 0);
            // 256: the columns shared with the other accumulator are groups 6 and 7 of
            // buf 0, 0 and 1 of buf 1.  The half that holds them reads them first; the
            // other has nothing to read before the next tile's MMAs, but has finished
            // the tile before this one.
            const bool shares = wide && half == (buf ^ 1);
            if (wide && !shares) {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(empty);
            }
            RowStore out = {box, args.ldc * 2, M - row0, nullptr, 0u};
            for (int i = 0; i < groups; ++i) {
                const int g = group0 + (shares && buf == 0 ? i ^ 2 : i);
                const int c0 = tn * bn + g * 32;
                uint32_t r[32];
                if (c0 < N) {  // warp-uniform
                    tmem_ld32(t_row + (uint32_t)(g * 32), r);
                    tmem_ld_wait();
                }
                if (wide ? shares && i == 1 : i == groups - 1) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(empty);
                }
                if (c0 >= N) continue;
                if (lane == 0 && args.tma_store) tma_stores_read_wait0();  // the last store has read the box
                __syncwarp();
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float2 v = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    if (NV) v = mul2(mul2(v, first), second);
                    w[j] = pack2(v.x, v.y, (T *)nullptr);
                }
                if (args.tma_store) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)  // the 64-byte swizzle
                        *reinterpret_cast<uint4 *>(rowp + ((c ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && row0 < M) tma_store_3d(&tmC, box, c0, row0, 0);
                } else {
                    uint16_t *corner = static_cast<uint16_t *>(args.C) + (long long)row0 * args.ldc + c0;
                    if (c0 + 32 <= N) {  // warp-uniform
                        out.put(reinterpret_cast<uint8_t *>(corner), w);
                    } else if (row0 + lane < M) {
                        uint16_t *crow = corner + lane * args.ldc;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < N) crow[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
                    }
                }
            }
            if (!args.tma_store) out.flush();
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
}

template <typename T, bool NV>
int clusters_max(int dev) {
    static std::atomic<int> known[kMaxDevices];
    return cluster_limit(known[dev], reinterpret_cast<const void *>(fp4_pair_kernel<T, NV>), THREADS,
                         smem_bytes(NV), 2);
}

template <typename T, bool NV>
cudaError_t launch_pair(const Fp4Problem &p, int *status, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const int cmax = clusters_max<T, NV>(dev);
    if (cmax <= 0) return cudaErrorNotSupported;
    // The tile's width: the least waves x time of a tile.  A tile takes the longer
    // of its stages (measured 0.25 us each at 192, 0.31 at 256, 0.22 at 128 and 0.205
    // at 64, with the 1 us in which 256's accumulators change hands) and its writing
    // (2.2, 2.5, 1.7 and 1.5 us).  Measured, NV, at 192 and 256: 8192^3 157 and 159 us,
    // 2048 x 12288 x 4096 38.2 and 42.1, 2048 x 4096 x 4096 18.1 and 16.7, 8192 x 12288
    // x 512 59.7 and 53.5; 1000 x 1001 x 4100 17.1, 18.7, 13.2 at 128; that in MX 10.8 at
    // 128 and 9.4 at 64, 200 x 2000 x 1000 4.7 and 4.3, 300 x 4096 x 4096 7.7 and 10.4.
    const long long tiles_m = (p.M + 255LL) / 256, kbs = (p.K + KB - 1LL) / KB;
    int bn = 0;
    long long tiles = 0, best = 0;
    for (int c : {192, 256, 128, 64}) {
        const long long t = tiles_m * ((p.N + c - 1LL) / c);
        const long long ns = c == 192   ? std::max(250 * kbs, 2200LL)
                             : c == 256 ? std::max(310 * kbs + 1000, 2500LL)
                             : c == 128 ? std::max(220 * kbs, 1700LL)
                                        : std::max(205 * kbs, 1500LL);
        const long long cost = (t + cmax - 1) / cmax * ns;
        if (bn == 0 || cost < best) { bn = c; tiles = t; best = cost; }
    }
    if (tiles > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const long long rb = fp4_row_bytes(p.K);
    const long long chunks = (long long)fp4_atoms(NV, p.K) / 2;  // of 1024 bytes, a tile of 128 rows
    constexpr int SFC = sf_stage(NV) / 1024;
    CUtensorMap ta, tsa, tb, tsb, tc;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    if (!make_map3(&ta, p.Qa, u8, rb, p.M, 1, p.pitch_a, p.pitch_a * p.M, 128, 128, 1, 128) ||
        !make_map3(&tb, p.Qb, u8, rb, p.N, 1, p.pitch_b, p.pitch_b * p.N, 128, bn / 2, 1, 128) ||
        !make_map3(&tsa, p.Sa, u32, 256, chunks, fp4_row_tiles(p.M), 1024, chunks * 1024, 256, SFC, 1, 0) ||
        !make_map3(&tsb, p.Sb, u32, 256, chunks, fp4_row_tiles(p.N), 1024, chunks * 1024, 256, SFC, bn <= 128 ? 1 : 2, 0))
        return cudaErrorInvalidValue;
    Args a = {};
    a.C = p.C;
    a.ldc = p.ldc;
    a.ga = p.ga;
    a.gb = p.gb;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.bn = bn;
    a.status = status;
    // TMA stores write whole 16-byte pieces of rows that start on 16 bytes.
    a.tma_store = ((uintptr_t)p.C & 15u) == 0 && p.ldc % 8 == 0 && p.N % 8 == 0;
    if (a.tma_store) {
        const auto dt = p.elt == Elt::BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if (!make_map3(&tc, p.C, dt, p.N, p.M, 1, p.ldc * 2, p.ldc * 2 * p.M, 32, 32, 1, 64)) a.tma_store = 0;
    }
    if (!a.tma_store) tc = tb;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(tiles, cmax)), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(NV);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    pdl_attr(attr[1]);
    cfg.attrs = attr;
    cfg.numAttrs = g_pdl ? 2 : 1;
    return launch_counted(&cfg, fp4_pair_kernel<T, NV>, ta, tsa, tb, tsb, tc, a);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Problem &p, int *status, cudaStream_t s) {
    if (p.elt == Elt::BF16)
        return p.nv ? launch_pair<__nv_bfloat16, true>(p, status, s) : launch_pair<__nv_bfloat16, false>(p, status, s);
    return p.nv ? launch_pair<__half, true>(p, status, s) : launch_pair<__half, false>(p, status, s);
}

}  // namespace gemm_gb300
