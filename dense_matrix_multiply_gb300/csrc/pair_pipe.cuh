// The tensor-core pipeline of the head's cross entropy (cross_entropy.cu) and of the
// orthogonalised update (orthogonalize.cu): D = A B of 16-bit operands, FP32 sums, whose
// tiles are handed to an epilogue of the caller's.
//
// A 256 x bn tile (bn 128, 192 or 256; 192 only where B lies K-major) belongs to a cluster of
// two CTAs (tcgen05 cta_group::2), 128 rows of A and half of B's columns loaded by each, K in
// stages of 64; up to 128 rows may go in 128 x 256 tiles, 64 of them to a CTA.  Either
// operand may lie K-major (rows of adjacent k) or MN-major (k by k, adjacent rows or
// columns), as its tensor map and the flags say.  Warp 0 loads, warp 1 of the leader issues
// the MMAs -- both converged, one elected lane for the instructions -- and warps 2-9 write
// out, 32 rows and half of the columns to each.  Two accumulators, so that a tile is
// written while the next is computed.  Clusters walk over the units (a tile, or one of its
// K ranges) in the same order.
//
// Where there are few tiles of a long K, two pairs of one cluster are joined on a tile of
// 256 x 128, half of K each: every CTA stores the FP32 sums of the other pair's 64 columns
// to the shared memory of its counterpart there and writes out its own 64.  (All of a
// tile's sums through the cluster, among four pairs: 7 us a tile; this way about 1.)
//
// Classes (Epi::CLASSES): a B whose rows lie off 16 bytes, K-major, which TMA cannot describe,
// is read in place.  Every eighth row (fourth, second: G = 8 / gcd(K, 8)) lies alike to 16
// bytes, so that rows r, r + G, ... make a matrix of their own whose rows are a multiple of
// 16 bytes apart.  It starts at the 16-byte piece that holds its first element, s_r elements
// before it; A has s_r zeros in front of its rows, a copy for each class, and before their
// first use the s_r elements in front of B's rows -- the ends of the rows before -- are
// overwritten with zeros in shared memory (0 times an infinity is a NaN).  A tile's columns
// are of one class.  Or the rows are K and B lies MN-major: a K range is of one class, A has a
// matrix for each, and D's columns are s_r too far right.
//
// Every wait is bounded; on expiry a code goes to the status word, both CTAs give up,
// their loads and MMAs are waited for, and the tensor memory is released.
#pragma once

#include "tc_ptx.cuh"

namespace gemm_gb300 {
namespace pair {

using namespace tc;

constexpr int THREADS = 320, EPI_WARPS = 8;
constexpr int BK = 64;                 // 16-bit k per stage: 128 bytes a row
constexpr int A_STAGE = 128 * BK * 2;  // 16 KiB per CTA
constexpr int B_STAGE = 128 * BK * 2;  // up to 128 of the tile's columns
constexpr int BOX64 = 64 * BK * 2;     // 64 columns x 64 k of an MN-major tile
constexpr int STG_BOX = 4096;          // 32 rows x 128 bytes: an epilogue warp's output
// Boxes of a warp, 1 or 2, and stages.
constexpr int stages_of(int boxes) { return 7 - boxes; }
constexpr int smem_of(int boxes) { return 1024 + stages_of(boxes) * (A_STAGE + B_STAGE) + boxes * EPI_WARPS * STG_BOX + 256; }
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP_M = 8;
static_assert(smem_of(1) <= 232448 && smem_of(2) <= 232448, "shared memory budget");

struct Bars {
    uint64_t full[6];
    uint64_t empty[6];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t joined;  // the other pair's sums are here
    uint64_t drain;
    uint64_t peer_done;
    long long peer_issued;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Args {
    int M, N;        // of D
    int num_kb;      // K blocks of 64
    int bn;
    int a_mn, b_mn;  // operands that lie MN-major
    int tiles;
    int splits;      // K ranges of a tile, each a unit of its own
    int joined;      // pairs on a tile: 1, or 2 (bn 128, splits 1, a cluster to each tile)
    // Rows of A's boxes.  For M up to half of a tile's rows those that there are, up to eights:
    // the leader's, the peer loads none (zeros behind the matrix cost a load as much time as
    // its elements: M = 1, N = 32000, K = 4096 84 us with boxes of 128 rows); what the rows
    // behind them hold reaches no row of D but theirs.
    int a_rows;
    // k that a stage's boxes hold, 64, where both operands lie MN-major and K is less 16, 32
    // or 48 at least as many: the rest of the only block is neither loaded nor multiplied.
    int k_rows;
    // Rows of a tile: 256, or 128 where M is no more (A K-major, pairs not joined): half the
    // MMAs' time.  A CTA then has 64 rows, and its accumulator those of the first half of the
    // columns in tensor-memory lanes 0-63, of the second half in lanes 64-127.
    int rows;
    // Classes: tiles (columns of them) of each, K ranges of each (0: the classes are of
    // columns), and s_r, four bits each.
    int class_tiles, class_splits;
    uint32_t shifts;
    int b_rows;  // rows of D to a matrix of B, MN-major (0: one for all)
    int *status;
};
// B's tensor maps, one of each class.
template <bool CLASSES>
struct BMaps {
    CUtensorMap m[CLASSES ? 8 : 1];
};

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// FP32 accumulator, A and B of one 16-bit type (0 f16, 1 bf16).
__device__ __forceinline__ uint32_t make_idesc(uint32_t format, uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
    return (1u << 4) | (format << 7) | (format << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((n >> 3) << 17) | ((m >> 4) << 24);
}

// The first s elements (s < 8) of the rows of a K-major operand, 128-byte swizzle, set to
// zero: whole warp, in either CTA's shared memory.
__device__ __forceinline__ void zero_front(uint32_t cluster_addr, int rows, uint32_t s, int lane) {
    for (int r = lane; r < rows; r += 32) {
        const uint32_t at = cluster_addr + (uint32_t)(r * 128 + ((r & 7) << 4));
        for (uint32_t i = 0; i + 1 < s; i += 2) st_cluster_u32(at + 2 * i, 0u);
        if (s & 1) asm volatile("st.shared::cluster.b16 [%0], %1;" ::"r"(at + 2 * (s - 1)), "h"((uint16_t)0) : "memory");
    }
}

// An accumulator's columns are in registers (tcgen05.wait::ld has returned) and may be
// overwritten.  Nothing in memory is handed over, so the arrival is relaxed: one that
// releases waits for the warp's output on its way to memory, 1700 cycles, and with it the
// accumulator's next tile (dW of 8 x 32000 x 4096 54 us against 77).
__device__ __forceinline__ void arrive_read(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// On the barrier at this offset in both CTAs of the pair whose leader is CTA `lead`.
__device__ __forceinline__ void commit_to_pair(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)(3u << lead))
        : "memory");
}

struct Tile {
    int m, n;
};
// Tiles in groups of GROUP_M rows of them, column by column within a group.  LOWER: only
// those of a square D that hold an element on or below its diagonal block of 256, row
// after row: (m + 1) 256 / bn of them in row m (fewer in the last).
template <bool LOWER>
__device__ __forceinline__ Tile tile_at(int t, const Args &a) {
    if constexpr (LOWER) {
        const int q = 256 / a.bn;
        int m = (int)((sqrtf(8.0f * (float)(t / q) + 1.0f) - 1.0f) * 0.5f);
        while (q * (m + 1) * (m + 2) / 2 <= t) ++m;
        while (q * m * (m + 1) / 2 > t) --m;
        return {m, t - q * m * (m + 1) / 2};
    }
    const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + a.bn - 1) / a.bn;
    const int group = t / (GROUP_M * tiles_n), first = group * GROUP_M, size = min(tiles_m - first, GROUP_M);
    const int q = t - group * GROUP_M * tiles_n;
    return {first + q % size, q / size};
}
inline long long lower_tiles(int n, int bn) {
    const long long rows = (n + 255LL) / 256, q = 256 / bn;
    return q * (rows - 1) * rows / 2 + (n + bn - 1LL) / bn;
}

// Joined pairs: the sums that come in, 32 columns after 32, of those four columns of all
// 128 rows after four -- a warp's stores, a row to a lane, are of 512 adjacent bytes
// (stores of 16 bytes to rows apart cross the cluster one by one).  They lie in the boxes
// of the warps that have no columns to write.
constexpr int JOIN_QUAD = 128 * 16, JOIN_CHUNK = 8 * JOIN_QUAD, JOIN_AT = EPI_WARPS * STG_BOX;
static_assert(JOIN_AT + 2 * JOIN_CHUNK <= 2 * EPI_WARPS * STG_BOX, "two boxes a warp");
// Four sums to another CTA, counted on a barrier there: the barrier's phase ends when all
// have arrived, without a fence at the sender.
__device__ __forceinline__ void send4(uint32_t cluster_addr, const uint32_t *r, uint32_t cluster_bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(cluster_bar)
                 : "memory");
}

// What an epilogue warp sees of a unit: 32 rows of D and columns [first, first + width) of
// a tile, multiples of 64.
struct Part {
    uint32_t tmem;          // this warp's rows, the tile's first column
    int row0, col0;         // of D: the warp's first row, the tile's first column (of its class)
    int tile_n, cls;        // the tile's index in a row of them; its class
    int first, width;
    int range, ranges;      // these columns are the tile's range-th of so many
    int split;              // which K range
    int bn, lane;
    uint8_t *box;           // STG_BOX bytes of this warp's, once or twice
    int turn;               // which of two is next (box_next)
    const uint8_t *joined;  // null, or this lane's row of the other pair's sums from column `first` on

    // Columns c .. c + 31 of the tile, this lane's row.
    template <bool JOIN>
    __device__ __forceinline__ void load(int c, uint32_t (&r)[32]) const {
        tmem_ld32(tmem + (uint32_t)c, r);
        tmem_ld_wait();
        if (JOIN && joined) {
            const uint8_t *at = joined + ((c - first) >> 5) * JOIN_CHUNK;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(at + j * JOIN_QUAD);
                r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + v.x);
                r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + v.y);
                r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + v.z);
                r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + v.w);
            }
        }
    }
};

// 32 registers of this lane's row to a box of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ void box_put(uint8_t *box, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
}
// Half h of them: sixteen registers.
__device__ __forceinline__ void box_put_half(uint8_t *box, int lane, int h, const uint32_t (&r)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(box + lane * 128 + (((h * 4 + c) ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
}
// The boxes once the stores that last read them have done so.
__device__ __forceinline__ void box_begin(int lane) {
    if (lane == 0) tma_stores_read_wait0();
    __syncwarp();
}
// One box, or two in turn: the next one, once the store that last read it has done so.  Of two
// all groups of stores but the youngest are waited for, so that every turn has to commit one
// group: box_store, or box_unstored in a turn that stores nothing.
template <int BOXES>
__device__ __forceinline__ uint8_t *box_next(Part &p) {
    if (BOXES == 1) {
        box_begin(p.lane);
        return p.box;
    }
    if (p.lane == 0) tma_stores_read_wait1();
    __syncwarp();
    uint8_t *box = p.box + p.turn * STG_BOX;
    p.turn ^= 1;
    return box;
}
__device__ __forceinline__ void box_store(const CUtensorMap *map, const uint8_t *box, int lane, int x, int y, int z) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, box, x, y, z);
}
__device__ __forceinline__ void box_unstored(int lane) {
    if (lane == 0) tma_store_none();
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// A box of 64 16-bit columns to a matrix that TMA cannot describe: by the element.
__device__ __forceinline__ void box_scatter(const uint8_t *box, int lane, uint16_t *out, long long ld, int row0, int col0,
                                            int M, int N) {
    __syncwarp();
    for (int r = 0; r < 32 && row0 + r < M; ++r) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        uint16_t *p = out + (row0 + r) * ld + col0 + 2 * lane;
        if (col0 + 2 * lane < N) p[0] = (uint16_t)v;
        if (col0 + 2 * lane + 1 < N) p[1] = (uint16_t)(v >> 16);
    }
    __syncwarp();
}

// Epi: static constexpr bool LOWER, JOIN (whether pairs may be joined) and CLASSES (whether B
// is of classes); int BOXES, 2 with JOIN; a type Pre and prefetch(Part, Pre), for what a
// unit's writing reads from memory, before its sums are waited for; run(Part, Pre); both
// called by whole warps with row0 < M.
template <uint32_t FORMAT, typename Epi>
__global__ void __launch_bounds__(THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BMaps<Epi::CLASSES> mapsB,
            const __grid_constant__ Epi epi, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int STAGES = stages_of(Epi::BOXES);
    static_assert(!Epi::JOIN || Epi::BOXES == 2, "room for the other pair's sums");
    uint8_t *a_tiles = smem;
    uint8_t *b_tiles = a_tiles + STAGES * A_STAGE;
    uint8_t *staging = b_tiles + STAGES * B_STAGE;
    Bars *bars = reinterpret_cast<Bars *>(staging + Epi::BOXES * EPI_WARPS * STG_BOX);
    volatile int *abort_flag = &bars->abort;

    const int bn = args.bn;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank(), rank = cta & 1, lead = cta & ~1u;
    const bool leader = rank == 0;
    const int cluster = (int)cluster_id_x(), nclusters = (int)cluster_count_x();
    const int units = args.tiles * args.splits;
    const bool joined = Epi::JOIN && args.joined > 1;
    // bytes of a stage that this CTA loads, and its peer
    const uint32_t a_bytes = args.a_mn ? 2u * (uint32_t)args.k_rows * 128u : (uint32_t)args.a_rows * 128u;
    const uint32_t b_bytes = args.b_mn ? (uint32_t)(bn >> 7) * (uint32_t)args.k_rows * 128u : (uint32_t)(bn >> 1) * 128u;
    const bool few = !args.a_mn && args.M <= args.rows / 2;  // none of the rows are the peer's
    const uint32_t peer_tx = b_bytes + (few ? 0u : a_bytes), stage_tx = a_bytes + b_bytes + peer_tx;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 2 * EPI_WARPS);
        }
        mbar_init(&bars->joined, 1);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->peer_done, 1);
        bars->abort = 0;
        mbar_init_fence();
        if (joined) mbar_arrive_expect_tx(&bars->joined, 2 * JOIN_CHUNK);
        prefetch_desc(&tmA);
        prefetch_desc(&mapsB.m[0]);
    }
    if (warp == 1) tmem_alloc<2>(&bars->tmem_base, TMEM_COLS);
    fence_before();
    cluster_sync();  // barriers of both CTAs initialised before any cross-CTA use
    fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    // The previous grid is waited for by the warps that touch global memory, once they know
    // their first unit: a few hundred cycles of index arithmetic, and the code itself, are
    // fetched while that grid drains.
    pdl_launch_dependents();

    // unit u: K range u / tiles of tile u % tiles (clusters share a range's operands); joined
    // pairs: a half of K each
    auto range = [&](int u, int &kb0, int &kb1) {
        const int j = u / args.tiles, own = Epi::CLASSES ? args.class_splits : 0;
        const int at = joined ? (int)(cta >> 1) : own ? j % own : j, n = joined ? 2 : own ? own : args.splits;
        kb0 = args.num_kb * at / n;  // (num_kb < 2^26, n <= 16)
        kb1 = args.num_kb * (at + 1) / n;
        return tile_at<Epi::LOWER>(u - j * args.tiles, args);
    };

    // the class of a unit's tile, and the tile's first column of it
    auto class_of = [&](int u, const Tile &t, int &col0) {
        int cls = 0;
        if (Epi::CLASSES) cls = args.class_splits ? u / args.tiles / args.class_splits : t.n / args.class_tiles;
        col0 = (t.n - (Epi::CLASSES && !args.class_splits ? cls * args.class_tiles : 0)) * bn;
        return cls;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        const bool issuer = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        int kb0, kb1;
        Tile t = range(cluster, kb0, kb1);
        pdl_wait();
        for (int u = cluster; ok && u < units;) {
            int col0;
            const int cls = class_of(u, t, col0), row0 = t.m * 256 + (int)rank * (args.rows >> 1);
            col0 += (int)rank * (bn >> 1);
            const CUtensorMap *const tmB = &mapsB.m[cls];
            const int b_at = args.b_rows ? t.m * 256 / args.b_rows : 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag, true)) { ok = false; break; }
                const uint32_t full = map_to_rank(&bars->full[stage], lead);
                uint8_t *a = a_tiles + stage * A_STAGE, *b = b_tiles + stage * B_STAGE;
                if (issuer) {
                    if (leader) mbar_arrive_expect_tx(&bars->full[stage], stage_tx);
                    if (args.a_mn) {
                        tma_load_3d_pair(a, &tmA, full, row0, kb * BK, 0);
                        tma_load_3d_pair(a + BOX64, &tmA, full, row0 + 64, kb * BK, 0);
                    } else if (leader || !few) {
                        tma_load_3d_pair(a, &tmA, full, kb * BK, row0, cls);
                    }
                    if (args.b_mn) {
                        for (int c = 0; c < (bn >> 1); c += 64)
                            tma_load_3d_pair(b + (c >> 6) * BOX64, tmB, full, col0 + c, kb * BK, b_at);
                    } else {
                        tma_load_3d_pair(b, tmB, full, kb * BK, col0, 0);
                    }
                }
                ++issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            u += nclusters;
            if (u < units) t = range(u, kb0, kb1);
        }
        if (!ok && issuer) {
            atomicOr(args.status, ST_PRODUCER);
            raise_abort_pair(abort_flag, cta);
        }
        // No load is left in flight into either CTA when the pair ends: the peer tells the
        // leader how many stages it loaded, and the leader waits until every stage that
        // either loaded has landed (the half that a side which gave up never loaded is
        // counted as done, or never armed).
        if (!issuer) {
        } else if (!leader) {
            st_cluster_s64(map_to_rank(&bars->peer_issued, lead), issued);
            mbar_arrive_cluster(map_to_rank(&bars->peer_done, lead));  // release: the count is visible first
        } else {
            long long ip = issued;
            if (mbar_wait(&bars->peer_done, 0, abort_flag, false))
                ip = *reinterpret_cast<volatile long long *>(&bars->peer_issued);
            else
                atomicOr(args.status, ST_DRAIN);
            const long long hi = issued > ip ? issued : ip;
            for (long long i = (hi > STAGES ? hi - STAGES : 0); i < hi; ++i) {
                const int s = (int)(i % STAGES);
                if (i >= issued) mbar_arrive_expect_tx(&bars->full[s], peer_tx);
                else if (i >= ip) mbar_complete_tx(&bars->full[s], peer_tx);
                if (!mbar_wait(&bars->full[s], (uint32_t)((i / STAGES) & 1), abort_flag, false)) {
                    atomicOr(args.status, ST_DRAIN);
                    break;
                }
            }
        }
    } else if (warp == 1 && leader) {
        // ------------------------------------------------------------ MMA issuer (leader)
        const bool issuer = elect_one();
        // K-major: a K step of 16 is 32 bytes of a 128-byte row.  MN-major: 16 rows of
        // 128 bytes, 64-element boxes BOX64 bytes apart.
        const bool a_mn = args.a_mn != 0, b_mn = args.b_mn != 0;
        const uint32_t idesc = make_idesc(FORMAT, (uint32_t)args.rows, (uint32_t)bn, a_mn, b_mn);
        const uint64_t a_desc0 = desc_sw128(smem_u32(a_tiles), a_mn ? BOX64 : 16, 1024);
        const uint64_t b_desc0 = desc_sw128(smem_u32(b_tiles), b_mn ? BOX64 : 16, 1024);
        const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        int stage = 0;
        uint32_t phase = 0;
        int it = 0;
        bool ok = true;
        for (int u = cluster; ok && u < units; u += nclusters, ++it) {
            int kb0, kb1;
            const Tile t = range(u, kb0, kb1);
            int col0;
            const uint32_t front = Epi::CLASSES && !b_mn ? args.shifts >> (4 * class_of(u, t, col0)) & 7u : 0u;
            const int buf = it & 1;
            if (!mbar_wait(&bars->acc_empty[buf], (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag, true)) { ok = false; break; }
            fence_after();
            const uint32_t d = tmem_base + (uint32_t)(buf * 256);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&bars->full[stage], phase, abort_flag, true)) { ok = false; break; }
                if (Epi::CLASSES && kb == 0 && front) {
                    __syncwarp();
                    for (uint32_t c = lead; c < lead + 2; ++c) zero_front(map_to_rank(b_tiles + stage * B_STAGE, c), bn >> 1, front, lane);
                    asm volatile("fence.acq_rel.cluster;\n\tfence.proxy.async;" ::: "memory");
                    __syncwarp();
                }
                fence_after();
                const uint64_t ad = a_desc0 + (uint64_t)((stage * A_STAGE) >> 4);
                const uint64_t bd = b_desc0 + (uint64_t)((stage * B_STAGE) >> 4);
                if (issuer) {
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ++ks)
                        if (ks * 16 < args.k_rows) mma(d, ad + ks * a_step, bd + ks * b_step, idesc, (uint32_t)(kb != kb0 || ks != 0));
                    commit_to_pair(&bars->empty[stage], lead);
                }
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (issuer) commit_to_pair(&bars->acc_full[buf], lead);
        }
        if (issuer) {
            if (!ok) {
                atomicOr(args.status, ST_MMA);
                raise_abort_pair(abort_flag, cta);
            }
            commit<2>(&bars->drain);
            if (!mbar_wait(&bars->drain, 0, abort_flag, false)) atomicOr(args.status, ST_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const bool gives = joined && half != (int)(cta >> 1);  // its columns are the other pair's
        Part p;
        p.bn = bn;
        p.lane = lane;
        p.box = staging + (joined ? quarter : warp - 2) * Epi::BOXES * STG_BOX;
        const bool thin = args.rows == 128;
        const int all = thin ? bn >> 1 : bn, left = (all / 2 + 63) & ~63;
        p.range = thin ? (quarter >> 1) * 2 + half : half;
        p.ranges = thin ? 4 : 2;
        p.first = (p.range >> 1) * all + half * left;
        p.width = half ? all - left : left;
        p.joined = nullptr;
        p.turn = 0;
        int it = 0;
        bool ok = true;
        p.split = cluster / args.tiles;
        Tile t = tile_at<Epi::LOWER>(cluster - p.split * args.tiles, args);
        pdl_wait();
        for (int u = cluster; u < units; ++it) {
            const int buf = it & 1;
            p.row0 = t.m * 256 + (thin ? (int)rank * 64 + (quarter & 1) * 32 : (int)rank * 128 + quarter * 32);
            p.tile_n = t.n;
            p.cls = class_of(u, t, p.col0);
            p.tmem = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * 256 - (thin ? (quarter >> 1) * (bn >> 1) : 0));
            const bool some = p.row0 < args.M;
            typename Epi::Pre pre;
            if (some && !gives) epi.prefetch(p, pre);
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->acc_full[buf], (uint32_t)((it >> 1) & 1), abort_flag, true))) {
                ok = false;
                break;
            }
            fence_after();
            __syncwarp();
            if (joined) {
                uint8_t *in = staging + JOIN_AT + (quarter * 32 + lane) * 16;
                if (gives) {
                    const uint32_t at = map_to_rank(in, cta ^ 2u), bar = map_to_rank(&bars->joined, cta ^ 2u);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[32];
                        tmem_ld32(p.tmem + (uint32_t)(p.first + c * 32), r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j) send4(at + c * JOIN_CHUNK + j * JOIN_QUAD, r + 4 * j, bar);
                    }
                } else {
                    if (!__all_sync(0xffffffffu, mbar_wait(&bars->joined, 0, abort_flag, true))) {
                        ok = false;
                        break;
                    }
                    p.joined = in;
                }
            }
            if (some && !gives) epi.run(p, pre);
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_read(map_to_rank(&bars->acc_empty[buf], lead));
            u += nclusters;
            if (u < units) {
                p.split = u / args.tiles;
                t = tile_at<Epi::LOWER>(u - p.split * args.tiles, args);
            }
        }
        if (lane == 0) tma_stores_wait0();
        if (!ok && lane == 0) {
            atomicOr(args.status, ST_EPILOGUE);
            raise_abort_pair(abort_flag, cta);
            if (joined && !gives) mbar_wait(&bars->joined, 0, abort_flag, false);  // sums that are on their way here
        }
    }

    __syncwarp();
    fence_before();
    cluster_sync();  // no CTA leaves while another may still touch its memory
    if (warp == 1) {
        fence_after();
        tmem_dealloc<2>(tmem_base, TMEM_COLS);
    }
}

template <uint32_t FORMAT, typename Epi>
int clusters_max(int dev) {
    static std::atomic<int> known[kMaxDevices];
    return cluster_limit(known[dev], reinterpret_cast<const void *>(pair_kernel<FORMAT, Epi>), THREADS, smem_of(Epi::BOXES), 2);
}
// The same of clusters of two joined pairs.
template <uint32_t FORMAT, typename Epi>
int joined_max(int dev) {
    static std::atomic<int> known[kMaxDevices];
    return cluster_limit(known[dev], reinterpret_cast<const void *>(pair_kernel<FORMAT, Epi>), THREADS, smem_of(Epi::BOXES), 4);
}

template <uint32_t FORMAT, typename Epi>
cudaError_t launch(const CUtensorMap &ta, const BMaps<Epi::CLASSES> &tb, const Epi &epi, const Args &args, int cmax, cudaStream_t s) {
    const long long units = (long long)args.tiles * args.splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(args.joined > 1 ? 4 * units : 2 * (units < cmax ? units : cmax)), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_of(Epi::BOXES);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)(2 * args.joined);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    pdl_attr(attr[1]);
    cfg.attrs = attr;
    cfg.numAttrs = g_pdl ? 2 : 1;
    return launch_counted(&cfg, pair_kernel<FORMAT, Epi>, ta, tb, epi, args);
}

template <uint32_t FORMAT, typename Epi>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const Epi &epi, const Args &args, int cmax, cudaStream_t s) {
    return launch<FORMAT>(ta, BMaps<false>{{tb}}, epi, args, cmax, s);
}

constexpr CUtensorMapDataType map_type(uint32_t format) {
    return format == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
// A row-major 16-bit matrix [rows, cols], rows ld elements apart, in boxes of box_rows x box_cols.
inline bool map16(CUtensorMap *m, const void *p, uint32_t format, long long rows, long long cols, long long ld, int box_rows,
                  int box_cols) {
    return make_map3(m, p, map_type(format), cols, rows, 1, ld * 2, rows * ld * 2, box_cols, box_rows, 1, 128);
}
// Rows of the tiles, where the caller takes Args::rows of 128, and of the left operand's boxes
// in tiles of `rows`, K-major.
inline int tile_rows(long long m) { return m <= 128 ? 128 : 256; }
inline int left_rows(long long m, int rows) { return m <= rows / 2 ? (int)(m + 7) / 8 * 8 : rows / 2; }
// An operand of the product from its stored matrix: mn: [K, MN] in k_rows x 64 boxes, else
// [MN, K] in boxes of `rows` x 64.
inline bool map_operand(CUtensorMap *m, const void *p, uint32_t format, bool mn, long long mn_size, long long k, long long ld,
                        int rows, int k_rows = BK) {
    return mn ? map16(m, p, format, k, mn_size, ld, k_rows, 64) : map16(m, p, format, mn_size, k, ld, rows, BK);
}

}  // namespace pair
}  // namespace gemm_gb300
