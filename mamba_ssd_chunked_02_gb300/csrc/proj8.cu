// proj8.cu -- matrix product of e4m3 operands with power-of-two scales (include/mamba2_proj.h).
//
//   out[i, j] = sum_k A[i, k] sA[i, k / 128] B[j, k] sB[j, k / 128]
//
// The scales are e8m0 bytes, which the block-scaled tcgen05.mma applies inside the tensor
// core: they are staged in shared memory four contracted blocks at a time (one 32-bit word a
// row), copied to tensor memory (tcgen05.cp) and picked by the instruction's scale id.
//
// Operands are read in place in either order (the contracted index inside or outside), so that
// no transposed copy is made: the forward product takes x and w with the contracted index
// inside, dx = dy w takes w with it outside, dw = dy^T x both.
//
// proj8_kernel: pairs of blocks whose two tensor cores work on one tile of 256 x BN (cta_group::2),
// each block with 128 rows of A and half of B's columns in its shared memory, one pair of blocks to two SMs,
// over tiles in panels.  Two accumulators in tensor memory: one tile's result leaves while the next is summed.
// Warp roles: 0 TMA, 1 MMA (and tensor memory), 2 scales of A, 3 scales of B, 4-11 epilogue,
// 12 hands the scales to the tensor cores.
//
// Bound by the tensor cores where sums are long: 32768 x 2560 x 10576 517 us in a burst (3.43 PFLOP/s; twice
// the measured bf16 rate is 3.91), 600 us when it runs on (the power limit; 464 us on zeros); by the result's
// bytes where they are short (13764 x 69 x 5968 bf16: 38 us, 4.3 TB/s); by the launch and memory's latency
// where all is small.  Single blocks with 128 x 128 tiles took 983 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "proj.cuh"
#include "tc5.cuh"
#include "tmap.h"

namespace m2 {
namespace {

using namespace tc;

constexpr int kThreads = 416;
constexpr int kDevices = 64;
// Columns of tiles a panel (32768 x 2560 x 10576: 8 528 us, 12 516, 16 511, 24 506, all 48 513; 16384 x 8192 x
// 8192: 12 608 us, 16 606, 24 612, 48 651).
constexpr int kPanel = 16;
constexpr int BM = 128, BK = 128;
constexpr int kMostPairs = 8;   // pairs that share a tile: 1, 2, 4 or 8

// D[tmem] (+)= A B with block scales (kind::mxf8f6f4: one scale per 32 contracted values).
// PAIR: two blocks' tensor cores on one tile, issued by the even one; every address holds for
// both blocks' shared and tensor memory.
template <bool PAIR>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// 32 rows of 16 bytes to 4 columns of tensor memory, the same for each 32 lanes.
template <bool PAIR> __device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Arrives at `bar` of this block, or of the pair's blocks in `mask`, when what was issued is done.
template <bool PAIR> __device__ __forceinline__ void commit(uint64_t* bar, uint32_t mask = 1) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"((uint16_t)mask)
            : "memory");
    else mma_commit(bar);
}
template <bool PAIR> __device__ __forceinline__ void alloc_tmem(uint32_t* dst, uint32_t cols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    }
}
template <bool PAIR> __device__ __forceinline__ void free_tmem(uint32_t at, uint32_t cols) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
    else tmem_dealloc(at, cols);
}
__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster's blocks meets; what they wrote before is visible behind it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void send(uint32_t at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
// This block's shared address, in the block of the cluster that has the given rank.
__device__ __forceinline__ uint32_t of_block(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same where tensor memory has been read and is given back: nothing is written that the waiter reads, and what
// orders the reads before the other block's later products are tcgen05.wait::ld, tcgen05.fence::before_thread_sync in
// front of the arrival and ::after_thread_sync behind the wait, which hold with a relaxed arrival; its scope, like that
// of the waits in proj8_kernel, is the cluster's.  The release above waits for the thread's stores, copies out among
// them, some 2000 cycles.  (Waits that all acquire at that scope: 4096 x 768 x 768 7.8 us instead of 7.5.)
__device__ __forceinline__ void arrive_read_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A tile into this block's shared memory, its bytes counted at a barrier of the pair's even block.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(m), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* m, const void* src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
// A warp whose wait ran out stays a millisecond before it goes where the block, or the cluster, meets: what other
// warps asked for and no one waits for any more (copies, products) ends within microseconds.
__device__ __noinline__ void stay() {   // once: apart from what runs when all is well
    for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < 1000000;) __nanosleep(1000);
}
__device__ __forceinline__ void linger(bool ok) {
    if (!ok) stay();
}
// Waits until the copies that were asked for, the last of each stage, have landed: at most limit_ns for all of them.
template <Scope S> __device__ __forceinline__ void land(uint64_t* full, int issued, int stages, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer();
    for (int i = issued - 1; i >= 0 && i >= issued - stages; --i) {
        const uint64_t gone = globaltimer() - t0;
        if (!mbar_wait<S>(&full[i % stages], i / stages & 1, gone < limit_ns ? limit_ns - gone : 0)) return;
    }
}
// Where a wait has run out in this block, every block of the cluster is told so: before the barrier at which they
// all meet, so that behind it all know, and none joins sums that are not there.
__device__ __forceinline__ void tell_abort(int* abort, int lane, uint32_t blocks) {
    if (lane == 0 && *reinterpret_cast<volatile int*>(abort))
        for (uint32_t r = 0; r < blocks; ++r) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(of_block(abort, r)), "r"(1) : "memory");
}
// One lane of a warp that is whole.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// 32 rows of 16 bytes: groups of 8 rows 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// kind::mxf8f6f4: e4m3 by e4m3, scales e8m0; the scale ids (bits 4 and 29) are added per block.
constexpr uint32_t idesc_mx(int M, int N, int a_mn, int b_mn) {
    return ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24);
}

struct Scales {
    const uint8_t* p;
    int64_t rs, ks;
    int shift, rows;
    bool words;   // a row's four blocks are one aligned word
};
struct Shape {
    int R, C, kb;          // rows, columns, contracted blocks
    int tr, tiles;         // tiles along the rows, in all
    int chunk;             // contracted blocks summed in tensor memory before they are added to the result
    bool copied;           // the result's rows are whole 16 bytes, and start there
    int64_t ldo;
    int split, share;      // pairs of a tile, contracted blocks of each
    Proj8Watch watch;
};

// A pair's tile of 256 x BN: a block has 128 rows of A and BN / 2 columns of B.
template <int BN, bool B_MN, int ES> struct Cfg {
    static constexpr int HALF = BN / 2;
    static constexpr int A_BYTES = BM * BK;
    // columns of B in a stage: MN-major copies are whole boxes of 128
    static constexpr int B_BYTES = (B_MN ? 128 : HALF) * BK;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    // Two accumulators and the scales of NSF sets in 512 columns.  At 256 columns the accumulators
    // share 32: a tile's products begin when those of the tile before have been read.
    static constexpr bool SHARED = BN == 256;
    static constexpr int NSF = SHARED ? 2 : 4;
    static constexpr int SFB = (BN + 127) / 128;                 // scale tiles of B
    static constexpr int SF_BYTES = 512 * (1 + SFB);
    // a part on its way out, of each of the epilogue's 8 warps: 32 rows of 128 bytes
    static constexpr int PART = 128 / ES, OUT = 32 * 128, OUT_BYTES = 8 * OUT;
    static constexpr int SPAN = (BN / 2 + 63) / 64 * 64;         // columns of the epilogue's first four warps
    static constexpr int FIXED = 1024 + NSF * SF_BYTES + OUT_BYTES;
    static constexpr int NS = (227 * 1024 - FIXED - 512) / STAGE < 6 ? (227 * 1024 - FIXED - 512) / STAGE : 6;
    static constexpr int SMEM = FIXED + NS * STAGE;
    static constexpr uint32_t ACC = SHARED ? BN - 32 : BN;       // from one accumulator to the other
    static constexpr uint32_t SF_COL = ACC + BN, SF_COLS = 4 * (1 + SFB);
    static constexpr uint32_t COLS = 512;
    static_assert(SF_COL + NSF * SF_COLS <= COLS, "tensor memory");
    static_assert(STAGE % 1024 == 0 && HALF <= 128, "tiles");
};

struct Bars {
    uint64_t full[6], empty[6];
    uint64_t sf_there[4], sf_full[4], sf_empty[4];
    uint64_t acc_full[2], acc_empty[2], acc_shared;
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// The scales of four rows (32 apart) for the contracted blocks k0 .. k0 + 3, as the 16 bytes that
// a lane of the tensor memory's copy holds.  Rows and blocks behind the ends read the last one's:
// what they scale is zero or not stored.  No branches, so that all loads are in flight at once.
__device__ __forceinline__ uint4 gather_scales(const Scales& s, bool words, const uint8_t* const* at, int k0, int kb) {
    uint32_t w[4];
    if (words) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(at[j] + k0));
    } else {
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t off = min(k0 + k, kb - 1) * s.ks;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j][k] = __ldg(at[j] + off);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j][0] | v[j][1] << 8 | v[j][2] << 16 | v[j][3] << 24;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// SPLIT: a cluster of q.split pairs takes one tile, a share of the contracted blocks each.
template <int BN, bool A_MN, bool B_MN, typename TO, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
proj8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
             const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_half, const Scales sa,
             const Scales sb, TO* __restrict__ out, const Shape q,
             int32_t* err) {
    using C = Cfg<BN, B_MN, sizeof(TO)>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* sout = smem + C::NS * C::STAGE;
    uint8_t* ssf = sout + C::OUT_BYTES;
    __shared__ Bars bars;
    volatile int* abort = &bars.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the even block (rank 0 of the pair) counts the copies and issues the products of both
    const int in_cluster = (int)block_rank(), rank = SPLIT ? in_cluster & 1 : in_cluster, even = in_cluster - rank;
    const uint32_t both = 3u << even;
    const int first = blockIdx.x / (SPLIT ? 2 * q.split : 2), step = SPLIT ? q.tiles : gridDim.x / 2;
    const int from_k = SPLIT ? (even >> 1) * q.share : 0, to_k = SPLIT ? min(q.kb, from_k + q.share) : q.kb;
    constexpr int kRows = 2 * BM;
    // Tiles go down panels of kPanel columns of tiles, a row of the panel at a time: the clusters that
    // run side by side then share few rows of A and of B.
    const auto place = [&](int tile, int* r, int* c) {
        const int tc = q.tiles / q.tr, each = kPanel * q.tr, p = tile / each, in = tile - p * each,
                  w = min(kPanel, tc - p * kPanel);
        *r = in / w;
        *c = p * kPanel + in - *r * w;
    };
    const auto row_of = [&](int r) { return r * kRows + rank * BM; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < C::NSF; ++i) {
            mbar_init(&bars.sf_there[i], 2);   // warps 2 and 3
            mbar_init(&bars.sf_full[i], 2);    // two blocks
            mbar_init(&bars.sf_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 16);   // eight warps of two blocks
        }
        mbar_init(&bars.acc_shared, 8);         // the four warps of two blocks that read the shared columns
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) alloc_tmem<true>(&bars.tmem, C::COLS);
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    grid_dep_wait();   // what is read was written by the kernel before
    [[maybe_unused]] float sum[SPLIT ? 64 : 1] = {};   // of a row, 64 columns: a warp's of the pair's share
    // The producing and the issuing warp run whole, with one lane elected for each instruction: what
    // the loop counts then stays in uniform registers, where the copies and products take it from
    // (issued from a loop of one lane, four products took 650 cycles instead of 450).
    if (warp == 0) {
        if (elected()) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
        }
        int it = 0, st = 0;
        uint32_t phase = 1;
        bool ok = true;
        const uint32_t full0 = of_block(&bars.full[0], even);
        for (int tile = first; tile < q.tiles && ok; tile += step) {
            int r, c;
            place(tile, &r, &c);
            const int r0 = row_of(r), c0 = c * BN + rank * C::HALF;
            for (int kb = from_k; kb < to_k; ++kb, ++it) {
                ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.empty[st], phase, abort, q.watch.limit_ns));
                if (!ok) break;
                if (elected()) {
                    uint8_t* a = smem + st * C::STAGE;
                    uint8_t* b = a + C::A_BYTES;
                    if (rank == 0) mbar_arrive_expect_tx(&bars.full[st], 2 * C::STAGE);
                    const uint32_t bar = full0 + 8 * st;
                    tma_load_pair(a, &tm_a, bar, A_MN ? r0 : kb * BK, A_MN ? kb * BK : r0);
                    tma_load_pair(b, &tm_b, bar, B_MN ? c0 : kb * BK, B_MN ? kb * BK : c0);
                }
                __syncwarp();
                if (++st == C::NS) st = 0, phase ^= 1;
            }
        }
        grid_dep_launch();   // all copies are asked for: the next kernel may set itself up as blocks end
        // the even block's barriers count both blocks' copies
        if (!ok && rank == 0 && lane == 0) land<kClusterBare>(bars.full, it, C::NS, q.watch.limit_ns);
        linger(ok);
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = idesc_mx(kRows, BN, A_MN, B_MN);
            constexpr uint32_t a_step = (A_MN ? 32 * 128 : 32) >> 4, b_step = (B_MN ? 32 * 128 : 32) >> 4;
            // K-major: 8-row groups 1024 bytes apart; MN-major: the same between 8 contracted rows (one
            // block of 128 m or n)
            const uint64_t a0 = smem_desc_sw128(smem_u32(smem), A_MN ? 128 * BK : 16, 1024);
            const uint64_t b0 = smem_desc_sw128(smem_u32(smem) + C::A_BYTES, B_MN ? 128 * BK : 16, 1024);
            const uint64_t s0 = scale_desc(smem_u32(ssf));
            int st = 0, sf = 0, t = 0;
            uint32_t phase = 0, sf_phase = 0;
            bool ok = true;
            for (int tile = first; tile < q.tiles && ok; tile += step)
                for (int k0 = from_k; k0 < to_k && ok; k0 += q.chunk, ++t) {
                    const int acc = t & 1, k1 = min(to_k, k0 + q.chunk);
                    ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.acc_empty[acc], (t / 2 & 1) ^ 1, abort, q.watch.limit_ns));
                    if (C::SHARED && ok && t > 0)
                        ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.acc_shared, (t - 1) & 1, abort, q.watch.limit_ns));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + acc * C::ACC;
                    bool there = false;   // the next stage's operands, asked for ahead
                    for (int kb = k0; kb < k1 && ok; kb += 4) {
                        const uint32_t ta = tmem + C::SF_COL + sf * C::SF_COLS;
                        ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kCluster>(&bars.sf_full[sf], sf_phase, abort, q.watch.limit_ns));
                        if (!ok) break;
                        tc_fence_after();
                        if (elected()) {
                            const uint64_t from = s0 + (uint32_t)(sf * (C::SF_BYTES >> 4));
#pragma unroll
                            for (int h = 0; h <= C::SFB; ++h) copy_scales<true>(ta + 4 * h, from + h * (512 >> 4));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (kb + i >= k1) break;
                            if (!there) {
                                ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.full[st], phase, abort, q.watch.limit_ns));
                                if (!ok) break;
                            }
                            tc_fence_after();
                            const int now = st;
                            if (++st == C::NS) st = 0, phase ^= 1;
                            const bool last = kb + i + 1 == k1;
                            there = !last && mbar_test_wait<kClusterBare>(smem_u32(&bars.full[st]), phase);
                            if (elected()) {
                                const uint32_t at = now * (C::STAGE >> 4);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_scaled<true>(d, a0 + at + k * a_step, b0 + at + k * b_step, idesc | i << 4 | i << 29, ta,
                                                     ta + 4, kb > k0 || i > 0 || k > 0);
                                commit<true>(&bars.empty[now], both);
                                if (i == 3 || last) commit<true>(&bars.sf_empty[sf], both);
                                if (last) commit<true>(&bars.acc_full[acc], both);
                            }
                            there = __all_sync(0xffffffffu, there);
                        }
                        if (++sf == C::NSF) sf = 0, sf_phase ^= 1;
                    }
                }
            if (!ok && elected()) {
                commit<true>(&bars.drain, 1u << even);
                mbar_wait(&bars.drain, 0, q.watch.limit_ns);
            }
            linger(ok);
        }
    } else if (warp < 4) {
        // The scales of the next kFly sets are on their way while this set's room is waited for (a load
        // takes 2000 cycles beside the copies, a set's products 1800), and places are worked out once a
        // tile: what a set costs this warp is on the products' path.
        constexpr int kFly = 3;
        const Scales& s = warp == 2 ? sa : sb;
        const int parts = warp == 2 ? 1 : C::SFB;
        const uint8_t* at[4 * C::SFB];   // scales of rows lane + 32 j of the tile
        uint4 next[kFly][C::SFB];
        int tile = first, kb = from_k;
        const auto begin = [&] {
            int r, c;
            place(tile, &r, &c);
            const int r0 = warp == 2 ? row_of(r) : c * BN;
#pragma unroll
            for (int j = 0; j < 4 * C::SFB; ++j)
                at[j] = s.p + (int64_t)(min(r0 + lane + 32 * j, s.rows - 1) >> s.shift) * s.rs;
        };
        const auto gather = [&](uint4 (&to)[C::SFB]) {   // the set at (tile, kb), and on to the one after it
            if (tile >= q.tiles) return;
#pragma unroll
            for (int h = 0; h < C::SFB; ++h)
                if (h < parts) to[h] = gather_scales(s, s.words, at + 4 * h, kb, q.kb);
            if ((kb += 4) >= to_k) {
                kb = from_k;
                if ((tile += step) < q.tiles) begin();
            }
        };
        int left = first < q.tiles ? (q.tiles - 1 - first) / step + 1 : 0;
        left *= (to_k - from_k + 3) / 4;
        int sf = 0;
        uint32_t phase = 1;
        if (left) begin();
#pragma unroll
        for (int u = 0; u < kFly; ++u) gather(next[u]);
        bool ok = true;
        while (left > 0 && ok) {
#pragma unroll
            for (int u = 0; u < kFly; ++u) {
                if (left <= 0 || !ok) break;
                uint4 w[C::SFB];
#pragma unroll
                for (int h = 0; h < C::SFB; ++h) w[h] = next[u][h];
                ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kCluster>(&bars.sf_empty[sf], phase, abort, q.watch.limit_ns));
                if (!ok) break;
                uint4* to = reinterpret_cast<uint4*>(ssf + sf * C::SF_BYTES) + (warp == 2 ? 0 : 32) + lane;
#pragma unroll
                for (int h = 0; h < C::SFB; ++h)
                    if (h < parts) to[32 * h] = w[h];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.sf_there[sf]);
                gather(next[u]);
                if (++sf == C::NSF) sf = 0, phase ^= 1;
                --left;
            }
        }
        linger(ok);
    } else if (warp == 12) {
        // Scales in shared memory to the tensor cores' proxy.  A warp of its own, as the fence waits for
        // all that its warp has in flight: behind the loads of later sets it took 2000 cycles.
        if (lane == 0) {
            const uint32_t full0 = of_block(&bars.sf_full[0], even);
            int left = first < q.tiles ? ((q.tiles - 1 - first) / step + 1) * ((to_k - from_k + 3) / 4) : 0;
            if (q.watch.withhold && in_cluster == 1) left = 0;
            int sf = 0;
            for (uint32_t phase = 0; left > 0; --left) {
                if (!mbar_wait_or_abort(&bars.sf_there[sf], phase, abort, q.watch.limit_ns)) break;
                fence_proxy_async_smem();
                arrive_at(full0 + 8 * sf);
                if (++sf == C::NSF) sf = 0, phase ^= 1;
            }
            linger(left <= 0);
        }
    } else if constexpr (SPLIT) {
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        int t = 0;
        for (int k0 = from_k; k0 < to_k; k0 += q.chunk, ++t) {
            const int acc = t & 1;
            ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.acc_full[acc], t / 2 & 1, abort, q.watch.limit_ns));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t v[32];
                tmem_ld32_sync(tmem + acc * C::ACC + lanes + 64 * ((warp - 4) >> 2) + 32 * u, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[32 * u + j] += __uint_as_float(v[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_read_at(of_block(&bars.acc_empty[acc], even));
        }
        linger(ok);
    } else {
        // A warp has 32 lanes of tensor memory, the tile's rows, and moves lines of 128 bytes of half the
        // columns: rounded, into shared memory, and by TMA to the result (coalesced stores where the result's
        // rows are not whole pieces of 16 bytes: 13764 x 69 x 5967 bf16 70 us, x 5968 38 us).
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int begin = half * C::SPAN, end = half ? BN : C::SPAN;
        uint8_t* part = sout + (warp - 4) * C::OUT;
        int t = 0;
        bool ok = true;
        for (int tile = first; tile < q.tiles && ok; tile += step) {
            int rt, ct;
            place(tile, &rt, &ct);
            for (int k0 = 0; k0 < q.kb; k0 += q.chunk, ++t) {
                const int acc = t & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_or_abort<kClusterBare>(&bars.acc_full[acc], t / 2 & 1, abort, q.watch.limit_ns));
                if (!ok) break;
                tc_fence_after();
                const int r0 = row_of(rt) + quad * 32, c0 = ct * BN;
                const uint32_t from = tmem + acc * C::ACC + ((uint32_t)(quad * 32) << 16);
                if (k0 > 0) {   // what is added to has been written
                    if (elected()) bulk_wait<0>();
                    __syncwarp();
                }
                // the columns that the next tile's accumulator shares come first: the last 32 of the even
                // accumulator, the first of the odd one
                const bool back = C::SHARED && acc == 0 && half == 1;
#pragma unroll 1
                for (int at = begin; at < end; at += C::PART) {
                    const int c = back ? begin + end - C::PART - at : at;
                    const bool wide = C::PART == 64 && c + 64 <= end;
                    uint32_t v[C::PART / 32][32];
                    tmem_ld32(from + c, v[0]);
                    if (C::PART == 64 && wide) tmem_ld32(from + c + 32, v[C::PART / 32 - 1]);
#pragma unroll
                    for (int h = 0; h < C::PART / 32; ++h) tmem_wait_ld_regs(v[h]);
                    if (C::SHARED && at == begin && half != acc) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_read_at(of_block(&bars.acc_shared, even));
                    }
                    if (r0 >= q.R || c0 + c >= q.C) continue;
                    if (elected()) bulk_wait_read<0>();   // the last copy has read the part
                    __syncwarp();
                    // 16-byte pieces in the places where a swizzled copy looks for them
                    const int line = sizeof(TO) == 2 && !wide ? 64 : 128;
                    uint4* row = reinterpret_cast<uint4*>(part + lane * line);
                    const int turn = line == 64 ? lane >> 1 & 3 : lane & 7;
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        if constexpr (sizeof(TO) == 2) {
                            if (p >= 4 && !wide) break;
                            const uint32_t* f = v[p / 4] + 8 * (p & 3);
                            row[p ^ turn] = make_uint4(pack_bf16x2(__uint_as_float(f[0]), __uint_as_float(f[1])),
                                                       pack_bf16x2(__uint_as_float(f[2]), __uint_as_float(f[3])),
                                                       pack_bf16x2(__uint_as_float(f[4]), __uint_as_float(f[5])),
                                                       pack_bf16x2(__uint_as_float(f[6]), __uint_as_float(f[7])));
                        } else {
                            row[p ^ turn] = make_uint4(v[0][4 * p], v[0][4 * p + 1], v[0][4 * p + 2], v[0][4 * p + 3]);
                        }
                    }
                    if (q.copied) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (elected()) {
                            if (k0 > 0) tma_reduce_add_2d(&tm_o, part, c0 + c, r0);
                            else tma_store_2d(C::PART == 64 && !wide ? &tm_half : &tm_o, part, c0 + c, r0);
                            bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        const int rows = min(32, q.R - r0);
                        constexpr int E = 16 / sizeof(TO);
#pragma unroll
                        for (int h = 0; h < C::PART / 32; ++h) {
                            const int col = 32 * h + lane;
                            if (c0 + c + col >= q.C || col >= end - c) break;
                            TO* o = out + (int64_t)r0 * q.ldo + c0 + c + col;
#pragma unroll 8
                            for (int r = 0; r < rows; ++r, o += q.ldo) {
                                const int piece = col / E ^ (line == 64 ? r >> 1 & 3 : r & 7);
                                const TO w = reinterpret_cast<const TO*>(part + r * line)[piece * E + col % E];
                                if (sizeof(TO) == 2 || k0 == 0) *o = w;
                                else atomicAdd(reinterpret_cast<float*>(o), to_f32(w));   // this thread's alone: no load waited for
                            }
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_read_at(of_block(&bars.acc_empty[acc], even));
            }
        }
        __syncwarp();
        if (elected()) bulk_wait<0>();   // copies out of this block's shared memory
        linger(ok);
    }
    __syncwarp();
    if constexpr (SPLIT) {
        tell_abort(&bars.abort, lane, 2 * q.split);
        __syncwarp();
    }
    tc_fence_before();
    cluster_sync();
    if constexpr (SPLIT) {
        // Every pair is done with its operands, whose room takes the shares' sums: a block owns BN / split
        // of its 128 rows' columns, gets them from the blocks of its half of the rows, and adds them in the
        // order of the pairs.  In fours of a row's columns, a column of fours 129 rows apart from the next:
        // lanes are rows when they are sent, fours of a row when they are read.
        static_assert(BN == 128 && C::NS * C::STAGE >= BN / 4 * 129 * 16, "room for the sums");
        constexpr int P = BM + 1;
        const int own = BN / q.split, fours = own / 4, tid = threadIdx.x - 128;   // powers of two
        float4* join = reinterpret_cast<float4*>(smem);   // [pair][four][row]
        if (warp >= 4 && warp < 12 && !*abort) {
            const int row = (warp & 3) * 32 + lane, c0 = 64 * ((warp - 4) >> 2);
#pragma unroll
            for (int g = 0; g < 4; ++g) {   // sixteen columns have one owner
                const int c = c0 + 16 * g;
                uint32_t to = of_block(join + ((even >> 1) * fours + (c & (own - 1)) / 4) * P + row, 2 * (c / own) + rank);
#pragma unroll
                for (int j = 0; j < 16; j += 4, to += P * 16)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(sum[16 * g + j]),
                                 "f"(sum[16 * g + j + 1]), "f"(sum[16 * g + j + 2]), "f"(sum[16 * g + j + 3])
                                 : "memory");
            }
        }
        cluster_sync();
        if (warp >= 4 && warp < 12 && !*abort) {
            int rt, ct;
            place(first, &rt, &ct);
            const int four = tid & (fours - 1), r0 = row_of(rt), c0 = ct * BN + (even >> 1) * own + 4 * four;
            const int rows = min(BM, q.R - r0), cols = q.C - c0;
            if (cols > 0)
#pragma unroll 2
                for (int row = tid / fours; row < rows; row += 256 / fours) {
                    const float4* at = join + four * P + row;
                    float4 v = at[0];
#pragma unroll
                    for (int s = 1; s < kMostPairs; ++s)
                        if (s < q.split) {
                            const float4 w = at[s * fours * P];
                            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                        }
                    TO* o = out + (int64_t)(r0 + row) * q.ldo + c0;
                    if (q.copied) {   // whole pieces of 16 bytes
                        if constexpr (sizeof(TO) == 2)
                            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(o) = v;
                    } else {
                        o[0] = from_f32<TO>(v.x);
                        if (cols > 1) o[1] = from_f32<TO>(v.y);
                        if (cols > 2) o[2] = from_f32<TO>(v.z);
                        if (cols > 3) o[3] = from_f32<TO>(v.w);
                    }
                }
        }
    }
    if (threadIdx.x == 0 && *abort) record_error(err, kErrTimeoutProj8);
    if (warp == 1) {
        tc_fence_after();
        free_tmem<true>(tmem, C::COLS);
    }
}

// ---- few rows --------------------------------------------------------------------------
// Where the result's rows are few (single tokens), the operand that is read once is the large one:
// its rows are the accumulator's lanes, 128 a tile, and BN columns hold the few.  A cluster of
// blocks splits a tile's contracted blocks; each column of the tile belongs to one of them, to
// which the others send their parts through the cluster's shared memory, and which adds them in the
// order of the blocks.
// Warp roles: 0 TMA, 1 MMA (and tensor memory), 2-5 scales, then the epilogue.
constexpr int kFewThreads = 192;
constexpr int kFewRows = 128;
constexpr int kFewBlocks = 32;   // contracted blocks a block: its scales stay in tensor memory

template <int BN> struct Few {
    static constexpr int A_BYTES = BM * BK, STAGE = A_BYTES + BN * BK;
    static constexpr int SETS = kFewBlocks / 4;
    static constexpr int SF_BYTES = 1024;                // of a set: 128 rows of A and of B
    static constexpr uint32_t COLS = 128;
    static_assert(BN + SETS * 8 <= 128, "tensor memory");
    // parts of the block's own columns, from every block of the cluster
    static int join_bytes(int split) { return split > 1 ? (BN + split - 1) / split * split * BM * 4 : 0; }
    // stages of a block that shares its SM with `others`
    static int stages(int split, int others) {
        return (227 * 1024 / (1 + others) - 2048 - 1024 - SETS * SF_BYTES - join_bytes(split)) / STAGE;
    }
    static int smem(int split, int ns) { return 1024 + ns * STAGE + SETS * SF_BYTES + join_bytes(split); }
};
constexpr int kFewStages = 8;
// Shared memory that leaves room for no more blocks on an SM than its tensor memory has columns for: a block that
// waits for columns never holds up one of another cluster, which may hold the columns that its own cluster waits for.
constexpr int kFewLeast = 47 * 1024;
static_assert(4 * Few<64>::COLS <= 512 && 5 * (kFewLeast + 1024) > 228 * 1024, "four blocks an SM");

struct FewShape {
    int R, C, kb;     // lanes' rows, few rows, contracted blocks
    int ns;           // stages
    int64_t ldo;
    Proj8Watch watch;
};

template <int BN, bool A_MN, typename TO>
__global__ void __launch_bounds__(kFewThreads, 2)
proj8_few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Scales sa,
                 const Scales sb, TO* __restrict__ out, const FewShape q, int32_t* err) {
    using C = Few<BN>;
    constexpr int STAGE = C::STAGE;
    const int ns = q.ns;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ssf = smem + ns * STAGE;
    float* join = reinterpret_cast<float*>(ssf + C::SETS * C::SF_BYTES);   // [block][own column][128]
    struct FewBars {
        uint64_t full[kFewStages], empty[kFewStages], sf_full, acc_full, drain;
        uint32_t tmem;
        int abort;
    };
    __shared__ FewBars bars;
    volatile int* abort = &bars.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const uint32_t rank = block_rank();
    const int r0 = (int)(blockIdx.x / split) * BM, c0 = blockIdx.y * BN;
    const int k0 = (int)((int64_t)q.kb * rank / split), n = (int)((int64_t)q.kb * (rank + 1) / split) - k0;

    // Warps 2 to 5 ask for their first set's scales before anything is set up: what the products wait
    // for longest (2 us after the others were ready).
    const uint8_t *at[4], *bt[4];
    uint4 sets[2];
    const bool whole = k0 % 4 == 0;   // words start where the block's share does
    const auto gather = [&](int set) {
        sets[0] = gather_scales(sa, sa.words && whole, at, k0 + 4 * set, k0 + n);
        sets[1] = gather_scales(sb, sb.words && whole, bt, k0 + 4 * set, k0 + n);
    };
    if (warp >= 2) {
        grid_dep_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            at[j] = sa.p + (int64_t)(min(r0 + lane + 32 * j, sa.rows - 1) >> sa.shift) * sa.rs;
            bt[j] = sb.p + (int64_t)(min(c0 + lane + 32 * j, sb.rows - 1) >> sb.shift) * sb.rs;
        }
        if (4 * (warp - 2) < n) gather(warp - 2);
    } else if (warp == 0) {
        if (elected()) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
        }
        if (lane < ns) {
            mbar_init(&bars.full[lane], 1);
            mbar_init(&bars.empty[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&bars.sf_full, 128);
            mbar_init(&bars.acc_full, 1);
            mbar_init(&bars.drain, 1);
            bars.abort = 0;
        }
        fence_barrier_init();
    } else {
        alloc_tmem<false>(&bars.tmem, C::COLS);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    if (split > 1) cluster_arrive();   // this block has begun
    bool ok = true;

    if (warp == 0) {
        grid_dep_wait();     // what is read was written by the kernel before
        grid_dep_launch();   // the next one may set itself up beside this one
        int st = 0, it = 0;
        for (uint32_t phase = 1; it < n; ++it) {
            ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars.empty[st], phase, abort, q.watch.limit_ns));
            if (!ok) break;
            if (elected()) {
                const int k = (k0 + it) * BK;
                uint8_t* a = smem + st * STAGE;
                mbar_arrive_expect_tx(&bars.full[st], STAGE);
                tma_load_2d(a, &tm_a, &bars.full[st], A_MN ? r0 : k, A_MN ? k : r0);
                tma_load_2d(a + C::A_BYTES, &tm_b, &bars.full[st], k, c0);
            }
            __syncwarp();
            if (++st == ns) st = 0, phase ^= 1;
        }
        if (!ok && lane == 0) land<kBlock>(bars.full, it, ns, q.watch.limit_ns);
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_mx(BM, BN, A_MN, 0);
        constexpr uint32_t a_step = (A_MN ? 32 * 128 : 32) >> 4, b_step = 32 >> 4;
        const uint64_t a0 = smem_desc_sw128(smem_u32(smem), A_MN ? 128 * BK : 16, 1024);
        const uint64_t b0 = smem_desc_sw128(smem_u32(smem) + C::A_BYTES, 16, 1024);
        const uint64_t s0 = scale_desc(smem_u32(ssf));
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars.sf_full, 0, abort, q.watch.limit_ns));
        tc_fence_after();
        int st = 0;
        uint32_t phase = 0;
        for (int i = 0; i < n && ok; ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars.full[st], phase, abort, q.watch.limit_ns));
            if (!ok) break;
            tc_fence_after();
            if (elected()) {
                const uint32_t set = i / 4, id4 = i & 3, ta = tmem + BN + set * 8;
                if (id4 == 0) {
                    copy_scales<false>(ta, s0 + set * (C::SF_BYTES >> 4));
                    copy_scales<false>(ta + 4, s0 + set * (C::SF_BYTES >> 4) + (512 >> 4));
                }
                const uint32_t at = st * (STAGE >> 4), id = idesc | id4 << 4 | id4 << 29;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_scaled<false>(tmem, a0 + at + k * a_step, b0 + at + k * b_step, id, ta, ta + 4, i > 0 || k > 0);
                commit<false>(&bars.empty[st]);
                if (i + 1 == n) commit<false>(&bars.acc_full);
            }
            __syncwarp();
            if (++st == ns) st = 0, phase ^= 1;
        }
        if (!ok && elected()) {   // products in flight are done before the block ends
            commit<false>(&bars.drain);
            mbar_wait(&bars.drain, 0, q.watch.limit_ns);
        }
    }
    const int quad = warp & 3, row = quad * 32 + lane;   // of the tile, where the warp is an epilogue's
    const int cols = min(BN, q.C - c0);
    const uint32_t own = (BN + split - 1) / split;   // columns a block
    if (warp >= 2) {
        for (int set = warp - 2; 4 * set < n; set += 4) {
            if (set > warp - 2) gather(set);
            uint4* to = reinterpret_cast<uint4*>(ssf + set * C::SF_BYTES) + lane;
            to[0] = sets[0];
            to[32] = sets[1];
        }
        fence_proxy_async_smem();
        if (!(q.watch.withhold && rank == 0 && warp == 2)) mbar_arrive(&bars.sf_full);
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars.acc_full, 0, abort, q.watch.limit_ns));
        tc_fence_after();
        if (split > 1) cluster_wait();   // the others have begun
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16);
        TO* o = out + (int64_t)c0 * q.ldo + r0 + row;
        uint32_t owner = 0, slot = 0;   // of column c + j
        uint32_t part = split > 1 ? of_block(join + rank * own * BM + row, 0) : 0;
#pragma unroll 1
        for (int c = 0; c < cols && ok; c += 16) {
            uint32_t v[16];
            tmem_ld16_sync(from + c, v);
            if (split > 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (c + j < cols) send(part, __uint_as_float(v[j]));
                    part += BM * 4;
                    if (++slot == own && ++owner < split) slot = 0, part = of_block(join + rank * own * BM + row, owner);
                }
            } else if (r0 + row < q.R) {
#pragma unroll
                for (int j = 0; j < 16; ++j, o += q.ldo)
                    if (c + j < cols) *o = from_f32<TO>(__uint_as_float(v[j]));
            }
        }
    } else if (split > 1) {
        __syncwarp();
        cluster_wait();
    }
    linger(ok);
    __syncwarp();
    if (split > 1) tell_abort(&bars.abort, lane, split);
    __syncwarp();
    tc_fence_before();
    if (split > 1) {
        cluster_sync();   // the parts are there
        if (warp >= 2 && r0 + row < q.R && !*abort) {
            const int from_c = rank * own, to_c = min(cols, from_c + (int)own);
            TO* o = out + (int64_t)(c0 + from_c) * q.ldo + r0 + row;
            const float* from = join + row;
#pragma unroll 2
            for (int c = from_c; c < to_c; ++c, from += BM, o += q.ldo) {
                float sum = from[0];
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    if (s < (int)split) sum += from[s * own * BM];
                *o = from_f32<TO>(sum);
            }
        }
    } else {
        __syncthreads();
    }
    if (threadIdx.x == 0 && *abort) record_error(err, kErrTimeoutProj8);
    if (warp == 1) {
        tc_fence_after();
        free_tmem<false>(tmem, C::COLS);
    }
}

// `across` contracted values (MN-major) or rows (K-major) a copy; 128 of the inner index.
bool map_of(CUtensorMap* m, const Operand& o, int64_t rows, int64_t depth, int across) {
    const uint64_t dims[2] = {(uint64_t)(o.mn ? rows : depth), (uint64_t)(o.mn ? depth : rows)};
    const uint64_t strides[1] = {(uint64_t)o.pitch};
    const uint32_t box[2] = {128, (uint32_t)across};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.q, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A launch in clusters of `blocks` along x (a lone block is one of its own).
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(int threads, int smem, int blocks, cudaStream_t st) {
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    // May begin while the kernel before it ends (and waits for it before it reads anything).
    void early() {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
};
// Clusters of `blocks` that the device holds at once (`known`: what was found before, by device).
template <typename K> int resident_clusters(K k, cudaLaunchConfig_t cfg, int blocks, std::atomic<int>* known) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return std::max(1, sm_count() / blocks);
    if ((n = known[dev].load(std::memory_order_relaxed))) return n;
    cfg.gridDim = dim3((unsigned)(sm_count() / blocks * blocks));
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = std::max(1, sm_count() / blocks);
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

Scales scales_of(const Operand& o, int64_t rows, int kb) {
    const bool words = o.ks == 1 && o.rs % 4 == 0 && kb <= o.rs && reinterpret_cast<uintptr_t>(o.s) % 4 == 0;
    return Scales{o.s, o.rs, o.ks, o.shift, (int)rows, words};
}

// Contracted blocks whose sum may stay in tensor memory for an fp32 result.  The tensor cores'
// sums lose up to 2^-23 of the sum a step, toward zero: 47 steps of 32 are off by 1.6e-7 of a
// result's norm, 1024 by 3.5e-6 where sums in fp32 registers are off by 5e-7.
constexpr int kChunk = 32;

// Contracted blocks of a pair, where a tile's are split: whole words of scales each.
int share_of(int kb, int split) { return split == 1 ? kb : ((kb + split - 1) / split + 3) / 4 * 4; }

// Clusters of `split` pairs with a tile of 128 columns each that the device holds at once.
template <bool A_MN, bool B_MN, typename TO> int split_clusters(int split) {
    using C = Cfg<128, B_MN, sizeof(TO)>;
    auto k = proj8_kernel<128, A_MN, B_MN, TO, true>;
    static std::atomic<uint64_t> done;
    static std::atomic<int> known[kMostPairs + 1][kDevices];
    if (allow_smem(k, C::SMEM, done, true) != cudaSuccess) return 0;
    const Launch l(kThreads, C::SMEM, 2 * split, nullptr);
    return resident_clusters(k, l.cfg, 2 * split, known[split]);
}

template <int BN, bool A_MN, bool B_MN, typename TO, bool SPLIT = false>
cudaError_t go(const Operand& A, const Operand& B, int64_t R, int64_t Cn, int64_t depth, TO* out, int64_t ldo,
               const Proj8Watch& watch, cudaStream_t st, int split = 1) {
    using C = Cfg<BN, B_MN, sizeof(TO)>;
    CUtensorMap ma, mb, mo, mh;
    if (!map_of(&ma, A, R, depth, 128) || !map_of(&mb, B, Cn, depth, B_MN ? BK : C::HALF))
        return cudaErrorInvalidValue;
    // the result by copies of 32 lines, where its rows start on 16 bytes and are whole ones (a copy out
    // is clipped to 16 bytes, not to elements: it would write behind the row's end)
    const uint64_t dims[2] = {(uint64_t)Cn, (uint64_t)R};
    const uint64_t strides[1] = {(uint64_t)((R == 1 ? Cn : ldo) * sizeof(TO))};
    const uint32_t box[2] = {C::PART, 32}, half[2] = {32, 32};
    const CUtensorMapDataType type = sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const bool copied = reinterpret_cast<uintptr_t>(out) % 16 == 0 && strides[0] % 16 == 0 && Cn * sizeof(TO) % 16 == 0 &&
                        make_tmap(&mo, type, out, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
                        (C::PART == 32 || make_tmap(&mh, type, out, 2, dims, strides, half, CU_TENSOR_MAP_SWIZZLE_64B));
    if (!copied) mo = ma;   // not used
    if (!copied || C::PART == 32) mh = ma;
    constexpr int kRows = 2 * BM;
    const int64_t tr = (R + kRows - 1) / kRows, tiles = tr * ((Cn + BN - 1) / BN);
    if (tiles >= (int64_t(1) << 30)) return kGridLimit;
    const int kb = (int)((depth + BK - 1) / BK);
    if ((int64_t)(split - 1) * share_of(kb, split) >= kb) return cudaErrorInvalidValue;   // a pair without blocks
    const Shape q{(int)R, (int)Cn, kb, (int)tr, (int)tiles, sizeof(TO) == 4 ? kChunk : kb, copied, ldo, split, share_of(kb, split),
                  watch};
    const Scales sa = scales_of(A, R, kb), sb = scales_of(B, Cn, kb);
    auto k = proj8_kernel<BN, A_MN, B_MN, TO, SPLIT>;
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(k, C::SMEM, done, SPLIT);
    if (e != cudaSuccess) return e;
    Launch l(kThreads, C::SMEM, 2 * split, st);
    l.early();
    static std::atomic<int> known[kDevices];
    const int64_t most = SPLIT ? tiles : resident_clusters(k, l.cfg, 2, known);
    l.cfg.gridDim = dim3((unsigned)(2 * split * (tiles < most ? tiles : most)));
    return cudaLaunchKernelEx(&l.cfg, k, ma, mb, mo, mh, sa, sb, out, q, device_error_word());
}

// A's rows to the lanes, B's few to the columns: out[j * ldo + i].
template <int BN, bool A_MN, typename TO>
cudaError_t go_few(const Operand& A, const Operand& B, int64_t R, int64_t Cn, int64_t depth, TO* out, int64_t ldo,
                   const Proj8Watch& watch, cudaStream_t st) {
    using C = Few<BN>;
    CUtensorMap ma, mb;
    if (!map_of(&ma, A, R, depth, 128) || !map_of(&mb, B, Cn, depth, BN)) return cudaErrorInvalidValue;
    const int64_t tr = (R + BM - 1) / BM, tc = (Cn + BN - 1) / BN;
    if (tr * 8 >= (int64_t(1) << 31) || tc > 65535) return kGridLimit;
    FewShape q{(int)R, (int)Cn, (int)((depth + BK - 1) / BK), 0, ldo, watch};
    auto k = proj8_few_kernel<BN, A_MN, TO>;
    constexpr int most = 226 * 1024;
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(k, most, done);
    if (e != cudaSuccess) return e;
    // The most blocks a tile with which all run at once, an SM to each (with w in L2: 10576 x 2560, 83 tiles, one
    // token: 8.5 us with one block a tile, 8.9 with three, two to an SM; 2560 x 5120, 20 tiles: 9.0 with
    // two, 6.5 with five, 10.7 with seven, of which some clusters wait); fewer where the largest share
    // stays the same.  A block's share is at most kFewBlocks.
    static std::atomic<int> known[9][kDevices];
    int split = (q.kb + kFewBlocks - 1) / kFewBlocks;
    for (int n = std::min(8, q.kb); n > split; --n) {
        const Launch l(kFewThreads, most, n, st);
        if (tr * tc > resident_clusters(k, l.cfg, n, known[n])) continue;
        const int share = (q.kb + n - 1) / n;
        split = (q.kb + share - 1) / share;
    }
    const int others = tr * tc * split > sm_count();
    q.ns = std::min({C::stages(split, others), kFewStages, (q.kb + split - 1) / split});
    Launch l(kFewThreads, std::max(C::smem(split, q.ns), kFewLeast), split, st);
    l.early();
    l.cfg.gridDim = dim3((unsigned)(tr * split), (unsigned)tc);
    return cudaLaunchKernelEx(&l.cfg, k, ma, mb, scales_of(A, R, q.kb), scales_of(B, Cn, q.kb), out, q, device_error_word());
}

// Whether the few rows' kernel takes a product.
bool few(int64_t R, int64_t depth) { return R <= kFewRows && (depth + BK - 1) / BK <= 8 * kFewBlocks; }

template <bool A_MN, bool B_MN, typename TO>
cudaError_t pick(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, TO* out, int64_t ldo,
                 const Proj8Watch& watch, cudaStream_t st) {
    if constexpr (!A_MN)
        if (few(R, depth))
            return R <= 16   ? go_few<16, B_MN, TO>(B, A, C, R, depth, out, ldo, watch, st)
                   : R <= 32 ? go_few<32, B_MN, TO>(B, A, C, R, depth, out, ldo, watch, st)
                             : go_few<64, B_MN, TO>(B, A, C, R, depth, out, ldo, watch, st);
    // Tiles of 224 columns, whose two accumulators lie apart; of 256 where B is MN-major, so that a
    // block's half of the columns is whole lines of memory (dx of 32768 x 10576 x 2560: 676 us at 224, of
    // which half the rows of a copy lie across two lines); of 128 where the pairs' rounds come out
    // shorter.  A round takes what its contracted blocks take, and what its ends take.
    constexpr int kWide = B_MN ? 256 : 224;
    const int64_t pairs = sm_count() / 2, tr = (R + 255) / 256, kb = (depth + BK - 1) / BK;
    const auto cycles = [&](int64_t bn, int64_t block, int64_t ends) {
        return (tr * ((C + bn - 1) / bn) + pairs - 1) / pairs * (kb * block + ends);
    };
    // Few tiles: the pairs to each with which a block's share and the join take least, of those that run side
    // by side (256 x 8192 x 256: 18.0 us with one pair a tile, 13.2 with two, 9.9 with four, 10.0 with eight;
    // 256 x 2048 x 256: 7.8, 7.7, 7.5; all gradients of 30490 x 192 x 80: 126 us, now 41).  A single pair's
    // blocks wait for memory longer where both operands are MN-major.
    const int64_t t128 = tr * ((C + 127) / 128), block = B_MN ? 800 : 380;
    int split = 1;
    int64_t least = kb * block;
    for (int n = 2; n <= kMostPairs; n *= 2) {
        const int64_t share = share_of((int)kb, n), take = share * block + (n < 8 ? 3000 : 6000);
        if (t128 * n > pairs || (n - 1) * share >= kb) break;
        if (take < least && t128 <= split_clusters<A_MN, B_MN, TO>(n)) split = n, least = take;
    }
    if (split > 1) return go<128, A_MN, B_MN, TO, true>(A, B, R, C, depth, out, ldo, watch, st, split);
    if (cycles(128, 330, 3000) < cycles(kWide, 2 * kWide + 40, 4000))
        return go<128, A_MN, B_MN, TO>(A, B, R, C, depth, out, ldo, watch, st);
    return go<kWide, A_MN, B_MN, TO>(A, B, R, C, depth, out, ldo, watch, st);
}

template <typename TO>
cudaError_t pick(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, TO* out, int64_t ldo,
                 const Proj8Watch& watch, cudaStream_t st) {
    if (A.mn && B.mn) return pick<true, true, TO>(A, B, R, C, depth, out, ldo, watch, st);
    if (B.mn) return pick<false, true, TO>(A, B, R, C, depth, out, ldo, watch, st);
    return pick<false, false, TO>(A, B, R, C, depth, out, ldo, watch, st);
}

}  // namespace

cudaError_t launch_proj8(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, void* out,
                         int64_t ldo, bool bf16, cudaStream_t st, const Proj8Watch& watch) {
    if (R == 0 || C == 0) return cudaSuccess;
    return bf16 ? pick(A, B, R, C, depth, static_cast<__nv_bfloat16*>(out), ldo, watch, st)
                : pick(A, B, R, C, depth, static_cast<float*>(out), ldo, watch, st);
}

}  // namespace m2
