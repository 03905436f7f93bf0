// proj8.cu -- matrix product of e4m3 operands with power-of-two scales (include/mamba2_proj.h).
//
//   out[j, i] = sum_k A[i, k] sA[i, k / 128] B[j, k] sB[j, k / 128]
//
// The scales are e8m0 bytes, which the block-scaled tcgen05.mma applies inside the tensor
// core: they are staged in shared memory four contracted blocks at a time (one 32-bit word a
// row), copied to tensor memory (tcgen05.cp) and picked by the instruction's scale id.
//
// i, the index that is contiguous in the result, is the accumulator's lane, so that a warp
// stores 32 neighbours; A is therefore the weight (forward: rows of W; dx: columns of W, read
// in place as an MN-major operand; dw: columns of x).
//
// Warp roles: 0 TMA, 1 MMA (and tensor memory), 2 scales of A, 3 scales of B, 4-7 epilogue.
#include <cuda_bf16.h>

#include "internal.h"
#include "proj.cuh"
#include "tc5.cuh"
#include "tmap.h"

namespace m2 {
namespace {

using namespace tc;

constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s: far beyond any legitimate wait
constexpr int kThreads = 256;
constexpr int BM = 128, BK = 128;

// D[tmem] (+)= A B with block scales (kind::mxf8f6f4: one scale per 32 contracted values).
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 32 rows of 16 bytes to 4 columns of tensor memory, the same for each 32 lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
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
};
struct Shape {
    int R, C, kb;          // rows, columns, contracted blocks
    int tr, tiles;         // tiles along the rows, in all
    int64_t ldo;
};

template <int BN> struct Cfg {
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    static constexpr int NS = 6, NSF = 4;
    static constexpr int SFB = (BN + 127) / 128;                 // scale tiles of B
    static constexpr int SF_BYTES = 512 * (1 + SFB);
    static constexpr int SMEM = 1024 + NS * STAGE + NSF * SF_BYTES;
    static constexpr uint32_t SF_COL = 2 * BN, SF_COLS = 4 * (1 + SFB);
    static constexpr uint32_t COLS = 512;
    static_assert(2 * BN + NSF * SF_COLS <= COLS, "tensor memory");
};

struct Bars {
    uint64_t full[6], empty[6];
    uint64_t sf_full[4], sf_empty[4];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// The scales of rows r0 + lane + 32 j (j < 4) for the contracted blocks 4 set .. 4 set + 3, as
// the 16 bytes that lane `lane` of the tensor memory's copy holds.  Behind the ends: 1.
__device__ __forceinline__ uint4 gather_scales(const Scales& s, int r0, int set, int kb, int lane) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + lane + 32 * j;
        w[j] = 0x7f7f7f7fu;
        if (r < s.rows) {
            const uint8_t* p = s.p + (int64_t)(r >> s.shift) * s.rs + (int64_t)set * 4 * s.ks;
            uint32_t v = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) v |= (uint32_t)(4 * set + k < kb ? __ldg(p + k * s.ks) : 0x7f) << (8 * k);
            w[j] = v;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int BN, bool A_MN, bool B_MN, typename TO>
__global__ void __launch_bounds__(kThreads, 1)
proj8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Scales sa,
             const Scales sb, TO* __restrict__ out, const Shape q, int32_t* err) {
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ssf = smem + C::NS * C::STAGE;
    __shared__ Bars bars;
    volatile int* abort = &bars.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < C::NSF; ++i) {
            mbar_init(&bars.sf_full[i], 64);
            mbar_init(&bars.sf_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 128);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem, C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    const int sets = (q.kb + 3) / 4;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
            int it = 0;
            for (int tile = blockIdx.x; tile < q.tiles; tile += gridDim.x) {
                const int r0 = tile % q.tr * BM, c0 = tile / q.tr * BN;
                for (int kb = 0; kb < q.kb; ++kb, ++it) {
                    const int st = it % C::NS;
                    if (!mbar_wait_or_abort(&bars.empty[st], (it / C::NS & 1) ^ 1, abort, kWaitNs)) goto loaded;
                    uint8_t* a = smem + st * C::STAGE;
                    uint8_t* b = a + C::A_BYTES;
                    mbar_arrive_expect_tx(&bars.full[st], C::STAGE);
                    if (A_MN) tma_load_2d(a, &tm_a, &bars.full[st], r0, kb * BK);
                    else tma_load_2d(a, &tm_a, &bars.full[st], kb * BK, r0);
                    if (B_MN) {
#pragma unroll
                        for (int h = 0; h < (BN + 127) / 128; ++h)
                            tma_load_2d(b + h * 128 * BK, &tm_b, &bars.full[st], c0 + h * 128, kb * BK);
                    } else {
                        tma_load_2d(b, &tm_b, &bars.full[st], kb * BK, c0);
                    }
                }
            }
        loaded:
            if (*abort)   // copies in flight land before the block ends
                for (int i = it - 1; i >= 0 && i >= it - C::NS; --i) mbar_wait(&bars.full[i % C::NS], i / C::NS & 1, kWaitNs);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_mx(BM, BN, A_MN, B_MN);
            constexpr uint32_t a_step = (A_MN ? 32 * 128 : 32) >> 4, b_step = (B_MN ? 32 * 128 : 32) >> 4;
            int it = 0, sit = 0, t = 0;
            for (int tile = blockIdx.x; tile < q.tiles; tile += gridDim.x, ++t) {
                const int acc = t & 1;
                if (!mbar_wait_or_abort(&bars.acc_empty[acc], (t / 2 & 1) ^ 1, abort, kWaitNs)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                bool ok = true;
                for (int set = 0; set < sets && ok; ++set, ++sit) {
                    const int sf = sit % C::NSF;
                    if (!(ok = mbar_wait_or_abort(&bars.sf_full[sf], sit / C::NSF & 1, abort, kWaitNs))) break;
                    tc_fence_after();
                    const uint32_t at = smem_u32(ssf + sf * C::SF_BYTES), ta = tmem + C::SF_COL + sf * C::SF_COLS, tb = ta + 4;
                    copy_scales(ta, scale_desc(at));
#pragma unroll
                    for (int h = 0; h < C::SFB; ++h) copy_scales(tb + 4 * h, scale_desc(at + 512 * (1 + h)));
                    const int end = min(q.kb, 4 * set + 4);
                    for (int kb = 4 * set; kb < end; ++kb, ++it) {
                        const int st = it % C::NS;
                        if (!(ok = mbar_wait_or_abort(&bars.full[st], it / C::NS & 1, abort, kWaitNs))) break;
                        tc_fence_after();
                        const uint32_t a = smem_u32(smem + st * C::STAGE), b = a + C::A_BYTES;
                        // K-major: 8-row groups 1024 bytes apart; MN-major: the same between 8 contracted
                        // rows, blocks of 128 m or n one operand tile of 128 rows apart
                        const uint64_t da = smem_desc_sw128(a, A_MN ? 128 * BK : 16, 1024);
                        const uint64_t db = smem_desc_sw128(b, B_MN ? 128 * BK : 16, 1024);
                        const uint32_t id = idesc | (uint32_t)(kb & 3) << 4 | (uint32_t)(kb & 3) << 29;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_scaled(d, da + k * a_step, db + k * b_step, id, ta, tb, kb > 0 || k > 0);
                        mma_commit(&bars.empty[st]);
                    }
                    if (ok) mma_commit(&bars.sf_empty[sf]);
                }
                if (!ok) break;
                mma_commit(&bars.acc_full[acc]);
            }
            if (*abort) {
                mma_commit(&bars.drain);
                mbar_wait(&bars.drain, 0, kWaitNs);
            }
        }
    } else if (warp < 4) {
        const Scales& s = warp == 2 ? sa : sb;
        int sit = 0;
        for (int tile = blockIdx.x; tile < q.tiles; tile += gridDim.x) {
            const int r0 = warp == 2 ? tile % q.tr * BM : tile / q.tr * BN;
            for (int set = 0; set < sets; ++set, ++sit) {
                const int sf = sit % C::NSF;
                uint4 w[C::SFB];
#pragma unroll
                for (int h = 0; h < C::SFB; ++h)
                    if (h == 0 || warp == 3) w[h] = gather_scales(s, r0 + 128 * h, set, q.kb, lane);
                if (!mbar_wait_or_abort(&bars.sf_empty[sf], (sit / C::NSF & 1) ^ 1, abort, kWaitNs)) goto scaled;
                uint4* to = reinterpret_cast<uint4*>(ssf + sf * C::SF_BYTES) + (warp == 2 ? 0 : 32) + lane;
#pragma unroll
                for (int h = 0; h < C::SFB; ++h)
                    if (h == 0 || warp == 3) to[32 * h] = w[h];
                fence_proxy_async_smem();
                mbar_arrive(&bars.sf_full[sf]);
            }
        }
    scaled:;
    } else {
        const int quad = warp & 3;
        int t = 0;
        for (int tile = blockIdx.x; tile < q.tiles; tile += gridDim.x, ++t) {
            const int acc = t & 1;
            if (!mbar_wait_or_abort(&bars.acc_full[acc], t / 2 & 1, abort, kWaitNs)) break;
            tc_fence_after();
            const int r = tile % q.tr * BM + quad * 32 + lane, c0 = tile / q.tr * BN;
            const uint32_t from = tmem + acc * BN + ((uint32_t)(quad * 32) << 16);
            TO* o = out + (int64_t)c0 * q.ldo + r;
            const int cols = min(BN, q.C - c0);
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
                uint32_t v[32];
                tmem_ld32_sync(from + c, v);
                if (r < q.R)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < cols) o[(int64_t)(c + j) * q.ldo] = from_f32<TO>(__uint_as_float(v[j]));
            }
            tc_fence_before();
            mbar_arrive(&bars.acc_empty[acc]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort) record_error(err, kErrTimeoutProj8);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

bool map_of(CUtensorMap* m, const Operand& o, int64_t rows, int64_t depth, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)(o.mn ? rows : depth), (uint64_t)(o.mn ? depth : rows)};
    const uint64_t strides[1] = {(uint64_t)o.pitch};
    const uint32_t box[2] = {128, (uint32_t)(o.mn ? BK : box_rows)};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.q, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int BN, bool A_MN, bool B_MN, typename TO>
cudaError_t go(const Operand& A, const Operand& B, int64_t R, int64_t Cn, int64_t depth, TO* out, int64_t ldo,
               cudaStream_t st) {
    using C = Cfg<BN>;
    CUtensorMap ma, mb;
    if (!map_of(&ma, A, R, depth, BM) || !map_of(&mb, B, Cn, depth, BN)) return cudaErrorInvalidValue;
    const int64_t tr = (R + BM - 1) / BM, tiles = tr * ((Cn + BN - 1) / BN);
    if (tiles >= (int64_t(1) << 30)) return kGridLimit;
    const Shape q{(int)R, (int)Cn, (int)((depth + BK - 1) / BK), (int)tr, (int)tiles, ldo};
    const Scales sa{A.s, A.rs, A.ks, A.shift, (int)R}, sb{B.s, B.rs, B.ks, B.shift, (int)Cn};
    auto k = proj8_kernel<BN, A_MN, B_MN, TO>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)(tiles < sm_count() ? tiles : sm_count()), kThreads, C::SMEM, st>>>(ma, mb, sa, sb, out, q,
                                                                                     device_error_word());
    return cudaGetLastError();
}

template <typename TO>
cudaError_t pick(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, TO* out, int64_t ldo,
                 cudaStream_t st) {
    if (A.mn && B.mn) return go<128, true, true, TO>(A, B, R, C, depth, out, ldo, st);
    if (A.mn) return go<128, true, false, TO>(A, B, R, C, depth, out, ldo, st);
    return go<128, false, false, TO>(A, B, R, C, depth, out, ldo, st);
}

}  // namespace

cudaError_t launch_proj8(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, void* out,
                         int64_t ldo, bool bf16, cudaStream_t st) {
    if (R == 0 || C == 0) return cudaSuccess;
    return bf16 ? pick(A, B, R, C, depth, static_cast<__nv_bfloat16*>(out), ldo, st)
                : pick(A, B, R, C, depth, static_cast<float*>(out), ldo, st);
}

}  // namespace m2
