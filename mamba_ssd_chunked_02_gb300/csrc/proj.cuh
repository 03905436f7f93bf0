// proj.cuh -- argument structs and launchers of the projection operators
// (include/mamba2_proj.h), and the e4m3 quantisation they share.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "layer.cuh"

namespace m2 {

constexpr int kGroup = 128;   // values that share a scale

// Whether a kernel of so many blocks is launched to begin while the one before it ends: small ones,
// of which the launch is a good part (quant8 of one token behind another kernel 1.7 us, else 2.3).
// Large ones lose by it (the gradients of 32768 x 10576 x 2560 with every kernel early 1635 us, with
// the products alone 1527).
inline bool early(int64_t blocks) { return blocks <= 2 * (int64_t)sm_count(); }

// Lets a kernel have `bytes` of dynamic shared memory (and clusters of 16 blocks); asked for once a device (`done`: devices
// where it has been, a word of one kernel's own).
template <typename K> cudaError_t allow_smem(K k, int bytes, std::atomic<uint64_t>& done, bool wide_clusters = false) {
    int dev = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
    const uint64_t bit = known ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && wide_clusters) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---- quantisation -----------------------------------------------------------------
// A group's scale is 2^e with the smallest e >= -127 for which its largest magnitude is at
// most 448 * 2^e (448 = 1.75 * 2^8, e4m3's largest value), held as the byte e + 127.  With
// the magnitude 1.m * 2^E as fp32 bits: e = E - 8, one more where 1.m > 1.75; both of a
// subnormal and of zero E <= -127, whose e falls below the bound.
__device__ __forceinline__ uint32_t scale_byte(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 0 ? 0 : e);
}
// 2^-e for the byte e + 127 (at most 247): an exact factor, in [2^-120, 2^127].
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// A group's scale is that of its finite values; what is not finite becomes e4m3's NaN.  fmaxf
// leaves NaN out and the conversion keeps it, so that infinities alone need a second look: a
// group whose largest magnitude is one is gone over again with CLEAN.
__device__ __forceinline__ bool infinite(float top) { return top > 3.402823466e38f; }
template <bool CLEAN> __device__ __forceinline__ float top_of(float top, float v) {
    const float a = fabsf(v);
    return CLEAN && infinite(a) ? top : fmaxf(top, a);
}
// Two values (low byte first) rounded to nearest even.
template <bool CLEAN> __device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t v = r;
    if (CLEAN) {   // the conversion takes infinities to the largest value
        if (infinite(fabsf(lo))) v |= 0x7fu;
        if (infinite(fabsf(hi))) v |= 0x7f00u;
    }
    return v;
}
// How a thread's values lie in a row of D: its unit u is V neighbours (VEC: D is a multiple of V
// and every access aligned), or lane + 32 j of a group of 128, each in its own access.  Either
// way kLanes neighbouring lanes hold a group.
template <int WIDE, bool VEC> struct Units {
    static constexpr int V = VEC ? WIDE : 4, kLanes = kGroup / V;
    static __host__ __device__ int count(int D) { return VEC ? D / V : (D + kGroup - 1) / kGroup * 32; }
    static __device__ __forceinline__ int at(int u, int j) { return VEC ? u * V + j : (u >> 5) * kGroup + (u & 31) + 32 * j; }

    // Unit u of a row (0 behind its end).
    template <typename E> static __device__ __forceinline__ void load(const E* row, int u, int D, float (&o)[V]) {
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = at(u, j) < D ? to_f32(row[at(u, j)]) : 0.f;
        } else if constexpr (sizeof(E) == 2) {
            float t[V];
            Conv<E, V>::to(*reinterpret_cast<const typename Pack<E, V>::Raw*>(row + u * V), t);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = t[j];
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 t = *reinterpret_cast<const float4*>(row + u * V + j);
                o[j] = t.x, o[j + 1] = t.y, o[j + 2] = t.z, o[j + 3] = t.w;
            }
        }
    }
    template <typename E> static __device__ __forceinline__ void store(E* row, int u, int D, const float (&v)[V]) {
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (at(u, j) < D) row[at(u, j)] = from_f32<E>(v[j]);
        } else if constexpr (sizeof(E) == 2) {
            *reinterpret_cast<typename Pack<E, V>::Raw*>(row + u * V) = Conv<E, V>::from(v);
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 4)
                *reinterpret_cast<float4*>(row + u * V + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    }
    // Rounds the unit with its group's scale; the whole warp calls it.
    static __device__ __forceinline__ void quantise(uint8_t* q, uint8_t* s, int u, int D, const float (&v)[V]) {
        const float top = group_top<false>(v);
        if (__any_sync(0xffffffffu, infinite(top))) put<true>(q, s, u, D, v, group_top<true>(v));
        else put<false>(q, s, u, D, v, top);
    }
    template <bool CLEAN> static __device__ __forceinline__ float group_top(const float (&v)[V]) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) top = top_of<CLEAN>(top, v[j]);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        return top;
    }
    template <bool CLEAN>
    static __device__ __forceinline__ void put(uint8_t* q, uint8_t* s, int u, int D, const float (&v)[V], float top) {
        const uint32_t byte = scale_byte(top);
        const float inv = scale_inverse(byte);
        if (u >= count(D)) return;
        if (u % kLanes == 0) s[u / kLanes] = (uint8_t)byte;
        uint32_t p[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) p[j] = e4m3_pair<CLEAN>(v[2 * j] * inv, v[2 * j + 1] * inv);
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (at(u, j) < D) q[at(u, j)] = (uint8_t)(p[j / 2] >> (j & 1 ? 8 : 0));
        } else if constexpr (V == 8) {
            *reinterpret_cast<uint2*>(q + u * V) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
        } else {
            *reinterpret_cast<uint32_t*>(q + u * V) = p[0] | p[1] << 16;
        }
    }
};

struct AddNormArgs {
    int64_t b, T, D;
    float eps;
    bool bf16, res_bf16;   // types of x and y, of the residual and the total
    bool quant;
    Tok sx, sres, sy, st;
};
// y: io, or e4m3 with `scales`.
cudaError_t launch_add_norm_fwd(const AddNormArgs& a, const void* x, const void* residual, const float* w,
                                void* y, uint8_t* scales, void* total, cudaStream_t st);
int64_t add_norm_bwd_slots(const AddNormArgs& a);
// sx of dtotal in sres, of dy in sy, of total in st.
cudaError_t launch_add_norm_bwd(const AddNormArgs& a, const void* total, const float* w, const void* dy,
                                const void* dtotal, void* dx, void* dresidual, float* dw, float* part,
                                cudaStream_t st);

struct Quant8Args {
    int64_t b, T, D;
    bool bf16, block;
    Tok sx, sq;
};
cudaError_t launch_quant8(const Quant8Args& a, const void* x, uint8_t* q, uint8_t* s, cudaStream_t st);
// The backward product's operands: dy [M, N] in groups along its rows (dyr, sr [M, ps]) and along its
// columns (dyc, sc [M / 128, N]), x [M, K] in groups along its columns (xc, sx [M / 128, K]).  pn, pk:
// pitches, whole lines of 128 bytes, so that a line of a copy is one of memory.
struct Quant8Operands {
    int64_t pn, pk, ps;
    uint8_t *dyr, *sr, *dyc, *sc, *xc, *sx;
};
// dy's for the gradients that are wanted.  Small calls make x's in the same launch (`turned`; 1500 x 1095 x
// 1002: all of the gradients 31 -> 28 us); others leave it to launch_quant8_turn, beside the product that reads it.
cudaError_t launch_quant8_operands(bool bf16, int64_t M, int64_t N, int64_t K, const void* dy, int64_t py, const uint8_t* x,
                                   int64_t px, const uint8_t* s, const Quant8Operands& o, bool dx, bool dw, bool* turned,
                                   cudaStream_t st);
// x [M, K] in e4m3, groups along its rows.  Rows start on 16 bytes.
cudaError_t launch_quant8_turn(int64_t M, int64_t K, const uint8_t* x, int64_t px, const uint8_t* s, const Quant8Operands& o,
                               cudaStream_t st);

// A matrix operand of the product: `rows` of the result's rows (or columns) by `depth`
// contracted values.  mn: the contracted index is the outer one in memory (pitch between
// its values), else the inner one.  The scale of row r and contracted block k is the byte
// s[(r >> shift) * rs + k * ks].
struct Operand {
    const uint8_t* q;
    int64_t pitch;
    bool mn;
    const uint8_t* s;
    int64_t rs, ks;
    int shift;
};
// How long the product's kernels wait at a barrier; withhold: a self-test, in which one block of each cluster keeps its
// scales back.
struct Proj8Watch {
    uint64_t limit_ns = 2000000000ull;   // 2 s: far beyond any legitimate wait
    bool withhold = false;
};
// out[i * ldo + j] = sum_k A[i, k] B[j, k], i < R, j < C, in bf16 or fp32.
cudaError_t launch_proj8(const Operand& A, const Operand& B, int64_t R, int64_t C, int64_t depth, void* out,
                         int64_t ldo, bool bf16, cudaStream_t st, const Proj8Watch& watch = {});

}  // namespace m2
