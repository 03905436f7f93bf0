// layer.cuh -- device helpers and launchers of the layer operators (conv, scan, norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace m2 {

// {batch, token} element strides of a token tensor.
struct Tok {
    int64_t b, t;
};

// Packed fp32 pairs: one instruction for two fp32 operations (the rate per
// operation is the plain one's; what it saves is issue slots).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 dup2(float a) { return pack2(a, a); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + exp(-v)); exp overflows to infinity and the result to 0 as it should.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }

// log(1 + exp(v)) = max(v, 0) + log1p(exp(-|v|)).  log1p(e) / e on [0, 1] is a
// degree-8 polynomial in e, a least-squares fit at 400 Chebyshev nodes: relative
// error below 1.7e-7 in fp32, at small e too (where log(1 + e) would lose bits).
__device__ __forceinline__ float softplus(float v) {
    const float e = ex2(-kLog2e * fabsf(v));
    float p = 0.005253457929939032f;
    p = fmaf(p, e, -0.02958850748836994f);
    p = fmaf(p, e, 0.07836166769266129f);
    p = fmaf(p, e, -0.13674770295619965f);
    p = fmaf(p, e, 0.19111430644989014f);
    p = fmaf(p, e, -0.24844369292259216f);
    p = fmaf(p, e, 0.33319270610809326f);
    p = fmaf(p, e, -0.49999502301216125f);
    p = fmaf(p, e, 1.f);
    return fmaf(p, e, v > 0.f ? v : 0.f);
}

// The same for a pair: two scalar chains, whose constants are immediates (packed, each
// constant takes a register pair that is set anew where registers are short).
__device__ __forceinline__ f2 softplus2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(softplus(a), softplus(b));
}

// V elements of type TI moved as one access (V * sizeof(TI) is 2, 4, 8 or 16 bytes).
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { typedef unsigned short type; };
template <> struct RawOf<4> { typedef uint32_t type; };
template <> struct RawOf<8> { typedef uint2 type; };
template <> struct RawOf<16> { typedef uint4 type; };

template <typename TI, int V> struct Pack {
    typedef typename RawOf<V * (int)sizeof(TI)>::type Raw;
};

template <typename TI, int V>
__device__ __forceinline__ typename Pack<TI, V>::Raw load_raw(const TI* p) {
    return __ldg(reinterpret_cast<const typename Pack<TI, V>::Raw*>(p));
}
template <typename Raw> __device__ __forceinline__ Raw zero_raw();
template <> __device__ __forceinline__ unsigned short zero_raw<unsigned short>() { return 0; }
template <> __device__ __forceinline__ uint32_t zero_raw<uint32_t>() { return 0u; }
template <> __device__ __forceinline__ uint2 zero_raw<uint2>() { return make_uint2(0, 0); }
template <> __device__ __forceinline__ uint4 zero_raw<uint4>() { return make_uint4(0, 0, 0, 0); }

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// A raw access to V floats and back.
template <typename TI, int V> struct Conv;
template <> struct Conv<float, 1> {
    static __device__ __forceinline__ void to(uint32_t r, float* o) { o[0] = __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t from(const float* o) { return __float_as_uint(o[0]); }
};
template <> struct Conv<float, 2> {
    static __device__ __forceinline__ void to(uint2 r, float* o) {
        o[0] = __uint_as_float(r.x);
        o[1] = __uint_as_float(r.y);
    }
    static __device__ __forceinline__ uint2 from(const float* o) {
        return make_uint2(__float_as_uint(o[0]), __float_as_uint(o[1]));
    }
};
template <> struct Conv<float, 4> {
    static __device__ __forceinline__ void to(uint4 r, float* o) {
        o[0] = __uint_as_float(r.x);
        o[1] = __uint_as_float(r.y);
        o[2] = __uint_as_float(r.z);
        o[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 from(const float* o) {
        return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                          __float_as_uint(o[3]));
    }
};
template <> struct Conv<__nv_bfloat16, 1> {
    static __device__ __forceinline__ void to(unsigned short r, float* o) {
        o[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ unsigned short from(const float* o) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(o[0]));
    }
};
template <> struct Conv<__nv_bfloat16, 2> {
    static __device__ __forceinline__ void to(uint32_t r, float* o) {
        o[0] = bf_lo(r);
        o[1] = bf_hi(r);
    }
    static __device__ __forceinline__ uint32_t from(const float* o) { return bf_pack(o[0], o[1]); }
};
template <> struct Conv<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void to(uint2 r, float* o) {
        o[0] = bf_lo(r.x);
        o[1] = bf_hi(r.x);
        o[2] = bf_lo(r.y);
        o[3] = bf_hi(r.y);
    }
    static __device__ __forceinline__ uint2 from(const float* o) {
        return make_uint2(bf_pack(o[0], o[1]), bf_pack(o[2], o[3]));
    }
};
template <> struct Conv<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void to(uint4 r, float* o) {
        o[0] = bf_lo(r.x);
        o[1] = bf_hi(r.x);
        o[2] = bf_lo(r.y);
        o[3] = bf_hi(r.y);
        o[4] = bf_lo(r.z);
        o[5] = bf_hi(r.z);
        o[6] = bf_lo(r.w);
        o[7] = bf_hi(r.w);
    }
    static __device__ __forceinline__ uint4 from(const float* o) {
        return make_uint4(bf_pack(o[0], o[1]), bf_pack(o[2], o[3]), bf_pack(o[4], o[5]),
                          bf_pack(o[6], o[7]));
    }
};

// A raw access as packed pairs and back; one value is a pair with an idle half.
template <typename TI, int V>
__device__ __forceinline__ void to_pairs(typename Pack<TI, V>::Raw r, f2 (&o)[(V + 1) / 2]) {
    float f[V];
    Conv<TI, V>::to(r, f);
    if constexpr (V == 1) {
        o[0] = pack2(f[0], 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o[i] = pack2(f[2 * i], f[2 * i + 1]);
    }
}
template <typename TI, int V>
__device__ __forceinline__ typename Pack<TI, V>::Raw from_pairs(const f2 (&v)[(V + 1) / 2]) {
    float f[V + 1];
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    return Conv<TI, V>::from(f);
}
__device__ __forceinline__ f2 sigmoid2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(sigmoid(a), sigmoid(b));
}

template <typename TI, int V>
__device__ __forceinline__ void store_raw(TI* p, typename Pack<TI, V>::Raw r) {
    *reinterpret_cast<typename Pack<TI, V>::Raw*>(p) = r;
}

// BYTES from global to shared memory without registers, zeros when !real.  Two bytes
// (one bf16) are too few for an asynchronous copy.
template <int BYTES> __device__ __forceinline__ void stage_copy(void* dst, const void* src, bool real) {
    if constexpr (BYTES >= 4) {
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES),
                     "r"(real ? BYTES : 0)
                     : "memory");
    } else {
        *static_cast<unsigned short*>(dst) = real ? *static_cast<const unsigned short*>(src) : 0;
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most PENDING of this thread's committed groups are in flight.
template <int PENDING = 0> __device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Host: true when every access of V elements at base + i * strides + k * V is aligned.
inline bool vec_ok(const void* p, const Tok& s, int64_t bytes, int64_t esize) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s.b * esize) % bytes == 0 &&
           (s.t * esize) % bytes == 0;
}

// A launcher's own refusal, before its first launch: the shape takes more blocks than a
// grid has.  Not a value of CUDA's, whose errors (an invalid value among them) may come from
// any of a call's launches.
constexpr cudaError_t kGridLimit = static_cast<cudaError_t>(12289);

struct ConvArgs {
    int64_t b, T, D;
    int W, dtype;
    bool silu;
    Tok sx, sy;
};
cudaError_t launch_conv_fwd(const ConvArgs& a, const void* x, const float* w, const float* bias,
                            const void* init, const int32_t* lengths, void* y, void* final_state,
                            cudaStream_t st);
cudaError_t launch_conv_step(const ConvArgs& a, void* state, const void* x, const float* w,
                             const float* bias, void* y, cudaStream_t st);
int64_t conv_bwd_slots(const ConvArgs& a);
cudaError_t launch_conv_bwd(const ConvArgs& a, const void* x, const float* w, const float* bias,
                            const void* init, const void* dy, const void* dfinal,
                            const int32_t* lengths, void* dx, float* dw, float* dbias, void* dinit,
                            float* part, cudaStream_t st);

struct NormArgs {
    int64_t b, T, D, G;
    float eps;
    int dtype;
    bool after;
    Tok sx, sz, sy;
};
cudaError_t launch_norm_fwd(const NormArgs& a, const void* x, const float* w, const void* z,
                            void* y, cudaStream_t st);
int64_t norm_bwd_slots(const NormArgs& a);
cudaError_t launch_norm_bwd(const NormArgs& a, const void* x, const float* w, const void* z,
                            const void* dy, void* dx, void* dz, float* dw, float* part,
                            cudaStream_t st);

struct ScanArgs {
    int64_t b, T, D, N, G;
    int dtype;
    bool softplus;
    Tok sx, sdt, sB, sC, sz, sy;
};
size_t scan_fwd_workspace(const ScanArgs& a);
bool scan_fwd_turns(const ScanArgs& a);   // rows take turns over slices of the token axis
// starve_ns: for a shape that takes turns, the first slice is launched behind the others,
// whose waits run out after that time (0: the ordinary call).
cudaError_t launch_scan_fwd(const ScanArgs& a, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z,
                            const float* dt_bias, const float* init, const int32_t* lengths,
                            void* y, float* final_state, void* ws, cudaStream_t st,
                            uint64_t starve_ns = 0);
cudaError_t launch_scan_step(const ScanArgs& a, float* state, const void* x, const void* dt,
                             const float* A, const void* B, const void* C, const float* D,
                             const void* z, const float* dt_bias, void* y, cudaStream_t st);
struct ScanGrads {
    void *dx, *ddt;
    float* dA;
    void *dB, *dC;
    float* dD;
    void* dz;
    float *ddt_bias, *dinit;
};
size_t scan_bwd_workspace(const ScanArgs& a);
cudaError_t launch_scan_bwd(const ScanArgs& a, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z,
                            const float* dt_bias, const float* init, const void* dy,
                            const float* dfinal, const int32_t* lengths, const ScanGrads& g,
                            void* ws, cudaStream_t st);

// out[c] = sum over slots s of part[s * cols + c], for c < n1 into out1 and for
// n1 <= c < cols into out2 (null: not wanted); the order of the sum is fixed.
cudaError_t launch_column_sum(const float* part, int64_t slots, int64_t cols, float* out1,
                              int64_t n1, float* out2, cudaStream_t st);

}  // namespace m2
