// add_norm.cu -- RMS norm of a sum with the residual (include/mamba2_proj.h).
//
//   t = x + residual (rounded to the residual's type);  y = t r w,  r = 1 / sqrt(mean(t^2) + eps)
//
// y in the io type or, rounded once from fp32, as e4m3 with a scale for each 128 channels.
// Backward, with g = dy w and n = t r:
//   dt = r (g - n mean(g n)) + dtotal;  dx = dresidual = dt;  dw = sum over tokens of dy n
//
// Bytes bound: every tensor moves once.  A team (a warp for narrow rows, else a block) holds its
// row in registers between the sum and the result; what wide rows do not fit is read again.
#include <algorithm>
#include <initializer_list>
#include <utility>

#include "common.cuh"
#include "internal.h"
#include "proj.cuh"

namespace m2 {
namespace {

struct Rows {
    uint32_t T;
    int D;
    int64_t rows;
    float eps;
    Tok sx, sres, sy, st;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sum over the team; `red` is not in use by an earlier call when a block's threads come here.
template <bool WARP> __device__ __forceinline__ float2 team_sum(float a, float b, float2* red) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (WARP) return make_float2(a, b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < nw ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

constexpr int kTeams = 8;   // warps a block when a team is a warp

// VPT units a thread; 0: any number, the total read again for the result.
template <typename TI, typename TR, bool VEC, int VPT, bool WARP, bool QUANT>
__global__ void __launch_bounds__(WARP ? kTeams * 32 : 1024)
fwd_kernel(const TI* __restrict__ x, const TR* res, const float* __restrict__ w, TI* __restrict__ y,
           uint8_t* __restrict__ s, TR* total, Rows q) {
    using U = Units<TI, VEC>;
    constexpr int V = U::V;
    __shared__ float2 red[32];
    const int64_t row = WARP ? (int64_t)blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    grid_dep_wait();
    grid_dep_launch();
    if (row >= q.rows) return;
    const int64_t b = (uint32_t)row / q.T, t = (uint32_t)row - (uint32_t)b * q.T;
    const TI* xr = x + b * q.sx.b + t * q.sx.t;
    const TR* rr = res ? res + b * q.sres.b + t * q.sres.t : nullptr;
    TR* tr = total + b * q.st.b + t * q.st.t;
    const int units = U::count(q.D);
    float ss = 0.f;
    auto sum = [&](int u, float (&v)[V]) {
        U::load(xr, u, q.D, v);
        if (rr) {
            float a[V];
            U::load(rr, u, q.D, a);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] += a[j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = to_f32(from_f32<TR>(v[j]));
            ss = fmaf(v[j], v[j], ss);
        }
        U::store(tr, u, q.D, v);
    };
    const auto scale = [&] { return __frsqrt_rn(team_sum<WARP>(ss, 0.f, red).x / (float)q.D + q.eps); };
    auto result = [&](int u, float (&v)[V], float r) {
        float f[V];
        if (u < units) {
            if (w) {
                U::load(w, u, q.D, f);
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = v[j] * r * f[j];
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] *= r;
            }
        }
        if constexpr (QUANT) {
            U::quantise(reinterpret_cast<uint8_t*>(y) + b * q.sy.b + t * q.sy.t, s + row * ((q.D + kGroup - 1) / kGroup), u, q.D, v);
        } else if (u < units) {
            U::store(y + b * q.sy.b + t * q.sy.t, u, q.D, v);
        }
    };
    if constexpr (VPT > 0) {
        float v[VPT][V];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[k][j] = 0.f;
            if (tid + k * nt < units) sum(tid + k * nt, v[k]);
        }
        const float r = scale();
#pragma unroll
        for (int k = 0; k < VPT; ++k) result(tid + k * nt, v[k], r);
    } else {
        float v[V];
        for (int u = tid; u < units; u += nt) sum(u, v);
        const float r = scale();
        for (int u = tid; u - tid < units; u += nt) {   // whole warps: groups are joined by shuffles
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = 0.f;
            if (u < units) U::load(tr, u, q.D, v);
            result(u, v, r);
        }
    }
}

// Team `slot` of `slots` has tokens slot, slot + slots, ...; its dw goes to part[slot].
template <typename TI, typename TR, bool VEC, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? kTeams * 32 : 1024)
bwd_kernel(const TR* __restrict__ total, const float* __restrict__ w, const TI* __restrict__ dy,
           const TR* __restrict__ dtotal, TI* __restrict__ dx, TR* __restrict__ dres, float* __restrict__ part, int slots,
           Rows q) {
    using U = Units<TI, VEC>;
    constexpr int V = U::V, K = VPT > 0 ? VPT : 1;
    __shared__ float2 red[2][32];
    const int slot = WARP ? (int)blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    grid_dep_wait();
    grid_dep_launch();
    if (slot >= slots) return;
    const int units = U::count(q.D);
    float* pr = part ? part + (int64_t)slot * q.D : nullptr;
    const float inv = 1.f / (float)q.D;
    float acc[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[k][j] = 0.f;
    int parity = 0;
    for (int64_t row = slot; row < q.rows; row += slots) {
        const int64_t b = (uint32_t)row / q.T, t = (uint32_t)row - (uint32_t)b * q.T;
        const TR* tr = total + b * q.st.b + t * q.st.t;
        const TI* dr = dy + b * q.sy.b + t * q.sy.t;
        const TR* er = dtotal ? dtotal + b * q.sres.b + t * q.sres.t : nullptr;
        float ss = 0.f, gv = 0.f;
        auto sums = [&](int u, float (&v)[V], float (&d)[V]) {
            U::load(tr, u, q.D, v);
            U::load(dr, u, q.D, d);
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = 1.f;
            if (w) U::load(w, u, q.D, f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                ss = fmaf(v[j], v[j], ss);
                gv = fmaf(d[j] * f[j], v[j], gv);
            }
        };
        float r, m;
        auto scales = [&] {
            // two halves of red in turn: the next token's sums do not overwrite one being read
            const float2 s = team_sum<WARP>(ss, gv, red[parity]);
            parity ^= 1;
            r = __frsqrt_rn(s.x * inv + q.eps);
            m = r * (s.y * inv);
        };
        // a: this unit's part of dw, added to
        auto result = [&](int u, const float (&v)[V], const float (&d)[V], float (&a)[V]) {
            float f[V], e[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = 1.f, e[j] = 0.f;
            if (w) U::load(w, u, q.D, f);
            if (er) U::load(er, u, q.D, e);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = v[j] * r;
                a[j] = fmaf(d[j], n, a[j]);
                e[j] = fmaf(r, fmaf(-n, m, d[j] * f[j]), e[j]);
            }
            U::store(dx + row * q.D, u, q.D, e);
            if (dres) U::store(dres + row * q.D, u, q.D, e);
        };
        if constexpr (VPT > 0) {
            float v[K][V], d[K][V];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < units) sums(tid + k * nt, v[k], d[k]);
            scales();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < units) result(tid + k * nt, v[k], d[k], acc[k]);
        } else {
            float v[V], d[V];
            for (int u = tid; u < units; u += nt) sums(u, v, d);
            scales();
            for (int u = tid; u < units; u += nt) {
                U::load(tr, u, q.D, v);
                U::load(dr, u, q.D, d);
                float a[V];
#pragma unroll
                for (int j = 0; j < V; ++j) a[j] = 0.f;
                if (pr && row != slot) U::load(pr, u, q.D, a);
                result(u, v, d, a);
                if (pr) U::store(pr, u, q.D, a);
            }
        }
    }
    if (VPT > 0 && pr)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (tid + k * nt < units) U::store(pr, tid + k * nt, q.D, acc[k]);
}

Rows rows_of(const AddNormArgs& a) {
    return Rows{(uint32_t)a.T, (int)a.D, a.b * a.T, a.eps, a.sx, a.sres, a.sy, a.st};
}
int threads_of(int64_t units, int vpt) { return (int)std::min<int64_t>(1024, (units + vpt * 32 - 1) / (vpt * 32) * 32); }

template <typename TI, typename TR, bool VEC, bool QUANT>
cudaError_t fwd_go(const AddNormArgs& a, const void* x_, const void* res_, const float* w, void* y_, uint8_t* s, void* t_,
                   cudaStream_t st) {
    const Rows q = rows_of(a);
    if (q.rows >= (int64_t(1) << 31)) return kGridLimit;
    const TI* x = static_cast<const TI*>(x_);
    const TR* res = static_cast<const TR*>(res_);
    TI* y = static_cast<TI*>(y_);
    TR* t = static_cast<TR*>(t_);
    const int64_t n = Units<TI, VEC>::count((int)a.D);
    const unsigned wb = (unsigned)((q.rows + kTeams - 1) / kTeams), bb = (unsigned)q.rows;
    const auto go = [&](auto k, unsigned blocks, int threads) {
        return launch_kernel(k, dim3(blocks), dim3((unsigned)threads), 0, st, early(blocks), x, res, w, y, s, t, q);
    };
    cudaError_t e;
    if (n <= 32) e = go(fwd_kernel<TI, TR, VEC, 1, true, QUANT>, wb, kTeams * 32);
    else if (n <= 64) e = go(fwd_kernel<TI, TR, VEC, 2, true, QUANT>, wb, kTeams * 32);
    else if (n <= 512) e = go(fwd_kernel<TI, TR, VEC, 1, false, QUANT>, bb, threads_of(n, 1));
    else if (n <= 2048) e = go(fwd_kernel<TI, TR, VEC, 2, false, QUANT>, bb, threads_of(n, 2));
    else e = go(fwd_kernel<TI, TR, VEC, 0, false, QUANT>, bb, 1024);
    return e;
}

template <typename TI, typename TR, bool VEC>
cudaError_t bwd_go(const AddNormArgs& a, const void* t_, const float* w, const void* dy_, const void* dt_, void* dx_,
                   void* dr_, float* part, cudaStream_t st) {
    const Rows q = rows_of(a);
    if (q.rows >= (int64_t(1) << 31)) return kGridLimit;
    const TR *t = static_cast<const TR*>(t_), *dt = static_cast<const TR*>(dt_);
    const TI* dy = static_cast<const TI*>(dy_);
    TI* dx = static_cast<TI*>(dx_);
    TR* dr = static_cast<TR*>(dr_);
    const int64_t n = Units<TI, VEC>::count((int)a.D);
    const int slots = (int)add_norm_bwd_slots(a);
    const unsigned wb = (unsigned)((slots + kTeams - 1) / kTeams), bb = (unsigned)slots;
    const auto go = [&](auto k, unsigned blocks, int threads) {
        return launch_kernel(k, dim3(blocks), dim3((unsigned)threads), 0, st, early(blocks), t, w, dy, dt, dx, dr, part, slots, q);
    };
    cudaError_t e;
    if (n <= 32) e = go(bwd_kernel<TI, TR, VEC, 1, true>, wb, kTeams * 32);
    else if (n <= 64) e = go(bwd_kernel<TI, TR, VEC, 2, true>, wb, kTeams * 32);
    else if (n <= 512) e = go(bwd_kernel<TI, TR, VEC, 1, false>, bb, threads_of(n, 1));
    else if (n <= 2048) e = go(bwd_kernel<TI, TR, VEC, 2, false>, bb, threads_of(n, 2));
    else e = go(bwd_kernel<TI, TR, VEC, 0, false>, bb, 1024);
    return e;
}

// Every access of a unit is aligned.
bool vec(const AddNormArgs& a, const float* w, std::initializer_list<std::pair<const void*, Tok>> io,
         std::initializer_list<std::pair<const void*, Tok>> res, const void* q8) {
    const int64_t es = a.bf16 ? 2 : 4, rs = a.res_bf16 ? 2 : 4, V = a.bf16 ? 8 : 4;
    if (a.D % V || reinterpret_cast<uintptr_t>(w) % 16) return false;
    for (const auto& t : io)
        if (!vec_ok(t.first, t.second, 16, es)) return false;
    for (const auto& t : res)
        if (t.first && !vec_ok(t.first, t.second, 16, rs)) return false;
    return !q8 || vec_ok(q8, a.sy, V, 1);
}

}  // namespace

cudaError_t launch_add_norm_fwd(const AddNormArgs& a, const void* x, const void* residual, const float* w, void* y,
                                uint8_t* s, void* total, cudaStream_t st) {
    if (a.b * a.T == 0 || a.D == 0) return cudaSuccess;
    const bool v = a.quant ? vec(a, w, {{x, a.sx}}, {{residual, a.sres}, {total, a.st}}, y)
                           : vec(a, w, {{x, a.sx}, {y, a.sy}}, {{residual, a.sres}, {total, a.st}}, nullptr);
    const auto go = [&](auto f) { return f(a, x, residual, w, y, s, total, st); };
    typedef __nv_bfloat16 bf;
    if (!a.bf16)
        return v ? (a.quant ? go(fwd_go<float, float, true, true>) : go(fwd_go<float, float, true, false>))
                 : (a.quant ? go(fwd_go<float, float, false, true>) : go(fwd_go<float, float, false, false>));
    if (!a.res_bf16)
        return v ? (a.quant ? go(fwd_go<bf, float, true, true>) : go(fwd_go<bf, float, true, false>))
                 : (a.quant ? go(fwd_go<bf, float, false, true>) : go(fwd_go<bf, float, false, false>));
    return v ? (a.quant ? go(fwd_go<bf, bf, true, true>) : go(fwd_go<bf, bf, true, false>))
             : (a.quant ? go(fwd_go<bf, bf, false, true>) : go(fwd_go<bf, bf, false, false>));
}

int64_t add_norm_bwd_slots(const AddNormArgs& a) {
    // the threads an SM holds, in teams of a row's width
    const int64_t units = a.bf16 ? (a.D + 7) / 8 : (a.D + 3) / 4;
    const int64_t per_sm = units <= 64 ? 64 : std::max<int64_t>(1, 2048 / threads_of(units, units <= 512 ? 1 : 2));
    return std::max<int64_t>(1, std::min<int64_t>(a.b * a.T, (int64_t)sm_count() * per_sm));
}

cudaError_t launch_add_norm_bwd(const AddNormArgs& a, const void* total, const float* w, const void* dy,
                                const void* dtotal, void* dx, void* dres, float* dw, float* part, cudaStream_t st) {
    if (a.D == 0) return cudaSuccess;
    const bool none = a.b * a.T == 0;
    if (!dw) part = nullptr;
    if (!none) {
        const Tok row{0, a.D};
        const bool v = vec(a, w, {{dy, a.sy}, {dx, row}}, {{total, a.st}, {dtotal, a.sres}, {dres, row}}, nullptr) &&
                       reinterpret_cast<uintptr_t>(part) % 16 == 0;
        const auto go = [&](auto f) { return f(a, total, w, dy, dtotal, dx, dres, part, st); };
        typedef __nv_bfloat16 bf;
        const cudaError_t e = !a.bf16     ? (v ? go(bwd_go<float, float, true>) : go(bwd_go<float, float, false>))
                              : !a.res_bf16 ? (v ? go(bwd_go<bf, float, true>) : go(bwd_go<bf, float, false>))
                                            : (v ? go(bwd_go<bf, bf, true>) : go(bwd_go<bf, bf, false>));
        if (e != cudaSuccess) return e;
    }
    return dw ? launch_column_sum(part, none ? 0 : add_norm_bwd_slots(a), a.D, dw, a.D, nullptr, st) : cudaSuccess;
}

}  // namespace m2
