// norm.cu -- RMS norm over groups of channels with a SiLU gate (include/mamba2_layer.h).
//
//   gate first:  v = x silu(z),  y = v r w            r = 1 / sqrt(mean(v^2) + eps)
//   gate after:  v = x,          y = v r w silu(z)
//
// Backward, with q = dy w (times silu(z) when the gate comes after):
//   dv = r q - v r^3 mean(q v);   dw = sum over tokens of dy (..) v r
//   gate first: dx = dv silu(z), dz = dv x silu'(z);  after: dx = dv, dz = dy v r w silu'(z)
//
// Bytes bound: every tensor moves once.  A team (a warp for groups that fit its
// registers, else a block) holds a group's row in registers between the sums and
// the result; the backward's two sums need one pass (mean(q v) does not need r).
// A backward team keeps its group and walks over tokens, so that its part of dw
// stays in registers; the parts are summed by a second kernel, in a fixed order.
#include <algorithm>

#include "internal.h"
#include "layer.cuh"

namespace m2 {
namespace {

struct Rows {
    int T, G, S;     // tokens per sequence, groups, channels per group
    int64_t rows;    // tokens in all
    float eps;
    Tok sx, sz, sy;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of (a, b) over the team: the warp, or the block (every thread calls it).
template <bool WARP>
__device__ __forceinline__ float2 team_sum(float a, float b, float2* red) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (WARP) return make_float2(a, b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < nw ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

enum { kNone = 0, kFirst = 1, kAfter = 2 };

// V weights from w (ones when null), 16 bytes at a time where V allows (w is then
// 16-byte aligned: scalar loads of 8 neighbouring weights a lane cost four times
// the load unit's time).
template <int V> __device__ __forceinline__ void load_weights(const float* w, float (&o)[V]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 1.f;
    } else if constexpr (V == 1) {
        o[0] = __ldg(w);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(w + j));
            o[j] = v.x;
            o[j + 1] = v.y;
            o[j + 2] = v.z;
            o[j + 3] = v.w;
        }
    }
}

// silu(z) and its derivative.
__device__ __forceinline__ void silu_d(float z, float& s, float& d) {
    const float sg = sigmoid(z);
    s = z * sg;
    d = sg * fmaf(z, 1.f - sg, 1.f);
}

constexpr int kWarpTeams = 4;   // warps a block when a team is a warp

// VPT vectors of V channels a thread; VPT = 0: any number, read again for the result.
template <typename TI, int V, int VPT, int GATE, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : 1024)
norm_fwd_kernel(const TI* __restrict__ x, const float* __restrict__ w, const TI* __restrict__ z,
                TI* __restrict__ y, Rows q) {
    __shared__ float2 red[32];
    const int64_t id = WARP ? (int64_t)blockIdx.x * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    if (WARP && id >= q.rows * q.G) return;
    const int64_t row = id / q.G;
    const int g = (int)(id - row * q.G);
    const int64_t b = row / q.T, t = row - b * q.T;
    const TI* xr = x + b * q.sx.b + t * q.sx.t + (int64_t)g * q.S;
    const TI* zr = z + b * q.sz.b + t * q.sz.t + (int64_t)g * q.S;
    TI* yr = y + b * q.sy.b + t * q.sy.t + (int64_t)g * q.S;
    const float* wr = w ? w + (int64_t)g * q.S : nullptr;
    const int nv = q.S / V;
    typedef typename Pack<TI, V>::Raw Raw;
    constexpr int K = VPT > 0 ? VPT : 1;
    Raw rx[K], rz[K];
    float ss = 0.f;
    auto square = [&](Raw vx, Raw vz) {
        float fx[V], fz[V];
        Conv<TI, V>::to(vx, fx);
        if (GATE == kFirst) Conv<TI, V>::to(vz, fz);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float v = GATE == kFirst ? fx[j] * fz[j] * sigmoid(fz[j]) : fx[j];
            ss = fmaf(v, v, ss);
        }
    };
    auto result = [&](int i, Raw vx, Raw vz, float r) {
        float fx[V], fz[V], o[V], fw[V];
        Conv<TI, V>::to(vx, fx);
        if (GATE != kNone) Conv<TI, V>::to(vz, fz);
        load_weights<V>(wr ? wr + i * V : nullptr, fw);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float v = fx[j] * r;
            if (GATE != kNone) v *= fz[j] * sigmoid(fz[j]);
            o[j] = v * fw[j];
        }
        store_raw<TI, V>(yr + i * V, Conv<TI, V>::from(o));
    };
    if (VPT > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * nt;
            rx[k] = rz[k] = zero_raw<Raw>();
            if (i < nv) {
                rx[k] = load_raw<TI, V>(xr + i * V);
                if (GATE != kNone) rz[k] = load_raw<TI, V>(zr + i * V);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) square(rx[k], rz[k]);   // absent vectors are zeros
    } else {
        for (int i = tid; i < nv; i += nt)
            square(load_raw<TI, V>(xr + i * V),
                   GATE == kFirst ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>());
    }
    const float r = rsqrtf(team_sum<WARP>(ss, 0.f, red).x / (float)q.S + q.eps);
    if (VPT > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * nt;
            if (i < nv) result(i, rx[k], rz[k], r);
        }
    } else {
        for (int i = tid; i < nv; i += nt)
            result(i, load_raw<TI, V>(xr + i * V),
                   GATE != kNone ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>(), r);
    }
}

// Team `team` of `teams` (a multiple of G) has group team % G and tokens team / G,
// + teams / G, ...; its dw goes to slot team / G of part ([slots][D]).
template <typename TI, int V, int VPT, int GATE, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : 1024)
norm_bwd_kernel(const TI* __restrict__ x, const float* __restrict__ w, const TI* __restrict__ z,
                const TI* __restrict__ dy, TI* __restrict__ dx, TI* __restrict__ dz,
                float* __restrict__ part, int teams, Rows q) {
    __shared__ float2 red[2][32];
    const int team = WARP ? (int)blockIdx.x * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    if (WARP && team >= teams) return;
    const int g = team % q.G, slot = team / q.G, nslot = teams / q.G;
    const int nv = q.S / V;
    const int64_t D = (int64_t)q.G * q.S;
    const float* wr = w ? w + (int64_t)g * q.S : nullptr;
    float* pr = part ? part + slot * D + (int64_t)g * q.S : nullptr;
    typedef typename Pack<TI, V>::Raw Raw;
    constexpr int K = VPT > 0 ? VPT : 1;
    Raw rx[K], rz[K], rd[K];
    float acc[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[k][j] = 0.f;
    int parity = 0;
    bool begun = false;   // VPT = 0: the slot holds a sum already
    const float inv = 1.f / (float)q.S;
    for (int64_t row = slot; row < q.rows; row += nslot) {
        const int64_t b = row / q.T, t = row - b * q.T;
        const TI* xr = x + b * q.sx.b + t * q.sx.t + (int64_t)g * q.S;
        const TI* zr = z + b * q.sz.b + t * q.sz.t + (int64_t)g * q.S;
        const TI* dr = dy + b * q.sy.b + t * q.sy.t + (int64_t)g * q.S;
        TI* ox = dx + row * D + (int64_t)g * q.S;
        TI* oz = dz + row * D + (int64_t)g * q.S;
        float ss = 0.f, qv = 0.f;
        auto sums = [&](int i, Raw vx, Raw vz, Raw vd) {
            float fx[V], fz[V], fd[V], fw[V];
            Conv<TI, V>::to(vx, fx);
            if (GATE != kNone) Conv<TI, V>::to(vz, fz);
            Conv<TI, V>::to(vd, fd);
            load_weights<V>(wr ? wr + i * V : nullptr, fw);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gate = GATE != kNone ? fz[j] * sigmoid(fz[j]) : 1.f;
                const float v = GATE == kFirst ? fx[j] * gate : fx[j];
                float d = fd[j] * fw[j];
                if (GATE == kAfter) d *= gate;
                ss = fmaf(v, v, ss);
                qv = fmaf(d, v, qv);
            }
        };
        // dx, dz; returns this token's part of dw in p
        auto result = [&](int i, Raw vx, Raw vz, Raw vd, float r, float m, float* p) {
            float fx[V], fz[V], fd[V], ax[V], az[V], fw[V];
            Conv<TI, V>::to(vx, fx);
            if (GATE != kNone) Conv<TI, V>::to(vz, fz);
            Conv<TI, V>::to(vd, fd);
            load_weights<V>(wr ? wr + i * V : nullptr, fw);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float gate = 1.f, slope = 0.f;
                if (GATE != kNone) silu_d(fz[j], gate, slope);
                const float v = GATE == kFirst ? fx[j] * gate : fx[j];
                const float wj = fw[j];
                const float n = v * r;
                const float d = GATE == kAfter ? fd[j] * gate : fd[j];
                const float dv = fmaf(r, d * wj, -v * m);
                p[j] = d * n;
                ax[j] = GATE == kFirst ? dv * gate : dv;
                az[j] = GATE == kFirst ? dv * fx[j] * slope : fd[j] * n * wj * slope;
            }
            store_raw<TI, V>(ox + i * V, Conv<TI, V>::from(ax));
            if (GATE != kNone) store_raw<TI, V>(oz + i * V, Conv<TI, V>::from(az));
        };
        if (VPT > 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int i = tid + k * nt;
                rx[k] = rz[k] = rd[k] = zero_raw<Raw>();
                if (i < nv) {
                    rx[k] = load_raw<TI, V>(xr + i * V);
                    if (GATE != kNone) rz[k] = load_raw<TI, V>(zr + i * V);
                    rd[k] = load_raw<TI, V>(dr + i * V);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < nv) sums(tid + k * nt, rx[k], rz[k], rd[k]);
        } else {
            for (int i = tid; i < nv; i += nt)
                sums(i, load_raw<TI, V>(xr + i * V),
                     GATE != kNone ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>(),
                     load_raw<TI, V>(dr + i * V));
        }
        // two halves of red in turn: the next token's sums do not overwrite one being read
        const float2 s = team_sum<WARP>(ss, qv, red[parity]);
        parity ^= 1;
        const float r = rsqrtf(s.x * inv + q.eps);
        const float m = r * r * r * (s.y * inv);
        if (VPT > 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int i = tid + k * nt;
                float p[V];
                if (i < nv) {
                    result(i, rx[k], rz[k], rd[k], r, m, p);
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[k][j] += p[j];
                }
            }
        } else {
            for (int i = tid; i < nv; i += nt) {
                float p[V];
                result(i, load_raw<TI, V>(xr + i * V),
                       GATE != kNone ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>(),
                       load_raw<TI, V>(dr + i * V), r, m, p);
                if (pr)
#pragma unroll
                    for (int j = 0; j < V; ++j) pr[i * V + j] = begun ? pr[i * V + j] + p[j] : p[j];
            }
            begun = true;
        }
    }
    if (!pr) return;
    if (VPT > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * nt;
            if (i < nv) {
                if constexpr (V == 1) {
                    pr[i] = acc[k][0];
                } else {
#pragma unroll
                    for (int j = 0; j < V; j += 4)
                        *reinterpret_cast<float4*>(pr + i * V + j) =
                            make_float4(acc[k][j], acc[k][j + 1], acc[k][j + 2], acc[k][j + 3]);
                }
            }
        }
    } else if (!begun) {
        for (int i = tid; i < nv * V; i += nt) pr[i] = 0.f;
    }
}

Rows rows_of(const NormArgs& a) {
    return Rows{(int)a.T, (int)a.G, (int)(a.D / a.G), a.b * a.T, a.eps, a.sx, a.sz, a.sy};
}

// Threads of a block team for nv vectors at VPT vectors a thread.
int team_threads(int64_t nv, int vpt) {
    return (int)std::min<int64_t>(1024, std::max<int64_t>(1, (nv + vpt * 32 - 1) / (vpt * 32)) * 32);
}

// Backward teams: enough to fill the GPU (1024 threads an SM), at most one per
// token of each group, a multiple of G; the warp teams are the bound for slots.
int64_t bwd_team_slots(const NormArgs& a) {
    const int64_t teams = (int64_t)sm_count() * 16;
    return std::max<int64_t>(1, std::min<int64_t>(a.b * a.T, (teams + a.G - 1) / a.G));
}

template <typename TI, int V, int GATE>
cudaError_t fwd_go(const NormArgs& a, const TI* x, const float* w, const TI* z, TI* y, cudaStream_t st) {
    const Rows q = rows_of(a);
    const int64_t items = q.rows * q.G, nv = q.S / V;
    if (items >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const unsigned wb = (unsigned)((items + kWarpTeams - 1) / kWarpTeams);
    const unsigned bb = (unsigned)items;
    if (nv <= 32) norm_fwd_kernel<TI, V, 1, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (nv <= 64) norm_fwd_kernel<TI, V, 2, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (nv <= 128) norm_fwd_kernel<TI, V, 4, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (nv <= 2048) norm_fwd_kernel<TI, V, 2, GATE, false><<<bb, team_threads(nv, 2), 0, st>>>(x, w, z, y, q);
    else norm_fwd_kernel<TI, V, 0, GATE, false><<<bb, 1024, 0, st>>>(x, w, z, y, q);
    return cudaGetLastError();
}

template <typename TI, int V, int GATE>
cudaError_t bwd_go(const NormArgs& a, const TI* x, const float* w, const TI* z, const TI* dy, TI* dx,
                   TI* dz, float* part, cudaStream_t st) {
    const Rows q = rows_of(a);
    const int64_t nv = q.S / V;
    const int64_t slots = bwd_team_slots(a), teams64 = slots * q.G;
    if (teams64 >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const int teams = (int)teams64;
    const unsigned wb = (unsigned)((teams64 + kWarpTeams - 1) / kWarpTeams);
    const unsigned bb = (unsigned)teams;
    if (nv <= 32) norm_bwd_kernel<TI, V, 1, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, dy, dx, dz, part, teams, q);
    else if (nv <= 96) norm_bwd_kernel<TI, V, 3, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, dy, dx, dz, part, teams, q);
    else if (nv <= 1024) norm_bwd_kernel<TI, V, 1, GATE, false><<<bb, team_threads(nv, 1), 0, st>>>(x, w, z, dy, dx, dz, part, teams, q);
    else if (nv <= 2048) norm_bwd_kernel<TI, V, 2, GATE, false><<<bb, team_threads(nv, 2), 0, st>>>(x, w, z, dy, dx, dz, part, teams, q);
    else norm_bwd_kernel<TI, V, 0, GATE, false><<<bb, 1024, 0, st>>>(x, w, z, dy, dx, dz, part, teams, q);
    return cudaGetLastError();
}

template <typename TI, int V>
cudaError_t fwd_gate(const NormArgs& a, const void* x, const float* w, const void* z, void* y,
                     cudaStream_t st) {
    auto go = [&](auto f) {
        return f(a, static_cast<const TI*>(x), w, static_cast<const TI*>(z), static_cast<TI*>(y), st);
    };
    return !z ? go(fwd_go<TI, V, kNone>) : a.after ? go(fwd_go<TI, V, kAfter>) : go(fwd_go<TI, V, kFirst>);
}
template <typename TI, int V>
cudaError_t bwd_gate(const NormArgs& a, const void* x, const float* w, const void* z, const void* dy,
                     void* dx, void* dz, float* part, cudaStream_t st) {
    auto go = [&](auto f) {
        return f(a, static_cast<const TI*>(x), w, static_cast<const TI*>(z), static_cast<const TI*>(dy),
                 static_cast<TI*>(dx), static_cast<TI*>(dz), part, st);
    };
    return !z ? go(bwd_go<TI, V, kNone>) : a.after ? go(bwd_go<TI, V, kAfter>) : go(bwd_go<TI, V, kFirst>);
}

bool wide(const NormArgs& a, int64_t V, const void* x, const float* w, const void* z, const void* y,
          const void* o1, const void* o2) {
    const int64_t es = a.dtype == 1 ? 2 : 4;
    const Tok row{0, a.D};
    return (a.D / a.G) % V == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0 && vec_ok(x, a.sx, 16, es) && (!z || vec_ok(z, a.sz, 16, es)) &&
           vec_ok(y, a.sy, 16, es) && vec_ok(o1, row, 16, es) && vec_ok(o2, row, 16, es);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, const void* x, const float* w, const void* z, void* y,
                            cudaStream_t st) {
    if (a.b * a.T == 0 || a.D == 0) return cudaSuccess;
    if (a.dtype == 1)
        return wide(a, 8, x, w, z, y, nullptr, nullptr) ? fwd_gate<__nv_bfloat16, 8>(a, x, w, z, y, st)
                                                     : fwd_gate<__nv_bfloat16, 1>(a, x, w, z, y, st);
    return wide(a, 4, x, w, z, y, nullptr, nullptr) ? fwd_gate<float, 4>(a, x, w, z, y, st)
                                                 : fwd_gate<float, 1>(a, x, w, z, y, st);
}

int64_t norm_bwd_slots(const NormArgs& a) { return bwd_team_slots(a); }

cudaError_t launch_norm_bwd(const NormArgs& a, const void* x, const float* w, const void* z,
                            const void* dy, void* dx, void* dz, float* dw, float* part,
                            cudaStream_t st) {
    if (a.D == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (!dw) part = nullptr;
    const bool none = a.b * a.T == 0;
    if (!none) {
        const bool v = wide(a, a.dtype == 1 ? 8 : 4, x, w, z, dy, dx, dz);
        if (a.dtype == 1)
            e = v ? bwd_gate<__nv_bfloat16, 8>(a, x, w, z, dy, dx, dz, part, st)
                  : bwd_gate<__nv_bfloat16, 1>(a, x, w, z, dy, dx, dz, part, st);
        else
            e = v ? bwd_gate<float, 4>(a, x, w, z, dy, dx, dz, part, st)
                  : bwd_gate<float, 1>(a, x, w, z, dy, dx, dz, part, st);
    }
    if (e != cudaSuccess || !dw) return e;
    return launch_column_sum(part, none ? 0 : norm_bwd_slots(a), a.D, dw, a.D, nullptr, st);
}

}  // namespace m2
