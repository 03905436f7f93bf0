// norm.cu -- RMS norm over groups of channels with a SiLU gate (include/mamba2_layer.h).
//
//   gate first:  v = x silu(z),  y = v r w            r = 1 / sqrt(mean(v^2) + eps)
//   gate after:  v = x,          y = v r w silu(z)
//
// Backward, with q = dy w (times silu(z) when the gate comes after):
//   dv = r q - v r^3 mean(q v);   dw = sum over tokens of dy (..) v r
//   gate first: dx = dv silu(z), dz = dv x silu'(z);  after: dx = dv, dz = dy v r w silu'(z)
//
// Bytes bound: every tensor moves once.  b8 T4096 C5120 bf16: forward 159 us (6.3 TB/s,
// 0.93 of the measured copy rate), backward in groups of 640 296 us (5.7 TB/s, 0.83, its
// issue slots at 0.64); one token of 64 sequences 2.5 us on the GPU, the launch.
//
// A team (a warp for groups that fit its registers, else a block) holds a group's row in
// registers between the sums and the result; the backward's two sums need one pass (mean(q v)
// does not need r).  A backward team keeps its group and walks over tokens, so that its part of
// dw stays in registers; the parts are summed by a second kernel, in a fixed order.
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

// V weights from w (ones when null) as pairs, 16 bytes at a time where V allows (w is
// then 16-byte aligned: scalar loads of 8 neighbouring weights a lane cost four times the
// load unit's time).
template <int V> __device__ __forceinline__ void load_weights(const float* w, f2 (&o)[(V + 1) / 2]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) o[i] = dup2(1.f);
    } else if constexpr (V == 1) {
        o[0] = pack2(__ldg(w), 0.f);
    } else if constexpr (V == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(w));
        o[0] = pack2(v.x, v.y);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; i += 2) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(w + 2 * i));
            o[i] = pack2(v.x, v.y);
            o[i + 1] = pack2(v.z, v.w);
        }
    }
}

constexpr int kWarpTeams = 4;   // warps a block when a team is a warp

// VPT vectors of V channels a thread; VPT = 0: any number, read again for the result.
template <typename TI, int V, int VPT, int GATE, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : 1024)
norm_fwd_kernel(const TI* __restrict__ x, const float* __restrict__ w, const TI* __restrict__ z,
                TI* __restrict__ y, Rows q) {
    __shared__ float2 red[32];
    // rows and row groups fit 32 bits (the launcher checks): a 64-bit division costs 100 instructions
    const uint32_t id = WARP ? blockIdx.x * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    if (WARP && id >= (uint32_t)q.rows * q.G) return;
    const uint32_t row = id / q.G;
    const int g = (int)(id - row * q.G);
    const int64_t b = row / (uint32_t)q.T, t = row - (uint32_t)b * q.T;
    const TI* xr = x + b * q.sx.b + t * q.sx.t + (int64_t)g * q.S;
    const TI* zr = z + b * q.sz.b + t * q.sz.t + (int64_t)g * q.S;
    TI* yr = y + b * q.sy.b + t * q.sy.t + (int64_t)g * q.S;
    const float* wr = w ? w + (int64_t)g * q.S : nullptr;
    const int nv = q.S / V;
    typedef typename Pack<TI, V>::Raw Raw;
    constexpr int K = VPT > 0 ? VPT : 1, H = (V + 1) / 2;
    f2 ss = dup2(0.f);
    // v = x or x silu(z), kept in fp32 for the result; the gate that comes after waits as raw z
    auto value = [&](Raw vx, Raw vz, f2 (&v)[H]) {
        to_pairs<TI, V>(vx, v);
        if (GATE == kFirst) {
            f2 fz[H];
            to_pairs<TI, V>(vz, fz);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = mul2(v[i], mul2(fz[i], sigmoid2(fz[i])));
        }
    };
    auto square = [&](const f2 (&v)[H]) {
#pragma unroll
        for (int i = 0; i < H; ++i) ss = fma2(v[i], v[i], ss);
    };
    auto result = [&](int at, f2 (&v)[H], Raw vz, f2 r) {
        f2 fw[H];
        load_weights<V>(wr ? wr + at * V : nullptr, fw);
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = mul2(mul2(v[i], r), fw[i]);
        if (GATE == kAfter) {
            f2 fz[H];
            to_pairs<TI, V>(vz, fz);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = mul2(v[i], mul2(fz[i], sigmoid2(fz[i])));
        }
        store_raw<TI, V>(yr + at * V, from_pairs<TI, V>(v));
    };
    const auto scale = [&] { return dup2(rsqrtf(team_sum<WARP>(sum2(ss), 0.f, red).x / (float)q.S + q.eps)); };
    if constexpr (VPT > 0) {
        Raw rx[K], rz[K];
        f2 v[K][H];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * nt;
            rx[k] = rz[k] = zero_raw<Raw>();   // absent vectors are zeros
            if (i < nv) {
                rx[k] = load_raw<TI, V>(xr + i * V);
                if (GATE != kNone) rz[k] = load_raw<TI, V>(zr + i * V);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            value(rx[k], rz[k], v[k]);
            square(v[k]);
        }
        const f2 r = scale();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (tid + k * nt < nv) result(tid + k * nt, v[k], rz[k], r);
    } else {
        f2 v[H];
        const auto zraw = [&](int i) { return GATE != kNone ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>(); };
        for (int i = tid; i < nv; i += nt) {
            value(load_raw<TI, V>(xr + i * V), zraw(i), v);
            square(v);
        }
        const f2 r = scale();
        for (int i = tid; i < nv; i += nt) {
            const Raw z0 = zraw(i);
            value(load_raw<TI, V>(xr + i * V), z0, v);
            result(i, v, z0, r);
        }
    }
}

// Warps an SM of the backward's warp teams: four blocks, or five where the registers of a
// lane's `each` channels allow it.
constexpr int bwd_warps(int each) { return each > 20 ? 16 : 20; }

// Team `team` of `teams` (a multiple of G) has group team % G and tokens team / G,
// + teams / G, ...; its dw goes to slot team / G of part ([slots][D]).
template <typename TI, int V, int VPT, int GATE, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : 1024, WARP ? bwd_warps(VPT * V) / kWarpTeams : 1)
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
    constexpr int K = VPT > 0 ? VPT : 1, H = (V + 1) / 2;
    f2 acc[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) acc[k][i] = dup2(0.f);
    int parity = 0;
    bool begun = false;   // VPT = 0: the slot holds a sum already
    const float inv = 1.f / (float)q.S;
    const f2 one = dup2(1.f), minus = dup2(-1.f);
    // The next token's row is copied into the other half of a thread's own room in shared
    // memory while this one is summed and applied.
    constexpr bool STAGE = VPT > 0 && V * sizeof(TI) >= 4;
    extern __shared__ __align__(16) unsigned char smem[];
    const int bt = blockDim.x;
    Raw* st = reinterpret_cast<Raw*>(smem) + threadIdx.x;   // [2][K][3 tensors][threads]
    Raw own[1][STAGE ? 1 : K][3];
    int half = 0;
    auto copy = [&](int64_t row, int to) {
        const int64_t b = (uint32_t)row / (uint32_t)q.T, t = row - b * q.T;
        const TI* xr = x + b * q.sx.b + t * q.sx.t + (int64_t)g * q.S;
        const TI* zr = z + b * q.sz.b + t * q.sz.t + (int64_t)g * q.S;
        const TI* dr = dy + b * q.sy.b + t * q.sy.t + (int64_t)g * q.S;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (tid + k * nt < nv) {
                const int at = (tid + k * nt) * V;
                Raw* d = st + (to * K + k) * 3 * bt;
                stage_copy<V * (int)sizeof(TI)>(d, xr + at, true);
                if (GATE != kNone) stage_copy<V * (int)sizeof(TI)>(d + bt, zr + at, true);
                stage_copy<V * (int)sizeof(TI)>(d + 2 * bt, dr + at, true);
            }
        stage_commit();
    };
    if (STAGE && slot < q.rows) copy(slot, 0);
    for (int64_t row = slot; row < q.rows; row += nslot) {
        const int64_t b = (uint32_t)row / (uint32_t)q.T, t = row - b * q.T;
        const TI* xr = x + b * q.sx.b + t * q.sx.t + (int64_t)g * q.S;
        const TI* zr = z + b * q.sz.b + t * q.sz.t + (int64_t)g * q.S;
        const TI* dr = dy + b * q.sy.b + t * q.sy.t + (int64_t)g * q.S;
        TI* ox = dx + row * D + (int64_t)g * q.S;
        TI* oz = dz + row * D + (int64_t)g * q.S;
        f2 ss = dup2(0.f), qv = dup2(0.f);
        // sg = sigmoid(z), kept for the result
        auto sums = [&](int at, Raw vx, Raw vz, Raw vd, f2 (&sg)[H]) {
            f2 v[H], fz[H], d[H], fw[H];
            to_pairs<TI, V>(vx, v);
            to_pairs<TI, V>(vd, d);
            load_weights<V>(wr ? wr + at * V : nullptr, fw);
            if (GATE != kNone) to_pairs<TI, V>(vz, fz);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                d[i] = mul2(d[i], fw[i]);
                if (GATE != kNone) {
                    sg[i] = sigmoid2(fz[i]);
                    const f2 gate = mul2(fz[i], sg[i]);
                    if (GATE == kFirst) v[i] = mul2(v[i], gate);
                    else d[i] = mul2(d[i], gate);
                }
                ss = fma2(v[i], v[i], ss);
                qv = fma2(d[i], v[i], qv);
            }
        };
        // dx, dz; adds this token's part of dw to p
        auto result = [&](int at, Raw vx, Raw vz, Raw vd, const f2 (&sg)[H], f2 r, f2 m, f2 (&p)[H]) {
            f2 fx[H], fz[H], d[H], fw[H], ax[H], az[H];
            to_pairs<TI, V>(vx, fx);
            to_pairs<TI, V>(vd, d);
            load_weights<V>(wr ? wr + at * V : nullptr, fw);
            if (GATE != kNone) to_pairs<TI, V>(vz, fz);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                f2 v = fx[i], gate = one, slope = one;
                if (GATE != kNone) {   // slope = silu'(z) = sg + z sg (1 - sg)
                    gate = mul2(fz[i], sg[i]);
                    slope = fma2(gate, fma2(sg[i], minus, one), sg[i]);
                }
                if (GATE == kFirst) v = mul2(v, gate);
                const f2 n = mul2(v, r);
                if (GATE == kAfter) az[i] = mul2(mul2(d[i], n), mul2(fw[i], slope));
                if (GATE == kAfter) d[i] = mul2(d[i], gate);
                const f2 dv = fma2(r, mul2(d[i], fw[i]), mul2(n, m));
                p[i] = fma2(d[i], n, p[i]);
                ax[i] = GATE == kFirst ? mul2(dv, gate) : dv;
                if (GATE == kFirst) az[i] = mul2(mul2(dv, fx[i]), slope);
            }
            store_raw<TI, V>(ox + at * V, from_pairs<TI, V>(ax));
            if (GATE != kNone) store_raw<TI, V>(oz + at * V, from_pairs<TI, V>(az));
        };
        f2 r2, m2;
        auto scales = [&] {
            // two halves of red in turn: the next token's sums do not overwrite one being read
            const float2 s = team_sum<WARP>(sum2(ss), sum2(qv), red[parity]);
            parity ^= 1;
            const float r = rsqrtf(s.x * inv + q.eps);
            r2 = dup2(r);
            m2 = dup2(-r * (r * (s.y * inv)));   // dv = r q - (v r) r (r mean(q v)): no r^3 to underflow
        };
        if constexpr (VPT > 0) {
            f2 sg[K][H];
            Raw rx, rz, rd;
            if (STAGE) {
                stage_wait();
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (tid + k * nt < nv) {
                        const int at = (tid + k * nt) * V;
                        own[0][k][0] = load_raw<TI, V>(xr + at);
                        if (GATE != kNone) own[0][k][1] = load_raw<TI, V>(zr + at);
                        own[0][k][2] = load_raw<TI, V>(dr + at);
                    }
            }
            auto get = [&](int k, int w) {
                if constexpr (STAGE) return st[((half * K + k) * 3 + w) * bt];
                else return own[0][k][w];
            };
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < nv) {
                    rz = zero_raw<Raw>();
                    if (GATE != kNone) rz = get(k, 1);
                    sums(tid + k * nt, get(k, 0), rz, get(k, 2), sg[k]);
                }
            if (STAGE && row + nslot < q.rows) copy(row + nslot, half ^ 1);
            scales();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < nv) {
                    rx = get(k, 0);
                    rd = get(k, 2);
                    rz = zero_raw<Raw>();
                    if (GATE != kNone) rz = get(k, 1);
                    result(tid + k * nt, rx, rz, rd, sg[k], r2, m2, acc[k]);
                }
            half ^= 1;
        } else {
            f2 sg[H];
            const auto zraw = [&](int i) { return GATE != kNone ? load_raw<TI, V>(zr + i * V) : zero_raw<Raw>(); };
            for (int i = tid; i < nv; i += nt)
                sums(i, load_raw<TI, V>(xr + i * V), zraw(i), load_raw<TI, V>(dr + i * V), sg);
            scales();
            for (int i = tid; i < nv; i += nt) {
                const Raw z0 = zraw(i);
                f2 p[H], fz[H];
                to_pairs<TI, V>(z0, fz);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    p[j] = dup2(0.f);
                    sg[j] = sigmoid2(fz[j]);
                }
                result(i, load_raw<TI, V>(xr + i * V), z0, load_raw<TI, V>(dr + i * V), sg, r2, m2, p);
                if (pr)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float lo, hi;
                        unpack2(p[j / 2], lo, hi);
                        const float add = j & 1 ? hi : lo;
                        pr[i * V + j] = begun ? pr[i * V + j] + add : add;
                    }
            }
            begun = true;
        }
    }
    if (!pr) return;
    if (VPT > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = tid + k * nt;
            if (at < nv) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float lo, hi;
                    unpack2(acc[k][j / 2], lo, hi);
                    pr[at * V + j] = j & 1 ? hi : lo;
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

// bf16 groups of 513 to 640 channels, backward: five rounds of four a lane instead of three of
// eight, the last of them half idle (b8 T4096 G8: groups of 520 294 against 305 us, 576 296
// against 309, 640 298 against 313).
bool five_of_four(const NormArgs& a) { return a.dtype == 1 && a.D / a.G > 512 && a.D / a.G <= 640; }

// Backward slots of dw: 16 or 20 warp teams an SM, or blocks of 1024 threads in all, each with an
// equal share of the tokens, over the groups.  An SM holds that many at once, except in fp32 at
// groups of 385 to 640: three blocks of 61,440 bytes of shared memory where five are counted, so
// that the shares run in two waves.
int64_t bwd_team_slots(const NormArgs& a) {
    const int64_t S = a.D / a.G, full = a.dtype == 1 ? 8 : 4;
    const int64_t V = S % full == 0 && !five_of_four(a) ? full : a.dtype != 1 ? 1 : S % 4 == 0 ? 4 : S % 2 == 0 ? 2 : 1;
    const int64_t nv = S / V, each = (nv + 31) / 32 * V;
    const int64_t per_sm = nv <= 96 || (V == 4 && nv <= 160)
                               ? bwd_warps((int)each)
                               : std::max<int64_t>(1, 1024 / team_threads(nv, V <= 2 ? 4 : nv <= 1024 ? 1 : 2));
    const int64_t teams = (int64_t)sm_count() * per_sm;
    return std::max<int64_t>(1, std::min<int64_t>(a.b * a.T, teams / a.G));
}

template <typename TI, int V, int GATE>
cudaError_t fwd_go(const NormArgs& a, const TI* x, const float* w, const TI* z, TI* y, cudaStream_t st) {
    const Rows q = rows_of(a);
    const int64_t items = q.rows * q.G, nv = q.S / V;
    if (items >= (int64_t(1) << 31)) return kGridLimit;
    const unsigned wb = (unsigned)((items + kWarpTeams - 1) / kWarpTeams);
    const unsigned bb = (unsigned)items;
    if (nv <= 32) norm_fwd_kernel<TI, V, 1, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (nv <= 64) norm_fwd_kernel<TI, V, 2, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (nv <= 128) norm_fwd_kernel<TI, V, 4, GATE, true><<<wb, kWarpTeams * 32, 0, st>>>(x, w, z, y, q);
    else if (V <= 2 && nv <= 8192)   // narrow accesses: more of them a thread, fewer warps to join
        norm_fwd_kernel<TI, V, V <= 2 ? 8 : 1, GATE, false><<<bb, team_threads(nv, 8), 0, st>>>(x, w, z, y, q);
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
    if (teams64 >= (int64_t(1) << 31) || q.rows >= (int64_t(1) << 31)) return kGridLimit;
    const int teams = (int)teams64;
    const unsigned wb = (unsigned)((teams64 + kWarpTeams - 1) / kWarpTeams);
    const unsigned bb = (unsigned)teams;
    // [2 halves][vectors a thread][3 tensors] of up to 16 bytes a thread: at most 192 KB a block
    auto go = [&](auto k, unsigned blocks, int threads, int vpt) {
        const size_t bytes = V * sizeof(TI), smem = bytes >= 4 ? (size_t)2 * vpt * 3 * bytes * threads : 0;
        constexpr size_t kRed = 2 * 32 * sizeof(float2);   // the kernel's static room counts against the limit too
        if (smem + kRed > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        k<<<blocks, threads, smem, st>>>(x, w, z, dy, dx, dz, part, teams, q);
        return cudaSuccess;
    };
    cudaError_t e;
    if (nv <= 32) e = go(norm_bwd_kernel<TI, V, 1, GATE, true>, wb, kWarpTeams * 32, 1);
    else if (nv <= 64) e = go(norm_bwd_kernel<TI, V, 2, GATE, true>, wb, kWarpTeams * 32, 2);
    else if (nv <= 96) e = go(norm_bwd_kernel<TI, V, 3, GATE, true>, wb, kWarpTeams * 32, 3);
    else if (V == 4 && nv <= 160)
        e = go(norm_bwd_kernel<TI, V, V == 4 ? 5 : 1, GATE, true>, wb, kWarpTeams * 32, 5);
    else if (V <= 2 && nv <= 4096)
        e = go(norm_bwd_kernel<TI, V, V <= 2 ? 4 : 1, GATE, false>, bb, team_threads(nv, 4), 4);
    else if (nv <= 1024) e = go(norm_bwd_kernel<TI, V, 1, GATE, false>, bb, team_threads(nv, 1), 1);
    else if (nv <= 2048) e = go(norm_bwd_kernel<TI, V, 2, GATE, false>, bb, team_threads(nv, 2), 2);
    else e = go(norm_bwd_kernel<TI, V, 0, GATE, false>, bb, 1024, 0);
    if (e != cudaSuccess) return e;
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

// Channels an access: the most of 16, 8 and 4 bytes at which every tensor's rows and the
// groups are aligned, else one.
int vec_of(const NormArgs& a, bool back, const void* x, const float* w, const void* z, const void* y,
           const void* o1, const void* o2) {
    const int64_t es = a.dtype == 1 ? 2 : 4;
    const Tok row{0, a.D};
    for (int V : {8, 4, 2}) {
        if (a.dtype != 1 && V != 4) continue;
        const int64_t by = V * es;
        if (back && V == 8 && five_of_four(a)) continue;
        if ((a.D / a.G) % V == 0 && reinterpret_cast<uintptr_t>(w) % (V > 2 ? 16 : 8) == 0 && vec_ok(x, a.sx, by, es) &&
            (!z || vec_ok(z, a.sz, by, es)) && vec_ok(y, a.sy, by, es) && vec_ok(o1, row, by, es) &&
            vec_ok(o2, row, by, es))
            return V;
    }
    return 1;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, const void* x, const float* w, const void* z, void* y,
                            cudaStream_t st) {
    if (a.b * a.T == 0 || a.D == 0) return cudaSuccess;
    const int V = vec_of(a, false, x, w, z, y, nullptr, nullptr);
    if (a.dtype != 1) return V == 4 ? fwd_gate<float, 4>(a, x, w, z, y, st) : fwd_gate<float, 1>(a, x, w, z, y, st);
    return V == 8   ? fwd_gate<__nv_bfloat16, 8>(a, x, w, z, y, st)
           : V == 4 ? fwd_gate<__nv_bfloat16, 4>(a, x, w, z, y, st)
           : V == 2 ? fwd_gate<__nv_bfloat16, 2>(a, x, w, z, y, st)
                    : fwd_gate<__nv_bfloat16, 1>(a, x, w, z, y, st);
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
        const int V = vec_of(a, true, x, w, z, dy, dx, dz);
        if (a.dtype != 1)
            e = V == 4 ? bwd_gate<float, 4>(a, x, w, z, dy, dx, dz, part, st)
                       : bwd_gate<float, 1>(a, x, w, z, dy, dx, dz, part, st);
        else
            e = V == 8   ? bwd_gate<__nv_bfloat16, 8>(a, x, w, z, dy, dx, dz, part, st)
                : V == 4 ? bwd_gate<__nv_bfloat16, 4>(a, x, w, z, dy, dx, dz, part, st)
                : V == 2 ? bwd_gate<__nv_bfloat16, 2>(a, x, w, z, dy, dx, dz, part, st)
                         : bwd_gate<__nv_bfloat16, 1>(a, x, w, z, dy, dx, dz, part, st);
    }
    if (e != cudaSuccess || !dw) return e;
    return launch_column_sum(part, none ? 0 : norm_bwd_slots(a), a.D, dw, a.D, nullptr, st);
}

}  // namespace m2
