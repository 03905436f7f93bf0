// scan_bwd.cuh -- gradients of the selective scan (include/mamba2_layer.h).
//
// With dY = dy silu(z) (or dy) and g_t the adjoint of h_t:
//   g_t = C_t dY_t + a_{t+1} g_{t+1},  a_t = exp(d_t A)      (last: + dfinal)
//   dC_t[n] = sum_c dY_t h_t           dB_t[n] = sum_c d_t x_t g_t
//   q_t = sum_n g_t B_t[n]             e_t = a_t g_t h_{t-1}
//   dx_t = d_t q_t + D dY_t            dd_t = x_t q_t + sum_n A e_t     ddt = dd (softplus')
//   dA = sum_t d_t e_t                 dD = sum_t dY_t x_t              dz = dy silu'(z) (C.h + D x)
//
// Three kernels.  (1) scan_local_kernel runs every stretch of the token axis from a
// zero state, forwards only: it stores the state every kL tokens, the stretch's
// final state S, its adjoint G = sum_t (prod_{s <= t} a_s) dY_t C_t of the state that
// enters it, and the sums of d.  (2) scan_join2_kernel carries the true states
// forwards and the true adjoints backwards over the stretches.  (3) scan_grad_kernel
// takes kL tokens at a time, last first: state = stored local state + exp(A sum d) x
// entering state, recomputed token by token into registers, then the adjoint walks
// back over them.  A lane does KK channels in turn, so that dB and dC are summed over
// them in registers before the warp's lanes, the block's warps and (through memory,
// by a last kernel in a fixed order) the blocks.
//
// b4 T4096 C5120 N16 bf16, gated: 1.95 ms, of which (1) 0.48, (2) 0.02, (3) 1.42 ms.  (3)
// needs 12 fp32 operations and one exponential per (t, c, n), about 0.55 ms of the pipes;
// it runs two warps a quarter of an SM (252 registers: 64 of dB and dC, 36 of states),
// with the issue slots at 0.53 and the load unit's data path at 0.62.  Three blocks an SM
// spill (2.45 to 2.9 ms), as do two channels at once (2.13 ms); stretches of four tokens
// double the stored states (2.3 to 2.6 ms); eight channels in turn leave one block an SM
// (3.0 ms).
#pragma once

#include <algorithm>

#include "internal.h"
#include "scan.cuh"

namespace m2 {
namespace scan_bwd {

constexpr int kL = 8;      // tokens between stored states = tokens of a gradient tile
constexpr int kGT = 128;   // threads of the gradient kernel

struct BwdP {
    const void *x, *dt, *B, *C, *z, *dy;
    const float *A, *D, *bias;
    const int32_t* lengths;
    const float *h_in, *g_in;   // [nseg][b][D][N] or null (zeros)
    float* ck;                  // [b][nck][D][N]
    float* ck_d;                // [b][nck][D]: sum of d from the stretch's start
    float *seg_h, *seg_g, *seg_d;
    void *dx, *ddt, *dz;
    float *dinit;
    float* part_bc;             // [ncb][b T G][2 N]
    float* part_A;              // [b nseg][D][N]
    float* part_v;              // [b nseg][2][D]: dD, ddt_bias
    int T, Dch, G, Dg, ncb, nseg, SL, nck, softplus;
    int64_t b;
    Tok sx, sdt, sB, sC, sz, sy;
};

// (1) Each stretch from zero, with the forward's lanes and tiles.  ADJ: also its adjoint
// (only needed when there are several stretches).
template <typename TI, int N, int V, bool ADJ>
__global__ void __launch_bounds__(Cfg<N>::NT, (min_blocks<TI, N, V>() < 8 ? min_blocks<TI, N, V>() : 8))
scan_local_kernel(const BwdP p) {
    using K = Cfg<N>;
    constexpr int NT = K::NT, LPC = K::LPC, CB = K::CB, TT = K::TT;
    constexpr int PR = CB / V, RS = NT / PR, IT = TT / RS;
    constexpr int BI = TT * N / V / NT, VB = V * (int)sizeof(TI);
    static_assert(TT % kL == 0, "whole stored states");
    extern __shared__ __align__(16) unsigned char smem[];
    float2* sP = reinterpret_cast<float2*>(smem);                         // [TT][CB] (d, dx)
    float* sB = reinterpret_cast<float*>(smem + (size_t)TT * CB * 8);     // [TT][N]
    float* sC = sB + TT * N;                                              // [TT][N]
    float* sY = sC + TT * N;                                              // [TT][CB] dY
    TI* sS = reinterpret_cast<TI*>(sY + TT * CB);                         // staged: x, dt, dy, z [TT][CB], B, C [TT][N]
    typedef typename Pack<TI, V>::Raw Raw;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int id = blockIdx.x;
    const int cb = id % p.ncb;
    id /= p.ncb;
    const int g = id % p.G;
    id /= p.G;
    const int seg = id % p.nseg, b = id / p.nseg;
    const int n = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.T) : p.T;
    const int s0 = seg * p.SL, s1 = min(s0 + p.SL, p.T), sn = min(s1, n);
    const int lc = (tid % PR) * V, r0 = tid / PR;
    const bool con = cb * CB + lc < p.Dg;
    const int64_t c = (int64_t)g * p.Dg + cb * CB + lc;
    // pointers to this thread's first row of the tile to load next, and the steps to its others
    const int64_t tr = s0 + r0;
    const TI* xp = static_cast<const TI*>(p.x) + (int64_t)b * p.sx.b + tr * p.sx.t + c;
    const TI* dp = static_cast<const TI*>(p.dt) + (int64_t)b * p.sdt.b + tr * p.sdt.t + c;
    const TI* zp = static_cast<const TI*>(p.z) + (int64_t)b * p.sz.b + tr * p.sz.t + c;
    const TI* yp = static_cast<const TI*>(p.dy) + (int64_t)b * p.sy.b + tr * p.sy.t + c;
    constexpr int BR = NT * V / N;     // rows of B between a thread's accesses
    static_assert(BR * N == NT * V, "B tile shape");
    const int br = tid * V / N;
    const TI* Bp = static_cast<const TI*>(p.B) + (int64_t)b * p.sB.b + (s0 + br) * p.sB.t + g * N + tid * V % N;
    const TI* Cp = static_cast<const TI*>(p.C) + (int64_t)b * p.sC.b + (s0 + br) * p.sC.t + g * N + tid * V % N;
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = p.bias && con ? __ldg(p.bias + c + j) : 0.f;

    const int q = lane % LPC, ch = 2 * (warp * K::CPW + lane / LPC);
    const int64_t cg = (int64_t)g * p.Dg + cb * CB + ch;
    bool on[2];
    f2 A2[2][2], h[2][2], G[2][2], P[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        on[j] = cb * CB + ch + j < p.Dg;
        h[j][0] = h[j][1] = G[j][0] = G[j][1] = A2[j][0] = A2[j][1] = dup2(0.f);
        P[j][0] = P[j][1] = dup2(1.f);
        if (on[j]) {
            const float* Ap = p.A + (cg + j) * N + q * kNS;
            A2[j][0] = pack2(__ldg(Ap) * kLog2e, __ldg(Ap + 1) * kLog2e);
            A2[j][1] = pack2(__ldg(Ap + 2) * kLog2e, __ldg(Ap + 3) * kLog2e);
        }
    }
    float dsum[2] = {0.f, 0.f};
    float* ck = p.ck + ((int64_t)b * p.nck * p.Dch + cg) * N + q * kNS;
    float* ckd = p.ck_d + (int64_t)b * p.nck * p.Dch + cg;

    const int own = r0 * CB + lc;   // this thread's first element of a staged tile
    const bool whole = cb * CB + CB <= p.Dg;   // every channel of the block exists
    auto stage_tile = [&](const bool FULL, int lim) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const bool real = FULL || (con && r0 + i * RS < lim);
            TI* d = sS + own + i * RS * CB;
            stage_copy<VB>(d, real ? xp + i * (RS * p.sx.t) : p.x, real);
            stage_copy<VB>(d + TT * CB, real ? dp + i * (RS * p.sdt.t) : p.x, real);
            if (ADJ) stage_copy<VB>(d + 2 * TT * CB, real ? yp + i * (RS * p.sy.t) : p.x, real);
            if (ADJ && p.z) stage_copy<VB>(d + 3 * TT * CB, real ? zp + i * (RS * p.sz.t) : p.x, real);
        }
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const bool real = FULL || br + i * BR < lim;
            TI* d = sS + 4 * TT * CB + (tid + i * NT) * V;
            stage_copy<VB>(d, real ? Bp + i * (BR * p.sB.t) : p.x, real);
            if (ADJ) stage_copy<VB>(d + TT * N, real ? Cp + i * (BR * p.sC.t) : p.x, real);
        }
    };
    auto stage = [&](int t0) {      // tile after tile; whole tiles without the edges' checks
        const int lim = sn - t0;
        if (whole && lim >= TT) stage_tile(true, lim);
        else stage_tile(false, lim);
        stage_commit();
        xp += TT * p.sx.t;
        dp += TT * p.sdt.t;
        zp += TT * p.sz.t;
        yp += TT * p.sy.t;
        Bp += TT * p.sB.t;
        Cp += TT * p.sC.t;
    };
    stage(s0);
    for (int t0 = s0; t0 < s1; t0 += TT) {
        stage_wait();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = r0 + i * RS;
            const bool real = con && t0 + r < sn;
            const TI* st = sS + own + i * RS * CB;
            f2 fx[1], fd[1], fz[1], fy[1];
            to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st), fx);
            to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st + TT * CB), fd);
            f2 d = add2(fd[0], pack2(bias[0], bias[V - 1]));
            if (p.softplus) d = softplus2(d);
            if (!real) d = dup2(0.f);
            float d0, d1, u0, u1;
            unpack2(d, d0, d1);
            unpack2(mul2(d, fx[0]), u0, u1);
            if constexpr (V == 2)
                *reinterpret_cast<float4*>(sP + r * CB + lc) = make_float4(d0, u0, d1, u1);
            else
                sP[r * CB + lc] = make_float2(d0, u0);
            if (ADJ) {
                to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st + 2 * TT * CB), fy);
                if (p.z) {
                    to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st + 3 * TT * CB), fz);
                    fy[0] = mul2(fy[0], mul2(fz[0], sigmoid2(fz[0])));
                }
                unpack2(fy[0], u0, u1);
                if constexpr (V == 2)
                    *reinterpret_cast<float2*>(sY + r * CB + lc) = make_float2(u0, u1);
                else
                    sY[r * CB + lc] = u0;
            }
        }
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const int e = (tid + i * NT) * V;
            const TI* st = sS + 4 * TT * CB + e;
            float f[V];
            Conv<TI, V>::to(*reinterpret_cast<const Raw*>(st), f);
#pragma unroll
            for (int j = 0; j < V; ++j) sB[e + j] = f[j];
            if (ADJ) {
                Conv<TI, V>::to(*reinterpret_cast<const Raw*>(st + TT * N), f);
#pragma unroll
                for (int j = 0; j < V; ++j) sC[e + j] = f[j];
            }
        }
        __syncthreads();
        if (t0 + TT < s1) stage(t0 + TT);
        const float4* pP = reinterpret_cast<const float4*>(sP + ch);
        const float2* pY = reinterpret_cast<const float2*>(sY + ch);
#pragma unroll 1
        for (int tb = 0; tb < TT; tb += kL) {
            if (t0 + tb >= s1) break;
            const int64_t at = (int64_t)((t0 + tb) / kL) * p.Dch;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (on[j]) {
                    float4 v;
                    unpack2(h[j][0], v.x, v.y);
                    unpack2(h[j][1], v.z, v.w);
                    *reinterpret_cast<float4*>(ck + (at + j) * N) = v;
                    if (q == 0) ckd[at + j] = dsum[j];
                }
#pragma unroll
            for (int u = 0; u < kL; ++u) {
                const int t = tb + u;
                const float4 w = pP[t * (CB / 2)];
                const ulonglong2 Bv = *reinterpret_cast<const ulonglong2*>(sB + t * N + q * kNS);
                ulonglong2 Cv = {0, 0};
                float2 yv = make_float2(0.f, 0.f);
                if (ADJ) {
                    Cv = *reinterpret_cast<const ulonglong2*>(sC + t * N + q * kNS);
                    yv = pY[t * (CB / 2)];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const f2 d = dup2(j ? w.z : w.x), dx = dup2(j ? w.w : w.y);
                    const f2 a0 = ex2_2(mul2(d, A2[j][0])), a1 = ex2_2(mul2(d, A2[j][1]));
                    h[j][0] = fma2(a0, h[j][0], mul2(dx, Bv.x));
                    h[j][1] = fma2(a1, h[j][1], mul2(dx, Bv.y));
                    dsum[j] += j ? w.z : w.x;
                    if (ADJ) {
                        const f2 y2 = dup2(j ? yv.y : yv.x);
                        P[j][0] = mul2(P[j][0], a0);
                        P[j][1] = mul2(P[j][1], a1);
                        G[j][0] = fma2(P[j][0], mul2(y2, Cv.x), G[j][0]);
                        G[j][1] = fma2(P[j][1], mul2(y2, Cv.y), G[j][1]);
                    }
                }
            }
        }
        __syncthreads();
    }
    if constexpr (ADJ)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!on[j]) continue;
        const int64_t at = ((int64_t)seg * p.b + b) * p.Dch + cg + j;
        float4 v;
        unpack2(h[j][0], v.x, v.y);
        unpack2(h[j][1], v.z, v.w);
        *reinterpret_cast<float4*>(p.seg_h + at * N + q * kNS) = v;
        unpack2(G[j][0], v.x, v.y);
        unpack2(G[j][1], v.z, v.w);
        *reinterpret_cast<float4*>(p.seg_g + at * N + q * kNS) = v;
        if (q == 0) p.seg_d[at] = dsum[j];
    }
}

// Sum of 2^k-strided lanes: v[0 .. M) over the CPW lanes lane, lane ^ LPC, ...; each
// lane ends with M / CPW of the sums, those of values  sel + CPW * j  where sel is the
// lane's channel index within the warp.
template <int M, int CPW, int LPC> __device__ __forceinline__ void channel_sum(float (&v)[M]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1, m = M; o < CPW; o <<= 1, m >>= 1) {
        const bool hi = lane & (o * LPC);
#pragma unroll
        for (int i = 0; i < M / 2; ++i)
            if (i < m / 2) {
                const float give = hi ? v[2 * i] : v[2 * i + 1], keep = hi ? v[2 * i + 1] : v[2 * i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * LPC);
            }
    }
}

// KK = 4: dB and dC leave the registers once for four channels (the sum over the lanes is a
// tenth of the work instead of a third).  KK = 1: a quarter of the channels a block, for
// problems that leave SMs without a block otherwise.
template <typename TI, int N, int KK> struct GCfg {
    static constexpr int LPC = N / kNS, CPW = 32 / LPC, WARPS = kGT / 32;
    static constexpr int CK = WARPS * CPW;       // channels of one turn
    static constexpr int CB = CK * KK;           // channels of the block
    static constexpr int U = LPC < 8 ? LPC : 8;
    static constexpr int QP = CB + (CPW < 2 ? 2 : CPW);   // pitch of the q, r, y tiles
    // shared memory, in bytes
    static constexpr size_t lane16 = (size_t)KK * kGT * 16;                   // a float4 a channel and lane
    static constexpr size_t raw = (size_t)kL * CB * sizeof(TI), rawBC = (size_t)kL * N * sizeof(TI);
    static constexpr size_t stage = 4 * raw + 2 * rawBC + lane16 + (size_t)KK * kGT * 4;
    static constexpr size_t smem = (size_t)kL * CB * 12 + 3 * (size_t)kL * QP * 4 + 2 * (size_t)kL * N * 4 +
                                   (size_t)WARPS * 2 * kL * N * 4 + 4 * lane16 + stage;
};

// (3) Gradients.  Block: CB channels of one group, one stretch of one sequence.  What a
// thread stages for the tile before (inputs, stored states) only it reads, so the copies
// need no barrier; they run under the arithmetic of the tile at hand.
template <typename TI, int N, int V, bool GATE, int kK>
__global__ void __launch_bounds__(kGT)
scan_grad_kernel(const BwdP p) {
    using K = GCfg<TI, N, kK>;
    constexpr int LPC = K::LPC, CPW = K::CPW, CB = K::CB, QP = K::QP, U = K::U;
    constexpr int PR0 = CB / V, PR = PR0 < kGT ? PR0 : kGT;          // threads a row
    constexpr int RS = kGT / PR, CI = PR0 / PR, RI = RS < kL ? kL / RS : 1;   // rows a pass, column passes, row passes
    static_assert(RS * RI >= kL && CI * PR == PR0, "tile shape");    // RS > kL: the last threads have no row
    constexpr int BI = (kL * N / V + kGT - 1) / kGT;                 // accesses of B (and of C) a thread
    constexpr int VB = V * (int)sizeof(TI);
    extern __shared__ __align__(16) unsigned char smem[];
    float2* sP = reinterpret_cast<float2*>(smem);                         // [kL][CB] (d, dx)
    float4* sA = reinterpret_cast<float4*>(sP + kL * CB);                 // [kK][kGT] A log2(e)
    float4* sH = sA + kK * kGT;                                           // entering state
    float4* sG = sH + kK * kGT;                                           // adjoint carried back
    float4* sD = sG + kK * kGT;                                           // dA
    float4* stK = sD + kK * kGT;                                          // staged: stored state
    float* stD = reinterpret_cast<float*>(stK + kK * kGT);                // staged: its sum of d
    TI* stX = reinterpret_cast<TI*>(stD + kK * kGT);                      // staged: x, dt, dy, z [kL][CB], B, C [kL][N]
    TI* stT = stX + kL * CB;
    TI* stY = stT + kL * CB;
    TI* stZ = stY + kL * CB;
    TI* stB = stZ + kL * CB;
    TI* stC = stB + kL * N;
    float* sY = reinterpret_cast<float*>(stC + kL * N);                   // [kL][CB] dY
    float* sB = sY + kL * CB;                                             // [kL][N]
    float* sC = sB + kL * N;
    float* sR = sC + kL * N;                                              // [WARPS][2 kL N]
    float* sQ = sR + K::WARPS * 2 * kL * N;                               // [kL][QP] q; then r, then C.h
    float* sE = sQ + kL * QP;
    float* sO = sE + kL * QP;
    typedef typename Pack<TI, V>::Raw Raw;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int id = blockIdx.x;
    const int cb = id % p.ncb;
    id /= p.ncb;
    const int g = id % p.G;
    id /= p.G;
    const int seg = id % p.nseg, b = id / p.nseg;
    const int n = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.T) : p.T;
    const int s0 = seg * p.SL, s1 = min(s0 + p.SL, p.T), sn = min(s1, n);
    const int64_t cg0 = (int64_t)g * p.Dg + cb * CB;   // first channel of the block
    const int left = p.Dg - cb * CB;                    // channels of the block that exist

    const int lc0 = (tid % PR) * V, r0 = tid / PR;
    f2 bias[CI], skip[CI], accD[CI], accB[CI];
#pragma unroll
    for (int ci = 0; ci < CI; ++ci) {
        const int lc = lc0 + ci * PR * V;
        const bool in = lc < left;
        const float* pb = p.bias && in ? p.bias + cg0 + lc : nullptr;
        const float* pd = p.D && in ? p.D + cg0 + lc : nullptr;
        bias[ci] = pb ? pack2(__ldg(pb), __ldg(pb + V - 1)) : dup2(0.f);
        skip[ci] = pd ? pack2(__ldg(pd), __ldg(pd + V - 1)) : dup2(0.f);
        accD[ci] = accB[ci] = dup2(0.f);
    }
    const int q = lane % LPC, cw = lane / LPC;
    const int64_t seg_at = ((int64_t)seg * p.b + b) * p.Dch;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        const int ch = k * K::CK + warp * CPW + cw;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), h = a, gg = a;
        if (ch < left) {
            const float* Ap = p.A + (cg0 + ch) * N + q * kNS;
            a = make_float4(__ldg(Ap) * kLog2e, __ldg(Ap + 1) * kLog2e, __ldg(Ap + 2) * kLog2e, __ldg(Ap + 3) * kLog2e);
            const int64_t o = (seg_at + cg0 + ch) * N + q * kNS;
            if (p.h_in) h = make_float4(p.h_in[o], p.h_in[o + 1], p.h_in[o + 2], p.h_in[o + 3]);
            if (p.g_in) gg = make_float4(p.g_in[o], p.g_in[o + 1], p.g_in[o + 2], p.g_in[o + 3]);
        }
        sA[k * kGT + tid] = a;
        sH[k * kGT + tid] = h;
        sG[k * kGT + tid] = gg;
        sD[k * kGT + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // pointers to this thread's first element of the tile to stage next (the last tile first)
    const int tiles = (s1 - s0 + kL - 1) / kL, tl = s0 + (tiles - 1) * kL;
    const int64_t tr = tl + r0;
    const TI* xp = static_cast<const TI*>(p.x) + (int64_t)b * p.sx.b + tr * p.sx.t + cg0 + lc0;
    const TI* dp = static_cast<const TI*>(p.dt) + (int64_t)b * p.sdt.b + tr * p.sdt.t + cg0 + lc0;
    const TI* zp = static_cast<const TI*>(p.z) + (int64_t)b * p.sz.b + tr * p.sz.t + cg0 + lc0;
    const TI* yp = static_cast<const TI*>(p.dy) + (int64_t)b * p.sy.b + tr * p.sy.t + cg0 + lc0;
    constexpr int BR = kGT * V / N > 0 ? kGT * V / N : 1;   // rows of B between a thread's accesses
    const int br = tid * V / N;
    const TI* Bp = static_cast<const TI*>(p.B) + (int64_t)b * p.sB.b + (tl + br) * p.sB.t + g * N + tid * V % N;
    const TI* Cp = static_cast<const TI*>(p.C) + (int64_t)b * p.sC.b + (tl + br) * p.sC.t + g * N + tid * V % N;
    const int ch0 = warp * CPW + cw;   // the lane's channel of turn 0
    // stored states and outputs: a base the block shares, and the thread's offset in it
    const float* ckb = p.ck + (((int64_t)b * p.nck + tl / kL) * p.Dch + cg0) * N;
    const float* ckdb = p.ck_d + ((int64_t)b * p.nck + tl / kL) * p.Dch + cg0;
    const int64_t out0 = ((int64_t)b * p.T + tl) * p.Dch + cg0;
    TI* oxb = static_cast<TI*>(p.dx) + out0;
    TI* odb = static_cast<TI*>(p.ddt) + out0;
    TI* ozb = static_cast<TI*>(p.dz) + out0;
    const int oat = r0 * p.Dch + lc0;   // rows r0 < 8, channels < 2^24
    float* bcp = p.part_bc + (((int64_t)cb * p.b * p.T + (int64_t)b * p.T + tl) * p.G + g) * (2 * N);

    auto stage_tile = [&](const bool FULL, int lim) {
#pragma unroll
        for (int ci = 0; ci < CI; ++ci)
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int r = r0 + i * RS, off = ci * PR * V, at = r * CB + lc0 + off;
                if (r >= kL) continue;
                const bool real = FULL || (lc0 + off < left && r < lim);
                stage_copy<VB>(stX + at, real ? xp + i * (RS * p.sx.t) + off : p.x, real);
                stage_copy<VB>(stT + at, real ? dp + i * (RS * p.sdt.t) + off : p.x, real);
                stage_copy<VB>(stY + at, real ? yp + i * (RS * p.sy.t) + off : p.x, real);
                if (GATE) stage_copy<VB>(stZ + at, real ? zp + i * (RS * p.sz.t) + off : p.x, real);
            }
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const int e = (tid + i * kGT) * V;
            if (e >= kL * N) continue;
            const bool real = FULL || br + i * BR < lim;
            stage_copy<VB>(stB + e, real ? Bp + i * (BR * p.sB.t) : p.x, real);
            stage_copy<VB>(stC + e, real ? Cp + i * (BR * p.sC.t) : p.x, real);
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const bool real = FULL || ch0 + k * K::CK < left;
            stage_copy<16>(stK + k * kGT + tid, real ? ckb + ((ch0 + k * K::CK) * N + q * kNS) : p.ck, real);
            stage_copy<4>(stD + k * kGT + tid, real ? ckdb + (ch0 + k * K::CK) : p.ck, real);
        }
    };
    auto stage = [&](int t0) {   // tile before tile; whole tiles without the edges' checks
        const int lim = sn - t0;
        if (left >= CB && lim >= kL) stage_tile(true, lim);
        else stage_tile(false, lim);
        stage_commit();
        xp -= kL * p.sx.t;
        dp -= kL * p.sdt.t;
        zp -= kL * p.sz.t;
        yp -= kL * p.sy.t;
        Bp -= kL * p.sB.t;
        Cp -= kL * p.sC.t;
        ckb -= (int64_t)p.Dch * N;
        ckdb -= p.Dch;
    };

    stage(tl);
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const int t0 = s0 + ti * kL;
        stage_wait();
        Raw kx[CI][RI], kd[CI][RI], kz[CI][RI], ky[CI][RI];
#pragma unroll
        for (int ci = 0; ci < CI; ++ci)
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int r = r0 + i * RS, lc = lc0 + ci * PR * V, at = r * CB + lc;
                if (r >= kL) continue;
                const bool real = lc < left && t0 + r < sn;
                kx[ci][i] = *reinterpret_cast<const Raw*>(stX + at);
                kd[ci][i] = *reinterpret_cast<const Raw*>(stT + at);
                ky[ci][i] = *reinterpret_cast<const Raw*>(stY + at);
                if (GATE) kz[ci][i] = *reinterpret_cast<const Raw*>(stZ + at);
                f2 fx[1], fd[1], fz[1], fy[1];
                to_pairs<TI, V>(kx[ci][i], fx);
                to_pairs<TI, V>(kd[ci][i], fd);
                to_pairs<TI, V>(ky[ci][i], fy);
                f2 d = add2(fd[0], bias[ci]);
                if (p.softplus) d = softplus2(d);
                if (!real) d = dup2(0.f);
                if (GATE) {
                    to_pairs<TI, V>(kz[ci][i], fz);
                    fy[0] = mul2(fy[0], mul2(fz[0], sigmoid2(fz[0])));
                }
                float d0, d1, u0, u1, y0, y1;
                unpack2(d, d0, d1);
                unpack2(mul2(d, fx[0]), u0, u1);
                unpack2(fy[0], y0, y1);
                if constexpr (V == 2) {
                    *reinterpret_cast<float4*>(sP + at) = make_float4(d0, u0, d1, u1);
                    *reinterpret_cast<float2*>(sY + at) = make_float2(y0, y1);
                } else {
                    sP[at] = make_float2(d0, u0);
                    sY[at] = y0;
                }
            }
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const int e = (tid + i * kGT) * V;
            if (e >= kL * N) continue;
            float f[V];
            Conv<TI, V>::to(*reinterpret_cast<const Raw*>(stB + e), f);
#pragma unroll
            for (int j = 0; j < V; ++j) sB[e + j] = f[j];
            Conv<TI, V>::to(*reinterpret_cast<const Raw*>(stC + e), f);
#pragma unroll
            for (int j = 0; j < V; ++j) sC[e + j] = f[j];
        }
        // the stored states, brought to the true ones (the staging room is then free)
        f2 h0[kK][2];
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const float4 v = stK[k * kGT + tid];
            const f2 c2 = dup2(stD[k * kGT + tid]);
            const ulonglong2 A2 = *reinterpret_cast<const ulonglong2*>(sA + k * kGT + tid);
            const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(sH + k * kGT + tid);
            h0[k][0] = fma2(ex2_2(mul2(c2, A2.x)), hi.x, pack2(v.x, v.y));
            h0[k][1] = fma2(ex2_2(mul2(c2, A2.y)), hi.y, pack2(v.z, v.w));
        }
        __syncthreads();
        if (ti > 0) stage(t0 - kL);

        f2 dBC[2][kL][2];   // dB, dC of the lane's states, summed over its channels
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int t = 0; t < kL; ++t) dBC[w][t][0] = dBC[w][t][1] = 0;
#pragma unroll 1
        for (int k = 0; k < kK; ++k) {
            const int ch = k * K::CK + warp * CPW + cw;
            const float2* pP = sP + ch;
            const float* pY = sY + ch;
            const ulonglong2 A2 = *reinterpret_cast<const ulonglong2*>(sA + k * kGT + tid);
            f2 hs[kL + 1][2];
            hs[0][0] = h0[0][0];
            hs[0][1] = h0[0][1];
#pragma unroll
            for (int i = 0; i + 1 < kK; ++i) {   // the loop over k is not unrolled: the next one moves up
                h0[i][0] = h0[i + 1][0];
                h0[i][1] = h0[i + 1][1];
            }
#pragma unroll
            for (int t = 0; t < kL; ++t) {
                const float2 w = pP[t * CB];
                const ulonglong2 Bv = *reinterpret_cast<const ulonglong2*>(sB + t * N + q * kNS);
                const f2 d = dup2(w.x), dx = dup2(w.y);
                hs[t + 1][0] = fma2(ex2_2(mul2(d, A2.x)), hs[t][0], mul2(dx, Bv.x));
                hs[t + 1][1] = fma2(ex2_2(mul2(d, A2.y)), hs[t][1], mul2(dx, Bv.y));
            }
            ulonglong2 G = *reinterpret_cast<const ulonglong2*>(sG + k * kGT + tid);
            ulonglong2 dA = *reinterpret_cast<const ulonglong2*>(sD + k * kGT + tid);
#pragma unroll
            for (int tb = kL - U; tb >= 0; tb -= U) {
                float vq[U], ve[U], vo[U];
#pragma unroll
                for (int u = U - 1; u >= 0; --u) {
                    const int t = tb + u;
                    const float2 w = pP[t * CB];
                    const ulonglong2 Bv = *reinterpret_cast<const ulonglong2*>(sB + t * N + q * kNS);
                    const ulonglong2 Cv = *reinterpret_cast<const ulonglong2*>(sC + t * N + q * kNS);
                    // The decays are taken a second time: kept from the pass above they cost 32
                    // registers and spills (2.07 ms against 1.95 ms, b4 T4096 C5120 N16 bf16).
                    // The compiler is kept from keeping them.
                    float dt_ = w.x;
                    asm volatile("" : "+f"(dt_));
                    const f2 y2 = dup2(pY[t * CB]), d = dup2(dt_), dx = dup2(w.y);
                    G.x = fma2(y2, Cv.x, G.x);
                    G.y = fma2(y2, Cv.y, G.y);
                    dBC[1][t][0] = fma2(y2, hs[t + 1][0], dBC[1][t][0]);
                    dBC[1][t][1] = fma2(y2, hs[t + 1][1], dBC[1][t][1]);
                    dBC[0][t][0] = fma2(dx, G.x, dBC[0][t][0]);
                    dBC[0][t][1] = fma2(dx, G.y, dBC[0][t][1]);
                    vq[u] = sum2(fma2(G.y, Bv.y, mul2(G.x, Bv.x)));
                    if (GATE) vo[u] = sum2(fma2(hs[t + 1][1], Cv.y, mul2(hs[t + 1][0], Cv.x)));
                    G.x = mul2(G.x, ex2_2(mul2(d, A2.x)));
                    G.y = mul2(G.y, ex2_2(mul2(d, A2.y)));
                    const f2 e0 = mul2(G.x, hs[t][0]), e1 = mul2(G.y, hs[t][1]);
                    ve[u] = sum2(fma2(e1, A2.y, mul2(e0, A2.x)));
                    dA.x = fma2(d, e0, dA.x);
                    dA.y = fma2(d, e1, dA.y);
                }
                const int at = (tb + (lane & (U - 1))) * QP + ch;
                const float fq = lanes_sum<LPC, U>(vq), fe = lanes_sum<LPC, U>(ve);
                float fo = 0.f;
                if (GATE) fo = lanes_sum<LPC, U>(vo);
                if (LPC <= U || q < U) {
                    sQ[at] = fq;
                    sE[at] = fe;
                    if (GATE) sO[at] = fo;
                }
            }
            *reinterpret_cast<ulonglong2*>(sG + k * kGT + tid) = G;
            *reinterpret_cast<ulonglong2*>(sD + k * kGT + tid) = dA;
        }
        // dB, dC: over the warp's channels, then its warps.  Values are numbered
        // ((which kL) + t) 4 + state.
        {
            float v[8 * kL];
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int t = 0; t < kL; ++t) {
                    unpack2(dBC[w][t][0], v[(w * kL + t) * 4], v[(w * kL + t) * 4 + 1]);
                    unpack2(dBC[w][t][1], v[(w * kL + t) * 4 + 2], v[(w * kL + t) * 4 + 3]);
                }
            channel_sum<8 * kL, CPW, LPC>(v);
#pragma unroll
            for (int i = 0; i < 8 * kL / CPW; ++i) {
                const int e = cw + CPW * i, wt = e >> 2, s = e & 3;   // wt = which kL + t
                sR[(warp * 2 * kL + wt) * N + q * kNS + s] = v[i];
            }
        }
        __syncthreads();
        for (int e = tid; e < 2 * kL * N; e += kGT) {
            const int wt = e / N, r = wt % kL;
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < K::WARPS; ++w) a += sR[w * 2 * kL * N + e];
            if (t0 + r < s1) bcp[r * (p.G * 2 * N) + (wt / kL) * N + e % N] = a;
        }
        bcp -= kL * p.G * 2 * N;
#pragma unroll
        for (int ci = 0; ci < CI; ++ci)
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int r = r0 + i * RS, t = t0 + r, lc = lc0 + ci * PR * V;
                if (r >= kL || lc >= left || t >= s1) continue;
                const bool real = t < sn;
                f2 fx[1], fd[1], fz[1], fy[1], od[1], o[1], qv, ev, ov, d;
                to_pairs<TI, V>(kx[ci][i], fx);
                to_pairs<TI, V>(kd[ci][i], fd);
                to_pairs<TI, V>(ky[ci][i], fy);
                if constexpr (V == 2) {
                    const float4 w = *reinterpret_cast<const float4*>(sP + r * CB + lc);
                    const float2 a = *reinterpret_cast<const float2*>(sQ + r * QP + lc);
                    const float2 e = *reinterpret_cast<const float2*>(sE + r * QP + lc);
                    d = pack2(w.x, w.z);
                    qv = pack2(a.x, a.y);
                    ev = pack2(e.x, e.y);
                    if (GATE) {
                        const float2 h = *reinterpret_cast<const float2*>(sO + r * QP + lc);
                        ov = pack2(h.x, h.y);
                    }
                } else {
                    d = pack2(sP[r * CB + lc].x, 0.f);
                    qv = pack2(sQ[r * QP + lc], 0.f);
                    ev = pack2(sE[r * QP + lc], 0.f);
                    if (GATE) ov = pack2(sO[r * QP + lc], 0.f);
                }
                const int at = oat + i * RS * p.Dch + ci * PR * V;
                if (GATE) {
                    to_pairs<TI, V>(kz[ci][i], fz);
                    const f2 sg = sigmoid2(fz[0]);
                    // silu' = sg (1 + z (1 - sg))
                    const f2 slope = mul2(sg, fma2(fz[0], fma2(sg, dup2(-1.f), dup2(1.f)), dup2(1.f)));
                    o[0] = mul2(mul2(fy[0], slope), fma2(skip[ci], fx[0], ov));
                    store_raw<TI, V>(ozb + at, from_pairs<TI, V>(o));
                    fy[0] = mul2(fy[0], mul2(fz[0], sg));
                }
                o[0] = fma2(d, qv, mul2(skip[ci], fy[0]));
                store_raw<TI, V>(oxb + at, from_pairs<TI, V>(o));
                od[0] = fma2(fx[0], qv, mul2(dup2(0.6931471805599453f), ev));   // e was taken with A log2(e)
                if (p.softplus) od[0] = mul2(od[0], sigmoid2(add2(fd[0], bias[ci])));
                if (!real) od[0] = dup2(0.f);
                store_raw<TI, V>(odb + at, from_pairs<TI, V>(od));
                accD[ci] = fma2(fy[0], fx[0], accD[ci]);
                accB[ci] = add2(accB[ci], od[0]);
            }
        oxb -= (int64_t)kL * p.Dch;
        odb -= (int64_t)kL * p.Dch;
        ozb -= (int64_t)kL * p.Dch;
        __syncthreads();
    }
    // dA, dinit
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        const int ch = k * K::CK + warp * CPW + cw;
        if (ch < left) {
            const int64_t o = (((int64_t)b * p.nseg + seg) * p.Dch + cg0 + ch) * N + q * kNS;
            *reinterpret_cast<float4*>(p.part_A + o) = sD[k * kGT + tid];
            if (p.dinit && seg == 0) {
                const float4 v = sG[k * kGT + tid];
                float* f = p.dinit + ((int64_t)b * p.Dch + cg0 + ch) * N + q * kNS;
                f[0] = v.x;
                f[1] = v.y;
                f[2] = v.z;
                f[3] = v.w;
            }
        }
    }
    // dD, ddt_bias: over the block's rows, through the q and r tiles
    if (r0 < kL) {
#pragma unroll
        for (int ci = 0; ci < CI; ++ci) {
            const int at = r0 * QP + lc0 + ci * PR * V;
            float a, c;
            unpack2(accD[ci], a, c);
            sQ[at] = a;
            if (V == 2) sQ[at + 1] = c;
            unpack2(accB[ci], a, c);
            sE[at] = a;
            if (V == 2) sE[at + 1] = c;
        }
    }
    __syncthreads();
    for (int c = tid; c < CB && c < left; c += kGT) {
        float a = 0.f, d = 0.f;
#pragma unroll
        for (int r = 0; r < (RS < kL ? RS : kL); ++r) {
            a += sQ[r * QP + c];
            d += sE[r * QP + c];
        }
        float* o = p.part_v + ((int64_t)b * p.nseg + seg) * 2 * p.Dch + cg0 + c;
        o[0] = a;
        o[p.Dch] = d;
    }
}

// (2) The stretches' true entering states and leaving adjoints (scan_bwd.cu).
cudaError_t join(const BwdP& p, int N, const float* init, const float* dfinal, cudaStream_t st);

template <typename KT> cudaError_t allow(KT k, size_t smem) {
    return smem > 48 * 1024 ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                            : cudaSuccess;
}

template <typename TI, int N, int V>
cudaError_t bwd_v(const BwdP& p, int KK, int64_t lncb, const float* init, const float* dfinal, cudaStream_t st) {
    using L = Cfg<N>;
    const bool adj = p.nseg > 1;
    const size_t ls = (size_t)L::TT * (L::CB * (12 + 4 * sizeof(TI)) + 2 * N * (4 + sizeof(TI)));
    const int64_t lb = p.b * p.nseg * p.G * lncb, gb = p.b * p.nseg * p.G * p.ncb;
    const int64_t total = p.b * p.Dch * N;
    if (lb >= (int64_t(1) << 31) || gb >= (int64_t(1) << 31) || (total + 255) / 256 >= (int64_t(1) << 31))
        return kGridLimit;
    BwdP l = p;
    l.ncb = (int)lncb;
    auto lk = adj ? scan_local_kernel<TI, N, V, true> : scan_local_kernel<TI, N, V, false>;
    cudaError_t e = allow(lk, ls);
    if (e != cudaSuccess) return e;
    lk<<<(unsigned)lb, L::NT, ls, st>>>(l);
    BwdP m = p;
    if (adj) {
        e = join(p, N, init, dfinal, st);
        if (e != cudaSuccess) return e;
        m.h_in = p.seg_h;
        m.g_in = p.seg_g;
    } else {
        m.h_in = init;
        m.g_in = dfinal;
    }
    auto go = [&](auto gk, size_t smem) {
        const cudaError_t e = allow(gk, smem);
        if (e == cudaSuccess) gk<<<(unsigned)gb, kGT, smem, st>>>(m);
        return e;
    };
    if (KK == 4)
        e = go(p.z ? scan_grad_kernel<TI, N, V, true, 4> : scan_grad_kernel<TI, N, V, false, 4>, GCfg<TI, N, 4>::smem);
    else
        e = go(p.z ? scan_grad_kernel<TI, N, V, true, 1> : scan_grad_kernel<TI, N, V, false, 1>, GCfg<TI, N, 1>::smem);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename TI, int N>
cudaError_t bwd_n(const ScanArgs& a, const BwdP& p, int KK, const float* init, const float* dfinal, cudaStream_t st) {
    const int64_t es = sizeof(TI), by = 2 * es, lncb = (p.Dg + Cfg<N>::CB - 1) / Cfg<N>::CB;
    const Tok row{0, a.D};
    const bool two = p.Dg % 2 == 0 && vec_ok(p.x, a.sx, by, es) && vec_ok(p.dt, a.sdt, by, es) &&
                     vec_ok(p.B, a.sB, by, es) && vec_ok(p.C, a.sC, by, es) &&
                     (!p.z || (vec_ok(p.z, a.sz, by, es) && vec_ok(p.dz, row, by, es))) &&
                     vec_ok(p.dy, a.sy, by, es) && vec_ok(p.dx, row, by, es) && vec_ok(p.ddt, row, by, es);
    return two ? bwd_v<TI, N, 2>(p, KK, lncb, init, dfinal, st) : bwd_v<TI, N, 1>(p, KK, lncb, init, dfinal, st);
}


// By state size; one translation unit per element type (scan_bwd_bf16.cu, scan_bwd_f32.cu).
template <typename TI>
cudaError_t run_type(const ScanArgs& a, const BwdP& p, int KK, const float* init, const float* dfinal,
                     cudaStream_t st) {
    switch (a.N) {
        case 8: return bwd_n<TI, 8>(a, p, KK, init, dfinal, st);
        case 16: return bwd_n<TI, 16>(a, p, KK, init, dfinal, st);
        case 32: return bwd_n<TI, 32>(a, p, KK, init, dfinal, st);
        case 64: return bwd_n<TI, 64>(a, p, KK, init, dfinal, st);
        case 128: return bwd_n<TI, 128>(a, p, KK, init, dfinal, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace scan_bwd

cudaError_t scan_bwd_bf16(const ScanArgs& a, const scan_bwd::BwdP& p, int KK, const float* init,
                          const float* dfinal, cudaStream_t st);
cudaError_t scan_bwd_f32(const ScanArgs& a, const scan_bwd::BwdP& p, int KK, const float* init,
                         const float* dfinal, cudaStream_t st);

}  // namespace m2
