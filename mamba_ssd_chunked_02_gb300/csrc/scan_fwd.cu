// scan_fwd.cu -- selective scan with a decay per channel and state (include/mamba2_layer.h):
// the forward pass and the single-token step.
//
//   h_t[c,n] = exp(d_t[c] A[c,n]) h_{t-1}[c,n] + d_t[c] x_t[c] B_t[n]
//   y_t[c]   = sum_n C_t[n] h_t[c,n] + D[c] x_t[c]     (times silu(z_t[c]))
//
// Unlike the chunked scan's one decay per head, the decay differs for every (c, n),
// so there is no matrix product to regroup: per (t, c, n) the pass needs one
// exponential and four multiply-adds, and it is bound by those pipes and by the bytes
// that shared memory hands to registers, not by memory: b8 T4096 C5120 N16 bf16 takes
// 0.82 ms (1.65 TB/s; its bytes alone 0.20 ms, its exponentials 0.28 ms, its fp32
// operations about 0.4 ms), with the load unit's data path at 0.63.
//
// A block turns a tile's dt and x into (d, d x) once, in fp32 in shared memory, then each
// lane walks over the tile's tokens with its states in registers; the lanes' parts of y
// meet in shared memory, and the epilogue adds them, the skip and the gate.
#include <algorithm>

#include "internal.h"
#include "scan.cuh"
#include "tc5.cuh"

namespace m2 {
namespace {

struct FwdP {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias, *init;
    const int32_t* lengths;
    void* y;
    float* fin;
    float* seg_h;     // [nseg][b][D][N]: local final states, then incoming states
    float* seg_d;     // [nseg][b][D]: sums of d
    int32_t* turns;   // slices: [rows] slices done of each row (-1: given up), then the ticket; or null
    int32_t* err;
    uint64_t turn_ns; // longest wait for a turn
    int slices, first;   // slices of the token axis, ticket of the first block
    int T, Dch, G, Dg, ncb, nseg, SL, softplus;
    int64_t b;
    Tok sx, sdt, sB, sC, sz, sy;
};

// Rows (blocks that walk over all tokens) that are a little more than the GPU holds at
// once would take two waves.  They take turns instead: the token axis is cut into
// slices, and blocks take (slice, row) in slice order from a ticket, so that a block
// only waits for one that started before it.  The state passes through final_state.
// A wait that runs out marks the row -1 for good: its later slices leave at once.
constexpr uint64_t kTurnNs = 2000000000ull;   // 2 s: far beyond any legitimate wait
__device__ bool await_turn(const int32_t* done, int slice, uint64_t limit_ns) {
    int v = tc::ld_acquire_gpu(done);
    const uint64_t t0 = tc::globaltimer();
    while (v >= 0 && v < slice) {
        if (tc::globaltimer() - t0 > limit_ns) return false;
        __nanosleep(100);
        v = tc::ld_acquire_gpu(done);
    }
    return v >= 0;
}

// STATES: only the segment's final state from zero and its sum of d (first of the
// two passes when the token axis is split).  V: channels per access of x, dt, z, y
// and elements per access of B, C.
template <typename TI, int N, int V, bool STATES>
__global__ void __launch_bounds__(Cfg<N>::NT, (min_blocks<TI, N, V>()))
scan_fwd_kernel(const FwdP p) {
    using K = Cfg<N>;
    constexpr int NT = K::NT, LPC = K::LPC, CB = K::CB, TT = K::TT, U = K::U, UT = K::UT, YP = K::YP;
    constexpr int PR = CB / V, RS = NT / PR, IT = TT / RS;        // threads a row, rows a pass, passes
    constexpr int BI = TT * N / V / NT;                            // accesses of B (and of C) a thread
    constexpr int VB = V * (int)sizeof(TI);
    static_assert(IT >= 1 && RS * IT == TT && BI >= 1, "tile shape");
    extern __shared__ __align__(16) unsigned char smem[];
    float2* sP = reinterpret_cast<float2*>(smem);                               // [TT][CB] (d, dx)
    // y of a tile: with up to four lanes a channel, each lane's part [TT][LPC][YP] (added by
    // the epilogue: fewer instructions than lane exchanges); else the sums [TT][YP]
    constexpr bool PART = LPC <= 4;
    float* sY = reinterpret_cast<float*>(smem + (size_t)TT * CB * 8);
    constexpr int ST = 3 * TT * CB + 2 * TT * N;                                // elements of a staged tile
    TI* sS = reinterpret_cast<TI*>(sY + K::YF);                               // [2] x, dt, z [TT][CB], B, C [TT][N]
    typedef typename Pack<TI, V>::Raw Raw;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int s_turn, s_go;
    int id = blockIdx.x, slice = 0;
    int32_t* done = nullptr;
    if (!STATES && p.turns) {
        const int rows = p.ncb * p.G * (int)p.b;
        if (tid == 0) s_turn = p.first + atomicAdd(p.turns + rows, 1);
        __syncthreads();
        slice = s_turn / rows;
        id = s_turn - slice * rows;
        done = p.turns + id;
    }
    const int cb = id % p.ncb;
    id /= p.ncb;
    const int g = id % p.G;
    id /= p.G;
    const int seg = done ? slice : id % p.nseg, b = done ? id : id / p.nseg;
    const int n = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.T) : p.T;
    const int s0 = seg * p.SL, s1 = min(s0 + p.SL, p.T), sn = min(s1, n);

    // tile duty: V channels of rows r0, r0 + RS, ...
    const int lc = (tid % PR) * V, r0 = tid / PR;
    const bool con = cb * CB + lc < p.Dg;
    const int64_t c = (int64_t)g * p.Dg + cb * CB + lc;
    // pointers to this thread's first row of the tile to load next, and the steps to its others
    const int64_t tr = s0 + r0;
    const TI* xp = static_cast<const TI*>(p.x) + (int64_t)b * p.sx.b + tr * p.sx.t + c;
    const TI* dp = static_cast<const TI*>(p.dt) + (int64_t)b * p.sdt.b + tr * p.sdt.t + c;
    const TI* zp = static_cast<const TI*>(p.z) + (int64_t)b * p.sz.b + tr * p.sz.t + c;
    TI* yp = static_cast<TI*>(p.y) + (int64_t)b * p.sy.b + tr * p.sy.t + c;
    constexpr int BR = NT * V / N;     // rows of B between a thread's accesses
    static_assert(BR * N == NT * V, "B tile shape");
    const int br = tid * V / N;
    const TI* Bp = static_cast<const TI*>(p.B) + (int64_t)b * p.sB.b + (s0 + br) * p.sB.t + g * N + tid * V % N;
    const TI* Cp = static_cast<const TI*>(p.C) + (int64_t)b * p.sC.b + (s0 + br) * p.sC.t + g * N + tid * V % N;
    float bias[V], skip[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bias[j] = p.bias && con ? __ldg(p.bias + c + j) : 0.f;
        skip[j] = p.D && con && !STATES ? __ldg(p.D + c + j) : 0.f;
    }

    // scan duty: states q kNS .. of channels ch, ch + 1
    const int q = lane % LPC, ch = 2 * (warp * K::CPW + lane / LPC);
    const int64_t sc = ((int64_t)b * p.Dch + (int64_t)g * p.Dg + cb * CB + ch) * N + q * kNS;   // in [b][D][N]
    const int64_t seg_off = (int64_t)seg * p.b * p.Dch * N;
    float dsum[2] = {0.f, 0.f};

    // What a thread stages for the next tile only it reads: the copies need no barrier and no
    // registers, and run under the scan of the tile at hand.
    const int own = r0 * CB + lc;   // this thread's first element of a staged tile
    const bool whole = cb * CB + CB <= p.Dg;   // every channel of the block exists
    auto stage_tile = [&](const bool FULL, int lim, TI* buf) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const bool real = FULL || (con && r0 + i * RS < lim);
            TI* d = buf + own + i * RS * CB;
            stage_copy<VB>(d, real ? xp + i * (RS * p.sx.t) : p.x, real);
            stage_copy<VB>(d + TT * CB, real ? dp + i * (RS * p.sdt.t) : p.x, real);
            if (!STATES && p.z) stage_copy<VB>(d + 2 * TT * CB, real ? zp + i * (RS * p.sz.t) : p.x, real);
        }
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const bool real = FULL || br + i * BR < lim;
            TI* d = buf + 3 * TT * CB + (tid + i * NT) * V;
            stage_copy<VB>(d, real ? Bp + i * (BR * p.sB.t) : p.x, real);
            if (!STATES) stage_copy<VB>(d + TT * N, real ? Cp + i * (BR * p.sC.t) : p.x, real);
        }
    };
    auto stage = [&](int t0, TI* buf) {   // tile after tile; whole tiles without the edges' checks
        const int lim = sn - t0;
        if (whole && lim >= TT) stage_tile(true, lim, buf);
        else stage_tile(false, lim, buf);
        stage_commit();
        xp += TT * p.sx.t;
        dp += TT * p.sdt.t;
        zp += TT * p.sz.t;
        Bp += TT * p.sB.t;
        Cp += TT * p.sC.t;
    };
    TI *cur = sS, *nxt = sS + ST;
    stage(s0, cur);
    f2 A2[2][2], h[2][2];
    if (slice > 0) {   // the copies of the first tile are under way meanwhile
        if (tid == 0) s_go = await_turn(done, slice, p.turn_ns);
        __syncthreads();
        if (!s_go) {
            if (tid == 0) {
                record_error(p.err, kErrChainScan);
                tc::st_release_gpu(done, -1);
            }
            stage_wait();
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), v = a;
        if (cb * CB + ch + j < p.Dg) {
            const float* Ap = p.A + ((int64_t)g * p.Dg + cb * CB + ch + j) * N + q * kNS;
            a = make_float4(__ldg(Ap), __ldg(Ap + 1), __ldg(Ap + 2), __ldg(Ap + 3));
            const float* hp = STATES ? nullptr : slice > 0 ? p.fin + sc : p.seg_h ? p.seg_h + seg_off + sc : p.init ? p.init + sc : nullptr;
            if (hp) v = make_float4(__ldcg(hp + j * N), __ldcg(hp + j * N + 1), __ldcg(hp + j * N + 2), __ldcg(hp + j * N + 3));
        }
        A2[j][0] = pack2(a.x * kLog2e, a.y * kLog2e);
        A2[j][1] = pack2(a.z * kLog2e, a.w * kLog2e);
        h[j][0] = pack2(v.x, v.y);
        h[j][1] = pack2(v.z, v.w);
    }
    for (int t0 = s0; t0 < s1; t0 += TT) {
        if (t0 >= n) {   // padding only
            if (!STATES && con)
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    if (t0 + r0 + i * RS < s1) store_raw<TI, V>(yp + i * (RS * p.sy.t), zero_raw<Raw>());
            yp += TT * p.sy.t;
            continue;
        }
        stage_wait();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = r0 + i * RS;
            const bool real = con && t0 + r < sn;
            const TI* st = cur + own + i * RS * CB;
            f2 fx[1], fd[1];
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
        }
        __syncthreads();
        if (t0 + TT < s1) stage(t0 + TT, nxt);
        const float4* pP = reinterpret_cast<const float4*>(sP + ch);
        // B and C as they were staged, in the tensors' type: every thread's copies have arrived
        const TI* pB = cur + 3 * TT * CB + q * kNS;
        const TI* pC = pB + TT * N;
        constexpr int UN = 16;   // tokens unrolled
#pragma unroll 1
        for (int tb = 0; tb < TT; tb += UN) {
#pragma unroll
            for (int tu = 0; tu < UN; tu += UT) {
                f2 yp2[UT][2];
#pragma unroll
                for (int u = 0; u < UT; ++u) {
                    const int t = tb + tu + u;
                    const float4 w = pP[t * (CB / 2)];
                    const ulonglong2 Bv = states4(pB + t * N);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f2 d = dup2(j ? w.z : w.x), dx = dup2(j ? w.w : w.y);
                        h[j][0] = fma2(ex2_2(mul2(d, A2[j][0])), h[j][0], mul2(dx, Bv.x));
                        h[j][1] = fma2(ex2_2(mul2(d, A2[j][1])), h[j][1], mul2(dx, Bv.y));
                        if (STATES) dsum[j] += j ? w.z : w.x;
                    }
                    if (!STATES) {
                        const ulonglong2 Cv = states4(pC + t * N);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            yp2[u][j] = fma2(h[j][1], Cv.y, mul2(h[j][0], Cv.x));
                    }
                }
                if (!STATES && PART) {
#pragma unroll
                    for (int u = 0; u < UT; ++u)
                        *reinterpret_cast<float2*>(sY + ((tb + tu + u) * LPC + q) * YP + ch) =
                            make_float2(sum2(yp2[u][0]), sum2(yp2[u][1]));
                } else if (!STATES) {   // value 2 u + j: token u of the UT, channel ch + j
                    float yv[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) yv[u] = sum2(yp2[u / 2][u & 1]);
                    const float s = lanes_sum<LPC, U>(yv);
                    if (LPC <= U || q < U) sY[(tb + tu + ((lane & (U - 1)) >> 1)) * YP + ch + (lane & 1)] = s;
                }
            }
        }
        __syncthreads();
        if (!STATES && con) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * RS, t = t0 + r;
                f2 fx[1], o[1];
                const TI* st = cur + own + i * RS * CB;
                to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st), fx);
                constexpr int PARTS = PART ? LPC : 1;
                const float* ys = sY + r * PARTS * YP + lc;
                o[0] = dup2(0.f);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) {
                    f2 part;
                    if constexpr (V == 2) {
                        const float2 yv = *reinterpret_cast<const float2*>(ys + k * YP);
                        part = pack2(yv.x, yv.y);
                    } else {
                        part = pack2(ys[k * YP], 0.f);
                    }
                    o[0] = k ? add2(o[0], part) : part;
                }
                o[0] = fma2(pack2(skip[0], skip[V - 1]), fx[0], o[0]);
                if (p.z) {
                    f2 fz[1];
                    to_pairs<TI, V>(*reinterpret_cast<const Raw*>(st + 2 * TT * CB), fz);
                    o[0] = mul2(o[0], mul2(fz[0], sigmoid2(fz[0])));
                }
                if (t >= n) o[0] = dup2(0.f);
                if (t < s1) store_raw<TI, V>(yp + i * (RS * p.sy.t), from_pairs<TI, V>(o));
            }
        }
        yp += TT * p.sy.t;
        TI* was = cur;
        cur = nxt;
        nxt = was;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (cb * CB + ch + j >= p.Dg) continue;
        float4 v;
        unpack2(h[j][0], v.x, v.y);
        unpack2(h[j][1], v.z, v.w);
        if (STATES) {
            *reinterpret_cast<float4*>(p.seg_h + seg_off + sc + j * N) = v;
            if (q == 0)
                p.seg_d[((int64_t)seg * p.b + b) * p.Dch + (int64_t)g * p.Dg + cb * CB + ch + j] = dsum[j];
        } else if (done || seg == p.nseg - 1) {
            float* f = p.fin + sc + j * N;
            f[0] = v.x;
            f[1] = v.y;
            f[2] = v.z;
            f[3] = v.w;
        }
    }
    if (done && slice + 1 < p.slices) {
        __threadfence();
        __syncthreads();
        if (tid == 0) tc::cas_release_gpu(done, slice, slice + 1);   // not over the mark of a row given up
    }
}

// The states entering each segment: h = init; for each segment: in = h, h = exp(A
// sum d) h + local.  One thread per (b, c, n).
__global__ void __launch_bounds__(256)
scan_join_kernel(float* __restrict__ seg_h, const float* __restrict__ seg_d, const float* __restrict__ A,
                 const float* __restrict__ init, int64_t total, int64_t DN, int N, int nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const float a = __ldg(A + i % DN) * kLog2e;
    float h = init ? init[i] : 0.f;
    const int64_t bd = i / N, nbd = total / N;
    for (int s0 = 0; s0 < nseg; s0 += 4) {   // four stretches' loads in flight
        float local[4], d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s0 + k < nseg) local[k] = seg_h[(s0 + k) * total + i], d[k] = seg_d[(s0 + k) * nbd + bd];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s0 + k < nseg) {
                seg_h[(s0 + k) * total + i] = h;
                h = fmaf(ex2(a * d[k]), h, local[k]);
            }
    }
}

// One token.  A lane owns four states of a channel (one 16-byte access), N / 4
// neighbouring lanes a channel.
template <typename TI, int N>
__global__ void __launch_bounds__(256)
scan_step_kernel(float* __restrict__ state, const TI* __restrict__ x, const TI* __restrict__ dt,
                 const float* __restrict__ A, const TI* __restrict__ B, const TI* __restrict__ C,
                 const float* __restrict__ D, const TI* __restrict__ z, const float* __restrict__ bias,
                 TI* __restrict__ y, int64_t total, int Dch, int Dg, int softplus_on, int wide,
                 int64_t sx, int64_t sdt, int64_t sB, int64_t sC, int64_t sz, int64_t sy) {
    constexpr int LPC = N / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool on = i < total;                 // whole channels: total is a multiple of LPC
    const int64_t ch = on ? i / LPC : 0;
    const int qn = on ? (int)(i % LPC) * 4 : 0;
    const int64_t b = ch / Dch;
    const int c = (int)(ch - b * Dch), g = c / Dg;
    float* sp = state + ch * N + qn;
    const float* Ap = A + (int64_t)c * N + qn;
    float h[4], a[4], Bv[4], Cv[4];
    if (wide) {
        const float4 v = *reinterpret_cast<const float4*>(sp), w = __ldg(reinterpret_cast<const float4*>(Ap));
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        a[0] = w.x, a[1] = w.y, a[2] = w.z, a[3] = w.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = sp[k], a[k] = __ldg(Ap + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        Bv[k] = to_f32(B[b * sB + (int64_t)g * N + qn + k]);
        Cv[k] = to_f32(C[b * sC + (int64_t)g * N + qn + k]);
    }
    const float xv = to_f32(x[b * sx + c]), zv = z ? to_f32(z[b * sz + c]) : 0.f;
    const float raw = to_f32(dt[b * sdt + c]) + (bias ? __ldg(bias + c) : 0.f);
    const float skip = D ? __ldg(D + c) : 0.f;
    const float d = softplus_on ? softplus(raw) : raw, dx = d * xv;
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(ex2(d * (a[k] * kLog2e)), h[k], dx * Bv[k]);
        acc = fmaf(h[k], Cv[k], acc);
    }
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (!on) return;
    if (wide) {
        *reinterpret_cast<float4*>(sp) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) sp[k] = h[k];
    }
    if (qn == 0) {
        acc = fmaf(skip, xv, acc);
        if (z) acc *= zv * sigmoid(zv);
        y[b * sy + c] = from_f32<TI>(acc);
    }
}

// How the token axis is cut.
// nseg > 1: stretches side by side, for few rows; they cost a second pass (the first
//   without y), so only where one pass leaves most of the GPU without warps.
// slices > 1: rows in turns (see await_turn), for rows between one and a few waves of
//   the blocks the GPU holds.  b8 T4096 C5120 N16 bf16 (1280 rows, 1216 held): one slice
//   1.12 ms (0.99 with nine blocks an SM), 4 slices 0.87, 8 slices 0.86, 16 slices 0.88.
//   T2048, one / 8 / 16 slices: 1280 rows 526 / 426 / 442 us (fp32 603 / 506 / 519), 1760 rows
//   602 / 579 / 600, 2560 rows 883 / 832 / 865, 3840 rows 1244 / 1236 / 1288, 6400 rows
//   2056 / 2045 / 2135.
// Held: 8 blocks an SM (4 from N = 64) is what registers and shared memory allow for two
// channels an access at N = 32, and in bf16 at N = 16.  Others hold fewer: fp32 N16 and bf16
// N8 7, fp32 N8 5, one channel an access 5 to 7.  That costs them time, nothing else: rows
// between the true number and this one run in two waves without turns, and no wait depends
// on how many blocks are held.
struct Cut {
    int64_t nseg, slices, SL;
};
int64_t block_threads(const ScanArgs& a) { return a.N >= 64 ? 128 : 64; }
int64_t rows_of(const ScanArgs& a) {
    const int64_t Dg = a.D / a.G, CB = 2 * (block_threads(a) / (a.N / kNS));
    return a.b * a.G * ((Dg + CB - 1) / CB);
}
Cut cut_of(const ScanArgs& a) {
    const int64_t tt = a.N >= 128 ? 32 : 16, tiles = std::max<int64_t>(1, (a.T + tt - 1) / tt);
    const int64_t rows = std::max<int64_t>(1, rows_of(a)), held = (int64_t)sm_count() * (a.N >= 64 ? 4 : 8);
    Cut c{1, 1, tiles * tt};
    int64_t parts = 1;
    if (2 * rows <= held && tiles >= 8) {   // (fewer tiles: the two more launches cost as much)
        parts = std::min<int64_t>(held / rows, tiles / 2);
    } else if (rows > held && rows < 6 * held) {
        parts = std::min<int64_t>(8, tiles / 8);
    }
    if (parts <= 1) return c;
    c.SL = (tiles + parts - 1) / parts * tt;
    const int64_t n = (a.T + c.SL - 1) / c.SL;
    (2 * rows <= held ? c.nseg : c.slices) = n;
    return c;
}

template <typename TI, int N, int V>
cudaError_t fwd_v(const FwdP& p, bool starve, cudaStream_t st) {
    using K = Cfg<N>;
    const int64_t rows = p.b * p.G * p.ncb, blocks = rows * p.nseg * p.slices;
    constexpr size_t smem = (size_t)K::TT * K::CB * 8 + (size_t)K::YF * 4 +
                            2 * (size_t)K::TT * (3 * K::CB + 2 * N) * sizeof(TI);
    if (blocks >= (int64_t(1) << 31)) return kGridLimit;
    auto k = scan_fwd_kernel<TI, N, V, false>;
    auto s = scan_fwd_kernel<TI, N, V, true>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(s, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    if (p.turns) {
        cudaError_t e = cudaMemsetAsync(p.turns, 0, sizeof(int32_t) * (size_t)(rows + 1), st);
        if (e != cudaSuccess) return e;
    }
    if (p.nseg > 1) {
        s<<<(unsigned)blocks, K::NT, smem, st>>>(p);
        const int64_t total = p.b * p.Dch * N;
        scan_join_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(p.seg_h, p.seg_d, p.A, p.init, total,
                                                                         (int64_t)p.Dch * N, N, p.nseg);
    }
    if (starve) {   // all slices but the first, then the first
        FwdP later = p;
        later.first = (int)rows;
        k<<<(unsigned)(blocks - rows), K::NT, smem, st>>>(later);
        const cudaError_t e = cudaMemsetAsync(p.turns + rows, 0, sizeof(int32_t), st);
        if (e != cudaSuccess) return e;
        k<<<(unsigned)rows, K::NT, smem, st>>>(p);
        return cudaGetLastError();
    }
    k<<<(unsigned)blocks, K::NT, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename TI, int N> cudaError_t fwd_n(const ScanArgs& a, FwdP p, bool starve, cudaStream_t st) {
    p.ncb = (int)((p.Dg + Cfg<N>::CB - 1) / Cfg<N>::CB);
    const int64_t es = sizeof(TI), by = 2 * es;
    const bool two = p.Dg % 2 == 0 && vec_ok(p.x, a.sx, by, es) && vec_ok(p.dt, a.sdt, by, es) &&
                     vec_ok(p.B, a.sB, by, es) && vec_ok(p.C, a.sC, by, es) &&
                     (!p.z || vec_ok(p.z, a.sz, by, es)) && vec_ok(p.y, a.sy, by, es);
    return two ? fwd_v<TI, N, 2>(p, starve, st) : fwd_v<TI, N, 1>(p, starve, st);
}

}  // namespace

bool scan_fwd_turns(const ScanArgs& a) { return a.b * a.T * a.D && cut_of(a).slices > 1; }

size_t scan_fwd_workspace(const ScanArgs& a) {
    if (a.b * a.T * a.D == 0) return 0;
    const Cut c = cut_of(a);
    if (c.nseg > 1) return sizeof(float) * (size_t)(c.nseg * a.b * a.D * (a.N + 1));
    return c.slices > 1 ? sizeof(int32_t) * (size_t)(rows_of(a) + 1) : 0;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* D, const void* z, const float* dt_bias,
                            const float* init, const int32_t* lengths, void* y, float* fin, void* ws,
                            cudaStream_t st, uint64_t starve_ns) {
    if (a.b == 0 || a.D == 0) return cudaSuccess;
    if (a.T == 0) {
        const size_t bytes = sizeof(float) * (size_t)(a.b * a.D * a.N);
        return init ? cudaMemcpyAsync(fin, init, bytes, cudaMemcpyDeviceToDevice, st)
                    : cudaMemsetAsync(fin, 0, bytes, st);
    }
    FwdP p;
    p.x = x, p.dt = dt, p.B = B, p.C = C, p.z = z, p.A = A, p.D = D, p.bias = dt_bias, p.init = init;
    p.lengths = lengths, p.y = y, p.fin = fin;
    p.T = (int)a.T, p.Dch = (int)a.D, p.G = (int)a.G, p.Dg = (int)(a.D / a.G), p.softplus = a.softplus;
    const Cut cut = cut_of(a);
    p.SL = (int)cut.SL, p.nseg = (int)cut.nseg, p.b = a.b, p.ncb = 0;
    p.seg_h = cut.nseg > 1 ? static_cast<float*>(ws) : nullptr;
    p.seg_d = cut.nseg > 1 ? p.seg_h + cut.nseg * a.b * a.D * a.N : nullptr;
    p.turns = cut.slices > 1 ? static_cast<int32_t*>(ws) : nullptr;
    p.err = device_error_word();
    p.turn_ns = starve_ns ? starve_ns : kTurnNs, p.slices = (int)cut.slices, p.first = 0;
    p.sx = a.sx, p.sdt = a.sdt, p.sB = a.sB, p.sC = a.sC, p.sz = a.sz, p.sy = a.sy;
    auto go = [&](auto f16, auto f32) { return a.dtype == 1 ? f16(a, p, starve_ns != 0, st) : f32(a, p, starve_ns != 0, st); };
    switch (a.N) {
        case 8: return go(fwd_n<__nv_bfloat16, 8>, fwd_n<float, 8>);
        case 16: return go(fwd_n<__nv_bfloat16, 16>, fwd_n<float, 16>);
        case 32: return go(fwd_n<__nv_bfloat16, 32>, fwd_n<float, 32>);
        case 64: return go(fwd_n<__nv_bfloat16, 64>, fwd_n<float, 64>);
        case 128: return go(fwd_n<__nv_bfloat16, 128>, fwd_n<float, 128>);
        default: return cudaErrorInvalidValue;
    }
}

namespace {
template <typename TI>
cudaError_t step_t(const ScanArgs& a, float* state, const void* x, const void* dt, const float* A,
                   const void* B, const void* C, const float* D, const void* z, const float* bias, void* y,
                   cudaStream_t st) {
    const int64_t total = a.b * a.D * (a.N / 4), blocks = (total + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return kGridLimit;
    const int wide = reinterpret_cast<uintptr_t>(state) % 16 == 0 && reinterpret_cast<uintptr_t>(A) % 16 == 0;
    auto go = [&](auto k) {
        k<<<(unsigned)blocks, 256, 0, st>>>(
            state, static_cast<const TI*>(x), static_cast<const TI*>(dt), A, static_cast<const TI*>(B),
            static_cast<const TI*>(C), D, static_cast<const TI*>(z), bias, static_cast<TI*>(y), total, (int)a.D,
            (int)(a.D / a.G), (int)a.softplus, wide, a.sx.b, a.sdt.b, a.sB.b, a.sC.b, a.sz.b, a.sy.b);
        return cudaGetLastError();
    };
    switch (a.N) {
        case 8: return go(scan_step_kernel<TI, 8>);
        case 16: return go(scan_step_kernel<TI, 16>);
        case 32: return go(scan_step_kernel<TI, 32>);
        case 64: return go(scan_step_kernel<TI, 64>);
        case 128: return go(scan_step_kernel<TI, 128>);
        default: return cudaErrorInvalidValue;
    }
}
}  // namespace

cudaError_t launch_scan_step(const ScanArgs& a, float* state, const void* x, const void* dt, const float* A,
                             const void* B, const void* C, const float* D, const void* z,
                             const float* dt_bias, void* y, cudaStream_t st) {
    if (a.b == 0 || a.D == 0) return cudaSuccess;
    return a.dtype == 1 ? step_t<__nv_bfloat16>(a, state, x, dt, A, B, C, D, z, dt_bias, y, st)
                        : step_t<float>(a, state, x, dt, A, B, C, D, z, dt_bias, y, st);
}

}  // namespace m2
