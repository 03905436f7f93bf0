// conv.cu -- short causal depthwise convolution over tokens (include/mamba2_layer.h).
//
//   s[t] = bias + sum_k w[k] x[t - (W - 1) + k]      y = s or s sigmoid(s)
//
// Bytes bound: forward x in, y out; backward x, dy in, dx out.  A thread owns V
// neighbouring channels and walks a stretch of tokens with the last W - 1 inputs in
// registers, so each input is read once plus W - 1 tokens of overlap per stretch;
// neighbouring threads read neighbouring bytes of one token's row.  The tokens arrive
// through a ring of asynchronous copies in shared memory, which keeps enough bytes in
// flight without registers (forward 139 -> 117 us, backward 272 -> 195 us when it came).
//
// b8 T4096 C5376 W4 bf16, x a column slice: forward 114 us (6.2 TB/s, 0.91 of the
// measured copy rate), backward 185 us (5.7 TB/s, 0.84; 196 us with registers for four
// blocks an SM instead of three: the fp32 pipe at half, the issue slots at 0.55).  The
// forward with eight channels a thread 160 us, with blocks of 128 threads instead of
// 64 132 us (whole waves).  A step of 64 tokens takes 2.2 us on the GPU, the launch.
#include <algorithm>

#include "internal.h"
#include "layer.cuh"

namespace m2 {
namespace {

template <typename TI, int V>
__device__ __forceinline__ void load_2(const TI* p, f2 (&o)[(V + 1) / 2]) {
    to_pairs<TI, V>(load_raw<TI, V>(p), o);
}
template <int V, int W>
__device__ __forceinline__ void load_w(const float* w, const float* bias, int64_t c,
                                       f2 (&wk)[W][(V + 1) / 2], f2 (&bi)[(V + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
        const int64_t lo = c + 2 * i, hi = V == 1 ? lo : lo + 1;
        if (W == 4 && V > 1) {   // one 16-byte access a channel (the launcher checked w's alignment)
            const float4 a = __ldg(reinterpret_cast<const float4*>(w) + lo);
            const float4 b = __ldg(reinterpret_cast<const float4*>(w) + hi);
            wk[0][i] = pack2(a.x, b.x);
            wk[1][i] = pack2(a.y, b.y);
            wk[2][i] = pack2(a.z, b.z);
            wk[W - 1][i] = pack2(a.w, b.w);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) wk[k][i] = pack2(__ldg(w + lo * W + k), __ldg(w + hi * W + k));
        }
        bi[i] = bias ? pack2(__ldg(bias + lo), __ldg(bias + hi)) : dup2(0.f);
    }
}

constexpr int kFwdThreads = 64;
// Groups of four tokens in a thread's ring (four: 117 / 195 us forward / backward, six
// 117 / 202, eight 154 / 214); none where an element is too small for an asynchronous
// copy (single bf16 values).
template <typename TI, int V> constexpr int ring() {
    return V * sizeof(TI) < 4 ? 0 : V * sizeof(TI) > 8 ? 3 : 4;
}

// Block: one stretch of TS tokens of one sequence, kFwdThreads * V channels.
template <typename TI, int V, int W, bool SILU>
__global__ void __launch_bounds__(kFwdThreads)
conv_fwd_kernel(const TI* __restrict__ x, const float* __restrict__ w,
                const float* __restrict__ bias, const TI* __restrict__ init,
                const int32_t* __restrict__ lengths, TI* __restrict__ y, TI* __restrict__ fin,
                int T, int D, int TS, int nseg, int ncb, Tok sx, Tok sy) {
    const int cb = blockIdx.x % ncb, bs = blockIdx.x / ncb;
    const int seg = bs % nseg, b = bs / nseg;
    const int c = (cb * kFwdThreads + threadIdx.x) * V;
    if (c >= D) return;
    const int n = lengths ? min(max(__ldg(lengths + b), 0), T) : T;
    const TI* xb = x + (int64_t)b * sx.b + c;
    TI* yb = y + (int64_t)b * sy.b + c;
    const TI* ib = init ? init + ((int64_t)b * (W - 1)) * D + c : nullptr;
    typedef typename Pack<TI, V>::Raw Raw;
    if (seg == 0 && fin) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = n - (W - 1) + k;
            Raw r = zero_raw<Raw>();
            if (t >= 0) r = load_raw<TI, V>(xb + (int64_t)t * sx.t);
            else if (ib) r = load_raw<TI, V>(ib + (int64_t)(t + W - 1) * D);
            store_raw<TI, V>(fin + ((int64_t)b * (W - 1) + k) * D + c, r);
        }
    }
    constexpr int H = (V + 1) / 2;
    f2 wk[W][H], bi[H], win[W - 1][H];
    load_w<V, W>(w, bias, c, wk, bi);
    const int t0 = seg * TS, t1 = min(t0 + TS, T), tn = min(t1, n);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = t0 - (W - 1) + k;
#pragma unroll
        for (int i = 0; i < H; ++i) win[k][i] = dup2(0.f);
        if (t >= 0) {
            if (t < n) load_2<TI, V>(xb + (int64_t)t * sx.t, win[k]);
        } else if (ib) {
            load_2<TI, V>(ib + (int64_t)(t + W - 1) * D, win[k]);
        }
    }
    auto one = [&](Raw r, int t) {
        f2 cur[H], o[H];
        to_pairs<TI, V>(r, cur);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            f2 s = fma2(wk[W - 1][i], cur[i], bi[i]);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) s = fma2(wk[k][i], win[k][i], s);
            o[i] = SILU ? mul2(s, sigmoid2(s)) : s;
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
            win[W - 2][i] = cur[i];
        }
        store_raw<TI, V>(yb + (int64_t)t * sy.t, from_pairs<TI, V>(o));
    };
    // Whole groups of U tokens pass through a ring in shared memory, in which each thread
    // reads only what it copied: kRing - 1 groups in flight, without registers.
    constexpr int NB = ring<TI, V>(), U = NB ? 4 : 8;
    int t = t0;
    if constexpr (NB > 0) {
        extern __shared__ __align__(16) unsigned char smem[];
        Raw* mine = reinterpret_cast<Raw*>(smem) + threadIdx.x;
        const int groups = max(tn - t0, 0) / U;
        const TI* src = xb + (int64_t)t0 * sx.t;
        auto copy = [&](int g) {
            if (g < groups) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    stage_copy<V * (int)sizeof(TI)>(mine + ((g % NB) * U + u) * kFwdThreads, src, true);
                    src += sx.t;
                }
            }
            stage_commit();
        };
#pragma unroll
        for (int g = 0; g < NB - 1; ++g) copy(g);
        for (int g = 0; g < groups; ++g, t += U) {
            stage_wait<NB - 2>();
            Raw r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = mine[((g % NB) * U + u) * kFwdThreads];
            copy(g + NB - 1);   // into the group read in the round before
#pragma unroll
            for (int u = 0; u < U; ++u) one(r[u], t + u);
        }
    } else {
        for (; t + U <= tn; t += U) {
            Raw r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = load_raw<TI, V>(xb + (int64_t)(t + u) * sx.t);
#pragma unroll
            for (int u = 0; u < U; ++u) one(r[u], t + u);
        }
    }
    for (; t < tn; ++t) one(load_raw<TI, V>(xb + (int64_t)t * sx.t), t);
    for (t = max(tn, t0); t < t1; ++t) store_raw<TI, V>(yb + (int64_t)t * sy.t, zero_raw<Raw>());
}

// One token: the window is read, applied and moved on.
template <typename TI, int V, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_step_kernel(TI* __restrict__ state, const TI* __restrict__ x, const float* __restrict__ w,
                 const float* __restrict__ bias, TI* __restrict__ y, int D, int ncb, int64_t sxb,
                 int64_t syb) {
    const int cb = blockIdx.x % ncb, b = blockIdx.x / ncb;
    const int c = (cb * 128 + threadIdx.x) * V;
    if (c >= D) return;
    typedef typename Pack<TI, V>::Raw Raw;
    TI* sb = state + (int64_t)b * (W - 1) * D + c;
    Raw r[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) r[k] = *reinterpret_cast<const Raw*>(sb + (int64_t)k * D);
    r[W - 1] = load_raw<TI, V>(x + (int64_t)b * sxb + c);
    constexpr int H = (V + 1) / 2;
    f2 wk[W][H], o[H];
    load_w<V, W>(w, bias, c, wk, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        f2 v[H];
        to_pairs<TI, V>(r[k], v);
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = fma2(wk[k][i], v[i], o[i]);
    }
    if (SILU) {
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = mul2(o[i], sigmoid2(o[i]));
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<TI, V>(sb + (int64_t)k * D, r[k + 1]);
    store_raw<TI, V>(y + (int64_t)b * syb + c, from_pairs<TI, V>(o));
}

// Backward.  ds = dy silu'(s) with s recomputed;  dx[t] = sum_k w[k] ds[t + W-1 - k];
// dw[k] = sum_t ds[t] x[t - (W-1) + k];  dbias = sum_t ds[t].
// A thread walks its stretch and W - 1 tokens past it (whose ds its last dx need)
// with windows of x and ds in registers; at t it finishes dx[t - (W - 1)], which
// for the first stretch includes the gradients of the initial window.  The kBwdTY
// stretches of a block are summed in shared memory into one slot of dw and dbias.
constexpr int kBwdTX = 32, kBwdTY = 4;

template <typename TI, int V, int W, bool SILU>
__global__ void __launch_bounds__(kBwdTX * kBwdTY, 3)
conv_bwd_kernel(const TI* __restrict__ x, const float* __restrict__ w,
                const float* __restrict__ bias, const TI* __restrict__ init,
                const TI* __restrict__ dy, const TI* __restrict__ dfin,
                const int32_t* __restrict__ lengths, TI* __restrict__ dx, TI* __restrict__ dinit,
                float* __restrict__ part, int T, int D, int TS, int nblk, int ncb, Tok sx, Tok sdy) {
    typedef typename Pack<TI, V>::Raw Raw;
    // the ring, and after it in the same place the sums
    extern __shared__ __align__(16) unsigned char smem[];
    Raw* mine = reinterpret_cast<Raw*>(smem) + threadIdx.y * kBwdTX + threadIdx.x;
    constexpr int RW = kBwdTX * V * (W + 1);
    float* red = reinterpret_cast<float*>(smem);   // [kBwdTY][RW]
    const int cb = blockIdx.x % ncb, slot = blockIdx.x / ncb;
    const int tb = slot % nblk, b = slot / nblk;
    const int c = (cb * kBwdTX + threadIdx.x) * V;
    const int seg = tb * kBwdTY + threadIdx.y;
    const bool first = seg == 0;
    const int t0 = min(seg * TS, T), t1 = min(t0 + TS, T);
    constexpr int H = (V + 1) / 2;
    f2 dwk[W][H], dbi[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) dwk[k][i] = dup2(0.f);
        dbi[i] = dup2(0.f);
    }
    if (c < D && (t0 < t1 || first)) {
        const int n = lengths ? min(max(__ldg(lengths + b), 0), T) : T;
        const TI* xb = x + (int64_t)b * sx.b + c;
        const TI* db = dy + (int64_t)b * sdy.b + c;
        TI* ob = dx + (int64_t)b * T * D + c;
        const int64_t wrow = (int64_t)b * (W - 1) * D + c;
        f2 wk[W][H], bi[H], xw[W][H], dsw[W][H];   // xw[W-1], dsw[W-1]: the current token
        load_w<V, W>(w, bias, c, wk, bi);
#pragma unroll
        for (int k = 0; k < W; ++k) {
#pragma unroll
            for (int i = 0; i < H; ++i) dsw[k][i] = xw[k][i] = dup2(0.f);
            const int t = t0 - W + k;   // shifted once before use
            if (k > 0) {
                if (t >= 0) {
                    if (t < n) load_2<TI, V>(xb + (int64_t)t * sx.t, xw[k]);
                } else if (init) {
                    load_2<TI, V>(init + wrow + (int64_t)(t + W - 1) * D, xw[k]);
                }
            }
        }
        // Token t: its ds, its part of dw, and the finished dx[t - (W-1)] in o.  ANY: t may
        // be padding or past the stretch.
        auto one = [&](const bool ANY, Raw rx, Raw rd, int t, f2 (&o)[H]) {
            f2 cx[H], ds[H];
            to_pairs<TI, V>(rx, cx);
            to_pairs<TI, V>(rd, ds);
#pragma unroll
            for (int i = 0; i < H; ++i) {
#pragma unroll
                for (int k = 0; k + 1 < W; ++k) {
                    xw[k][i] = xw[k + 1][i];
                    dsw[k][i] = dsw[k + 1][i];
                }
                xw[W - 1][i] = cx[i];
                if (SILU) {
                    f2 s = bi[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) s = fma2(wk[k][i], xw[k][i], s);
                    const f2 sg = sigmoid2(s);   // silu' = sg (1 + s (1 - sg))
                    ds[i] = mul2(ds[i], mul2(sg, fma2(s, fma2(sg, dup2(-1.f), dup2(1.f)), dup2(1.f))));
                }
                f2 own = ds[i];
                if (ANY) {
                    if (t >= n) ds[i] = own = dup2(0.f);
                    if (t >= t1) own = dup2(0.f);
                }
                dsw[W - 1][i] = ds[i];
#pragma unroll
                for (int k = 0; k < W; ++k) dwk[k][i] = fma2(own, xw[k][i], dwk[k][i]);
                dbi[i] = add2(dbi[i], own);
                f2 a = mul2(wk[W - 1][i], dsw[0][i]);
#pragma unroll
                for (int k = 0; k + 1 < W; ++k) a = fma2(wk[k][i], dsw[W - 1 - k][i], a);
                o[i] = a;
            }
        };
        // Up to W - 1 tokens from t, before te, that may be anything; their loads together.
        const int te = t1 + W - 1, tf = min(t1, n);
        auto slow = [&](int t, int end) {
            Raw rx[W - 1], rd[W - 1];
#pragma unroll
            for (int u = 0; u < W - 1; ++u) {
                rx[u] = rd[u] = zero_raw<Raw>();
                if (t + u < min(end, n)) {
                    rx[u] = load_raw<TI, V>(xb + (int64_t)(t + u) * sx.t);
                    rd[u] = load_raw<TI, V>(db + (int64_t)(t + u) * sdy.t);
                }
            }
#pragma unroll
            for (int u = 0; u < W - 1; ++u) {
                if (t + u >= end) break;
                f2 o[H];
                one(true, rx[u], rd[u], t + u, o);
                const int tp = t + u - (W - 1);
                if (tp < t0 && !first) continue;
                if (dfin && tp < n && tp >= n - (W - 1)) {
                    f2 f[H];
                    load_2<TI, V>(dfin + wrow + (int64_t)(tp - (n - (W - 1))) * D, f);
#pragma unroll
                    for (int i = 0; i < H; ++i) o[i] = add2(o[i], f[i]);
                }
                if (tp >= 0) store_raw<TI, V>(ob + (int64_t)tp * D, from_pairs<TI, V>(o));
                else if (dinit)
                    store_raw<TI, V>(dinit + wrow + (int64_t)(tp + W - 1) * D, from_pairs<TI, V>(o));
            }
        };
        constexpr int NB = ring<TI, V>(), U = NB ? 4 : 8;
        int t = min(t0 + W - 1, te);
        slow(t0, t);
        // Whole groups of U real tokens of this stretch (dfinal only reaches tokens finished
        // at or after n), through a ring as in the forward.
        if constexpr (NB > 0) {
            const int groups = max(tf - t, 0) / U;
            const TI* srcx = xb + (int64_t)t * sx.t;
            const TI* srcd = db + (int64_t)t * sdy.t;
            TI* dst = ob + (int64_t)(t - (W - 1)) * D;
            auto copy = [&](int g) {
                if (g < groups) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        Raw* at = mine + ((g % NB) * U + u) * (2 * kBwdTX * kBwdTY);
                        stage_copy<V * (int)sizeof(TI)>(at, srcx, true);
                        stage_copy<V * (int)sizeof(TI)>(at + kBwdTX * kBwdTY, srcd, true);
                        srcx += sx.t;
                        srcd += sdy.t;
                    }
                }
                stage_commit();
            };
#pragma unroll
            for (int g = 0; g < NB - 1; ++g) copy(g);
            for (int g = 0; g < groups; ++g, t += U) {
                stage_wait<NB - 2>();
                copy(g + NB - 1);   // into the group read in the round before
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Raw* at = mine + ((g % NB) * U + u) * (2 * kBwdTX * kBwdTY);
                    f2 o[H];
                    one(false, at[0], at[kBwdTX * kBwdTY], t + u, o);
                    store_raw<TI, V>(dst, from_pairs<TI, V>(o));
                    dst += D;
                }
            }
        } else {
            for (; t + U <= tf; t += U) {
                Raw rx[U], rd[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rx[u] = load_raw<TI, V>(xb + (int64_t)(t + u) * sx.t);
                    rd[u] = load_raw<TI, V>(db + (int64_t)(t + u) * sdy.t);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    f2 o[H];
                    one(false, rx[u], rd[u], t + u, o);
                    store_raw<TI, V>(ob + (int64_t)(t + u - (W - 1)) * D, from_pairs<TI, V>(o));
                }
            }
        }
        for (; t < te; t += W - 1) slow(t, te);
    }
    __syncthreads();   // every thread is through with its ring
    float* mr = red + threadIdx.y * RW + threadIdx.x;
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            float lo, hi;
            unpack2(k < W ? dwk[k < W ? k : 0][i] : dbi[i], lo, hi);
            mr[(2 * i * (W + 1) + k) * kBwdTX] = lo;
            if (V > 1) mr[((2 * i + 1) * (W + 1) + k) * kBwdTX] = hi;
        }
    __syncthreads();
    const int tid = threadIdx.y * kBwdTX + threadIdx.x;
    for (int i = tid; i < RW; i += kBwdTX * kBwdTY) {
        const int cx = i % kBwdTX, jk = i / kBwdTX, j = jk / (W + 1), k = jk % (W + 1);
        const int64_t ch = (int64_t)(cb * kBwdTX + cx) * V + j;
        if (ch >= D) continue;
        float a = 0.f;
#pragma unroll
        for (int q = 0; q < kBwdTY; ++q) a += red[q * RW + i];
        float* row = part + (int64_t)slot * D * (W + 1);
        if (k < W) row[ch * W + k] = a;
        else row[(int64_t)D * W + ch] = a;
    }
}

// Stretch lengths: long ones amortise the start (weights, the tokens of overlap and,
// backward, the slots of dw); short ones fill the GPU when there are few rows, and spread
// the blocks evenly over it.  Picks the best share of time spent on whole tokens: `lanes`
// threads a token row, `start` tokens' worth of start, `resident` threads an SM.
int pick_ts(int64_t lanes, int64_t T, int start, int resident) {
    const double room = (double)sm_count() * resident;
    int best = 8;
    double top = 0.;
    for (int ts = 8; ts <= 256; ts *= 2) {
        const double waves = (double)lanes * (double)((T + ts - 1) / ts) / room;
        const double used = waves < 1. ? waves : waves / (double)(int64_t)(waves + 0.999);
        const double share = used * ts / (ts + start);
        if (share > top * 1.01) {
            top = share;
            best = ts;
        }
    }
    return best;
}

int bwd_vec(const ConvArgs& a) { return a.D % 4 == 0 ? 4 : a.dtype == 1 && a.D % 2 == 0 ? 2 : 1; }
int bwd_ts(const ConvArgs& a) {
    const int64_t lanes = (a.D + bwd_vec(a) - 1) / bwd_vec(a);
    return pick_ts(a.b * lanes, a.T, 40, 384);
}
int64_t bwd_blocks(const ConvArgs& a) {
    const int64_t per = (int64_t)bwd_ts(a) * kBwdTY;
    return std::max<int64_t>(1, (a.T + per - 1) / per);
}

template <typename TI, int V, int W>
cudaError_t fwd_w(const ConvArgs& a, const TI* x, const float* w, const float* bias, const TI* init,
                  const int32_t* lengths, TI* y, TI* fin, cudaStream_t st) {
    const int64_t lanes = (a.D + V - 1) / V, ncb = (lanes + kFwdThreads - 1) / kFwdThreads;
    const int ts = pick_ts(a.b * lanes, a.T, 6, 768);
    const int64_t nseg = std::max<int64_t>(1, (a.T + ts - 1) / ts);
    if (a.b * nseg * ncb >= (int64_t(1) << 31)) return kGridLimit;
    auto k = a.silu ? conv_fwd_kernel<TI, V, W, true> : conv_fwd_kernel<TI, V, W, false>;
    constexpr size_t smem = (size_t)ring<TI, V>() * 4 * kFwdThreads * V * sizeof(TI);
    static_assert(smem <= 48 * 1024, "the default limit");
    k<<<(unsigned)(a.b * nseg * ncb), kFwdThreads, smem, st>>>(
        x, w, bias, init, lengths, y, fin, (int)a.T, (int)a.D, ts, (int)nseg, (int)ncb, a.sx, a.sy);
    return cudaGetLastError();
}

template <typename TI, int V, int W>
cudaError_t step_w(const ConvArgs& a, TI* state, const TI* x, const float* w, const float* bias, TI* y,
                   cudaStream_t st) {
    const int64_t ncb = ((a.D + V - 1) / V + 127) / 128;
    if (a.b * ncb >= (int64_t(1) << 31)) return kGridLimit;
    auto k = a.silu ? conv_step_kernel<TI, V, W, true> : conv_step_kernel<TI, V, W, false>;
    k<<<(unsigned)(a.b * ncb), 128, 0, st>>>(state, x, w, bias, y, (int)a.D, (int)ncb, a.sx.b, a.sy.b);
    return cudaGetLastError();
}

template <typename TI, int V, int W>
cudaError_t bwd_w(const ConvArgs& a, const TI* x, const float* w, const float* bias, const TI* init,
                  const TI* dy, const TI* dfin, const int32_t* lengths, TI* dx, TI* dinit, float* part,
                  cudaStream_t st) {
    const int64_t ncb = ((a.D + V - 1) / V + kBwdTX - 1) / kBwdTX, nblk = bwd_blocks(a);
    if (a.b * nblk * ncb >= (int64_t(1) << 31)) return kGridLimit;
    auto k = a.silu ? conv_bwd_kernel<TI, V, W, true> : conv_bwd_kernel<TI, V, W, false>;
    constexpr size_t rings = (size_t)ring<TI, V>() * 4 * 2 * kBwdTX * kBwdTY * V * sizeof(TI);
    constexpr size_t sums = (size_t)kBwdTY * kBwdTX * V * (W + 1) * sizeof(float), smem = rings > sums ? rings : sums;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)(a.b * nblk * ncb), dim3(kBwdTX, kBwdTY), smem, st>>>(
        x, w, bias, init, dy, dfin, lengths, dx, dinit, part, (int)a.T, (int)a.D, bwd_ts(a), (int)nblk,
        (int)ncb, a.sx, a.sy);
    return cudaGetLastError();
}

template <typename TI, int V>
cudaError_t fwd_v(const ConvArgs& a, const void* x, const float* w, const float* bias, const void* init,
                  const int32_t* lengths, void* y, void* fin, cudaStream_t st) {
    auto go = [&](auto f) {
        return f(a, static_cast<const TI*>(x), w, bias, static_cast<const TI*>(init), lengths,
                 static_cast<TI*>(y), static_cast<TI*>(fin), st);
    };
    return a.W == 2 ? go(fwd_w<TI, V, 2>) : a.W == 3 ? go(fwd_w<TI, V, 3>) : go(fwd_w<TI, V, 4>);
}
template <typename TI, int V>
cudaError_t step_v(const ConvArgs& a, void* state, const void* x, const float* w, const float* bias,
                   void* y, cudaStream_t st) {
    auto go = [&](auto f) {
        return f(a, static_cast<TI*>(state), static_cast<const TI*>(x), w, bias, static_cast<TI*>(y), st);
    };
    return a.W == 2 ? go(step_w<TI, V, 2>) : a.W == 3 ? go(step_w<TI, V, 3>) : go(step_w<TI, V, 4>);
}
template <typename TI, int V>
cudaError_t bwd_v(const ConvArgs& a, const void* x, const float* w, const float* bias, const void* init,
                  const void* dy, const void* dfin, const int32_t* lengths, void* dx, void* dinit,
                  float* part, cudaStream_t st) {
    auto go = [&](auto f) {
        return f(a, static_cast<const TI*>(x), w, bias, static_cast<const TI*>(init),
                 static_cast<const TI*>(dy), static_cast<const TI*>(dfin), lengths, static_cast<TI*>(dx),
                 static_cast<TI*>(dinit), part, st);
    };
    return a.W == 2 ? go(bwd_w<TI, V, 2>) : a.W == 3 ? go(bwd_w<TI, V, 3>) : go(bwd_w<TI, V, 4>);
}

// Every access of the call is whole and aligned at V elements a piece.
bool wide(const ConvArgs& a, int64_t V, const float* w, const void* x, const void* y, const void* s0,
          const void* s1, const void* o) {
    const int64_t es = a.dtype == 1 ? 2 : 4, bytes = V * es;
    const Tok row{0, a.D};
    return a.D % V == 0 && (a.W != 4 || reinterpret_cast<uintptr_t>(w) % 16 == 0) && vec_ok(x, a.sx, bytes, es) && vec_ok(y, a.sy, bytes, es) &&
           vec_ok(s0, row, bytes, es) && vec_ok(s1, row, bytes, es) && vec_ok(o, row, bytes, es);
}

// Sum of one column of part over the slots: TX columns x 1024 / TX rows of slots a block.
template <int TX>
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float* __restrict__ part, int64_t slots, int64_t cols, float* __restrict__ out1,
                  int64_t n1, float* __restrict__ out2) {
    constexpr int TY = 1024 / TX;
    __shared__ float red[TY][TX + 1];
    const int64_t c = (int64_t)blockIdx.x * TX + threadIdx.x;
    float a = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int64_t s = threadIdx.y; s < slots; s += TY) a += __ldg(part + s * cols + c);
    red[threadIdx.y][threadIdx.x] = a;
    for (int q = TY / 2; q > 0; q /= 2) {
        __syncthreads();
        if (threadIdx.y < q) red[threadIdx.y][threadIdx.x] += red[threadIdx.y + q][threadIdx.x];
    }
    if (threadIdx.y == 0 && c < cols) {
        a = red[0][threadIdx.x];
        if (c < n1) {
            if (out1) out1[c] = a;
        } else if (out2) {
            out2[c - n1] = a;
        }
    }
}

}  // namespace

cudaError_t launch_column_sum(const float* part, int64_t slots, int64_t cols, float* out1, int64_t n1,
                              float* out2, cudaStream_t st) {
    if (cols == 0) return cudaSuccess;
    if ((cols + 7) / 8 >= (int64_t(1) << 31)) return kGridLimit;
    // few columns and many slots (a narrow layer): more rows of slots a block, so that a
    // thread's chain of loads stays short
    if (cols < (int64_t)sm_count() * 64 && slots > 64)
        column_sum_kernel<8><<<(unsigned)((cols + 7) / 8), dim3(8, 128), 0, st>>>(part, slots, cols, out1, n1, out2);
    else
        column_sum_kernel<32><<<(unsigned)((cols + 31) / 32), dim3(32, 32), 0, st>>>(part, slots, cols, out1, n1, out2);
    return cudaGetLastError();
}

cudaError_t launch_conv_fwd(const ConvArgs& a, const void* x, const float* w, const float* bias,
                            const void* init, const int32_t* lengths, void* y, void* fin,
                            cudaStream_t st) {
    if (a.b == 0 || a.D == 0) return cudaSuccess;
    if (a.dtype == 1)
        return wide(a, 4, w, x, y, init, fin, nullptr)
                   ? fwd_v<__nv_bfloat16, 4>(a, x, w, bias, init, lengths, y, fin, st)
               : wide(a, 2, w, x, y, init, fin, nullptr)
                   ? fwd_v<__nv_bfloat16, 2>(a, x, w, bias, init, lengths, y, fin, st)
                   : fwd_v<__nv_bfloat16, 1>(a, x, w, bias, init, lengths, y, fin, st);
    return wide(a, 4, w, x, y, init, fin, nullptr)
               ? fwd_v<float, 4>(a, x, w, bias, init, lengths, y, fin, st)
               : fwd_v<float, 1>(a, x, w, bias, init, lengths, y, fin, st);
}

cudaError_t launch_conv_step(const ConvArgs& a, void* state, const void* x, const float* w,
                             const float* bias, void* y, cudaStream_t st) {
    if (a.b == 0 || a.D == 0) return cudaSuccess;
    if (a.dtype == 1)
        return wide(a, 2, w, x, y, state, nullptr, nullptr)
                   ? step_v<__nv_bfloat16, 2>(a, state, x, w, bias, y, st)
                   : step_v<__nv_bfloat16, 1>(a, state, x, w, bias, y, st);
    return step_v<float, 1>(a, state, x, w, bias, y, st);
}

int64_t conv_bwd_slots(const ConvArgs& a) { return a.b * bwd_blocks(a); }

cudaError_t launch_conv_bwd(const ConvArgs& a, const void* x, const float* w, const float* bias,
                            const void* init, const void* dy, const void* dfin, const int32_t* lengths,
                            void* dx, float* dw, float* dbias, void* dinit, float* part,
                            cudaStream_t st) {
    if (a.D == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (a.b > 0) {
        // dfin and dinit are rows of D like the initial window
        auto fits = [&](int64_t V) {
            return wide(a, V, w, x, dy, init, dfin, dinit) && wide(a, V, w, x, dy, dx, nullptr, nullptr);
        };
        const bool v4 = fits(4);
        if (a.dtype == 1)
            e = v4 ? bwd_v<__nv_bfloat16, 4>(a, x, w, bias, init, dy, dfin, lengths, dx, dinit, part, st)
                : fits(2)
                   ? bwd_v<__nv_bfloat16, 2>(a, x, w, bias, init, dy, dfin, lengths, dx, dinit, part, st)
                   : bwd_v<__nv_bfloat16, 1>(a, x, w, bias, init, dy, dfin, lengths, dx, dinit, part, st);
        else
            e = v4 ? bwd_v<float, 4>(a, x, w, bias, init, dy, dfin, lengths, dx, dinit, part, st)
                   : bwd_v<float, 1>(a, x, w, bias, init, dy, dfin, lengths, dx, dinit, part, st);
    }
    if (e != cudaSuccess) return e;
    return launch_column_sum(part, a.b ? conv_bwd_slots(a) : 0, a.D * (a.W + 1), dw, a.D * a.W, dbias, st);
}

}  // namespace m2
