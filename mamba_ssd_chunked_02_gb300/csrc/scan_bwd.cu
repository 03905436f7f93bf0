// scan_bwd.cu -- the selective scan's gradients: the cut of the token axis, the workspace,
// the small kernels between and after the ones of scan_bwd.cuh, and the call.
#include "scan_bwd.cuh"

namespace m2 {
namespace {
using namespace scan_bwd;

// (2) One thread per (b, c, n): seg_h becomes the state entering each stretch, seg_g
// the adjoint of the state leaving it.
__global__ void __launch_bounds__(256)
scan_join2_kernel(float* __restrict__ seg_h, float* __restrict__ seg_g, const float* __restrict__ seg_d,
                  const float* __restrict__ A, const float* __restrict__ init,
                  const float* __restrict__ dfinal, int64_t total, int64_t DN, int N, int nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const float a = __ldg(A + i % DN) * kLog2e;
    const int64_t bd = i / N, nbd = total / N;
    float h = init ? init[i] : 0.f, g = dfinal ? dfinal[i] : 0.f;
    for (int s0 = 0; s0 < nseg; s0 += 4) {   // four stretches' loads in flight
        float hl[4], gl[4], hd[4], gd[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s0 + k < nseg) {
                const int s = s0 + k, r = nseg - 1 - s;
                hl[k] = seg_h[s * total + i], gl[k] = seg_g[r * total + i];
                hd[k] = seg_d[s * nbd + bd], gd[k] = seg_d[r * nbd + bd];
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s0 + k < nseg) {
                const int s = s0 + k, r = nseg - 1 - s;
                seg_h[s * total + i] = h;
                seg_g[r * total + i] = g;
                h = fmaf(ex2(a * hd[k]), h, hl[k]);
                g = fmaf(ex2(a * gd[k]), g, gl[k]);
            }
    }
}

// dB, dC [b,T,G,N] in the I/O type: the sum over the channel blocks of a group.
template <typename TI>
__global__ void __launch_bounds__(256)
scan_bc_sum_kernel(const float* __restrict__ part, int ncb, int64_t rows, int N, TI* __restrict__ dB,
                   TI* __restrict__ dC) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = rows * 2 * N;
    if (i >= total) return;
    float a = 0.f;
    for (int s = 0; s < ncb; ++s) a += __ldg(part + s * total + i);
    const int64_t row = i / (2 * N);
    const int e = (int)(i - row * 2 * N);
    if (e < N) dB[row * N + e] = from_f32<TI>(a);
    else dC[row * N + e - N] = from_f32<TI>(a);
}

struct Plan {
    int KK;
    int64_t SL, nseg, nck, ncb;
    size_t ck, ck_d, seg, seg_d, bc, A, v, total;
};

// Stretches: as many as keep the gradient kernel's blocks (two an SM; one in fp32 at N = 8 with
// four channels in turn, for 129,536 bytes of shared memory) busiest, whole waves
// of them against the start of each; none shorter than two tiles of the first
// pass, and no more than 64 for the join.
Plan plan_of(const ScanArgs& a) {
    Plan p;
    const int64_t Dg = a.D / a.G, lpc = a.N / kNS;
    const int64_t tt = 32;   // a multiple of the first pass's tile and of kL
    const int64_t held = (int64_t)sm_count() * 2;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(64, a.T / tt));
    auto blocks = [&](int KK) { return (Dg + kGT / lpc * KK - 1) / (kGT / lpc * KK); };
    // Four channels in turn where that still fills the GPU.  b4 T2048, KK = 4 against 1: C2048 bf16 N16
    // 482 / 521 us, N32 867 / 1010, N64 1487 / 2339, N128 3359 / 5717, fp32 much the same.  Not everywhere: N8
    // 373 / 320 (fp32 415 / 325; its blocks hold 256 channels), C2047 N16 920 / 810 (N8 621 / 674, N32 1084 / 1397).
    // KK = 1 for small problems: b3 T1956 C320 in groups of 80, N8, fp32: 166 us with four in turn, 99 with one.
    p.KK = a.b * a.G * blocks(4) * most >= held && 2 * Dg > kGT / lpc * 4 ? 4 : 1;
    p.ncb = blocks(p.KK);
    const int64_t per = std::max<int64_t>(1, a.b * a.G * p.ncb);
    double top = 0.;
    p.SL = std::max<int64_t>(tt, (a.T + tt - 1) / tt * tt);
    for (int64_t n = 1; n <= most; ++n) {
        const int64_t SL = ((a.T + n - 1) / n + tt - 1) / tt * tt, segs = (a.T + SL - 1) / SL;
        // waves of blocks, each as long as a stretch and its start (about two tiles)
        const double waves = (double)((per * segs + held - 1) / held);
        const double share = (double)per * (double)a.T / (waves * (double)held * (double)(SL + 16));
        if (share > top * 1.01) {
            top = share;
            p.SL = SL;
        }
    }
    p.nseg = std::max<int64_t>(1, (a.T + p.SL - 1) / p.SL);
    p.nck = (a.T + kL - 1) / kL;
    auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
    const size_t f = sizeof(float);
    size_t o = 0;
    auto take = [&](size_t& at, size_t bytes) { at = o; o += al(bytes); };
    take(p.ck, f * (size_t)(a.b * p.nck * a.D * a.N));
    take(p.ck_d, f * (size_t)(a.b * p.nck * a.D));
    take(p.seg, p.nseg > 1 ? 2 * f * (size_t)(p.nseg * a.b * a.D * a.N) : 0);
    take(p.seg_d, p.nseg > 1 ? f * (size_t)(p.nseg * a.b * a.D) : 0);
    take(p.bc, f * (size_t)(p.ncb * a.b * a.T * a.G * 2 * a.N));
    take(p.A, f * (size_t)(p.nseg * a.b * a.D * a.N));
    take(p.v, f * (size_t)(p.nseg * a.b * 2 * a.D));
    p.total = o;
    return p;
}

}  // namespace

cudaError_t scan_bwd::join(const BwdP& p, int N, const float* init, const float* dfinal, cudaStream_t st) {
    const int64_t total = p.b * p.Dch * N;
    scan_join2_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
        p.seg_h, p.seg_g, p.seg_d, p.A, init, dfinal, total, (int64_t)p.Dch * N, N, p.nseg);
    return cudaGetLastError();
}

size_t scan_bwd_workspace(const ScanArgs& a) { return a.b * a.T * a.D ? plan_of(a).total : 0; }

cudaError_t launch_scan_bwd(const ScanArgs& a, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* D, const void* z, const float* dt_bias,
                            const float* init, const void* dy, const float* dfinal, const int32_t* lengths,
                            const ScanGrads& g, void* ws, cudaStream_t st) {
    if (a.D == 0) return cudaSuccess;
    const size_t f = sizeof(float), states = f * (size_t)(a.b * a.D * a.N);
    if (a.b * a.T == 0) {   // nothing was computed from the parameters; the state passes through
        cudaError_t e = cudaMemsetAsync(g.dA, 0, f * (size_t)(a.D * a.N), st);
        if (e == cudaSuccess && g.dD) e = cudaMemsetAsync(g.dD, 0, f * (size_t)a.D, st);
        if (e == cudaSuccess && g.ddt_bias) e = cudaMemsetAsync(g.ddt_bias, 0, f * (size_t)a.D, st);
        if (e == cudaSuccess && g.dinit && states)
            e = dfinal ? cudaMemcpyAsync(g.dinit, dfinal, states, cudaMemcpyDeviceToDevice, st)
                       : cudaMemsetAsync(g.dinit, 0, states, st);
        return e;
    }
    const int64_t rows = a.b * a.T * a.G, blocks = (rows * 2 * a.N + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return kGridLimit;   // before the first launch
    const Plan pl = plan_of(a);
    char* w = static_cast<char*>(ws);
    BwdP p = {};
    p.x = x, p.dt = dt, p.B = B, p.C = C, p.z = z, p.dy = dy, p.A = A, p.D = D, p.bias = dt_bias;
    p.lengths = lengths;
    p.ck = reinterpret_cast<float*>(w + pl.ck), p.ck_d = reinterpret_cast<float*>(w + pl.ck_d);
    p.seg_h = reinterpret_cast<float*>(w + pl.seg);
    p.seg_g = p.seg_h + pl.nseg * a.b * a.D * a.N;
    p.seg_d = reinterpret_cast<float*>(w + pl.seg_d);
    p.dx = g.dx, p.ddt = g.ddt, p.dz = g.dz, p.dinit = g.dinit;
    p.part_bc = reinterpret_cast<float*>(w + pl.bc), p.part_A = reinterpret_cast<float*>(w + pl.A);
    p.part_v = reinterpret_cast<float*>(w + pl.v);
    p.T = (int)a.T, p.Dch = (int)a.D, p.G = (int)a.G, p.Dg = (int)(a.D / a.G), p.ncb = (int)pl.ncb;
    p.nseg = (int)pl.nseg, p.SL = (int)pl.SL, p.nck = (int)pl.nck, p.softplus = a.softplus, p.b = a.b;
    p.sx = a.sx, p.sdt = a.sdt, p.sB = a.sB, p.sC = a.sC, p.sz = a.sz, p.sy = a.sy;
    cudaError_t e = a.dtype == 1 ? scan_bwd_bf16(a, p, pl.KK, init, dfinal, st) : scan_bwd_f32(a, p, pl.KK, init, dfinal, st);
    if (e != cudaSuccess) return e;
    if (a.dtype == 1)
        scan_bc_sum_kernel<<<(unsigned)blocks, 256, 0, st>>>(p.part_bc, p.ncb, rows, (int)a.N,
                                                            static_cast<__nv_bfloat16*>(g.dB),
                                                            static_cast<__nv_bfloat16*>(g.dC));
    else
        scan_bc_sum_kernel<<<(unsigned)blocks, 256, 0, st>>>(p.part_bc, p.ncb, rows, (int)a.N,
                                                            static_cast<float*>(g.dB), static_cast<float*>(g.dC));
    e = cudaGetLastError();
    const int64_t slots = pl.nseg * a.b;
    if (e == cudaSuccess) e = launch_column_sum(p.part_A, slots, a.D * a.N, g.dA, a.D * a.N, nullptr, st);
    if (e == cudaSuccess && (g.dD || g.ddt_bias))
        e = launch_column_sum(p.part_v, slots, 2 * a.D, g.dD, a.D, g.ddt_bias, st);
    return e;
}

}  // namespace m2
