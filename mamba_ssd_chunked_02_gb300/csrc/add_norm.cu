// add_norm.cu -- RMS norm of a sum with the residual (include/mamba2_proj.h).
//
//   t = x + residual (rounded to the residual's type);  y = t r w,  r = 1 / sqrt(mean(t^2) + eps)
//
// y in the io type or, rounded once from fp32, as e4m3 with a scale for each 128 channels.
// Backward, with g = dy w and n = t r:
//   dt = r (g - n mean(g n)) + dtotal;  dx = dresidual = dt;  dw = sum over tokens of dy n
//
// Bytes bound: every tensor moves once.  b8 T4096 D2560 bf16 with an fp32 residual: forward 145 us,
// in 8 bits 137 us (6.7 TB/s, the measured copy rate), backward 206 us (6.5 TB/s, 0.97), with a bf16
// residual 123 us (0.82: issue slots, twice the values a byte); one token 2.1 us, the launch.
//
// A team (a warp for narrow rows, else a block) holds a forward row in registers between the sum
// and the result; what wide rows do not fit is read again.  A backward team walks over tokens, so
// that its part of dw stays in registers; the parts are summed by a second kernel, in a fixed order.  Rows of more than
// 2048 units (8192 channels, 16384 with a bf16 residual) are read twice, and their part of dw stays in memory: as many
// values in rows of 16384 with an fp32 residual 259 us.
#include <algorithm>
#include <atomic>
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
    bool flat;   // rows lie at even distances in all of the backward's inputs
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sums over the team; `red` is not in use by an earlier call when a block's threads come here.
template <bool WARP> __device__ __forceinline__ float team_sum(float a, float* red) {
    a = warp_sum(a);
    if (WARP) return a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = a;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.f);
}
template <bool WARP> __device__ __forceinline__ float2 team_sum(float a, float b, float2* red) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (WARP) return make_float2(a, b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    if (nw <= 10) {   // few: every thread adds them all, two a load (rows of 1024: 94 us, by shuffles 107)
        const float4* all = reinterpret_cast<const float4*>(red);
        float2 s = nw & 1 ? red[nw - 1] : make_float2(0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < nw / 2; ++i) {
            const float4 v = all[i];
            s.x += v.x + v.z;
            s.y += v.y + v.w;
        }
        return s;
    }
    const float2 v = lane < nw ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

constexpr int kTeams = 8;   // warps a block when a team is a warp

// VPT units a thread; 0: any number, the total read again for the result.
template <typename TI, typename TR, bool VEC, int VPT, bool WARP, bool QUANT>
__global__ void __launch_bounds__(WARP ? kTeams * 32 : 1024)
fwd_kernel(const TI* __restrict__ x, const TR* res, const float* __restrict__ w, TI* __restrict__ y,
           uint8_t* __restrict__ s, TR* total, Rows q) {
    using U = Units<16 / sizeof(TI), VEC>;
    constexpr int V = U::V;
    __shared__ float red[32];
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
    const auto scale = [&] { return __frsqrt_rn(team_sum<WARP>(ss, red) / (float)q.D + q.eps); };
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

// A backward unit's V channels are 16 bytes of the residual's type, so that neighbouring lanes'
// accesses touch (with 8 channels of fp32 a lane, every access reads half of each sector).
template <typename TR, bool VEC> using BwdUnits = Units<16 / sizeof(TR), VEC>;
template <typename E, int V> __device__ __forceinline__ void fetch(const uint4* from, float (&o)[V]) {
    Conv<E, V>::to(*reinterpret_cast<const typename Pack<E, V>::Raw*>(from), o);
}

// Team `slot` of `slots` has tokens slot, slot + slots, ...; its dw goes to part[slot].
// AHEAD: the next row is copied into each thread's own room in shared memory while this one is
// summed and applied.
template <typename TI, typename TR, bool VEC, int VPT, bool WARP, bool AHEAD>
__global__ void __launch_bounds__(WARP ? kTeams * 32 : VPT == 1 ? 512 : 1024, WARP ? 3 : VPT == 1 ? 2 : 1)
bwd_kernel(const TR* __restrict__ total, const float* __restrict__ w, const TI* __restrict__ dy,
           const TR* __restrict__ dtotal, TI* __restrict__ dx, TR* __restrict__ dres, float* __restrict__ part, int slots,
           Rows q) {
    using U = BwdUnits<TR, VEC>;
    static_assert(!AHEAD || (VEC && VPT > 0), "copies are of whole units");
    constexpr int V = U::V, K = VPT > 0 ? VPT : 1;
    __shared__ __align__(16) float2 red[2][32];
    extern __shared__ __align__(16) uint4 room[];   // [2 rows][K][total, dtotal, dy][threads]
    constexpr int kD = V * (int)sizeof(TI), kUnit = 32 + kD;   // bytes of dy's piece, of a unit
    const int slot = WARP ? (int)blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    grid_dep_wait();
    grid_dep_launch();
    const int units = U::count(q.D), bt = blockDim.x;
    float* pr = part && slot < slots ? part + (int64_t)slot * q.D : nullptr;
    const float inv = 1.f / (float)q.D;
    constexpr int P = V / 2;   // pairs: the arithmetic is packed
    f2 acc[K][P];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) acc[k][j] = 0;
    int parity = 0;
    const auto place = [&](int64_t row, const Tok& s) {
        if (q.flat) return row * s.t;
        const uint32_t b = (uint32_t)row / q.T;
        return (int64_t)b * s.b + (int64_t)((uint32_t)row - b * q.T) * s.t;
    };
    const auto piece = [&](int at, int k, int i) {
        unsigned char* base = reinterpret_cast<unsigned char*>(room) + (at * K + k) * kUnit * bt;
        return reinterpret_cast<uint4*>(base + (i < 2 ? (i * bt + threadIdx.x) * 16 : 32 * bt + threadIdx.x * kD));
    };
    const auto copy = [&](int64_t row, int at) {   // a group of copies, empty behind the last row
        if (row >= q.rows) return stage_commit();
        const TR* tr = total + place(row, q.st);
        const TI* dr = dy + place(row, q.sy);
        const TR* er = dtotal ? dtotal + place(row, q.sres) : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = tid + k * nt;
            if (u >= units) continue;
            stage_copy<16>(piece(at, k, 0), tr + u * V, true);
            if (er) stage_copy<16>(piece(at, k, 1), er + u * V, true);
            stage_copy<kD>(piece(at, k, 2), dr + u * V, true);
        }
        stage_commit();
    };
    // a thread's channels are the same in every row: their weights stay in registers (read from L1, which the
    // copies push them out of, the rows took 222 us instead of 207; from shared memory 138 instead of 123 with a bf16 residual)
    f2 wr[K][P];
    const auto load_weights = [&](int u, f2 (&o)[P]) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = 1.f;
        if (w && u < units) U::load(w, u, q.D, f);
#pragma unroll
        for (int j = 0; j < P; ++j) o[j] = pack2(f[2 * j], f[2 * j + 1]);
    };
    if constexpr (VPT > 0)
#pragma unroll
        for (int k = 0; k < K; ++k) load_weights(tid + k * nt, wr[k]);
    const auto put = [&](int u, const f2 (&a)[P]) {
        float f[V];
#pragma unroll
        for (int j = 0; j < P; ++j) unpack2(a[j], f[2 * j], f[2 * j + 1]);
        U::store(pr, u, q.D, f);
    };
    if (slot >= slots) return;
    if constexpr (AHEAD) copy(slot, 0);
    for (int64_t row = slot; row < q.rows; row += slots) {
        f2 ss = 0, gv = 0, r, less;   // less: -mean(g n)
        const auto sums = [&](const f2 (&f)[P], const float (&v)[V], const float (&d)[V]) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const f2 x = pack2(v[2 * j], v[2 * j + 1]);
                ss = fma2(x, x, ss);
                gv = fma2(mul2(pack2(d[2 * j], d[2 * j + 1]), f[j]), x, gv);
            }
        };
        const auto scales = [&] {
            // two halves of red in turn: the next token's sums do not overwrite one being read
            const float2 s = team_sum<WARP>(sum2(ss), sum2(gv), red[parity]);
            const float one = __frsqrt_rn(s.x * inv + q.eps);
            r = dup2(one);
            less = dup2(-one * (s.y * inv));
        };
        // e: dtotal; a: this unit's part of dw, added to
        const auto result = [&](int u, const f2 (&f)[P], const float (&v)[V], const float (&d)[V], float (&e)[V], f2 (&a)[P]) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const f2 n = mul2(pack2(v[2 * j], v[2 * j + 1]), r), g = pack2(d[2 * j], d[2 * j + 1]);
                a[j] = fma2(g, n, a[j]);
                const f2 t = fma2(n, less, mul2(g, f[j]));
                unpack2(fma2(r, t, pack2(e[2 * j], e[2 * j + 1])), e[2 * j], e[2 * j + 1]);
            }
            U::store(dx + row * q.D, u, q.D, e);
            if (dres) U::store(dres + row * q.D, u, q.D, e);
        };
        const auto zero = [](float (&e)[V]) {
#pragma unroll
            for (int j = 0; j < V; ++j) e[j] = 0.f;
        };
        if constexpr (AHEAD) {
            copy(row + slots, parity ^ 1);
            stage_wait<1>();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < units) {
                    float v[V], d[V];
                    fetch<TR>(piece(parity, k, 0), v);
                    fetch<TI>(piece(parity, k, 2), d);
                    sums(wr[k], v, d);
                }
            scales();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * nt < units) {
                    float v[V], d[V], e[V];
                    fetch<TR>(piece(parity, k, 0), v);
                    fetch<TI>(piece(parity, k, 2), d);
                    if (dtotal) fetch<TR>(piece(parity, k, 1), e);
                    else zero(e);
                    result(tid + k * nt, wr[k], v, d, e, acc[k]);
                }
        } else {
            const TR* tr = total + place(row, q.st);
            const TI* dr = dy + place(row, q.sy);
            const TR* er = dtotal ? dtotal + place(row, q.sres) : nullptr;
            float v[K][V], d[K][V], e[V];
            const auto third = [&](int u) {
                if (er) U::load(er, u, q.D, e);
                else zero(e);
            };
            if constexpr (VPT > 0) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (tid + k * nt < units) {
                        U::load(tr, tid + k * nt, q.D, v[k]);
                        U::load(dr, tid + k * nt, q.D, d[k]);
                    }
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (tid + k * nt < units) sums(wr[k], v[k], d[k]);
                scales();
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (tid + k * nt < units) {
                        third(tid + k * nt);
                        result(tid + k * nt, wr[k], v[k], d[k], e, acc[k]);
                    }
            } else {
                for (int u = tid; u < units; u += nt) {
                    U::load(tr, u, q.D, v[0]);
                    U::load(dr, u, q.D, d[0]);
                    load_weights(u, wr[0]);
                    sums(wr[0], v[0], d[0]);
                }
                scales();
                for (int u = tid; u < units; u += nt) {
                    U::load(tr, u, q.D, v[0]);
                    U::load(dr, u, q.D, d[0]);
                    third(u);
                    float part_of[V];
                    zero(part_of);
                    if (pr && row != slot) U::load(pr, u, q.D, part_of);
                    f2 a[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) a[j] = pack2(part_of[2 * j], part_of[2 * j + 1]);
                    load_weights(u, wr[0]);
                    result(u, wr[0], v[0], d[0], e, a);
                    if (pr) put(u, a);
                }
            }
        }
        parity ^= 1;
    }
    if (VPT > 0 && pr)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (tid + k * nt < units) put(tid + k * nt, acc[k]);
}

Rows rows_of(const AddNormArgs& a) {
    const auto even = [&](const Tok& s) { return a.b <= 1 || s.b == a.T * s.t; };
    return Rows{(uint32_t)a.T, (int)a.D, a.b * a.T, a.eps, a.sx, a.sres, a.sy, a.st, even(a.sres) && even(a.sy) && even(a.st)};
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
    const int64_t n = Units<16 / sizeof(TI), VEC>::count((int)a.D);
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

constexpr int kDevices = 64;
constexpr int kSharedMost = 128 * 1024;   // bytes of an SM, for the rows copied ahead
constexpr int kRoomMost = 2 * 2 * 48 * 1024;   // of a block: two rows, two units of three pieces a thread

// Blocks of kernel k that an SM holds, having let it have its shared memory; asked for once for the
// sizes that were last asked for on a device (`known`: this kernel's threads, room and blocks, by device).
template <typename K> cudaError_t resident_blocks(K k, int threads, int room, std::atomic<uint64_t>* known, int* blocks) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = (uint64_t)threads << 32 | (uint64_t)room << 8;
    const uint64_t old = dev < kDevices ? known[dev].load(std::memory_order_relaxed) : 0;
    if ((old & ~uint64_t(255)) == key) return *blocks = (int)(old & 255), cudaSuccess;
    // the most that any size asks for, so that calls of two sizes at once do not take it from each other
    if (room && (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoomMost)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, k, threads, (size_t)room)) != cudaSuccess) return e;
    // Copies land by way of L1: with 228 KB of an SM taken from it they come at three quarters of the rate,
    // whatever is in flight (fp32, D 2560: 262 us, with 164 KB 200).
    *blocks = std::max(1, std::min(*blocks, kSharedMost / (room + 1536)));
    if (room && (e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 72)) != cudaSuccess) return e;
    if (dev < kDevices) known[dev].store(key | (uint64_t)*blocks, std::memory_order_relaxed);
    return cudaSuccess;
}

// *slots: the teams that it takes (rows of part).
template <typename TI, typename TR, bool VEC>
cudaError_t bwd_go(const AddNormArgs& a, const void* t_, const float* w, const void* dy_, const void* dt_, void* dx_,
                   void* dr_, float* part, int* slots, cudaStream_t st) {
    const Rows q = rows_of(a);
    if (q.rows >= (int64_t(1) << 31)) return kGridLimit;
    const TR *t = static_cast<const TR*>(t_), *dt = static_cast<const TR*>(dt_);
    const TI* dy = static_cast<const TI*>(dy_);
    TI* dx = static_cast<TI*>(dx_);
    TR* dr = static_cast<TR*>(dr_);
    const int64_t n = BwdUnits<TR, VEC>::count((int)a.D);
    const int64_t most = add_norm_bwd_slots(a);
    static std::atomic<uint64_t> known[5][kDevices];   // by form
    // ahead: units a thread, 0: none is copied
    const auto go = [&](int form, auto k, bool warp, int threads, int ahead) {
        const int room = ahead ? 2 * ahead * (32 + BwdUnits<TR, VEC>::V * (int)sizeof(TI)) * threads : 0;
        int per_sm;
        const cudaError_t e = resident_blocks(k, threads, room, known[form], &per_sm);
        if (e != cudaSuccess) return e;
        const int64_t teams = warp ? kTeams : 1;
        *slots = (int)std::min(most, (int64_t)sm_count() * per_sm * teams);
        const unsigned blocks = (unsigned)((*slots + teams - 1) / teams);
        return launch_kernel(k, dim3(blocks), dim3((unsigned)threads), (size_t)room, st, early(blocks), t, w, dy, dt, dx, dr, part,
                             *slots, q);
    };
    if (n <= 32) return go(0, bwd_kernel<TI, TR, VEC, 1, true, VEC>, true, kTeams * 32, VEC);
    if (n <= 64) return go(1, bwd_kernel<TI, TR, VEC, 2, true, VEC>, true, kTeams * 32, 2 * VEC);
    if (n <= 512) return go(2, bwd_kernel<TI, TR, VEC, 1, false, VEC>, false, threads_of(n, 1), VEC);
    if (n <= 2048) return go(3, bwd_kernel<TI, TR, VEC, 2, false, VEC>, false, threads_of(n, 2), 2 * VEC);
    return go(4, bwd_kernel<TI, TR, VEC, 0, false, false>, false, 1024, 0);
}

// Every access of a unit of V channels is aligned.
bool vec(const AddNormArgs& a, int64_t V, const float* w, std::initializer_list<std::pair<const void*, Tok>> io,
         std::initializer_list<std::pair<const void*, Tok>> res, const void* q8) {
    const int64_t es = a.bf16 ? 2 : 4, rs = a.res_bf16 ? 2 : 4;
    if (a.D % V || reinterpret_cast<uintptr_t>(w) % 16) return false;
    for (const auto& t : io)
        if (!vec_ok(t.first, t.second, V * es, es)) return false;
    for (const auto& t : res)
        if (t.first && !vec_ok(t.first, t.second, 16, rs)) return false;
    return !q8 || vec_ok(q8, a.sy, V, 1);
}

}  // namespace

cudaError_t launch_add_norm_fwd(const AddNormArgs& a, const void* x, const void* residual, const float* w, void* y,
                                uint8_t* s, void* total, cudaStream_t st) {
    if (a.b * a.T == 0 || a.D == 0) return cudaSuccess;
    const bool v = a.quant ? vec(a, a.bf16 ? 8 : 4, w, {{x, a.sx}}, {{residual, a.sres}, {total, a.st}}, y)
                           : vec(a, a.bf16 ? 8 : 4, w, {{x, a.sx}, {y, a.sy}}, {{residual, a.sres}, {total, a.st}}, nullptr);
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
    // what the workspace has room for: no fewer teams than any form of the kernel has on an SM at once
    const int64_t units = a.res_bf16 ? (a.D + 7) / 8 : (a.D + 3) / 4;
    const int64_t per_sm = units <= 64 ? 4 * kTeams : std::max<int64_t>(1, 2048 / threads_of(units, units <= 512 ? 1 : 2));
    return std::max<int64_t>(1, std::min<int64_t>(a.b * a.T, (int64_t)sm_count() * per_sm));
}

cudaError_t launch_add_norm_bwd(const AddNormArgs& a, const void* total, const float* w, const void* dy,
                                const void* dtotal, void* dx, void* dres, float* dw, float* part, cudaStream_t st) {
    if (a.D == 0) return cudaSuccess;
    const bool none = a.b * a.T == 0;
    int slots = 0;
    if (!dw) part = nullptr;
    if (!none) {
        const Tok row{0, a.D};
        const bool v = vec(a, a.res_bf16 ? 8 : 4, w, {{dy, a.sy}, {dx, row}}, {{total, a.st}, {dtotal, a.sres}, {dres, row}}, nullptr) &&
                       reinterpret_cast<uintptr_t>(part) % 16 == 0;
        const auto go = [&](auto f) { return f(a, total, w, dy, dtotal, dx, dres, part, &slots, st); };
        typedef __nv_bfloat16 bf;
        const cudaError_t e = !a.bf16     ? (v ? go(bwd_go<float, float, true>) : go(bwd_go<float, float, false>))
                              : !a.res_bf16 ? (v ? go(bwd_go<bf, float, true>) : go(bwd_go<bf, float, false>))
                                            : (v ? go(bwd_go<bf, bf, true>) : go(bwd_go<bf, bf, false>));
        if (e != cudaSuccess) return e;
    }
    return dw ? launch_column_sum(part, slots, a.D, dw, a.D, nullptr, st) : cudaSuccess;
}

}  // namespace m2
