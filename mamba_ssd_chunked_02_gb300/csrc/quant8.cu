// quant8.cu -- values to e4m3 with a power-of-two scale for each group of 128
// (include/mamba2_proj.h): groups along rows, along columns, or blocks of 128 x 128.
//
//   s = 2^e, e the smallest whole number >= -127 with max|x| <= 448 s;  q = x / s to nearest even
//
// Bytes bound: a block of 256 threads holds a tile of 128 x 128 in registers, 8 x 8 values a
// thread, so that both kinds of groups come from one reading (the backward product takes dy
// along its rows for dx and along its columns for dw).
#include <cuda_bf16.h>

#include "internal.h"
#include "proj.cuh"

namespace m2 {
namespace {

enum { kRow = 1, kCol = 2, kBlock = 4 };
constexpr int kThreads = 256;

struct Tile {
    int64_t M, N;
    uint32_t T, nb;          // rows of one sequence, groups along a row
    Tok sx;                  // elements
    Tok sq;                  // of q (both outputs)
    const uint8_t* s_in;     // scales of an e4m3 input [M, nb]
    uint8_t *qr, *sr, *qc, *sc;
    int64_t ps;              // bytes between the rows of sr
};

// Thread (tx, ty) has rows ty + 16 i and columns 8 tx + j (VEC: one access) or tx + 16 j.
template <typename TI, bool VEC, int MODE>
__global__ void __launch_bounds__(kThreads) quant8_kernel(const TI* __restrict__ x, const Tile p) {
    __shared__ float tops[8][kGroup];
    __shared__ uint8_t bytes[kGroup];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t m0 = (int64_t)(blockIdx.x / p.nb) * kGroup;
    const uint32_t nb = blockIdx.x % p.nb;
    const int64_t n0 = (int64_t)nb * kGroup;
    const int rows = (int)min((int64_t)kGroup, p.M - m0), cols = (int)min((int64_t)kGroup, p.N - n0);
    const auto col = [&](int j) { return VEC ? 8 * tx + j : tx + 16 * j; };
    const auto place = [&](int64_t m, const Tok& s) {
        const uint32_t b = (uint32_t)m / p.T;
        return (int64_t)b * s.b + (int64_t)((uint32_t)m - b * p.T) * s.t + n0;
    };
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty + 16 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (r >= rows) continue;
        const TI* from = x + place(m0 + r, p.sx);
        if constexpr (sizeof(TI) == 1) {
            const float s = scale_value(p.s_in[(m0 + r) * p.nb + nb]);
            if (VEC) {
                if (8 * tx < cols) {
                    const uint2 w = *reinterpret_cast<const uint2*>(from + 8 * tx);
                    e4m3_quad(w.x, v[i]);
                    e4m3_quad(w.y, v[i] + 4);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < cols) {
                        float f[4];
                        e4m3_quad(from[col(j)], f);
                        v[i][j] = f[0];
                    }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= s;
        } else if constexpr (VEC && sizeof(TI) == 2) {
            if (8 * tx < cols) Conv<TI, 8>::to(load_raw<TI, 8>(from + 8 * tx), v[i]);
        } else if constexpr (VEC) {
            if (8 * tx < cols) {
                Conv<TI, 4>::to(load_raw<TI, 4>(from + 8 * tx), v[i]);
                Conv<TI, 4>::to(load_raw<TI, 4>(from + 8 * tx + 4), v[i] + 4);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col(j) < cols) v[i][j] = to_f32(from[col(j)]);
        }
    }
    const auto store = [&](uint8_t* q, int i, auto inv) {
        const int r = ty + 16 * i;
        if (r >= rows) return;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e4m3_pair(v[i][2 * j] * inv(2 * j), v[i][2 * j + 1] * inv(2 * j + 1));
        uint8_t* to = q + place(m0 + r, p.sq);
        if (VEC) {
            if (8 * tx < cols) *reinterpret_cast<uint2*>(to + 8 * tx) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col(j) < cols) to[col(j)] = (uint8_t)(w[j / 2] >> (j & 1 ? 8 : 0));
        }
    };
    if constexpr (MODE & kRow) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = top_of(top, v[i][j]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t byte = scale_byte(top);
            const float f = scale_inverse(byte);
            if (tx == 0 && ty + 16 * i < rows) p.sr[(m0 + ty + 16 * i) * p.ps + nb] = (uint8_t)byte;
            store(p.qr, i, [&](int) { return f; });
        }
    }
    if constexpr (MODE & kCol) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = top_of(top, v[i][j]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (lane < 16) tops[warp][col(j)] = top;
        }
        __syncthreads();
        if (threadIdx.x < kGroup) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, tops[k][threadIdx.x]);
            bytes[threadIdx.x] = (uint8_t)scale_byte(top);
            if (threadIdx.x < cols) p.sc[m0 / kGroup * p.N + n0 + threadIdx.x] = bytes[threadIdx.x];
        }
        __syncthreads();
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scale_inverse(bytes[col(j)]);
#pragma unroll
        for (int i = 0; i < 8; ++i) store(p.qc, i, [&](int j) { return f[j]; });
    }
    if constexpr (MODE & kBlock) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = top_of(top, v[i][j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) tops[0][warp] = top;
        __syncthreads();
        top = tops[0][0];
#pragma unroll
        for (int k = 1; k < 8; ++k) top = fmaxf(top, tops[0][k]);
        const uint32_t byte = scale_byte(top);
        const float f = scale_inverse(byte);
        if (threadIdx.x == 0) p.sr[blockIdx.x] = (uint8_t)byte;
#pragma unroll
        for (int i = 0; i < 8; ++i) store(p.qr, i, [&](int) { return f; });
    }
}

template <typename TI, int MODE> cudaError_t go(const TI* x, Tile p, cudaStream_t st) {
    if (p.M == 0 || p.N == 0) return cudaSuccess;
    p.nb = (uint32_t)((p.N + kGroup - 1) / kGroup);
    const int64_t blocks = (p.M + kGroup - 1) / kGroup * p.nb;
    if (blocks >= (int64_t(1) << 31) || p.M >= (int64_t(1) << 31)) return kGridLimit;
    const int64_t es = sizeof(TI);
    const bool v = p.N % 8 == 0 && vec_ok(x, p.sx, es == 1 ? 8 : 16, es) && (!p.qr || vec_ok(p.qr, p.sq, 8, 1)) &&
                   (!p.qc || vec_ok(p.qc, p.sq, 8, 1));
    if (v) quant8_kernel<TI, true, MODE><<<(unsigned)blocks, kThreads, 0, st>>>(x, p);
    else quant8_kernel<TI, false, MODE><<<(unsigned)blocks, kThreads, 0, st>>>(x, p);
    return cudaGetLastError();
}

template <int MODE> cudaError_t go(bool bf16, const void* x, const Tile& p, cudaStream_t st) {
    return bf16 ? go<__nv_bfloat16, MODE>(static_cast<const __nv_bfloat16*>(x), p, st)
                : go<float, MODE>(static_cast<const float*>(x), p, st);
}

}  // namespace

cudaError_t launch_quant8(const Quant8Args& a, const void* x, uint8_t* q, uint8_t* s, cudaStream_t st) {
    const Tile p{a.b * a.T, a.D, (uint32_t)a.T, 0, a.sx, a.sq, nullptr, q, s, nullptr, nullptr, (a.D + kGroup - 1) / kGroup};
    return a.block ? go<kBlock>(a.bf16, x, p, st) : go<kRow>(a.bf16, x, p, st);
}

cudaError_t launch_quant8_both(bool bf16, int64_t M, int64_t N, const void* x, int64_t px, uint8_t* qr, uint8_t* sr,
                               int64_t ps, uint8_t* qc, uint8_t* sc, int64_t pq, cudaStream_t st) {
    const Tile p{M, N, (uint32_t)M, 0, Tok{0, px}, Tok{0, pq}, nullptr, qr, sr, qc, sc, ps};
    return !qc ? go<kRow>(bf16, x, p, st) : !qr ? go<kCol>(bf16, x, p, st) : go<kRow | kCol>(bf16, x, p, st);
}

cudaError_t launch_quant8_turn(int64_t M, int64_t N, const uint8_t* q, int64_t px, const uint8_t* s, uint8_t* qc,
                               uint8_t* sc, int64_t pq, cudaStream_t st) {
    const Tile p{M, N, (uint32_t)M, 0, Tok{0, px}, Tok{0, pq}, s, nullptr, nullptr, qc, sc, 0};
    return go<uint8_t, kCol>(q, p, st);
}

}  // namespace m2
