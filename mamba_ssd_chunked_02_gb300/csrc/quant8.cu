// quant8.cu -- values to e4m3 with a power-of-two scale for each group of 128
// (include/mamba2_proj.h): groups along rows, along columns, or blocks of 128 x 128.
//
//   s = 2^e, e the smallest whole number >= -127 with max|x| <= 448 s;  q = x / s to nearest even
//
// Bytes bound: a block of 512 threads holds a tile of 128 x 128 in registers, 4 x 8 values a
// thread, so that both kinds of groups come from one reading (the backward product takes dy
// along its rows for dx and along its columns for dw).  In a graph: bf16 rows 32768 x 5120 79 us, 6.4 TB/s
// (0.96 of the measured copy rate; a call 81); fp32 blocks 10576 x 2560 25 us (5.4; a call 26.7); dy of 32768 x 10576 both
// ways 283 us (4.9), issue slots at 0.56 (the next tile copied ahead: 300); x turned 46 us (3.6).  Kernels here and in add_norm.cu
// may begin while the one before them ends, and wait for it before they read.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "proj.cuh"

namespace m2 {
namespace {

enum { kRow = 1, kCol = 2, kBlock = 4 };
constexpr int kThreads = 512, kLines = kThreads / 16, kPer = kGroup / kLines, kWarps = kThreads / 32;

struct Tile {
    int64_t M, N;
    uint32_t T, nb;          // rows of one sequence, groups along a row
    Tok sx;                  // elements
    Tok sq;                  // of q (both outputs)
    const uint8_t* s_in;     // scales of an e4m3 input [M, nb]
    uint8_t *qr, *sr, *qc, *sc;
    int64_t ps;              // bytes between the rows of sr
    bool even;               // rows lie at even distances, sequences or not
};

// Two e4m3 pairs of products v f, v in fp32.
template <bool CLEAN> __device__ __forceinline__ uint32_t e4m3_four(const float* v, f2 lo, f2 hi) {
    float f[4];
    unpack2(mul2(pack2(v[0], v[1]), lo), f[0], f[1]);
    unpack2(mul2(pack2(v[2], v[3]), hi), f[2], f[3]);
    return e4m3_pair<CLEAN>(f[0], f[1]) | e4m3_pair<CLEAN>(f[2], f[3]) << 16;
}

// Eight neighbours of a row as they lie in memory, read by one access (VEC) or one by one, and
// Tops, the largest magnitudes in a column of such.
template <typename TI> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint32_t w[4];
    struct Tops {
        uint32_t w[4];   // of either sign
        __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
        __device__ __forceinline__ void join(const uint32_t (&o)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = larger(w[j], o[j]);
        }
        __device__ __forceinline__ void join_lane(int other) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = __shfl_xor_sync(0xffffffffu, w[j], other);
            join(o);
        }
        __device__ __forceinline__ void get(float (&t)[8]) const {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[2 * j] = fabsf(bf_lo(w[j])), t[2 * j + 1] = fabsf(bf_hi(w[j]));
        }
    };
    // max(|a|, |b|) of both halves, NaN left out, of either sign
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    template <bool VEC> __device__ __forceinline__ void load(const __nv_bfloat16* p, int count) {
        if constexpr (VEC) {
            if (count <= 0) return;
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
            if (count >= 8) {   // the widest accesses that the row's start allows (the same for all its lanes)
                const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(p);
                if (at % 16 == 0) return load<true>(p, count);
                if (at % 4 == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
                } else {   // a half, three words, a half
                    uint32_t v[5] = {(uint32_t)__ldg(u) << 16, 0, 0, 0, (uint32_t)__ldg(u + 7)};
#pragma unroll
                    for (int j = 0; j < 3; ++j) v[j + 1] = __ldg(reinterpret_cast<const uint32_t*>(u + 1) + j);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_l(v[j], v[j + 1], 16);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (2 * j < count ? __ldg(u + 2 * j) : 0) | (uint32_t)(2 * j + 1 < count ? __ldg(u + 2 * j + 1) : 0) << 16;
        }
    }
    __device__ __forceinline__ float top() const {
        const uint32_t m = larger(larger(w[0], w[1]), larger(w[2], w[3]));   // NaN only where all are
        return fmaxf(fmaxf(0.f, fabsf(bf_lo(m))), fabsf(bf_hi(m)));
    }
    __device__ __forceinline__ void into(Tops& t) const { t.join(w); }
    // Unpacked anew at each use (the statement hides what it was unpacked to before), so that the
    // packed words alone are kept from one pass over the tile to the next.
    __device__ __forceinline__ void get(float (&v)[8]) {
        asm volatile("" : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf_lo(w[j]), v[2 * j + 1] = bf_hi(w[j]);
    }
};
template <> struct Eight<float> {
    float f[8];
    struct Tops {
        float t[8];
        __device__ __forceinline__ void zero() {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = 0.f;
        }
        __device__ __forceinline__ void join_lane(int other) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = fmaxf(t[j], __shfl_xor_sync(0xffffffffu, t[j], other));
        }
        __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = t[j];
        }
    };
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.f;
    }
    template <bool VEC> __device__ __forceinline__ void load(const float* p, int count) {
        if constexpr (VEC) {
            if (count <= 0) return;
            const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p + 4));
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
            if (count >= 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) return load<true>(p, count);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = j < count ? __ldg(p + j) : 0.f;
        }
    }
    __device__ __forceinline__ float top() const {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = fmaxf(t, fabsf(f[j]));
        return t;
    }
    __device__ __forceinline__ void into(Tops& t) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) t.t[j] = fmaxf(t.t[j], fabsf(f[j]));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f[j];
    }
};

// Eight bytes of a row, `count` of them inside it.
template <bool VEC> __device__ __forceinline__ void store_eight(uint8_t* to, int count, uint32_t lo, uint32_t hi) {
    if (VEC ? count > 0 : count >= 8) {
        *reinterpret_cast<uint2*>(to) = make_uint2(lo, hi);
    } else if (!VEC) {   // the row's end: nothing behind it is written
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count) to[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// The largest magnitudes t of 8 columns a lane (lanes 0-15 of each warp) to the tile's column
// scales: written to p.sc, and the bytes left in shared memory.
__device__ __forceinline__ void column_scales(const Tile& p, float (*tops)[kGroup], uint8_t* bytes, uint32_t mb, int64_t n0, int cols) {
    if (threadIdx.x < kGroup) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, tops[k][threadIdx.x]);
        bytes[threadIdx.x] = (uint8_t)scale_byte(top);
        if (threadIdx.x < cols) p.sc[mb * p.N + n0 + threadIdx.x] = bytes[threadIdx.x];
    }
    __syncthreads();
}
__device__ __forceinline__ void column_inverses(const uint8_t* bytes, int tx, float (&t)[8]) {
    const uint2 w = *reinterpret_cast<const uint2*>(bytes + 8 * tx);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = scale_inverse((j < 4 ? w.x : w.y) >> (8 * (j & 3)) & 0xffu);
}
__device__ __forceinline__ void put_tops(float (*tops)[kGroup], int warp, int tx, const float (&t)[8]) {
    float4* to = reinterpret_cast<float4*>(&tops[warp][8 * tx]);
    to[0] = make_float4(t[0], t[1], t[2], t[3]);
    to[1] = make_float4(t[4], t[5], t[6], t[7]);
}

// Thread (tx, ty) has rows ty + 32 i and columns 8 tx + j.
template <typename TI, bool VEC, int MODE, int kThreads = 512>
__device__ __forceinline__ void quant_tile(const TI* __restrict__ x, const Tile& p, uint32_t tile) {
    constexpr int kLines = kThreads / 16, kPer = kGroup / kLines, kWarps = kThreads / 32;
    __shared__ __align__(16) float tops[kWarps][kGroup];
    __shared__ __align__(8) uint8_t bytes[kGroup];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t mb = tile / p.nb, nb = tile - mb * p.nb;
    const int64_t m0 = (int64_t)mb * kGroup, n0 = (int64_t)nb * kGroup;
    const int rows = (int)min((int64_t)kGroup, p.M - m0), cols = (int)min((int64_t)kGroup, p.N - n0), count = cols - 8 * tx;
    grid_dep_wait();
    grid_dep_launch();
    // where the rows' values lie, in x and in q
    int64_t from[kPer], to[kPer];
    if (p.even) {
        from[0] = (m0 + ty) * p.sx.t + n0 + 8 * tx, to[0] = (m0 + ty) * p.sq.t + n0 + 8 * tx;
#pragma unroll
        for (int i = 1; i < kPer; ++i) from[i] = from[i - 1] + kLines * p.sx.t, to[i] = to[i - 1] + kLines * p.sq.t;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t m = (uint32_t)(m0 + ty + kLines * i), b = m / p.T, t = m - b * p.T;
            from[i] = b * p.sx.b + t * p.sx.t + n0 + 8 * tx, to[i] = b * p.sq.b + t * p.sq.t + n0 + 8 * tx;
        }
    }
    Eight<TI> raw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        raw[i].zero();
        if (ty + kLines * i < rows) raw[i].template load<VEC>(x + from[i], count);
    }
    // largest magnitude of row i's eight values; with CLEAN, of those that are finite
    const auto top_in = [&](auto clean, int i) {
        if (!decltype(clean)::value) return raw[i].top();
        float v[8], top = 0.f;
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = top_of<true>(top, v[j]);
        return top;
    };
    const auto put = [&](auto clean, uint8_t* q, int i, auto inv) {
        constexpr bool CLEAN = decltype(clean)::value;
        if (ty + kLines * i >= rows) return;
        float v[8];
        raw[i].get(v);
        store_eight<VEC>(q + to[i], count, e4m3_four<CLEAN>(v, inv(0), inv(1)), e4m3_four<CLEAN>(v + 4, inv(2), inv(3)));
    };
    // each returns false where there are infinities to be looked for (and is called again with `clean`)
    const auto rows_go = [&](auto clean) {
        constexpr bool CLEAN = decltype(clean)::value;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float top = top_in(clean, i);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (!CLEAN && __any_sync(0xffffffffu, infinite(top))) return false;
            const uint32_t byte = scale_byte(top);
            const f2 f = dup2(scale_inverse(byte));
            if (tx == 0 && ty + kLines * i < rows) p.sr[(m0 + ty + kLines * i) * p.ps + nb] = (uint8_t)byte;
            put(clean, p.qr, i, [&](int) { return f; });
        }
        return true;
    };
    const auto cols_go = [&](auto clean) {
        constexpr bool CLEAN = decltype(clean)::value;
        float t[8];
        if constexpr (CLEAN) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                float v[8];
                raw[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = top_of<true>(t[j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = fmaxf(t[j], __shfl_xor_sync(0xffffffffu, t[j], 16));
        } else {
            typename Eight<TI>::Tops all;
            all.zero();
#pragma unroll
            for (int i = 0; i < kPer; ++i) raw[i].into(all);
            all.join_lane(16);
            all.get(t);
        }
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) bad |= infinite(t[j]);
        if (lane < 16) put_tops(tops, warp, tx, t);
        if (__syncthreads_or(bad) && !CLEAN) return false;
        column_scales(p, tops, bytes, mb, n0, cols);
        column_inverses(bytes, tx, t);
        f2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pack2(t[2 * j], t[2 * j + 1]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) put(clean, p.qc, i, [&](int j) { return f[j]; });
        return true;
    };
    const auto block_go = [&](auto clean) {
        constexpr bool CLEAN = decltype(clean)::value;
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) top = fmaxf(top, top_in(clean, i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) tops[CLEAN][warp] = top;
        __syncthreads();
        top = tops[CLEAN][0];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, tops[CLEAN][k]);
        if (!CLEAN && infinite(top)) return false;
        const uint32_t byte = scale_byte(top);
        const f2 f = dup2(scale_inverse(byte));
        if (threadIdx.x == 0) p.sr[tile] = (uint8_t)byte;
#pragma unroll
        for (int i = 0; i < kPer; ++i) put(clean, p.qr, i, [&](int) { return f; });
        return true;
    };
    const std::false_type plain{};
    const std::true_type clean{};
    if constexpr (MODE & kRow)
        if (!rows_go(plain)) rows_go(clean);
    if constexpr (MODE & kCol)
        if (!cols_go(plain)) cols_go(clean);
    if constexpr (MODE & kBlock)
        if (!block_go(plain)) block_go(clean);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// e4m3 in groups along rows to e4m3 in groups along columns.  The bits of an e4m3 number in the
// places of a bf16's (or fp32's) low exponent and high mantissa bits are its magnitude times 2^-120,
// subnormal ones too: a shift and a product by a power of two, where conversions by way of fp16 run at
// a quarter of the rate; the sign is put back as it was.  In bf16, two at a time, everything is exact but
// for values below 2^-126: rows of scales below 2^-111, 2^8 and up, and NaN take the way by whole numbers.
template <bool VEC> __device__ __forceinline__ void turn_tile(const uint8_t* __restrict__ x, const Tile& p, uint32_t tile) {
    __shared__ __align__(16) float tops[kWarps][kGroup];
    __shared__ __align__(8) uint8_t bytes[kGroup];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t mb = tile / p.nb, nb = tile - mb * p.nb;
    const int64_t m0 = (int64_t)mb * kGroup, n0 = (int64_t)nb * kGroup;
    const int rows = (int)min((int64_t)kGroup, p.M - m0), cols = (int)min((int64_t)kGroup, p.N - n0), count = cols - 8 * tx;
    const int64_t from = (m0 + ty) * p.sx.t + n0 + 8 * tx, to = (m0 + ty) * p.sq.t + n0 + 8 * tx;
    grid_dep_wait();
    grid_dep_launch();
    const auto scale_of = [&](int i) {   // row i's: 2^(e - 127)
        return ty + kLines * i < rows ? __ldg(p.s_in + (m0 + ty + kLines * i) * p.nb + nb) : 0;
    };
    const auto load = [&](int i, uint32_t (&o)[2]) {
        const uint8_t* f = x + from + i * (kLines * p.sx.t);
        o[0] = o[1] = 0;
        if (ty + kLines * i < rows && (VEC ? count > 0 : count >= 8)) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(f));
            o[0] = v.x, o[1] = v.y;
        } else if (!VEC && ty + kLines * i < rows) {   // the row's end
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < count) o[j / 4] |= (uint32_t)__ldg(f + j) << (8 * (j & 3));
        }
    };
    // all loads first: none waits for another
    uint32_t w[kPer][2], e[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = scale_of(i);
#pragma unroll
    for (int i = 0; i < kPer; ++i) load(i, w[i]);
    bool bad = false;   // what takes the careful way
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        bad |= e[i] > 134 || (e[i] < 16 && ((w[i][0] | w[i][1]) & 0x7f7f7f7fu) != 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) bad |= __vcmpeq4(w[i][h] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    }
    // A value as a number's bits, with 8 bits of exponent more than an fp32's sign leaves room for: the magnitude's
    // bits, its exponent moved on by the scale byte.  They order as the values do; what the scales stand for goes up
    // to 448 * 2^127, and an fp32 maximum rounds up to 2^128.  All ones: NaN, a NaN scale's among them.
    constexpr uint32_t kNaN = 0xffffffffu;
    const auto bits = [&](const uint32_t (&v)[2], uint32_t byte, int j) {
        const uint32_t k = 8 * (j & 3), b = (k < 20 ? v[j / 4] << (20 - k) : v[j / 4] >> (k - 20)) & 0x07f00000u;
        const uint32_t n = __float_as_uint(__uint_as_float(b) * 0x1p120f) + (byte << 23);
        return b == 0x07f00000u || byte == 255 ? kNaN : b ? n : 0u;
    };
    // Reads the rows again, one by one: the other way's registers are its own.
    const auto carefully = [&] {
        uint32_t t[8] = {}, v[2];
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
            load(i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t n = bits(v, scale_of(i), j);
                t[j] = max(t[j], n == kNaN ? 0u : n);
            }
        }
        float most[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) most[j] = __uint_as_float(max(t[j], __shfl_xor_sync(0xffffffffu, t[j], 16)));
        if (lane < 16) put_tops(tops, warp, tx, most);
        __syncthreads();
        if (threadIdx.x < kGroup) {   // as scale_byte, with 127 more in the exponent
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) m = max(m, __float_as_uint(tops[k][threadIdx.x]));
            bytes[threadIdx.x] = (uint8_t)max((int)(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
            if (threadIdx.x < cols) p.sc[mb * p.N + n0 + threadIdx.x] = bytes[threadIdx.x];
        }
        __syncthreads();
        const uint2 down = *reinterpret_cast<const uint2*>(bytes + 8 * tx);
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
            if (ty + kLines * i >= rows) break;
            load(i, v);
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t n = bits(v, scale_of(i), 4 * h + j), by = (h ? down.y : down.x) >> (8 * j) & 0xffu;
                    // below 2^-126 there is no e4m3 number
                    f[j] = n == kNaN ? __uint_as_float(0x7fffffffu) : n < (by + 1) << 23 ? 0.f : __uint_as_float(n - (by << 23));
                }
                o[h] = e4m3_pair<false>(f[0], f[1]) | e4m3_pair<false>(f[2], f[3]) << 16 | (v[h] & 0x80808080u);
            }
            store_eight<VEC>(p.qc + to + i * (kLines * p.sq.t), count, o[0], o[1]);
        }
    };
    if (__syncthreads_or(bad)) return carefully();
    // columns 0 and 2, 1 and 3, 4 and 6, 5 and 7 of each row
    uint32_t v[kPer][4], top[4] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t by = (e[i] + 120) * 0x00800080u;   // 2^120 times the row's scale, twice
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            v[i][h] = mul_bf16x2((h & 1 ? w[i][h / 2] >> 4 : w[i][h / 2] << 4) & 0x07f007f0u, by);
            top[h] = max_bf16x2(top[h], v[i][h]);
        }
    }
    float t[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        top[h] = max_bf16x2(top[h], __shfl_xor_sync(0xffffffffu, top[h], 16));
        t[4 * (h / 2) + (h & 1)] = bf_lo(top[h]), t[4 * (h / 2) + (h & 1) + 2] = bf_hi(top[h]);
    }
    if (lane < 16) put_tops(tops, warp, tx, t);
    __syncthreads();
    column_scales(p, tops, bytes, mb, n0, cols);
    column_inverses(bytes, tx, t);
    uint32_t inv[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
        inv[h] = __float_as_uint(t[4 * (h / 2) + (h & 1)]) >> 16 | (__float_as_uint(t[4 * (h / 2) + (h & 1) + 2]) & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (ty + kLines * i >= rows) continue;
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a = mul_bf16x2(v[i][2 * h], inv[2 * h]), b = mul_bf16x2(v[i][2 * h + 1], inv[2 * h + 1]);
            o[h] = e4m3_pair<false>(bf_lo(a), bf_lo(b)) | e4m3_pair<false>(bf_hi(a), bf_hi(b)) << 16 | (w[i][h] & 0x80808080u);
        }
        store_eight<VEC>(p.qc + to + i * (kLines * p.sq.t), count, o[0], o[1]);
    }
}

// bf16 rows: four blocks an SM, though of 32 registers 48 to 64 bytes spill (32768 x 5120: 78.8 us, three 81.8).  Both
// ways: two, at 64 registers, of which bf16 spills 12 to 32 bytes.
template <typename TI, bool VEC, int MODE, int kThreads = 512>
__global__ void __launch_bounds__(kThreads, sizeof(TI) == 2 && MODE == kRow ? 4 : 2) quant8_kernel(const TI* __restrict__ x, const Tile p) {
    quant_tile<TI, VEC, MODE, kThreads>(x, p, blockIdx.x);
}
// Three blocks an SM at 40 registers, none of them spilled where rows are whole units (20 bytes else; 264 and more
// where the careful way kept the rows in registers: 0.6 us).  32768 x 2560: 46 us, four blocks 47; where each row's
// loads waited for the last's 58, with two blocks then 75.
template <bool VEC> __global__ void __launch_bounds__(kThreads, 3) quant8_turn_kernel(const uint8_t* __restrict__ x, const Tile p) {
    turn_tile<VEC>(x, p, blockIdx.x);
}
// The backward product's operands in one launch: `tiles` of dy, then those of x.
template <typename TI, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
quant8_operands_kernel(const TI* __restrict__ dy, const Tile p, uint32_t tiles, const uint8_t* __restrict__ x, const Tile q) {
    if (blockIdx.x < tiles) quant_tile<TI, VEC, kRow | kCol>(dy, p, blockIdx.x);
    else turn_tile<false>(x, q, blockIdx.x - tiles);
}

int64_t blocks_of(Tile& p) {
    p.nb = (uint32_t)((p.N + kGroup - 1) / kGroup);
    p.even = p.M == p.T || (p.sx.b == p.T * p.sx.t && p.sq.b == p.T * p.sq.t);
    return (p.M + kGroup - 1) / kGroup * p.nb;
}

template <typename TI> bool vectors(const TI* x, const Tile& p) {
    return p.N % 8 == 0 && vec_ok(x, p.sx, 16, sizeof(TI)) && (!p.qr || vec_ok(p.qr, p.sq, 8, 1)) &&
           (!p.qc || vec_ok(p.qc, p.sq, 8, 1));
}

template <typename TI, int MODE> cudaError_t go(const TI* x, Tile p, cudaStream_t st) {
    if (p.M == 0 || p.N == 0) return cudaSuccess;
    const int64_t blocks = blocks_of(p);
    if (blocks >= (int64_t(1) << 31) || p.M >= (int64_t(1) << 31)) return kGridLimit;
    const bool v = vectors(x, p);
    // blocks of 128 x 128 by 1024 threads, of which an SM holds as many tiles' loads at once as fit it
    constexpr int T = MODE == kBlock ? 1024 : kThreads;
    return launch_kernel(v ? quant8_kernel<TI, true, MODE, T> : quant8_kernel<TI, false, MODE, T>, dim3((unsigned)blocks),
                         dim3(T), 0, st, early(blocks), x, p);
}

template <int MODE> cudaError_t go(bool bf16, const void* x, const Tile& p, cudaStream_t st) {
    return bf16 ? go<__nv_bfloat16, MODE>(static_cast<const __nv_bfloat16*>(x), p, st)
                : go<float, MODE>(static_cast<const float*>(x), p, st);
}

}  // namespace

cudaError_t launch_quant8(const Quant8Args& a, const void* x, uint8_t* q, uint8_t* s, cudaStream_t st) {
    const Tile p{a.b * a.T, a.D, (uint32_t)a.T, 0, a.sx, a.sq, nullptr, q, s, nullptr, nullptr, (a.D + kGroup - 1) / kGroup, false};
    return a.block ? go<kBlock>(a.bf16, x, p, st) : go<kRow>(a.bf16, x, p, st);
}

cudaError_t launch_quant8_operands(bool bf16, int64_t M, int64_t N, int64_t K, const void* dy, int64_t py, const uint8_t* x,
                                   int64_t px, const uint8_t* s, const Quant8Operands& o, bool dx, bool dw, bool* turned,
                                   cudaStream_t st) {
    Tile p{M, N, (uint32_t)M, 0, Tok{0, py}, Tok{0, o.pn}, nullptr, dx ? o.dyr : nullptr, o.sr, dw ? o.dyc : nullptr, o.sc, o.ps, false};
    Tile q{M, K, (uint32_t)M, 0, Tok{0, px}, Tok{0, o.pk}, s, nullptr, nullptr, o.xc, o.sx, 0, false};
    const int64_t tiles = blocks_of(p), all = tiles + blocks_of(q);
    *turned = dx && dw && early(all);
    if (!*turned) return !dw ? go<kRow>(bf16, dy, p, st) : !dx ? go<kCol>(bf16, dy, p, st) : go<kRow | kCol>(bf16, dy, p, st);
    const auto together = [&](auto* d) {
        using TI = std::remove_const_t<std::remove_pointer_t<decltype(d)>>;
        return launch_kernel(vectors(d, p) ? quant8_operands_kernel<TI, true> : quant8_operands_kernel<TI, false>,
                             dim3((unsigned)all), dim3(kThreads), 0, st, true, d, p, (uint32_t)tiles, x, q);
    };
    return bf16 ? together(static_cast<const __nv_bfloat16*>(dy)) : together(static_cast<const float*>(dy));
}

cudaError_t launch_quant8_turn(int64_t M, int64_t K, const uint8_t* x, int64_t px, const uint8_t* s, const Quant8Operands& o,
                               cudaStream_t st) {
    Tile q{M, K, (uint32_t)M, 0, Tok{0, px}, Tok{0, o.pk}, s, nullptr, nullptr, o.xc, o.sx, 0, false};
    const int64_t blocks = blocks_of(q);
    if (blocks >= (int64_t(1) << 31) || M >= (int64_t(1) << 31)) return kGridLimit;
    return launch_kernel(K % 8 == 0 ? quant8_turn_kernel<true> : quant8_turn_kernel<false>, dim3((unsigned)blocks), dim3(kThreads), 0,
                         st, early(blocks), x, q);
}

}  // namespace m2
