// scan.cuh -- lane and tile layout shared by the selective scan's kernels.
#pragma once

#include "layer.cuh"

namespace m2 {

// Lanes and tiles.  A lane keeps kNS states of each of two neighbouring channels, and
// N / kNS neighbouring lanes a pair of channels: shared memory hands 128 bytes a clock to
// an SM's registers whether lanes read the same address or not, so B and C (four states
// each per token and lane) are used twice per load.  Measured on the forward, b8 T4096
// C5120 N16 bf16: one channel a lane 1.40 ms (12 bytes per state update, the load unit the
// limit), two 1.09 ms (6 bytes), four 1.09 ms where two had come to 0.85 (fewer warps, and
// nothing to hide the latency of exponentials and loads).  A block holds CB channels of one
// group and one sequence and walks over tokens in tiles of TT (32 tokens: 1.35 against 1.05 ms).
constexpr int kNS = 4;
template <int N> struct Cfg {
    static constexpr int NT = N >= 64 ? 128 : 64;
    static constexpr int LPC = N / kNS;
    static constexpr int CPW = 32 / LPC;                  // pairs a warp
    static constexpr int CB = 2 * (NT / LPC);
    static constexpr int TT = N >= 128 ? 32 : 16;
    static constexpr int U = LPC < 8 ? LPC : 8;           // values reduced together: 2 channels x UT tokens
    static constexpr int UT = U / 2;
    static constexpr int YP = LPC <= 4 ? CB + CPW : CB + 2 * CPW;   // pitch of the y tile (bank-conflict free)
    static constexpr int YF = TT * (LPC <= 4 ? LPC : 1) * YP;       // floats of the y tile
};

// Four neighbouring states of B or C from shared memory.
__device__ __forceinline__ ulonglong2 states4(const float* p) { return *reinterpret_cast<const ulonglong2*>(p); }
__device__ __forceinline__ ulonglong2 states4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return ulonglong2{pack2(bf_lo(v.x), bf_hi(v.x)), pack2(bf_lo(v.y), bf_hi(v.y))};
}

// Blocks an SM the registers are kept to.  (Nine, 96 registers, is slower by a sixth than
// eight, 128: 0.24 against 0.20 ms for 16384 tokens of one sequence, C1280.)
template <typename TI, int N, int V> constexpr int min_blocks() {
    return N >= 64 ? 4 : V == 2 && N >= 16 ? 8 : 6;
}

// Sum v[u] over the LPC lanes of a channel for U values at once: at each step a lane
// hands over the half it does not keep.  On return v[0] is the sum for value
// (lane & (U - 1)).
template <int LPC, int U> __device__ __forceinline__ float lanes_sum(float (&v)[U]) {
    const int lane = threadIdx.x & 31;
    int off = 1;
#pragma unroll
    for (int n = U; n > 1; n >>= 1) {
        const bool hi = lane & off;
#pragma unroll
        for (int i = 0; i < U / 2; ++i)
            if (i < n / 2) {
                const float give = hi ? v[2 * i] : v[2 * i + 1], keep = hi ? v[2 * i + 1] : v[2 * i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        off <<= 1;
    }
#pragma unroll
    for (int o = U; o < LPC; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return v[0];
}

}  // namespace m2
