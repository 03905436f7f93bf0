// scan.cuh -- lane and tile layout shared by the selective scan's kernels.
#pragma once

#include "layer.cuh"

namespace m2 {

// Lanes and tiles.  A lane keeps kNS states of one channel; N / kNS neighbouring
// lanes make a channel.  A block holds CB channels of one group and one sequence
// and walks over tokens in tiles of TT.
constexpr int kNS = 4;
template <int N> struct Cfg {
    static constexpr int NT = N >= 64 ? 256 : 128;
    static constexpr int LPC = N / kNS;
    static constexpr int CPW = 32 / LPC;
    static constexpr int CB = NT / LPC;
    static constexpr int TT = N >= 128 ? 64 : 32;
    static constexpr int U = LPC < 8 ? LPC : 8;           // tokens reduced together
    static constexpr int YP = CB + (CPW < 2 ? 2 : CPW);   // pitch of the y tile (bank-conflict free)
    static constexpr size_t smem = (size_t)TT * (CB * 16 + 2 * N * 4 + YP * 4);
};

// Sum v[u] over the LPC lanes of a channel for U tokens at once: at each step a lane
// hands over the half it does not keep.  On return v[0] is the sum for token
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
