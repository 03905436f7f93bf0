// check.h -- what the C ABI of the layer and projection operators checks alike (host).
#pragma once

#include <stdint.h>

#include "layer.cuh"
#include "mamba2_layer.h"

namespace m2 {

constexpr int64_t kMaxT = int64_t(1) << 30, kMaxD = int64_t(1) << 24, kMaxStride = int64_t(1) << 40;

inline mamba2_status from_cuda(cudaError_t e) {
    return e == cudaSuccess ? MAMBA2_OK : e == kGridLimit ? MAMBA2_ERR_UNSUPPORTED : MAMBA2_ERR_CUDA;
}

// Pointers need their element type's alignment; a tensor without elements may be null.
inline bool req(const void* p, int64_t count, int64_t align) {
    return count == 0 || (p && reinterpret_cast<uintptr_t>(p) % align == 0);
}
inline bool opt(const void* p, int64_t align) { return !p || reinterpret_cast<uintptr_t>(p) % align == 0; }

inline bool dims(int64_t b, int64_t T, int64_t D, int32_t dtype, mamba2_status* st) {
    *st = MAMBA2_ERR_INVALID_ARG;
    if (b < 0 || T < 0 || D < 0 || (dtype != MAMBA2_F32 && dtype != MAMBA2_BF16)) return false;
    *st = MAMBA2_ERR_UNSUPPORTED;
    if (b > kMaxT || T > kMaxT || D > kMaxD) return false;
    if (b && T > (int64_t(1) << 40) / b) return false;
    *st = MAMBA2_OK;
    return true;
}

// Strides of a read tensor: anything that steps forward.
inline bool in_strides(const int64_t* s, int64_t T, int64_t width, Tok* out) {
    if (!s) {
        *out = Tok{T * width, width};
        return true;
    }
    if (s[0] < 0 || s[1] < 0 || s[0] >= kMaxStride || s[1] >= kMaxStride) return false;
    *out = Tok{s[0], s[1]};
    return true;
}
// n pieces of `width` elements, `near` apart, lie apart from each other and within `far`
// (divided, as near * n may pass 64 bits).
inline bool apart(int64_t near, int64_t n, int64_t width, int64_t far) {
    return near >= width && far >= width && n - 1 <= (far - width) / near;
}
// Strides of a written tensor: no two elements in one place.
inline bool out_strides(const int64_t* s, int64_t b, int64_t T, int64_t width, Tok* out) {
    if (!in_strides(s, T, width, out)) return false;
    const int64_t sb = out->b, st = out->t;
    if (b == 0 || T == 0 || width == 0 || (b == 1 && T == 1)) return true;
    if (b <= 1) return st >= width;
    if (T <= 1) return sb >= width;
    return apart(st, T, width, sb) || apart(sb, b, width, st);
}

inline bool space(const void* ws, size_t have, size_t need, int64_t align = 16) {
    return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % align == 0);
}

}  // namespace m2
