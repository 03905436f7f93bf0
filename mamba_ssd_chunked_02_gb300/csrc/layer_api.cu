// layer_api.cu -- the C ABI declared in include/mamba2_layer.h: argument validation.
// Nothing is launched before every argument has been checked.
#include <cuda_runtime.h>
#include <stdint.h>

#include "check.h"
#include "layer.cuh"
#include "mamba2_layer.h"

namespace {

using m2::dims;
using m2::from_cuda;
using m2::in_strides;
using m2::kMaxD;
using m2::opt;
using m2::out_strides;
using m2::req;
using m2::space;

bool conv_args(const mamba2_conv_shape* s, const mamba2_conv_strides* st, bool y_written, m2::ConvArgs* a,
               mamba2_status* e) {
    *e = MAMBA2_ERR_INVALID_ARG;
    if (!s || !dims(s->batch, s->seqlen, s->channels, s->dtype, e)) return false;
    *e = MAMBA2_ERR_INVALID_ARG;
    if (s->flags & ~MAMBA2_CONV_SILU) return false;
    if (s->width < 2 || s->width > 4) {
        *e = s->width <= 0 ? MAMBA2_ERR_INVALID_ARG : MAMBA2_ERR_UNSUPPORTED;
        return false;
    }
    a->b = s->batch, a->T = s->seqlen, a->D = s->channels, a->W = s->width;
    a->dtype = s->dtype == MAMBA2_BF16, a->silu = s->flags & MAMBA2_CONV_SILU;
    if (!in_strides(st ? st->x : nullptr, a->T, a->D, &a->sx)) return false;
    if (y_written ? !out_strides(st ? st->y : nullptr, a->b, a->T, a->D, &a->sy)
                  : !in_strides(st ? st->y : nullptr, a->T, a->D, &a->sy))
        return false;
    *e = MAMBA2_OK;
    return true;
}

bool scan_args(const mamba2_scan_shape* s, const mamba2_scan_strides* st, bool y_written, m2::ScanArgs* a,
               mamba2_status* e) {
    *e = MAMBA2_ERR_INVALID_ARG;
    if (!s || !dims(s->batch, s->seqlen, s->channels, s->dtype, e)) return false;
    *e = MAMBA2_ERR_INVALID_ARG;
    if ((s->flags & ~MAMBA2_SCAN_SOFTPLUS) || s->groups <= 0 || s->states <= 0 || s->channels % s->groups)
        return false;
    if (s->states != 8 && s->states != 16 && s->states != 32 && s->states != 64 && s->states != 128) {
        *e = MAMBA2_ERR_UNSUPPORTED;
        return false;
    }
    a->b = s->batch, a->T = s->seqlen, a->D = s->channels, a->N = s->states, a->G = s->groups;
    if (a->D == 0) a->G = 1;
    a->dtype = s->dtype == MAMBA2_BF16, a->softplus = s->flags & MAMBA2_SCAN_SOFTPLUS;
    if (s->groups > kMaxD / a->N) {   // a token's B and C: as wide as a token at most
        *e = MAMBA2_ERR_UNSUPPORTED;
        return false;
    }
    const int64_t w = s->groups * a->N;
    if (!in_strides(st ? st->x : nullptr, a->T, a->D, &a->sx) ||
        !in_strides(st ? st->dt : nullptr, a->T, a->D, &a->sdt) ||
        !in_strides(st ? st->B : nullptr, a->T, w, &a->sB) || !in_strides(st ? st->C : nullptr, a->T, w, &a->sC) ||
        !in_strides(st ? st->z : nullptr, a->T, a->D, &a->sz))
        return false;
    if (y_written ? !out_strides(st ? st->y : nullptr, a->b, a->T, a->D, &a->sy)
                  : !in_strides(st ? st->y : nullptr, a->T, a->D, &a->sy))
        return false;
    *e = MAMBA2_OK;
    return true;
}

bool norm_args(const mamba2_norm_shape* s, const mamba2_norm_strides* st, bool y_written, m2::NormArgs* a,
               mamba2_status* e) {
    *e = MAMBA2_ERR_INVALID_ARG;
    if (!s || !dims(s->batch, s->seqlen, s->channels, s->dtype, e)) return false;
    *e = MAMBA2_ERR_INVALID_ARG;
    if ((s->flags & ~MAMBA2_NORM_GATE_AFTER) || s->groups <= 0 || s->channels % s->groups || !(s->eps >= 0.f))
        return false;
    a->b = s->batch, a->T = s->seqlen, a->D = s->channels, a->G = s->groups, a->eps = s->eps;
    a->dtype = s->dtype == MAMBA2_BF16, a->after = s->flags & MAMBA2_NORM_GATE_AFTER;
    if (!in_strides(st ? st->x : nullptr, a->T, a->D, &a->sx) || !in_strides(st ? st->z : nullptr, a->T, a->D, &a->sz))
        return false;
    if (y_written ? !out_strides(st ? st->y : nullptr, a->b, a->T, a->D, &a->sy)
                  : !in_strides(st ? st->y : nullptr, a->T, a->D, &a->sy))
        return false;
    *e = MAMBA2_OK;
    return true;
}

}  // namespace

extern "C" {

mamba2_status mamba2_conv_fwd(const mamba2_conv_shape* shape, const mamba2_conv_strides* strides, const void* x,
                              const float* w, const float* bias, const void* initial_state,
                              const int32_t* lengths, void* y, void* final_state, void* stream) {
    m2::ConvArgs a;
    mamba2_status e;
    if (!conv_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(x, all, es) || !req(w, a.b * a.D, 4) || !opt(bias, 4) || !opt(initial_state, es) || !opt(lengths, 4) ||
        !req(y, all, es) || !opt(final_state, es))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(m2::launch_conv_fwd(a, x, w, bias, initial_state, lengths, y, final_state,
                                         static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_conv_step(const mamba2_conv_shape* shape, const mamba2_conv_strides* strides, void* state,
                               const void* x, const float* w, const float* bias, void* y, void* stream) {
    m2::ConvArgs a;
    mamba2_status e;
    if (!conv_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.D;
    if (a.T != 1 || !req(state, all, es) || !req(x, all, es) || !req(w, all, 4) || !opt(bias, 4) || !req(y, all, es))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(m2::launch_conv_step(a, state, x, w, bias, y, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_conv_bwd_workspace_size(const mamba2_conv_shape* shape) {
    m2::ConvArgs a;
    mamba2_status e;
    if (!conv_args(shape, nullptr, false, &a, &e)) return 0;
    return sizeof(float) * (size_t)(m2::conv_bwd_slots(a) * a.D * (a.W + 1));
}

mamba2_status mamba2_conv_bwd(const mamba2_conv_shape* shape, const mamba2_conv_strides* strides, const void* x,
                              const float* w, const float* bias, const void* initial_state, const void* dy,
                              const void* dfinal, const int32_t* lengths, void* dx, float* dw, float* dbias,
                              void* dinit, void* workspace, size_t workspace_bytes, void* stream) {
    m2::ConvArgs a;
    mamba2_status e;
    if (!conv_args(shape, strides, false, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(x, all, es) || !req(w, a.b * a.D, 4) || !opt(bias, 4) || !opt(initial_state, es) || !req(dy, all, es) ||
        !opt(dfinal, es) || !opt(lengths, 4) || !req(dx, all, es) || !req(dw, a.D, 4) || !opt(dbias, 4) ||
        !opt(dinit, es))
        return MAMBA2_ERR_INVALID_ARG;
    if (!space(workspace, workspace_bytes, mamba2_conv_bwd_workspace_size(shape))) return MAMBA2_ERR_WORKSPACE;
    return from_cuda(m2::launch_conv_bwd(a, x, w, bias, initial_state, dy, dfinal, lengths, dx, dw, dbias, dinit,
                                         static_cast<float*>(workspace), static_cast<cudaStream_t>(stream)));
}

size_t mamba2_scan_workspace_size(const mamba2_scan_shape* shape) {
    m2::ScanArgs a;
    mamba2_status e;
    return scan_args(shape, nullptr, false, &a, &e) ? m2::scan_fwd_workspace(a) : 0;
}

mamba2_status mamba2_scan_fwd(const mamba2_scan_shape* shape, const mamba2_scan_strides* strides, const void* x,
                              const void* dt, const float* A, const void* B, const void* C, const float* D,
                              const void* z, const float* dt_bias, const float* initial_state,
                              const int32_t* lengths, void* y, float* final_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
    m2::ScanArgs a;
    mamba2_status e;
    if (!scan_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D, bd = a.b * a.D;
    if (!req(x, all, es) || !req(dt, all, es) || !req(A, bd, 4) || !req(B, all, es) || !req(C, all, es) || !opt(D, 4) ||
        !opt(z, es) || !opt(dt_bias, 4) || !opt(initial_state, 4) || !opt(lengths, 4) || !req(y, all, es) ||
        !req(final_state, bd, 4))
        return MAMBA2_ERR_INVALID_ARG;
    if (!space(workspace, workspace_bytes, m2::scan_fwd_workspace(a))) return MAMBA2_ERR_WORKSPACE;
    return from_cuda(m2::launch_scan_fwd(a, x, dt, A, B, C, D, z, dt_bias, initial_state, lengths, y, final_state,
                                         workspace, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_scan_selftest_turn_timeout(const mamba2_scan_shape* shape, const void* x, const void* dt,
                                                const float* A, const void* B, const void* C, void* y,
                                                float* final_state, void* workspace, size_t workspace_bytes,
                                                uint32_t limit_us, void* stream) {
    m2::ScanArgs a;
    mamba2_status e;
    if (!scan_args(shape, nullptr, true, &a, &e)) return e;
    if (limit_us < 1 || limit_us > 100000) return MAMBA2_ERR_INVALID_ARG;
    if (!m2::scan_fwd_turns(a)) return MAMBA2_ERR_UNSUPPORTED;
    const int64_t es = a.dtype ? 2 : 4;
    if (!req(x, 1, es) || !req(dt, 1, es) || !req(A, 1, 4) || !req(B, 1, es) || !req(C, 1, es) || !req(y, 1, es) ||
        !req(final_state, 1, 4))
        return MAMBA2_ERR_INVALID_ARG;
    if (!space(workspace, workspace_bytes, m2::scan_fwd_workspace(a))) return MAMBA2_ERR_WORKSPACE;
    return from_cuda(m2::launch_scan_fwd(a, x, dt, A, B, C, nullptr, nullptr, nullptr, nullptr, nullptr, y, final_state,
                                         workspace, static_cast<cudaStream_t>(stream), (uint64_t)limit_us * 1000));
}

mamba2_status mamba2_scan_step(const mamba2_scan_shape* shape, const mamba2_scan_strides* strides, float* state,
                               const void* x, const void* dt, const float* A, const void* B, const void* C,
                               const float* D, const void* z, const float* dt_bias, void* y, void* stream) {
    m2::ScanArgs a;
    mamba2_status e;
    if (!scan_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, bd = a.b * a.D;
    if (a.T != 1 || !req(state, bd, 4) || !req(x, bd, es) || !req(dt, bd, es) || !req(A, bd, 4) || !req(B, bd, es) ||
        !req(C, bd, es) || !opt(D, 4) || !opt(z, es) || !opt(dt_bias, 4) || !req(y, bd, es))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(m2::launch_scan_step(a, state, x, dt, A, B, C, D, z, dt_bias, y,
                                          static_cast<cudaStream_t>(stream)));
}

size_t mamba2_scan_bwd_workspace_size(const mamba2_scan_shape* shape) {
    m2::ScanArgs a;
    mamba2_status e;
    return scan_args(shape, nullptr, false, &a, &e) ? m2::scan_bwd_workspace(a) : 0;
}

mamba2_status mamba2_scan_bwd(const mamba2_scan_shape* shape, const mamba2_scan_strides* strides, const void* x,
                              const void* dt, const float* A, const void* B, const void* C, const float* D,
                              const void* z, const float* dt_bias, const float* initial_state, const void* dy,
                              const float* dfinal, const int32_t* lengths, void* dx, void* ddt, float* dA, void* dB,
                              void* dC, float* dD, void* dz, float* ddt_bias, float* dinit, void* workspace,
                              size_t workspace_bytes, void* stream) {
    m2::ScanArgs a;
    mamba2_status e;
    if (!scan_args(shape, strides, false, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D, bd = a.b * a.D;
    if (!req(x, all, es) || !req(dt, all, es) || !req(A, bd, 4) || !req(B, all, es) || !req(C, all, es) || !opt(D, 4) ||
        !opt(z, es) || !opt(dt_bias, 4) || !opt(initial_state, 4) || !req(dy, all, es) || !opt(dfinal, 4) ||
        !opt(lengths, 4) || !req(dx, all, es) || !req(ddt, all, es) || !req(dA, a.D, 4) || !req(dB, all, es) ||
        !req(dC, all, es) || !opt(dD, 4) || !opt(dz, es) || !opt(ddt_bias, 4) || !opt(dinit, 4) ||
        (D && !dD && a.D) || (z && !dz && all) || (dt_bias && !ddt_bias && a.D))
        return MAMBA2_ERR_INVALID_ARG;
    if (!space(workspace, workspace_bytes, m2::scan_bwd_workspace(a))) return MAMBA2_ERR_WORKSPACE;
    const m2::ScanGrads g{dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit};
    return from_cuda(m2::launch_scan_bwd(a, x, dt, A, B, C, D, z, dt_bias, initial_state, dy, dfinal, lengths, g,
                                         workspace, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_norm_fwd(const mamba2_norm_shape* shape, const mamba2_norm_strides* strides, const void* x,
                              const float* w, const void* z, void* y, void* stream) {
    m2::NormArgs a;
    mamba2_status e;
    if (!norm_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(x, all, es) || !opt(w, 4) || !opt(z, es) || !req(y, all, es)) return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(m2::launch_norm_fwd(a, x, w, z, y, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_norm_bwd_workspace_size(const mamba2_norm_shape* shape) {
    m2::NormArgs a;
    mamba2_status e;
    if (!norm_args(shape, nullptr, false, &a, &e) || a.b * a.T * a.D == 0) return 0;
    return sizeof(float) * (size_t)(m2::norm_bwd_slots(a) * a.D);
}

mamba2_status mamba2_norm_bwd(const mamba2_norm_shape* shape, const mamba2_norm_strides* strides, const void* x,
                              const float* w, const void* z, const void* dy, void* dx, void* dz, float* dw,
                              void* workspace, size_t workspace_bytes, void* stream) {
    m2::NormArgs a;
    mamba2_status e;
    if (!norm_args(shape, strides, false, &a, &e)) return e;
    const int64_t es = a.dtype ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(x, all, es) || !opt(w, 4) || !opt(z, es) || !req(dy, all, es) || !req(dx, all, es) || !opt(dz, es) ||
        (z && !dz && all) || !opt(dw, 4))
        return MAMBA2_ERR_INVALID_ARG;
    if (dw && !space(workspace, workspace_bytes, mamba2_norm_bwd_workspace_size(shape))) return MAMBA2_ERR_WORKSPACE;
    return from_cuda(m2::launch_norm_bwd(a, x, w, z, dy, dx, dz, dw, static_cast<float*>(workspace),
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
