// proj_api.cu -- the C ABI declared in include/mamba2_proj.h: argument validation, and the
// backward product's sequence of launches.  Nothing is launched before every argument has
// been checked.
#include <cuda_runtime.h>
#include <stdint.h>

#include "check.h"
#include "mamba2_proj.h"
#include "proj.cuh"

namespace {

using namespace m2;

constexpr int64_t kMaxSide = int64_t(1) << 30;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t groups(int64_t n) { return (n + kGroup - 1) / kGroup; }

// Rows of e4m3 values start on 16-byte boundaries.
bool rows16(const void* p, const Tok& s, int64_t b, int64_t T) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (b <= 1 || s.b % 16 == 0) && (T <= 1 || s.t % 16 == 0);
}

bool norm_args(const mamba2_add_norm_shape* s, const mamba2_add_norm_strides* st, bool back, AddNormArgs* a,
               mamba2_status* e) {
    *e = MAMBA2_ERR_INVALID_ARG;
    if (!s || !dims(s->batch, s->seqlen, s->channels, s->dtype, e)) return false;
    *e = MAMBA2_ERR_INVALID_ARG;
    if ((s->flags & ~MAMBA2_ADD_NORM_QUANT) || !(s->eps >= 0.f) ||
        (s->res_dtype != MAMBA2_F32 && s->res_dtype != MAMBA2_BF16))
        return false;
    if (s->res_dtype == MAMBA2_BF16 && s->dtype != MAMBA2_BF16) {
        *e = MAMBA2_ERR_UNSUPPORTED;
        return false;
    }
    a->b = s->batch, a->T = s->seqlen, a->D = s->channels, a->eps = s->eps;
    a->bf16 = s->dtype == MAMBA2_BF16, a->res_bf16 = s->res_dtype == MAMBA2_BF16;
    a->quant = !back && (s->flags & MAMBA2_ADD_NORM_QUANT);
    const int64_t q_row = up(a->D, 16), q_strides[2] = {a->T * q_row, q_row};
    const int64_t* sy = st ? st->y : a->quant ? q_strides : nullptr;
    a->sx = Tok{0, 0};
    if ((!back && !in_strides(st ? st->x : nullptr, a->T, a->D, &a->sx)) ||
        !in_strides(st ? st->residual : nullptr, a->T, a->D, &a->sres))
        return false;
    if (back ? !in_strides(sy, a->T, a->D, &a->sy) || !in_strides(st ? st->total : nullptr, a->T, a->D, &a->st)
             : !out_strides(sy, a->b, a->T, a->D, &a->sy) || !out_strides(st ? st->total : nullptr, a->b, a->T, a->D, &a->st))
        return false;
    *e = MAMBA2_OK;
    return true;
}

struct Proj {
    int64_t M, K, N, px, pw, py;
    bool bf16;
};

// back: the pitch of y is that of dy, whose rows are read and may lie in one another.
bool proj_args(const mamba2_proj8_shape* s, const mamba2_proj8_pitches* p, bool back, Proj* a, mamba2_status* e) {
    *e = MAMBA2_ERR_INVALID_ARG;
    if (!s || s->tokens < 0 || s->inputs < 0 || s->outputs < 0 || s->flags ||
        (s->dtype != MAMBA2_F32 && s->dtype != MAMBA2_BF16))
        return false;
    *e = MAMBA2_ERR_UNSUPPORTED;
    if (s->tokens > kMaxSide || s->inputs > kMaxSide || s->outputs > kMaxSide || s->inputs == 0) return false;
    a->M = s->tokens, a->K = s->inputs, a->N = s->outputs, a->bf16 = s->dtype == MAMBA2_BF16;
    a->px = p ? p->x : up(a->K, 16), a->pw = p ? p->w : up(a->K, 16), a->py = p ? p->y : a->N;
    *e = MAMBA2_ERR_INVALID_ARG;
    // a single row's pitch is not used, but the copies' maps want one that could be
    if (a->M <= 1) a->px = up(a->K, 16), a->py = a->N;
    if (a->N <= 1) a->pw = up(a->K, 16);
    if (a->px < a->K || a->pw < a->K || a->py < (back ? 0 : a->N) || a->px % 16 || a->pw % 16 || a->px >= kMaxStride ||
        a->pw >= kMaxStride || a->py >= kMaxStride)
        return false;
    *e = MAMBA2_OK;
    return true;
}

cudaError_t forward(const Proj& a, const uint8_t* x, const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales,
                    void* y, cudaStream_t st, const Proj8Watch& watch) {
    const int64_t kb = groups(a.K);
    const Operand W{w, a.pw, false, w_scales, kb, 1, 7}, X{x, a.px, false, x_scales, kb, 1, 0};
    return launch_proj8(X, W, a.M, a.N, a.K, y, a.py, a.bf16, st, watch);
}

// The backward product's workspace.
size_t work_of(const Proj& a, void* base, Quant8Operands* w) {
    w->pn = up(a.N, 128), w->pk = up(a.K, 128), w->ps = up(groups(a.N), 4);
    size_t at = 0;
    const auto take = [&](int64_t n) {
        uint8_t* p = static_cast<uint8_t*>(base) + at;
        at += (size_t)up(n, 256);
        return p;
    };
    w->dyr = take(a.M * w->pn), w->sr = take(a.M * w->ps);
    w->dyc = take(a.M * w->pn), w->sc = take(groups(a.M) * a.N);
    w->xc = take(a.M * w->pk), w->sx = take(groups(a.M) * a.K);
    return at;
}

}  // namespace

extern "C" {

mamba2_status mamba2_add_norm_fwd(const mamba2_add_norm_shape* shape, const mamba2_add_norm_strides* strides,
                                  const void* x, const void* residual, const float* w, void* y, uint8_t* scales,
                                  void* total, void* stream) {
    AddNormArgs a;
    mamba2_status e;
    if (!norm_args(shape, strides, false, &a, &e)) return e;
    const int64_t es = a.bf16 ? 2 : 4, rs = a.res_bf16 ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(x, all, es) || !opt(residual, rs) || !opt(w, 4) || !req(y, all, a.quant ? 1 : es) ||
        !req(total, all, rs) || (a.quant ? !req(scales, all, 1) : scales != nullptr) ||
        (a.quant && all && !rows16(y, a.sy, a.b, a.T)))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(launch_add_norm_fwd(a, x, residual, w, y, scales, total, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_add_norm_bwd_workspace_size(const mamba2_add_norm_shape* shape) {
    AddNormArgs a;
    mamba2_status e;
    if (!norm_args(shape, nullptr, true, &a, &e) || a.b * a.T * a.D == 0) return 0;
    return sizeof(float) * (size_t)(add_norm_bwd_slots(a) * a.D);
}

mamba2_status mamba2_add_norm_bwd(const mamba2_add_norm_shape* shape, const mamba2_add_norm_strides* strides,
                                  const void* total, const float* w, const void* dy, const void* dtotal, void* dx,
                                  void* dresidual, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    AddNormArgs a;
    mamba2_status e;
    if (!norm_args(shape, strides, true, &a, &e)) return e;
    const int64_t es = a.bf16 ? 2 : 4, rs = a.res_bf16 ? 2 : 4, all = a.b * a.T * a.D;
    if (!req(total, all, rs) || !opt(w, 4) || !req(dy, all, es) || !opt(dtotal, rs) || !req(dx, all, es) ||
        !opt(dresidual, rs) || !opt(dw, 4))
        return MAMBA2_ERR_INVALID_ARG;
    if (dw && !space(workspace, workspace_bytes, mamba2_add_norm_bwd_workspace_size(shape))) return MAMBA2_ERR_WORKSPACE;
    return from_cuda(launch_add_norm_bwd(a, total, w, dy, dtotal, dx, dresidual, dw, static_cast<float*>(workspace),
                                         static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_quant8(const mamba2_quant8_shape* shape, const mamba2_quant8_strides* strides, const void* x,
                            uint8_t* q, uint8_t* scales, void* stream) {
    Quant8Args a;
    mamba2_status e;
    if (!shape || !dims(shape->batch, shape->seqlen, shape->channels, shape->dtype, &e))
        return shape ? e : MAMBA2_ERR_INVALID_ARG;
    a.b = shape->batch, a.T = shape->seqlen, a.D = shape->channels, a.bf16 = shape->dtype == MAMBA2_BF16;
    a.block = shape->flags & MAMBA2_QUANT8_BLOCK;
    const int64_t row = up(a.D, 16), sq[2] = {a.T * row, row}, es = a.bf16 ? 2 : 4, all = a.b * a.T * a.D;
    if ((shape->flags & ~MAMBA2_QUANT8_BLOCK) || (a.block && a.b != 1) ||
        !in_strides(strides ? strides->x : nullptr, a.T, a.D, &a.sx) ||
        !out_strides(strides ? strides->q : sq, a.b, a.T, a.D, &a.sq) || !req(x, all, es) || !req(q, all, 1) ||
        !req(scales, all, 1) || (all && !rows16(q, a.sq, a.b, a.T)))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(launch_quant8(a, x, q, scales, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_proj8_fwd(const mamba2_proj8_shape* shape, const mamba2_proj8_pitches* pitches, const uint8_t* x,
                               const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales, void* y,
                               void* stream) {
    Proj a;
    mamba2_status e;
    if (!proj_args(shape, pitches, false, &a, &e)) return e;
    const int64_t all = a.M * a.N;
    if (!req(x, all, 16) || !req(x_scales, all, 1) || !req(w, all, 16) || !req(w_scales, all, 1) ||
        !req(y, all, a.bf16 ? 2 : 4))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(forward(a, x, x_scales, w, w_scales, y, static_cast<cudaStream_t>(stream), Proj8Watch{}));
}

mamba2_status mamba2_proj8_selftest_timeout(const mamba2_proj8_shape* shape, const uint8_t* x, const uint8_t* x_scales,
                                            const uint8_t* w, const uint8_t* w_scales, void* y, uint32_t limit_us,
                                            void* stream) {
    Proj a;
    mamba2_status e;
    if (!proj_args(shape, nullptr, false, &a, &e)) return e;
    if (limit_us < 1 || limit_us > 100000 || a.M == 0 || a.N == 0 || !req(x, 1, 16) || !req(x_scales, 1, 1) ||
        !req(w, 1, 16) || !req(w_scales, 1, 1) || !req(y, 1, a.bf16 ? 2 : 4))
        return MAMBA2_ERR_INVALID_ARG;
    return from_cuda(forward(a, x, x_scales, w, w_scales, y, static_cast<cudaStream_t>(stream),
                             Proj8Watch{(uint64_t)limit_us * 1000, true}));
}

size_t mamba2_proj8_bwd_workspace_size(const mamba2_proj8_shape* shape) {
    Proj a;
    mamba2_status e;
    if (!proj_args(shape, nullptr, true, &a, &e) || a.M == 0 || a.N == 0) return 0;
    Quant8Operands w;
    return work_of(a, nullptr, &w);
}

mamba2_status mamba2_proj8_bwd(const mamba2_proj8_shape* shape, const mamba2_proj8_pitches* pitches, const void* dy,
                               const uint8_t* x, const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales,
                               void* dx, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    Proj a;
    mamba2_status e;
    if (!proj_args(shape, pitches, true, &a, &e)) return e;
    const int64_t all = a.M * a.N, es = a.bf16 ? 2 : 4;
    if (!req(dy, all, es) || !req(x, all, 16) || !req(x_scales, all, 1) || !req(w, all, 16) || !req(w_scales, all, 1) ||
        !opt(dx, es) || !opt(dw, 4))
        return MAMBA2_ERR_INVALID_ARG;
    if (!space(workspace, workspace_bytes, mamba2_proj8_bwd_workspace_size(shape), 256)) return MAMBA2_ERR_WORKSPACE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (all == 0) {   // sums of nothing
        cudaError_t c = cudaSuccess;
        if (dx && a.M) c = cudaMemsetAsync(dx, 0, (size_t)(a.M * a.K * es), st);
        if (c == cudaSuccess && dw && a.N) c = cudaMemsetAsync(dw, 0, (size_t)(a.N * a.K * 4), st);
        return from_cuda(c);
    }
    if (!dx && !dw) return MAMBA2_OK;
    Quant8Operands k;
    work_of(a, workspace, &k);
    const int64_t kb = groups(a.K);
    bool turned;
    cudaError_t c = launch_quant8_operands(a.bf16, a.M, a.N, a.K, dy, a.py, x, a.px, x_scales, k, dx, dw, &turned, st);
    if (c == cudaSuccess && dx) {
        const Operand W{w, a.pw, true, w_scales, 1, kb, 7}, D{k.dyr, k.pn, false, k.sr, k.ps, 1, 0};
        c = launch_proj8(D, W, a.M, a.K, a.N, dx, a.K, a.bf16, st);
    }
    if (c == cudaSuccess && dw) {
        if (!turned) c = launch_quant8_turn(a.M, a.K, x, a.px, x_scales, k, st);
        const Operand X{k.xc, k.pk, true, k.sx, 1, a.K, 0}, D{k.dyc, k.pn, true, k.sc, 1, a.N, 0};
        if (c == cudaSuccess) c = launch_proj8(D, X, a.N, a.K, a.M, dw, a.K, false, st);
    }
    return from_cuda(c);
}

}  // extern "C"
