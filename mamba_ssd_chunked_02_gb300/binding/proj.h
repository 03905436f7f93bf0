// proj.h -- Python binding of include/mamba2_proj.h, part of layer_ext.cpp.
#pragma once

#include "call.h"
#include "mamba2_proj.h"

namespace {

constexpr at::ScalarType kE4M3 = at::kFloat8_e4m3fn, kE8M0 = at::kFloat8_e8m0fnu;

int64_t groups(int64_t n) { return (n + 127) / 128; }

// A tensor of [.., width] in two or three dimensions as {batch, token, width}.
struct Lead {
    int64_t b, T, D;
    bool flat;   // two dimensions: [tokens, width]
};
Lead lead_of(const Tensor& t, const char* name) {
    if (t.dim() != 2 && t.dim() != 3) raise(PyExc_ValueError, std::string(name) + " must have 2 or 3 dimensions");
    if (t.dim() == 2) return {1, t.size(0), t.size(1), true};
    return {t.size(0), t.size(1), t.size(2), false};
}
// The caller's shape of a tensor that is `width` wide.
struct Sizes {
    int64_t n[3];
    int count;
    Sizes(const Lead& l, int64_t width) : n{l.b, l.T, width}, count(3) {
        if (l.flat) n[0] = l.T, n[1] = width, count = 2;
    }
    operator at::IntArrayRef() const { return at::IntArrayRef(n, (size_t)count); }
};

// Address and {batch, token} strides of a tensor [.., width] of type `type`.
void* token_of(const Call& c, PyObject* o, const char* name, at::ScalarType type, const Lead& l, int64_t width, int64_t* st,
               bool optional = false, bool written = false) {
    const Tensor* t = tensor(o, name);
    if (!t) {
        if (optional) return st[0] = st[1] = 0, nullptr;
        raise(PyExc_ValueError, std::string(name) + " is required");
    }
    c.fits(*t, name, type, Sizes(l, width));
    const at::IntArrayRef s = t->strides();
    const size_t k = l.flat ? 0 : 1;
    if (width > 1 && s[k + 1] != 1) raise(PyExc_ValueError, std::string(name) + ": each token's data must be contiguous");
    st[1] = l.T > 1 ? s[k] : width;
    st[0] = !l.flat && l.b > 1 ? s[0] : l.T * st[1];
    if (l.b > 1 && l.T <= 1) st[1] = st[0];   // one token a sequence: the batch's step is the token's
    return c.note(*t, name, written, width, l.b, st[0], l.T, st[1]);
}
// Rows of 8-bit values: addresses and strides in whole 16 bytes.
void* rows16(const Call& c, PyObject* o, const char* name, const Lead& l, int64_t width, int64_t* st, bool written = false) {
    void* p = token_of(c, o, name, kE4M3, l, width, st, false, written);
    if (l.b * l.T > 0 && width > 0 && (reinterpret_cast<uintptr_t>(p) % 16 || (l.b * l.T > 1 && (st[0] % 16 || st[1] % 16))))
        raise(PyExc_ValueError, std::string(name) + ": rows of 8-bit values must start on 16-byte boundaries (quant8 lays them out so)");
    return p;
}
// The distance between a tensor's tokens where it is the same throughout; at least `width`.
int64_t pitch_of(const char* name, const Lead& l, const int64_t* st, int64_t width) {
    if (l.b > 1 && l.T > 0 && st[0] != l.T * st[1]) raise(PyExc_ValueError, std::string(name) + ": tokens must lie at even distances");
    if (l.b * l.T > 1 && st[1] < width) raise(PyExc_ValueError, std::string(name) + ": rows must not overlap each other");
    return st[1];
}
void* scales_of(const Call& c, PyObject* o, const char* name, at::IntArrayRef shape, bool written = false) {
    const Tensor* t = tensor(o, name);
    if (!t) raise(PyExc_ValueError, std::string(name) + " is required");
    c.fits(*t, name, kE8M0, shape);
    if (!t->is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return c.note(*t, name, written, t->numel());
}
Tensor make(const Call& c, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(c.device));
}
Out wrap(Tensor t) {
    Out o;
    o.at = t.data_ptr();
    o.obj = THPVariable_Wrap(std::move(t));
    return o;
}
Out keep(PyObject* given, void* at) {
    Out o;
    Py_INCREF(given);
    o.obj = given;
    o.at = at;
    return o;
}
// A token output, given or new and contiguous.
Out token_new(const Call& c, PyObject* o, const char* name, at::ScalarType type, const Lead& l, int64_t width, int64_t* st) {
    if (given(o)) return keep(o, token_of(c, o, name, type, l, width, st, false, true));
    st[1] = width;
    st[0] = l.T * width;
    return wrap(make(c, Sizes(l, width), type));
}
// 8-bit rows, given or new: a new tensor's rows are padded to 16 bytes.
Out rows_new(const Call& c, PyObject* o, const char* name, const Lead& l, int64_t width, int64_t* st) {
    if (given(o)) return keep(o, rows16(c, o, name, l, width, st, true));
    const int64_t row = (width + 15) / 16 * 16;
    st[1] = row;
    st[0] = l.T * row;
    Tensor t = make(c, Sizes(l, row), kE4M3);
    return wrap(row == width ? std::move(t) : t.narrow(-1, 0, width));
}
Out scales_new(const Call& c, PyObject* o, const char* name, at::IntArrayRef shape) {
    if (given(o)) return keep(o, scales_of(c, o, name, shape, true));
    return wrap(make(c, shape, kE8M0));
}
// The residual's type: its own, or that asked for.
at::ScalarType res_type(const Call& c, PyObject* o, const char* name) {
    const Tensor* t = tensor(o, name);
    if (!t) return c.io;
    const at::ScalarType r = t->scalar_type();
    if (r != at::kFloat && r != c.io)
        raise(PyExc_TypeError, std::string(name) + " must be torch.float32 or of the input's type, got " + show(r));
    return r;
}
int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? MAMBA2_BF16 : MAMBA2_F32; }

// ---- add_norm: (x, residual, w, eps, quant, residual_f32, y, scales, total, stream)
PyObject* add_norm_fwd(Args a) {
    const Call c(a[0], "x");
    const OnStream on(c, a[9]);
    const Lead l = lead_of(THPVariable_Unpack(a[0]), "x");
    const bool quant = truth(a[4]);
    if (!quant && given(a[7])) raise(PyExc_ValueError, "scales are written with quant only");
    at::ScalarType rt =
        given(a[1]) ? res_type(c, a[1], "residual") : given(a[8]) ? res_type(c, a[8], "total") : c.io;
    if (truth(a[5])) {
        if (given(a[1]) && rt != at::kFloat) raise(PyExc_TypeError, "residual must be torch.float32 with residual_f32");
        rt = at::kFloat;
    }
    const mamba2_add_norm_shape sh{l.b, l.T, l.D, real(a[3]), c.dtype(), code(rt), quant ? MAMBA2_ADD_NORM_QUANT : 0};
    mamba2_add_norm_strides st;
    void* px = token_of(c, a[0], "x", c.io, l, l.D, st.x);
    void* pr = token_of(c, a[1], "residual", rt, l, l.D, st.residual, true);
    void* pw = c.dense(a[2], "w", at::kFloat, {l.D}, true);
    Out y = quant ? rows_new(c, a[6], "y", l, l.D, st.y) : token_new(c, a[6], "y", c.io, l, l.D, st.y);
    Out s;
    if (quant) s = scales_new(c, a[7], "scales", Sizes(l, groups(l.D)));
    Out t = token_new(c, a[8], "total", rt, l, l.D, st.total);
    c.distinct();
    check("mamba2_add_norm_fwd",
          mamba2_add_norm_fwd(&sh, &st, px, pr, (float*)pw, y.at, (uint8_t*)s.at, t.at, on.raw));
    if (!quant) return pair(y, t);
    PyObject *p = y.give(), *q = s.give(), *r = t.give(), *all = PyTuple_Pack(3, p, q, r);
    Py_DECREF(p);
    Py_DECREF(q);
    Py_DECREF(r);
    return all;
}

// Entry `name` of the dict of gradients, shaped as the caller's tensors.
void* grad_of(const Call& c, PyObject* out, PyObject* grads, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    PyObject* old = given(grads) ? PyDict_GetItemString(grads, name) : nullptr;   // borrowed
    Out o;
    if (given(old)) {
        const Tensor* t = tensor(old, name);
        c.fits(*t, name, type, shape);
        if (!t->is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
        o = keep(old, c.note(*t, name, true, t->numel()));
    } else {
        o = wrap(make(c, shape, type));
    }
    void* at = o.at;
    PyObject* v = o.give();
    const int rc = PyDict_SetItemString(out, name, v);
    Py_DECREF(v);
    if (rc) throw Raised();
    return at;
}
void set_none(PyObject* out, const char* name) {
    if (PyDict_SetItemString(out, name, Py_None)) throw Raised();
}

// (total, w, dy, dtotal, eps, grads, workspace, stream)
PyObject* add_norm_bwd(Args a) {
    const Call c(a[2], "dy");
    const OnStream on(c, a[7]);
    const Lead l = lead_of(THPVariable_Unpack(a[2]), "dy");
    if (!given(a[0])) raise(PyExc_ValueError, "total is required");
    const at::ScalarType rt = res_type(c, a[0], "total");
    const mamba2_add_norm_shape sh{l.b, l.T, l.D, real(a[4]), c.dtype(), code(rt), 0};
    mamba2_add_norm_strides st;
    st.x[0] = st.x[1] = 0;
    void* pt = token_of(c, a[0], "total", rt, l, l.D, st.total);
    void* pw = c.dense(a[1], "w", at::kFloat, {l.D}, true);
    void* py = token_of(c, a[2], "dy", c.io, l, l.D, st.y);
    void* pe = token_of(c, a[3], "dtotal", rt, l, l.D, st.residual, true);
    Dict g(a[5]);
    void* dx = grad_of(c, g.d, a[5], "dx", c.io, Sizes(l, l.D));
    void* dr = nullptr;
    if (rt != c.io) {
        dr = grad_of(c, g.d, a[5], "dresidual", rt, Sizes(l, l.D));
    } else {   // one tensor serves both
        PyObject* both = PyDict_GetItemString(g.d, "dx");   // borrowed
        PyObject* own = given(a[5]) ? PyDict_GetItemString(a[5], "dresidual") : nullptr;
        if (given(own) && own != both) dr = grad_of(c, g.d, a[5], "dresidual", rt, Sizes(l, l.D));
        else if (PyDict_SetItemString(g.d, "dresidual", both)) throw Raised();
    }
    void* dw = nullptr;
    if (given(a[1])) dw = grad_of(c, g.d, a[5], "dw", at::kFloat, at::IntArrayRef(&l.D, 1));
    else set_none(g.d, "dw");
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[6], dw ? mamba2_add_norm_bwd_workspace_size(&sh) : 0, hold, &bytes);
    c.distinct();
    check("mamba2_add_norm_bwd",
          mamba2_add_norm_bwd(&sh, &st, pt, (float*)pw, py, pe, dx, dr, (float*)dw, ws, bytes, on.raw));
    return g.give();
}

// ---- quant8: (x, block, q, scales, stream)
PyObject* quant8(Args a) {
    const Call c(a[0], "x");
    const OnStream on(c, a[4]);
    const Lead l = lead_of(THPVariable_Unpack(a[0]), "x");
    const bool block = truth(a[1]);
    if (block && !l.flat) raise(PyExc_ValueError, "x must have 2 dimensions for block groups");
    const mamba2_quant8_shape sh{l.b, l.T, l.D, c.dtype(), block ? MAMBA2_QUANT8_BLOCK : 0};
    mamba2_quant8_strides st;
    void* px = token_of(c, a[0], "x", c.io, l, l.D, st.x);
    Out q = rows_new(c, a[2], "q", l, l.D, st.q);
    const int64_t nb[2] = {groups(l.T), groups(l.D)};
    Out s = block ? scales_new(c, a[3], "scales", at::IntArrayRef(nb, 2)) : scales_new(c, a[3], "scales", Sizes(l, groups(l.D)));
    c.distinct();
    check("mamba2_quant8", mamba2_quant8(&sh, &st, px, (uint8_t*)q.at, (uint8_t*)s.at, on.raw));
    return pair(q, s);
}

// ---- proj8
// The operands of both directions: x in row groups, w in block groups.
struct Operands {
    Lead l;
    int64_t N;
    void *x, *xs, *w, *ws;
    mamba2_proj8_pitches p;
    Operands(const Call& c, PyObject* ox, PyObject* oxs, PyObject* ow, PyObject* ows) {
        l = lead_of(THPVariable_Unpack(ox), "x");
        const Tensor* t = tensor(ow, "w");
        if (!t || t->dim() != 2) raise(PyExc_ValueError, "w must be an [outputs, inputs] tensor");
        N = t->size(0);
        int64_t st[2];
        x = rows16(c, ox, "x", l, l.D, st);
        p.x = pitch_of("x", l, st, l.D);
        xs = scales_of(c, oxs, "x_scales", Sizes(l, groups(l.D)));
        const Lead lw{1, N, l.D, true};
        w = rows16(c, ow, "w", lw, l.D, st);
        p.w = pitch_of("w", lw, st, l.D);
        const int64_t nb[2] = {groups(N), groups(l.D)};
        ws = scales_of(c, ows, "w_scales", at::IntArrayRef(nb, 2));
    }
    int64_t tokens() const { return l.b * l.T; }
};

// (x, x_scales, w, w_scales, f32, y, stream)
PyObject* proj8_fwd(Args a) {
    const Call c(a[0], "x", {kE4M3});
    const OnStream on(c, a[6]);
    const Operands o(c, a[0], a[1], a[2], a[3]);
    const at::ScalarType type = truth(a[4]) ? at::kFloat : at::kBFloat16;
    int64_t st[2];
    Out y = token_new(c, a[5], "y", type, o.l, o.N, st);
    mamba2_proj8_pitches p = o.p;
    p.y = pitch_of("y", o.l, st, o.N);
    const mamba2_proj8_shape sh{o.tokens(), o.l.D, o.N, code(type), 0};
    c.distinct();
    check("mamba2_proj8_fwd", mamba2_proj8_fwd(&sh, &p, (uint8_t*)o.x, (uint8_t*)o.xs, (uint8_t*)o.w, (uint8_t*)o.ws, y.at, on.raw));
    return y.give();
}

// (dy, x, x_scales, w, w_scales, need_dx, need_dw, grads, workspace, stream)
PyObject* proj8_bwd(Args a) {
    const Call c(a[0], "dy");
    const OnStream on(c, a[9]);
    if (!tensor(a[1], "x")) raise(PyExc_ValueError, "x is required");
    const Operands o(c, a[1], a[2], a[3], a[4]);
    int64_t st[2];
    void* dy = token_of(c, a[0], "dy", c.io, o.l, o.N, st);
    mamba2_proj8_pitches p = o.p;
    p.y = pitch_of("dy", o.l, st, 0);
    const mamba2_proj8_shape sh{o.tokens(), o.l.D, o.N, c.dtype(), 0};
    Dict g(a[7]);
    void *dx = nullptr, *dw = nullptr;
    if (truth(a[5])) dx = grad_of(c, g.d, a[7], "dx", c.io, Sizes(o.l, o.l.D));
    else set_none(g.d, "dx");
    const int64_t nw[2] = {o.N, o.l.D};
    if (truth(a[6])) dw = grad_of(c, g.d, a[7], "dw", at::kFloat, at::IntArrayRef(nw, 2));
    else set_none(g.d, "dw");
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[8], mamba2_proj8_bwd_workspace_size(&sh), hold, &bytes);
    c.distinct();
    check("mamba2_proj8_bwd", mamba2_proj8_bwd(&sh, &p, dy, (uint8_t*)o.x, (uint8_t*)o.xs, (uint8_t*)o.w, (uint8_t*)o.ws, dx,
                                               (float*)dw, ws, bytes, on.raw));
    return g.give();
}

}  // namespace
