// layer_ext.cpp -- Python binding of include/mamba2_layer.h and include/mamba2_proj.h (proj.h).
//
// Native because the single-token calls take 3 us on the GPU: the same checks in
// Python (ctypes) cost 7 to 12 us a call, these about 1.
#include "call.h"
#include "proj.h"

namespace {

// A width as the C ABI takes it; one beyond 32 bits stays one that is refused.
int32_t width32(int64_t w) { return w > INT32_MAX ? INT32_MAX : (int32_t)w; }

// ---- conv: (x, w, bias, initial_state, lengths, silu, y, final_state, stream)
PyObject* conv_fwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[8]);
    const Tensor& x = THPVariable_Unpack(a[0]);
    const int64_t b = x.size(0), T = x.size(1), D = x.size(2), W = second_dim(a[1], "w", "width", D);
    const mamba2_conv_shape sh{b, T, D, width32(W), c.dtype(), truth(a[5]) ? MAMBA2_CONV_SILU : 0};
    mamba2_conv_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pw = c.dense(a[1], "w", at::kFloat, {D, W});
    void* pb = c.dense(a[2], "bias", at::kFloat, {D}, true);
    void* pi = c.dense(a[3], "initial_state", c.io, {b, W - 1, D}, true);
    void* pl = c.dense(a[4], "lengths", at::kInt, {b}, true);
    Out y = token_out(c, a[6], "y", {b, T, D}, st.y);
    Out f = dense_out(c, a[7], "final_state", c.io, {b, W > 0 ? W - 1 : 0, D});
    c.distinct();
    check("mamba2_conv_fwd", mamba2_conv_fwd(&sh, &st, px, (float*)pw, (float*)pb, pi, (int32_t*)pl, y.at, f.at,
                                             on.raw));
    return pair(y, f);
}

// (state, x, w, bias, silu, y, stream)
PyObject* conv_step(Args a) {
    const Call c(a[1], "x", 2);
    const OnStream on(c, a[6]);
    const Tensor& x = THPVariable_Unpack(a[1]);
    const int64_t b = x.size(0), D = x.size(1), W = second_dim(a[2], "w", "width", D);
    const mamba2_conv_shape sh{b, 1, D, width32(W), c.dtype(), truth(a[4]) ? MAMBA2_CONV_SILU : 0};
    mamba2_conv_strides st;
    void* ps = c.dense(a[0], "state", c.io, {b, W - 1, D}, false, true);
    void* px = c.token(a[1], "x", {b, D}, st.x, 1);
    void* pw = c.dense(a[2], "w", at::kFloat, {D, W});
    void* pb = c.dense(a[3], "bias", at::kFloat, {D}, true);
    Out y = token_out(c, a[5], "y", {b, D}, st.y, 1);
    c.distinct();
    check("mamba2_conv_step",
          mamba2_conv_step(&sh, &st, ps, px, (float*)pw, (float*)pb, y.at, on.raw));
    return y.give();
}

// (x, w, bias, initial_state, dy, dfinal, lengths, silu, grads, workspace, stream)
PyObject* conv_bwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[10]);
    const Tensor& x = THPVariable_Unpack(a[0]);
    const int64_t b = x.size(0), T = x.size(1), D = x.size(2), W = second_dim(a[1], "w", "width", D);
    const mamba2_conv_shape sh{b, T, D, width32(W), c.dtype(), truth(a[7]) ? MAMBA2_CONV_SILU : 0};
    mamba2_conv_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pw = c.dense(a[1], "w", at::kFloat, {D, W});
    void* pb = c.dense(a[2], "bias", at::kFloat, {D}, true);
    void* pi = c.dense(a[3], "initial_state", c.io, {b, W - 1, D}, true);
    void* py = c.token(a[4], "dy", {b, T, D}, st.y);
    void* pf = c.dense(a[5], "dfinal", c.io, {b, W - 1, D}, true);
    void* pl = c.dense(a[6], "lengths", at::kInt, {b}, true);
    Dict g(a[8]);
    void* dx = grad(c, g.d, a[8], "dx", c.io, {b, T, D});
    void* dw = grad(c, g.d, a[8], "dw", at::kFloat, {D, W});
    void* db = grad(c, g.d, a[8], "dbias", at::kFloat, {D}, given(a[2]));
    void* di = grad(c, g.d, a[8], "dinit", c.io, {b, W > 0 ? W - 1 : 0, D}, given(a[3]));
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[9], mamba2_conv_bwd_workspace_size(&sh), hold, &bytes);
    c.distinct();
    check("mamba2_conv_bwd", mamba2_conv_bwd(&sh, &st, px, (float*)pw, (float*)pb, pi, py, pf, (int32_t*)pl, dx, (float*)dw,
                                             (float*)db, di, ws, bytes, on.raw));
    return g.give();
}

// ---- scan
struct ScanCall {
    int64_t b, T, D, N, G;
    mamba2_scan_shape sh;
};
ScanCall scan_call(const Call& c, const Tensor& x, PyObject* A, PyObject* B, bool step, bool softplus) {
    ScanCall s;
    s.b = x.size(0);
    s.T = step ? 1 : x.size(1);
    s.D = x.size(step ? 1 : 2);
    s.N = second_dim(A, "A", "states", s.D);
    const Tensor* t = tensor(B, "B");
    if (!t || t->dim() != (step ? 3 : 4)) raise(PyExc_ValueError, "B must be a [.., groups, states] tensor");
    s.G = t->size(t->dim() - 2);
    s.sh = mamba2_scan_shape{s.b, s.T, s.D, s.N, s.G, c.dtype(), softplus ? MAMBA2_SCAN_SOFTPLUS : 0};
    return s;
}

// (x, dt, A, B, C, D, z, dt_bias, initial_state, lengths, dt_softplus, y, final_state, workspace, stream)
PyObject* scan_fwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[14]);
    const ScanCall s = scan_call(c, THPVariable_Unpack(a[0]), a[2], a[3], false, truth(a[10]));
    const int64_t b = s.b, T = s.T, D = s.D, N = s.N, G = s.G;
    mamba2_scan_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pt = c.token(a[1], "dt", {b, T, D}, st.dt);
    void* pA = c.dense(a[2], "A", at::kFloat, {D, N});
    void* pB = c.token(a[3], "B", {b, T, G, N}, st.B);
    void* pC = c.token(a[4], "C", {b, T, G, N}, st.C);
    void* pD = c.dense(a[5], "D", at::kFloat, {D}, true);
    st.z[0] = st.z[1] = 0;
    void* pz = c.token(a[6], "z", {b, T, D}, st.z, 2, true);
    void* pb = c.dense(a[7], "dt_bias", at::kFloat, {D}, true);
    void* pi = c.dense(a[8], "initial_state", at::kFloat, {b, D, N}, true);
    void* pl = c.dense(a[9], "lengths", at::kInt, {b}, true);
    Out y = token_out(c, a[11], "y", {b, T, D}, st.y);
    Out f = dense_out(c, a[12], "final_state", at::kFloat, {b, D, N});
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[13], mamba2_scan_workspace_size(&s.sh), hold, &bytes);
    c.distinct();
    check("mamba2_scan_fwd",
          mamba2_scan_fwd(&s.sh, &st, px, pt, (float*)pA, pB, pC, (float*)pD, pz, (float*)pb, (float*)pi, (int32_t*)pl,
                          y.at, (float*)f.at, ws, bytes, on.raw));
    return pair(y, f);
}

// (state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, y, stream)
PyObject* scan_step(Args a) {
    const Call c(a[1], "x", 2);
    const OnStream on(c, a[11]);
    const ScanCall s = scan_call(c, THPVariable_Unpack(a[1]), a[3], a[4], true, truth(a[9]));
    const int64_t b = s.b, D = s.D, N = s.N, G = s.G;
    mamba2_scan_strides st;
    void* ps = c.dense(a[0], "state", at::kFloat, {b, D, N}, false, true);
    void* px = c.token(a[1], "x", {b, D}, st.x, 1);
    void* pt = c.token(a[2], "dt", {b, D}, st.dt, 1);
    void* pA = c.dense(a[3], "A", at::kFloat, {D, N});
    void* pB = c.token(a[4], "B", {b, G, N}, st.B, 1);
    void* pC = c.token(a[5], "C", {b, G, N}, st.C, 1);
    void* pD = c.dense(a[6], "D", at::kFloat, {D}, true);
    st.z[0] = st.z[1] = 0;
    void* pz = c.token(a[7], "z", {b, D}, st.z, 1, true);
    void* pb = c.dense(a[8], "dt_bias", at::kFloat, {D}, true);
    Out y = token_out(c, a[10], "y", {b, D}, st.y, 1);
    c.distinct();
    check("mamba2_scan_step", mamba2_scan_step(&s.sh, &st, (float*)ps, px, pt, (float*)pA, pB, pC, (float*)pD, pz,
                                               (float*)pb, y.at, on.raw));
    return y.give();
}

// (x, dt, A, B, C, D, z, dt_bias, initial_state, dy, dfinal, lengths, dt_softplus, grads, workspace, stream)
PyObject* scan_bwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[15]);
    const ScanCall s = scan_call(c, THPVariable_Unpack(a[0]), a[2], a[3], false, truth(a[12]));
    const int64_t b = s.b, T = s.T, D = s.D, N = s.N, G = s.G;
    mamba2_scan_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pt = c.token(a[1], "dt", {b, T, D}, st.dt);
    void* pA = c.dense(a[2], "A", at::kFloat, {D, N});
    void* pB = c.token(a[3], "B", {b, T, G, N}, st.B);
    void* pC = c.token(a[4], "C", {b, T, G, N}, st.C);
    void* pD = c.dense(a[5], "D", at::kFloat, {D}, true);
    st.z[0] = st.z[1] = 0;
    void* pz = c.token(a[6], "z", {b, T, D}, st.z, 2, true);
    void* pb = c.dense(a[7], "dt_bias", at::kFloat, {D}, true);
    void* pi = c.dense(a[8], "initial_state", at::kFloat, {b, D, N}, true);
    void* py = c.token(a[9], "dy", {b, T, D}, st.y);
    void* pf = c.dense(a[10], "dfinal", at::kFloat, {b, D, N}, true);
    void* pl = c.dense(a[11], "lengths", at::kInt, {b}, true);
    Dict g(a[13]);
    PyObject* in = a[13];
    void* dx = grad(c, g.d, in, "dx", c.io, {b, T, D});
    void* ddt = grad(c, g.d, in, "ddt", c.io, {b, T, D});
    void* dA = grad(c, g.d, in, "dA", at::kFloat, {D, N});
    void* dB = grad(c, g.d, in, "dB", c.io, {b, T, G, N});
    void* dC = grad(c, g.d, in, "dC", c.io, {b, T, G, N});
    void* dD = grad(c, g.d, in, "dD", at::kFloat, {D}, given(a[5]));
    void* dz = grad(c, g.d, in, "dz", c.io, {b, T, D}, given(a[6]));
    void* db = grad(c, g.d, in, "ddt_bias", at::kFloat, {D}, given(a[7]));
    void* di = grad(c, g.d, in, "dinit", at::kFloat, {b, D, N}, given(a[8]));
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[14], mamba2_scan_bwd_workspace_size(&s.sh), hold, &bytes);
    c.distinct();
    check("mamba2_scan_bwd",
          mamba2_scan_bwd(&s.sh, &st, px, pt, (float*)pA, pB, pC, (float*)pD, pz, (float*)pb, (float*)pi, py, (float*)pf,
                          (int32_t*)pl, dx, ddt, (float*)dA, dB, dC, (float*)dD, dz, (float*)db, (float*)di, ws, bytes,
                          on.raw));
    return g.give();
}

// ---- norm: (x, w, z, ngroups, eps, gate_first, y, stream)
PyObject* norm_fwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[7]);
    const Tensor& x = THPVariable_Unpack(a[0]);
    const int64_t b = x.size(0), T = x.size(1), D = x.size(2);
    const mamba2_norm_shape sh{b, T, D, whole(a[3]), real(a[4]), c.dtype(), truth(a[5]) ? 0 : MAMBA2_NORM_GATE_AFTER};
    mamba2_norm_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pw = c.dense(a[1], "w", at::kFloat, {D}, true);
    st.z[0] = st.z[1] = 0;
    void* pz = c.token(a[2], "z", {b, T, D}, st.z, 2, true);
    Out y = token_out(c, a[6], "y", {b, T, D}, st.y);
    c.distinct();
    check("mamba2_norm_fwd", mamba2_norm_fwd(&sh, &st, px, (float*)pw, pz, y.at, on.raw));
    return y.give();
}

// (x, w, z, dy, ngroups, eps, gate_first, grads, workspace, stream)
PyObject* norm_bwd(Args a) {
    const Call c(a[0], "x", 3);
    const OnStream on(c, a[9]);
    const Tensor& x = THPVariable_Unpack(a[0]);
    const int64_t b = x.size(0), T = x.size(1), D = x.size(2);
    const mamba2_norm_shape sh{b, T, D, whole(a[4]), real(a[5]), c.dtype(), truth(a[6]) ? 0 : MAMBA2_NORM_GATE_AFTER};
    mamba2_norm_strides st;
    void* px = c.token(a[0], "x", {b, T, D}, st.x);
    void* pw = c.dense(a[1], "w", at::kFloat, {D}, true);
    st.z[0] = st.z[1] = 0;
    void* pz = c.token(a[2], "z", {b, T, D}, st.z, 2, true);
    void* py = c.token(a[3], "dy", {b, T, D}, st.y);
    Dict g(a[7]);
    void* dx = grad(c, g.d, a[7], "dx", c.io, {b, T, D});
    void* dz = grad(c, g.d, a[7], "dz", c.io, {b, T, D}, given(a[2]));
    void* dw = grad(c, g.d, a[7], "dw", at::kFloat, {D}, given(a[1]));
    Tensor hold;
    size_t bytes;
    void* ws = c.space(a[8], mamba2_norm_bwd_workspace_size(&sh), hold, &bytes);
    c.distinct();
    check("mamba2_norm_bwd", mamba2_norm_bwd(&sh, &st, px, (float*)pw, pz, py, dx, dz, (float*)dw, ws, bytes,
                                             on.raw));
    return g.give();
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define ENTRY(name, count) \
    { #name, (PyCFunction)(void (*)(void))entry<name, count>, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(conv_fwd, 9),  ENTRY(conv_step, 7), ENTRY(conv_bwd, 11), ENTRY(scan_fwd, 15),
                         ENTRY(scan_step, 12), ENTRY(scan_bwd, 16), ENTRY(norm_fwd, 8),  ENTRY(norm_bwd, 10),
                         ENTRY(add_norm_fwd, 10), ENTRY(add_norm_bwd, 8), ENTRY(quant8, 5), ENTRY(proj8_fwd, 7),
                         ENTRY(proj8_bwd, 10),
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "layer_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_layer_ext() { return PyModule_Create(&module); }
