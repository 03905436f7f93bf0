// layer_ext.cpp -- Python binding of include/mamba2_layer.h: checks torch tensors,
// allocates outputs and workspaces, and calls the C ABI on the caller's stream.
//
// An output given, a state or a workspace that shares memory with another tensor of the call
// is a ValueError: the kernels read inputs while they write, in no order.
//
// Native because the single-token calls take 3 us on the GPU: the same checks in
// Python (ctypes) cost 7 to 12 us a call, these about 1.  Every function takes its
// arguments by position (layer.py has the documented signatures) and raises TypeError
// or ValueError for a tensor that does not fit, and the package's Mamba2Error for a
// status of the library.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <utility>

#include "mamba2_layer.h"
#include "overlap.h"

namespace {

using at::Tensor;
typedef std::initializer_list<int64_t> Dims;

PyObject* g_error = nullptr;   // mamba_ssd_chunked_02_gb300.Mamba2Error

// An exception of Python's, thrown through the C++ frames to the entry point.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Raised();
}

std::string show(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const char* show(at::ScalarType t) {
    return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : c10::toString(t);
}

const Tensor* tensor(PyObject* o, const char* name) {
    if (!o || o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return &THPVariable_Unpack(o);
}

// One call's common facts, from its first input.
struct Call {
    at::ScalarType io;
    c10::Device device;
    // The caller's tensors, for distinct(); written: outputs given, a state, a workspace given.
    struct Held {
        const char* name;
        m2::Rows rows;
        int64_t end;
        bool written;
    };
    mutable Held held[24];
    mutable int count = 0;
    mutable bool writes = false;

    Call(PyObject* o, const char* name, int64_t rank) : io(at::kFloat), device(c10::DeviceType::CPU) {
        const Tensor* t = tensor(o, name);
        if (!t) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
        io = t->scalar_type();
        if (io != at::kFloat && io != at::kBFloat16)
            raise(PyExc_TypeError, std::string("unsupported element type ") + show(io) + ": " + name +
                                       " must be bfloat16 or float32");
        if (!t->is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (there is no CPU path)");
        if (t->dim() != rank)
            raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(rank) + " dimensions");
        device = t->device();
        if (device.index() != c10::cuda::current_device())
            raise(PyExc_ValueError, std::string(name) + " must be on the current CUDA device");
    }
    int32_t dtype() const { return io == at::kBFloat16 ? MAMBA2_BF16 : MAMBA2_F32; }

    void fits(const Tensor& t, const char* name, at::ScalarType type, Dims shape) const {
        if (t.device() != device)
            raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the same device as the input");
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, std::string(name) + " must be " + show(type) + ", got " + show(t.scalar_type()));
        if (t.sizes() != at::IntArrayRef(shape))
            raise(PyExc_ValueError, std::string(name) + " must have shape " + show(at::IntArrayRef(shape)) + ", got " +
                                        show(t.sizes()));
    }
    void* note(const Tensor& t, const char* name, bool written, int64_t row, int64_t n0 = 1, int64_t s0 = 0, int64_t n1 = 1,
               int64_t s1 = 0) const {
        void* p = t.data_ptr();
        if (row <= 0 || n0 <= 0 || n1 <= 0) return p;
        if (count == (int)(sizeof(held) / sizeof(*held))) raise(PyExc_SystemError, "more tensors than a call has");
        const int64_t e = (int64_t)t.element_size();
        Held& h = held[count++];
        h.name = name, h.written = written;
        h.rows = {(int64_t)reinterpret_cast<intptr_t>(p), row * e, {n0, n1}, {s0 * e, s1 * e}};
        h.end = h.rows.end();
        writes |= written;
        return p;
    }
    // Refuses a written tensor that shares memory with another of the call.
    void distinct() const {
        if (!writes) return;
        for (int i = 0; i < count; ++i)
            for (int j = 0; j < count && held[i].written; ++j)
                if (j != i && held[i].rows.at < held[j].end && held[j].rows.at < held[i].end &&
                    m2::overlap(held[i].rows, held[j].rows))
                    raise(PyExc_ValueError, std::string(held[i].name) + " must not overlap " + held[j].name);
    }
    // Address of a contiguous tensor; null for an absent optional one.
    void* dense(PyObject* o, const char* name, at::ScalarType type, Dims shape, bool optional = false,
                bool written = false) const {
        const Tensor* t = tensor(o, name);
        if (!t) {
            if (optional) return nullptr;
            raise(PyExc_ValueError, std::string(name) + " is required");
        }
        fits(*t, name, type, shape);
        if (!t->is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
        return note(*t, name, written, t->numel());
    }
    // Address of a token tensor and its {batch, token} strides (lead = 1: batch only).
    void* token(PyObject* o, const char* name, Dims shape, int64_t* st, size_t lead = 2, bool optional = false,
                bool written = false) const {
        const Tensor* t = tensor(o, name);
        if (!t) {
            if (optional) return nullptr;
            raise(PyExc_ValueError, std::string(name) + " is required");
        }
        fits(*t, name, io, shape);
        const at::IntArrayRef s = t->strides();
        const int64_t* n = shape.begin();
        int64_t width = 1;
        for (size_t k = shape.size(); k-- > lead;) {
            if (n[k] != 1 && s[k] != width)
                raise(PyExc_ValueError, std::string(name) + ": each token's data must be contiguous");
            width *= n[k];
        }
        // a dimension of one entry is never stepped over: any stride does
        st[0] = n[0] > 1 ? s[0] : width;
        st[1] = lead == 2 && n[1] > 1 ? s[1] : width;
        return note(*t, name, written, width, n[0], st[0], lead == 2 ? n[1] : 1, st[1]);
    }
    Tensor make(Dims shape, at::ScalarType type) const {
        return at::empty(at::IntArrayRef(shape), at::TensorOptions().dtype(type).device(device));
    }
    // The workspace given, or a new one of `need` bytes kept alive by `hold`.
    void* space(PyObject* o, size_t need, Tensor& hold, size_t* bytes) const {
        if (const Tensor* t = tensor(o, "workspace")) {
            if (t->device() != device || !t->is_contiguous())
                raise(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on the same device as the input");
            *bytes = t->nbytes();
            return note(*t, "workspace", true, t->numel());
        }
        *bytes = need;
        if (!need) return nullptr;
        hold = make({(int64_t)need}, at::kByte);
        return hold.data_ptr();
    }
};

// The stream of a call: the current one, or the one given, which is then the current one
// for what the call allocates (an output or a workspace of another stream's pool could
// still be in use there, or be handed out again before this call is through with it).
struct OnStream {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    void* raw;

    OnStream(const Call& c, PyObject* o) {
        if (!o || o == Py_None) {
            raw = c10::cuda::getCurrentCUDAStream(c.device.index()).stream();
            return;
        }
        PyObject* h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
        if (!h) throw Raised();
        raw = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (PyErr_Occurred()) throw Raised();
        guard.emplace(raw ? c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), c.device.index())
                          : c10::cuda::getDefaultCUDAStream(c.device.index()));
    }
};

void check(const char* fn, mamba2_status rc) {
    if (rc == MAMBA2_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)rc);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

bool truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Raised();
    return t;
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1. && PyErr_Occurred()) throw Raised();
    return (float)v;
}

// A new or given output and its address.
struct Out {
    PyObject* obj = nullptr;   // owned
    void* at = nullptr;
    Out() = default;
    Out(const Out&) = delete;
    Out(Out&& o) noexcept : obj(o.obj), at(o.at) { o.obj = nullptr; }
    Out& operator=(Out&& o) noexcept {
        std::swap(obj, o.obj);
        std::swap(at, o.at);
        return *this;
    }
    ~Out() { Py_XDECREF(obj); }
    PyObject* give() {
        PyObject* o = obj;
        obj = nullptr;
        if (o) return o;
        Py_RETURN_NONE;
    }
};
Out dense_out(const Call& c, PyObject* given, const char* name, at::ScalarType type, Dims shape) {
    Out o;
    if (given && given != Py_None) {
        o.at = c.dense(given, name, type, shape, false, true);
        Py_INCREF(given);
        o.obj = given;
    } else {
        Tensor t = c.make(shape, type);
        o.at = t.data_ptr();
        o.obj = THPVariable_Wrap(std::move(t));
    }
    return o;
}
Out token_out(const Call& c, PyObject* given, const char* name, Dims shape, int64_t* st, size_t lead = 2) {
    if (given && given != Py_None) {
        Out o;
        o.at = c.token(given, name, shape, st, lead, false, true);
        Py_INCREF(given);
        o.obj = given;
        return o;
    }
    Out o = dense_out(c, nullptr, name, c.io, shape);
    const int64_t* n = shape.begin();
    st[1] = n[lead];
    st[0] = lead == 2 ? n[1] * n[2] : n[1];
    return o;
}
// Entry `name` of the dict of gradients: given in `grads` or new; None when not wanted.
void* grad(const Call& c, PyObject* out, PyObject* grads, const char* name, at::ScalarType type, Dims shape,
           bool wanted = true) {
    Out o;
    if (wanted) {
        PyObject* given = nullptr;
        if (grads && grads != Py_None) given = PyDict_GetItemString(grads, name);   // borrowed
        o = dense_out(c, given, name, type, shape);
    }
    void* at = o.at;
    PyObject* v = o.give();
    const int rc = PyDict_SetItemString(out, name, v);
    Py_DECREF(v);
    if (rc) throw Raised();
    return at;
}
struct Dict {
    PyObject* d;
    explicit Dict(PyObject* grads) : d(PyDict_New()) {
        if (!d) throw Raised();
        if (grads && grads != Py_None) {
            if (!PyDict_Check(grads)) raise(PyExc_TypeError, "grads must be a dict");
            if (PyDict_Update(d, grads)) throw Raised();
        }
    }
    Dict(const Dict&) = delete;
    ~Dict() { Py_XDECREF(d); }
    PyObject* give() {
        PyObject* o = d;
        d = nullptr;
        return o;
    }
};
bool given(PyObject* o) { return o && o != Py_None; }

PyObject* pair(Out& a, Out& b) {
    PyObject *x = a.give(), *y = b.give(), *t = PyTuple_Pack(2, x, y);
    Py_DECREF(x);
    Py_DECREF(y);
    return t;
}

// Rows and columns of a parameter [channels, n].
int64_t second_dim(PyObject* o, const char* name, const char* what, int64_t channels) {
    const Tensor* t = tensor(o, name);
    if (!t || t->dim() != 2 || t->size(0) != channels)
        raise(PyExc_ValueError, std::string(name) + " must be a [channels, " + what + "] tensor with " +
                                    std::to_string(channels) + " channels");
    return t->size(1);
}

typedef PyObject* const* Args;

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

template <PyObject* (*F)(Args), Py_ssize_t COUNT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != COUNT) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
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
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "layer_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_layer_ext() { return PyModule_Create(&module); }
