// call.h -- what every function of the Python binding does with its arguments: torch tensors
// are checked, outputs and workspaces allocated, the caller's stream and the library's status
// taken over.
//
// An output given, a state or a workspace that shares memory with another tensor of the call
// is a ValueError: the kernels read inputs while they write, in no order.
//
// Functions take their arguments by position (layer.py and proj.py have the documented
// signatures) and raise TypeError or ValueError for a tensor that does not fit, and the
// package's Mamba2Error for a status of the library.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
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
    return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32"
           : t == at::kFloat8_e4m3fn ? "torch.float8_e4m3fn" : t == at::kFloat8_e8m0fnu ? "torch.float8_e8m0fnu" : c10::toString(t);
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

    // types: the element types the first input may have.
    Call(PyObject* o, const char* name, std::initializer_list<at::ScalarType> types = {at::kBFloat16, at::kFloat})
        : io(at::kFloat), device(c10::DeviceType::CPU) {
        const Tensor* t = tensor(o, name);
        if (!t) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
        io = t->scalar_type();
        if (std::find(types.begin(), types.end(), io) == types.end())
            raise(PyExc_TypeError, std::string("unsupported element type ") + show(io) + ": " + name + " must be " +
                                       (types.size() > 1 ? "bfloat16 or float32" : show(*types.begin())));
        if (!t->is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (there is no CPU path)");
        device = t->device();
        if (device.index() != c10::cuda::current_device())
            raise(PyExc_ValueError, std::string(name) + " must be on the current CUDA device");
    }
    Call(PyObject* o, const char* name, int64_t rank) : Call(o, name) {
        if (THPVariable_Unpack(o).dim() != rank)
            raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(rank) + " dimensions");
    }
    int32_t dtype() const { return io == at::kBFloat16 ? MAMBA2_BF16 : MAMBA2_F32; }

    void fits(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
        if (t.device() != device)
            raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the same device as the input");
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, std::string(name) + " must be " + show(type) + ", got " + show(t.scalar_type()));
        if (t.sizes() != shape)
            raise(PyExc_ValueError, std::string(name) + " must have shape " + show(shape) + ", got " +
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

}  // namespace
