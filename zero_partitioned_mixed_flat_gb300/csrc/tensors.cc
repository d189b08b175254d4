// tensors.cc -- the calls on torch tensors whose time is the host's (Python module _tensors):
// argument checks, allocations and the libzero call without the interpreter between them.
// gated_linear of one token took 13 us on the host, of which libzero 3.6; a list of 580
// tensors took adamw_step a microsecond each.  What is checked, and the messages, are those of
// head.py; a refusal raises the class that bind() was given.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "zero.h"

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <vector>

namespace {

PyObject *error_class = nullptr;

// raises error_class(code, where, message)
void raise(int code, const char *where, const char *message) {
    PyObject *e = PyObject_CallFunction(error_class, "iss", code, where, message);
    if (!e) return;
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
}

bool refuse(const char *where, const char *fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    raise(ZERO_EINVAL, where, text);
    return false;
}

const char *type_name(at::ScalarType t) { return t == at::kHalf ? "torch.float16" : t == at::kBFloat16 ? "torch.bfloat16" : at::toString(t); }

int lp_of(at::ScalarType t) { return t == at::kHalf ? ZERO_FP16 : t == at::kBFloat16 ? ZERO_BF16 : -1; }
int type_of(at::ScalarType t) { return t == at::kFloat ? ZERO_FP32 : lp_of(t); }

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool here(const at::Tensor &t, long device) { return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == device; }

// A call wrote to the tensor: a backward pass that saved it before has to find out.  (Inference
// tensors have no version.)
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

struct Matrix {
    const at::Tensor *t = nullptr;
    int64_t rows = 0, cols = 0, stride = 0;
    void *at = nullptr;

    // a 2-D tensor with contiguous rows on the device; like: of its type; rows, cols >= 0: of that shape
    bool take(const char *where, const char *name, PyObject *o, long device, const Matrix *like, int64_t want_rows, int64_t want_cols) {
        t = tensor(o);
        if (t && t->requires_grad() && at::GradMode::is_enabled())
            return refuse(where, "%s requires grad, and the call would record no graph: detach it, or call under torch.no_grad()", name);
        if (!t || t->dim() != 2 || lp_of(t->scalar_type()) < 0 || !here(*t, device))
            return refuse(where, "%s must be a 2-D float16 or bfloat16 tensor on the current CUDA device", name);
        if (like && t->scalar_type() != like->t->scalar_type())
            return refuse(where, "%s is %s, expected %s", name, type_name(t->scalar_type()), type_name(like->t->scalar_type()));
        rows = t->size(0);
        cols = t->size(1);
        if ((want_rows >= 0 && rows != want_rows) || (want_cols >= 0 && cols != want_cols))
            return refuse(where, "%s is %lld x %lld, expected %lld x %lld", name, (long long)rows, (long long)cols,
                          (long long)(want_rows >= 0 ? want_rows : rows), (long long)(want_cols >= 0 ? want_cols : cols));
        if (t->stride(1) != 1 && cols > 1) return refuse(where, "%s: the elements of a row must be contiguous", name);
        // the stride of a single row (or of none) says nothing
        stride = rows > 1 ? t->stride(0) : (cols + 7) / 8 * 8;
        at = t->data_ptr();
        return true;
    }
};

// the call's status, raised where it is none
bool called(int status, const char *name) {
    if (status == ZERO_OK) return true;
    raise(status, name, zero_last_error());
    return false;
}

struct Gated {
    Matrix x, gate, up;

    bool take(const char *where, PyObject *const *a, long device) {
        if (!x.take(where, "x", a[0], device, nullptr, -1, -1)) return false;
        // (libzero takes 32 bits of it)
        if (x.cols > ZERO_HEAD_MAX_DIM) return refuse(where, "x has %lld columns, at most %d are allowed", (long long)x.cols, ZERO_HEAD_MAX_DIM);
        return gate.take(where, "gate", a[1], device, &x, -1, x.cols) &&
               up.take(where, "up", a[2], device, &x, gate.rows, x.cols);
    }
};

bool arguments(const char *name, Py_ssize_t have, Py_ssize_t need) {
    if (have == need) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, need);
    return false;
}

// (x, gate, up, act, device, status address, stream) -> out
PyObject *gated_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("gated_forward", n, 7)) return nullptr;
    const long act = PyLong_AsLong(a[3]), device = PyLong_AsLong(a[4]);
    int32_t *status = static_cast<int32_t *>(PyLong_AsVoidPtr(a[5]));
    void *stream = PyLong_AsVoidPtr(a[6]);
    if (PyErr_Occurred()) return nullptr;
    Gated g;
    if (!g.take("gated_linear", a, device)) return nullptr;
    at::Tensor out = at::empty({g.x.rows, g.gate.rows}, g.x.t->options());
    int code;
    Py_BEGIN_ALLOW_THREADS  // (the forward call needs no workspace)
    code = zero_gated_forward(g.x.at, g.x.stride, g.gate.at, g.gate.stride, g.up.at, g.up.stride, (int32_t)act, g.x.rows, g.gate.rows,
                              (int32_t)g.x.cols, (zero_lp)lp_of(g.x.t->scalar_type()), out.data_ptr(), g.gate.rows, status, nullptr, 0, stream);
    Py_END_ALLOW_THREADS
    if (!called(code, "zero_gated_forward")) return nullptr;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// (x, gate, up, act, device, status address, stream, grad_out, grad_x, grad_gate, grad_up) -> the
// three gradients, new where they are None
PyObject *gated_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("gated_backward", n, 11)) return nullptr;
    const char *const where = "gated_linear_backward";
    const long act = PyLong_AsLong(a[3]), device = PyLong_AsLong(a[4]);
    int32_t *status = static_cast<int32_t *>(PyLong_AsVoidPtr(a[5]));
    void *stream = PyLong_AsVoidPtr(a[6]);
    if (PyErr_Occurred()) return nullptr;
    Gated g;
    Matrix grad;
    if (!g.take(where, a, device) || !grad.take(where, "grad_out", a[7], device, &g.x, g.x.rows, g.gate.rows)) return nullptr;
    const char *const names[3] = {"grad_x", "grad_gate", "grad_up"};
    const int64_t rows[3] = {g.x.rows, g.gate.rows, g.gate.rows};
    Matrix given[3];
    for (int i = 0; i < 3; ++i)
        if (a[8 + i] != Py_None && !given[i].take(where, names[i], a[8 + i], device, &g.x, rows[i], g.x.cols)) return nullptr;
    at::Tensor made[3];
    void *at[3];
    int64_t stride[3];
    for (int i = 0; i < 3; ++i) {
        if (!given[i].t) made[i] = at::empty({rows[i], g.x.cols}, g.x.t->options());
        at[i] = given[i].t ? given[i].at : made[i].data_ptr();
        stride[i] = given[i].t ? given[i].stride : g.x.cols;
    }
    int64_t need = 0;
    if (!called(zero_gated_workspace(g.x.rows, g.gate.rows, (int32_t)g.x.cols, nullptr, &need), "zero_gated_workspace")) return nullptr;
    at::Tensor space = at::empty({need}, g.x.t->options().dtype(at::kByte));
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = zero_gated_backward(g.x.at, g.x.stride, g.gate.at, g.gate.stride, g.up.at, g.up.stride, (int32_t)act, grad.at, grad.stride,
                               g.x.rows, g.gate.rows, (int32_t)g.x.cols, (zero_lp)lp_of(g.x.t->scalar_type()), at[0], stride[0], at[1],
                               stride[1], at[2], stride[2], status, space.data_ptr(), need, stream);
    Py_END_ALLOW_THREADS
    if (!called(code, "zero_gated_backward")) return nullptr;
    for (const Matrix &m : given)
        if (m.t) written(*m.t);
    PyObject *out = PyTuple_New(3);
    for (int i = 0; out && i < 3; ++i) {
        PyObject *t = a[8 + i];
        if (given[i].t) Py_INCREF(t);
        else t = THPVariable_Wrap(std::move(made[i]));
        if (!t) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, t);
    }
    return out;
    END_HANDLE_TH_ERRORS
}

// A list of contiguous tensors of one type on the device, which it holds until the call ends: an
// iterator's may be the last there are, and a list may be another thread's, too.
struct List {
    std::vector<int64_t> lens;
    std::vector<void *> at;
    at::ScalarType type = at::kFloat;
    PyObject *held = nullptr;

    List() = default;
    List(const List &) = delete;
    List &operator=(const List &) = delete;
    ~List() { Py_XDECREF(held); }

    void all_written() const {
        for (Py_ssize_t i = 0; held && i < PyTuple_GET_SIZE(held); ++i) written(*tensor(PyTuple_GET_ITEM(held, i)));
    }

    bool take(const char *where, const char *name, PyObject *list, const char *types, bool floats, bool lps, long device) {
        held = PySequence_Tuple(list);
        if (!held) return false;
        const Py_ssize_t n = PyTuple_GET_SIZE(held);
        lens.resize(n);
        at.resize(n);
        bool ok = true;
        for (Py_ssize_t i = 0; ok && i < n; ++i) {
            const at::Tensor *t = tensor(PyTuple_GET_ITEM(held, i));
            ok = t && here(*t, device) && t->is_contiguous() &&
                 (i == 0 ? (floats && t->scalar_type() == at::kFloat) || (lps && lp_of(t->scalar_type()) >= 0) : t->scalar_type() == type);
            if (!ok) break;
            type = t->scalar_type();
            lens[i] = t->numel();
            at[i] = t->data_ptr();
        }
        return ok || refuse(where, "%s must be contiguous tensors of one type (%s) on the current CUDA device", name, types);
    }
};

// one of a state's vectors, or one element that may be None
bool vector_at(const char *where, const char *name, PyObject *o, at::ScalarType type, int64_t n, long device, void **at) {
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != 1 || t->numel() != n || !here(*t, device) || !t->is_contiguous())
        return refuse(where, "the state's %s must be %lld contiguous %s on the current CUDA device", name, (long long)n, at::toString(type));
    *at = t->data_ptr();
    return true;
}

bool one_at(const char *where, const char *name, PyObject *o, at::ScalarType type, long device, void **at) {
    *at = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != type || t->numel() != 1 || !here(*t, device))
        return refuse(where, "%s must be one %s on the current CUDA device", name, at::toString(type));
    *at = t->data_ptr();
    return true;
}

// (params, grads, copies or None, (m, v, m_scales, v_scales, record), lr, beta1, beta2, eps,
// weight_decay, loss_scale, coef or None, skip or None, seed, device, stream)
PyObject *adamw_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("adamw_step", n, 15)) return nullptr;
    const char *const where = "adamw_step";
    double number[6];
    for (int i = 0; i < 6; ++i) number[i] = PyFloat_AsDouble(a[4 + i]);
    const long long seed = PyLong_AsLongLong(a[12]);
    const long device = PyLong_AsLong(a[13]);
    void *stream = PyLong_AsVoidPtr(a[14]);
    if (PyErr_Occurred()) return nullptr;
    if (seed < INT32_MIN || seed > INT32_MAX) {
        refuse(where, "seed outside 32 bits");
        return nullptr;
    }
    List params, grads, copies;
    const bool copied = a[2] != Py_None;
    if (!params.take(where, "params", a[0], "float32", true, false, device) ||
        !grads.take(where, "grads", a[1], "float16, bfloat16 or float32", true, true, device) ||
        (copied && !copies.take(where, "copies", a[2], "float16 or bfloat16", false, true, device)))
        return nullptr;
    if (params.lens.empty() || params.lens.size() > INT32_MAX) {
        refuse(where, params.lens.empty() ? "no parameters" : "more than 2^31 - 1 parameters");
        return nullptr;
    }
    if (grads.lens != params.lens || (copied && copies.lens != params.lens)) {
        refuse(where, "one gradient, and one copy if any, per parameter, each of its parameter's length");
        return nullptr;
    }
    std::vector<void *> seen;
    for (size_t i = 0; i < params.lens.size(); ++i)
        if (params.lens[i] > 0) seen.push_back(params.at[i]);
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) {
        refuse(where, "a parameter is listed twice");
        return nullptr;
    }
    int64_t total = 0;
    for (const int64_t len : params.lens) total += (len + ZERO_QUANT_BLOCK - 1) / ZERO_QUANT_BLOCK * ZERO_QUANT_BLOCK;
    if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 5) {
        refuse(where, "the state must be (m, v, m_scales, v_scales, record)");
        return nullptr;
    }
    PyObject **s = reinterpret_cast<PyTupleObject *>(a[3])->ob_item;
    const at::Tensor *first = tensor(s[0]);
    const bool eight = first && first->scalar_type() == at::kChar;
    void *m, *v, *m_scales = nullptr, *v_scales = nullptr, *record, *coef, *skip;
    if (!vector_at(where, "m", s[0], eight ? at::kChar : at::kFloat, total, device, &m) ||
        !vector_at(where, "v", s[1], eight ? at::kByte : at::kFloat, total, device, &v) ||
        (eight && (!vector_at(where, "m_scales", s[2], at::kFloat, total / ZERO_QUANT_BLOCK, device, &m_scales) ||
                   !vector_at(where, "v_scales", s[3], at::kFloat, total / ZERO_QUANT_BLOCK, device, &v_scales))) ||
        !vector_at(where, "record", s[4], at::kLong, 2, device, &record) || !one_at(where, "coef", a[10], at::kFloat, device, &coef) ||
        !one_at(where, "skip", a[11], at::kInt, device, &skip))
        return nullptr;
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = zero_adamw_step((int32_t)params.lens.size(), reinterpret_cast<float *const *>(params.at.data()), grads.at.data(),
                           type_of(grads.type), copied ? copies.at.data() : nullptr, (zero_lp)(copied ? lp_of(copies.type) : ZERO_BF16),
                           params.lens.data(), eight ? ZERO_MOMENTS_8BIT : ZERO_MOMENTS_FP32, m, v, static_cast<float *>(m_scales),
                           static_cast<float *>(v_scales), static_cast<int64_t *>(record), number[0], number[1], number[2], number[3],
                           number[4], (float)number[5], static_cast<const float *>(coef), static_cast<const int32_t *>(skip), (int32_t)seed,
                           stream);
    Py_END_ALLOW_THREADS
    if (!called(code, "zero_adamw_step")) return nullptr;
    params.all_written();
    copies.all_written();
    for (int i = 0; i < 5; ++i)
        if (i < 2 || i == 4 || eight) written(*tensor(s[i]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// the class of the errors: called with (status, where, message)
PyObject *bind(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F *f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"gated_forward", fast(gated_forward), METH_FASTCALL, nullptr},
                         {"gated_backward", fast(gated_backward), METH_FASTCALL, nullptr},
                         {"adamw_step", fast(adamw_step), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
