// binding.hpp -- what the Python bindings of the operators beside the layer
// share: checks of tensors, results, the call's device and stream, errors.
#pragma once

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "gdn.h"

namespace gdn_binding {

inline PyObject *error_class = nullptr;  // GDNError(code, where)

// Python's error `type` with `text`, through the entry's HANDLE_TH_ERRORS.
[[noreturn]] inline void raise(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw python_error();
}
[[noreturn]] inline void type_error(const std::string &text) { raise(PyExc_TypeError, text); }
[[noreturn]] inline void value_error(const std::string &text) { raise(PyExc_ValueError, text); }

inline std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The tensor of an argument; null for None where that is allowed.
inline const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

inline int32_t dtype_code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    type_error(std::string(name) + " must be bfloat16 or float32, got " + c10::toString(t.scalar_type()));
}

inline void check_type_and_shape(const at::Tensor &t, const char *name, at::ScalarType type,
                          at::IntArrayRef shape) {
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
                   c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                    shape_text(t.sizes()));
}

inline void check_device(const at::Tensor &t, const char *name, const at::Tensor &first) {
    if (!t.is_cuda() || t.device() != first.device())
        value_error(std::string(name) + " is on " + t.device().str() +
                    ": all tensors of a call must be on one CUDA device");
}

// Checks a token-major tensor, whose rows may be strided; its row stride.
inline int64_t rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
             const at::Tensor &first) {
    check_type_and_shape(t, name, type, shape);
    int64_t width = 1;
    bool whole = true;
    for (size_t i = shape.size(); --i > 0;) {
        whole &= shape[i] == 1 || t.stride(i) == width;
        width *= shape[i];
    }
    if (t.numel() > 0 && !(whole && (shape[0] == 1 || t.stride(0) >= width)))
        value_error(std::string(name) +
                    " must be contiguous within its rows, and its rows must not overlap (shape " +
                    shape_text(shape) + ", strides " + shape_text(t.strides()) + ")");
    check_device(t, name, first);
    return t.numel() > 0 ? t.stride(0) : width;
}

// Checks an optional contiguous tensor; its data.
inline void *data(const at::Tensor *t, const char *name, at::ScalarType type, at::IntArrayRef shape,
           const at::Tensor &first) {
    if (!t) return nullptr;
    check_type_and_shape(*t, name, type, shape);
    if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
    check_device(*t, name, first);
    return t->data_ptr();
}

inline const at::Tensor &with_dims(const at::Tensor &t, const char *name, int64_t dims) {
    if (t.dim() != dims)
        value_error(std::string(name) + " must have " + std::to_string(dims) +
                    " dimensions, got shape " + shape_text(t.sizes()));
    return t;
}

// A size for the C ABI, which refuses those that 32 bits do not hold.
inline int32_t narrow(int64_t v) { return (int32_t)std::min<int64_t>(v, INT32_MAX); }

// The number of sequences of cu_seqlens.
inline int64_t sequences(const at::Tensor &cu) {
    if (cu.size(0) < 1) value_error("cu_seqlens must have at least one element");
    return cu.size(0) - 1;
}

// The taps of a convolution's weight.
inline int64_t taps(const at::Tensor &w) {
    if (w.size(1) < 1) value_error("weight must have at least one tap per channel");
    return w.size(1);
}

// A new tensor beside `first`, without the dispatcher's detour.
inline at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &first) {
    return at::detail::empty_cuda(shape, type, first.device(), std::nullopt);
}

// The device and stream of a call.
struct Call {
    c10::cuda::CUDAGuard guard;
    gdn_stream_t stream;
    explicit Call(const at::Tensor &first)
        : guard(first.device()),
          stream(reinterpret_cast<gdn_stream_t>(
              c10::cuda::getCurrentCUDAStream(first.device().index()).stream())) {}
};

// Python's error for a status, or true.
inline bool fine(gdn_status status, const char *where) {
    if (status == GDN_OK) return true;
    if (PyObject *e = PyObject_CallFunction(error_class, "is", (int)status, where)) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return false;
}

inline PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
inline PyObject *wrap_pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *first = wrap(a);
    PyObject *second = b.defined() ? wrap(b) : Py_NewRef(Py_None);
    PyObject *pair = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return pair;
}

inline void check_count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("wrong number of arguments");
    if (!error_class) raise(PyExc_RuntimeError, "the entry points are not bound");
}

inline bool flag(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
inline int32_t integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return (int32_t)v;
}
inline float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

// The result tensor of an argument that may be None, and its row stride.
inline at::Tensor result(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape,
                  const at::Tensor &first, int64_t *stride) {
    if (const at::Tensor *t = tensor(o, name, true)) {
        *stride = rows(*t, name, type, shape, first);
        return *t;
    }
    *stride = shape[1];
    return make(shape, type, first);
}

}  // namespace gdn_binding
