// block_binding.cpp -- Python binding of the block operators (the C ABI of
// include/gdn_block.h) for PyTorch tensors.
//
// A single token's operator runs for a few microseconds, less than an
// interpreter takes to look over ten tensors: this module checks the tensors'
// types, shapes, strides and devices, allocates results, and calls the C entry
// points on the current stream.  It holds no kernel and no state but the entry
// points' addresses, which the Python module takes from libgdn and hands to
// bind() with its error class.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>

#include "gdn_block.h"

namespace {

decltype(&gdn_short_conv) short_conv_entry = nullptr;
decltype(&gdn_short_conv_step) short_conv_step_entry = nullptr;
decltype(&gdn_selective_scan) scan_entry = nullptr;
decltype(&gdn_selective_scan_step) scan_step_entry = nullptr;
decltype(&gdn_selective_scan_workspace_size) scan_workspace_entry = nullptr;
decltype(&gdn_norm_gate_residual) norm_entry = nullptr;
PyObject *error_class = nullptr;  // GDNError(code, where)

// Python's error `type` with `text`, through the entry's HANDLE_TH_ERRORS.
[[noreturn]] void raise(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw python_error();
}
[[noreturn]] void type_error(const std::string &text) { raise(PyExc_TypeError, text); }
[[noreturn]] void value_error(const std::string &text) { raise(PyExc_ValueError, text); }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The tensor of an argument; null for None where that is allowed.
const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

int32_t dtype_code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    type_error(std::string(name) + " must be bfloat16 or float32, got " + c10::toString(t.scalar_type()));
}

void check_type_and_shape(const at::Tensor &t, const char *name, at::ScalarType type,
                          at::IntArrayRef shape) {
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
                   c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                    shape_text(t.sizes()));
}

void check_device(const at::Tensor &t, const char *name, const at::Tensor &first) {
    if (!t.is_cuda() || t.device() != first.device())
        value_error(std::string(name) + " is on " + t.device().str() +
                    ": all tensors of a call must be on one CUDA device");
}

// Checks a token-major tensor, whose rows may be strided; its row stride.
int64_t rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
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
void *data(const at::Tensor *t, const char *name, at::ScalarType type, at::IntArrayRef shape,
           const at::Tensor &first) {
    if (!t) return nullptr;
    check_type_and_shape(*t, name, type, shape);
    if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
    check_device(*t, name, first);
    return t->data_ptr();
}

const at::Tensor &with_dims(const at::Tensor &t, const char *name, int64_t dims) {
    if (t.dim() != dims)
        value_error(std::string(name) + " must have " + std::to_string(dims) +
                    " dimensions, got shape " + shape_text(t.sizes()));
    return t;
}

// A size for the C ABI, which refuses those that 32 bits do not hold.
int32_t narrow(int64_t v) { return (int32_t)std::min<int64_t>(v, INT32_MAX); }

// The number of sequences of cu_seqlens.
int64_t sequences(const at::Tensor &cu) {
    if (cu.size(0) < 1) value_error("cu_seqlens must have at least one element");
    return cu.size(0) - 1;
}

// The taps of a convolution's weight.
int64_t taps(const at::Tensor &w) {
    if (w.size(1) < 1) value_error("weight must have at least one tap per channel");
    return w.size(1);
}

// A new tensor beside `first`, without the dispatcher's detour.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &first) {
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
bool fine(gdn_status status, const char *where) {
    if (status == GDN_OK) return true;
    if (PyObject *e = PyObject_CallFunction(error_class, "is", (int)status, where)) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return false;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap_pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *first = wrap(a);
    PyObject *second = b.defined() ? wrap(b) : Py_NewRef(Py_None);
    PyObject *pair = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return pair;
}

void check_count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("wrong number of arguments");
    if (!error_class) raise(PyExc_RuntimeError, "the entry points are not bound");
}

bool flag(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
int32_t integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return (int32_t)v;
}
float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

// The result tensor of an argument that may be None, and its row stride.
at::Tensor result(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape,
                  const at::Tensor &first, int64_t *stride) {
    if (const at::Tensor *t = tensor(o, name, true)) {
        *stride = rows(*t, name, type, shape, first);
        return *t;
    }
    *stride = shape[1];
    return make(shape, type, first);
}

// x, weight, cu_seqlens, bias, initial_state, activation, out, final_state, want_final
PyObject *short_conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 9);
    const at::Tensor &x = with_dims(*tensor(a[0], "x"), "x", 2);
    const at::Tensor &w = with_dims(*tensor(a[1], "weight"), "weight", 2);
    const at::Tensor &cu = with_dims(*tensor(a[2], "cu_seqlens"), "cu_seqlens", 1);
    const auto type = x.scalar_type();
    const int64_t T = x.size(0), C = x.size(1), K = taps(w), N = sequences(cu);
    gdn_conv_problem p{};
    p.dtype = dtype_code(x, "x");
    p.x_stride = rows(x, "x", type, x.sizes(), x);
    p.num_seqs = narrow(N);
    p.total_tokens = T;
    p.channels = narrow(C);
    p.width = narrow(K);
    p.activation = integer(a[5]);
    const int64_t state[3] = {N, K - 1, C};
    const void *weight = data(&w, "weight", at::kFloat, {C, K}, x);
    const void *bias = data(tensor(a[3], "bias", true), "bias", at::kFloat, {C}, x);
    const void *lens = data(&cu, "cu_seqlens", at::kInt, {N + 1}, x);
    const void *init = data(tensor(a[4], "initial_state", true), "initial_state", type, state, x);
    const at::Tensor *given = tensor(a[7], "final_state", true);
    void *fin = data(given, "final_state", type, state, x);
    const Call call(x);
    const at::Tensor out = result(a[6], "out", type, {T, C}, x, &p.out_stride);
    at::Tensor final_state;
    if (given) {
        final_state = *given;
    } else if (flag(a[8])) {
        final_state = make(state, type, x);
        fin = final_state.data_ptr();
    }
    if (!fine(short_conv_entry(&p, x.data_ptr(), static_cast<const float *>(weight),
                               static_cast<const float *>(bias),
                               static_cast<const int32_t *>(lens), init, out.data_ptr(), fin,
                               call.stream),
              "gdn_short_conv"))
        return nullptr;
    return wrap_pair(out, final_state);
    END_HANDLE_TH_ERRORS
}

// x, weight, state, bias, activation, out, new_state
PyObject *short_conv_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 7);
    const at::Tensor &x = with_dims(*tensor(a[0], "x"), "x", 2);
    const at::Tensor &w = with_dims(*tensor(a[1], "weight"), "weight", 2);
    const auto type = x.scalar_type();
    const int64_t N = x.size(0), C = x.size(1), K = taps(w);
    gdn_conv_problem p{};
    p.dtype = dtype_code(x, "x");
    p.x_stride = rows(x, "x", type, x.sizes(), x);
    p.num_seqs = narrow(N);
    p.total_tokens = N;
    p.channels = narrow(C);
    p.width = narrow(K);
    p.activation = integer(a[4]);
    const int64_t state[3] = {N, K - 1, C};
    const void *weight = data(&w, "weight", at::kFloat, {C, K}, x);
    void *old = data(tensor(a[2], "state"), "state", type, state, x);
    const void *bias = data(tensor(a[3], "bias", true), "bias", at::kFloat, {C}, x);
    const at::Tensor *given = tensor(a[6], "new_state", true);
    void *fresh = given ? data(given, "new_state", type, state, x) : old;
    const Call call(x);
    const at::Tensor out = result(a[5], "out", type, {N, C}, x, &p.out_stride);
    if (!fine(short_conv_step_entry(&p, x.data_ptr(), static_cast<const float *>(weight),
                                    static_cast<const float *>(bias), old, out.data_ptr(), fresh,
                                    call.stream),
              "gdn_short_conv_step"))
        return nullptr;
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// What the scan and its step share: x, dt, A, B, C of a[0 .. 4], D, z,
// dt_bias, softplus from a[s].
struct Scan {
    gdn_ssm_problem p{};
    const at::Tensor &x;
    const at::Tensor *z;
    const void *dt, *B, *C;
    const float *A, *D, *bias;
    int64_t states;
    Scan(PyObject *const *a, int s) : x(with_dims(*tensor(a[0], "x"), "x", 2)) {
        const at::Tensor &d = *tensor(a[1], "dt"), &b = with_dims(*tensor(a[3], "B"), "B", 3),
                         &c = *tensor(a[4], "C");
        const auto type = x.scalar_type();
        const int64_t T = x.size(0), ch = x.size(1), G = b.size(1), S = b.size(2);
        states = S;
        p.dtype = dtype_code(x, "x");
        p.total_tokens = T;
        p.channels = narrow(ch);
        p.num_groups = narrow(G);
        p.state_dim = narrow(S);
        p.dt_softplus = flag(a[s + 3]);
        p.x_stride = rows(x, "x", type, {T, ch}, x);
        p.dt_stride = rows(d, "dt", type, {T, ch}, x);
        p.b_stride = rows(b, "B", type, {T, G, S}, x);
        p.c_stride = rows(c, "C", type, {T, G, S}, x);
        z = tensor(a[s + 1], "z", true);
        if (z) p.z_stride = rows(*z, "z", type, {T, ch}, x);
        dt = d.data_ptr();
        B = b.data_ptr();
        C = c.data_ptr();
        A = static_cast<const float *>(data(tensor(a[2], "A"), "A", at::kFloat, {ch, S}, x));
        D = static_cast<const float *>(data(tensor(a[s], "D", true), "D", at::kFloat, {ch}, x));
        bias = static_cast<const float *>(
            data(tensor(a[s + 2], "dt_bias", true), "dt_bias", at::kFloat, {ch}, x));
    }
    const void *gate() const { return z ? z->data_ptr() : nullptr; }
};

// x, dt, A, B, C, cu_seqlens, D, z, dt_bias, softplus, initial_state, out,
// final_state, want_final, workspace
PyObject *selective_scan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 15);
    Scan s(a, 6);
    const at::Tensor &x = s.x, &cu = with_dims(*tensor(a[5], "cu_seqlens"), "cu_seqlens", 1);
    const int64_t N = sequences(cu), T = x.size(0), ch = x.size(1);
    s.p.num_seqs = narrow(N);
    const int64_t state[3] = {N, ch, s.states};
    const void *lens = data(&cu, "cu_seqlens", at::kInt, {N + 1}, x);
    const void *init =
        data(tensor(a[10], "initial_state", true), "initial_state", at::kFloat, state, x);
    const at::Tensor *given = tensor(a[12], "final_state", true);
    void *fin = data(given, "final_state", at::kFloat, state, x);
    const at::Tensor *scratch = tensor(a[14], "workspace", true);
    const Call call(x);
    const at::Tensor out = result(a[11], "out", x.scalar_type(), {T, ch}, x, &s.p.out_stride);
    at::Tensor final_state, own;
    if (given) {
        final_state = *given;
    } else if (flag(a[13])) {
        final_state = make(state, at::kFloat, x);
        fin = final_state.data_ptr();
    }
    if (scratch) {
        if (!scratch->is_contiguous()) value_error("workspace must be contiguous");
        check_device(*scratch, "workspace", x);
        s.p.workspace = scratch->data_ptr();
        s.p.workspace_bytes = scratch->nbytes();
    } else if (const size_t need = scan_workspace_entry(&s.p)) {
        // From the caching allocator, for this stream.
        own = make({(int64_t)need}, at::kByte, x);
        s.p.workspace = own.data_ptr();
        s.p.workspace_bytes = need;
    }
    if (!fine(scan_entry(&s.p, x.data_ptr(), s.dt, s.A, s.B, s.C, s.D, s.gate(), s.bias,
                         static_cast<const int32_t *>(lens), static_cast<const float *>(init),
                         out.data_ptr(), static_cast<float *>(fin), call.stream),
              "gdn_selective_scan"))
        return nullptr;
    return wrap_pair(out, final_state);
    END_HANDLE_TH_ERRORS
}

// x, dt, A, B, C, state, D, z, dt_bias, softplus, out, new_state
PyObject *selective_scan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 12);
    Scan s(a, 6);
    const at::Tensor &x = s.x;
    const int64_t N = x.size(0), ch = x.size(1);
    s.p.num_seqs = narrow(N);
    const int64_t state[3] = {N, ch, s.states};
    void *old = data(tensor(a[5], "state"), "state", at::kFloat, state, x);
    const at::Tensor *given = tensor(a[11], "new_state", true);
    void *fresh = given ? data(given, "new_state", at::kFloat, state, x) : old;
    const Call call(x);
    const at::Tensor out = result(a[10], "out", x.scalar_type(), {N, ch}, x, &s.p.out_stride);
    if (!fine(scan_step_entry(&s.p, x.data_ptr(), s.dt, s.A, s.B, s.C, s.D, s.gate(), s.bias,
                              static_cast<const float *>(old), out.data_ptr(),
                              static_cast<float *>(fresh), call.stream),
              "gdn_selective_scan_step"))
        return nullptr;
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// y, weight, gate, residual, next_weight, activation, gate_first, scale, eps, out, next_out
PyObject *norm_gate_residual(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 11);
    const at::Tensor &y = with_dims(*tensor(a[0], "y"), "y", 2);
    const at::Tensor *w = tensor(a[1], "weight", true), *g = tensor(a[2], "gate", true),
                     *r = tensor(a[3], "residual", true),
                     *nw = tensor(a[4], "next_weight", true), *o = tensor(a[9], "out", true),
                     *no = tensor(a[10], "next_out", true);
    const auto type = y.scalar_type();
    const int64_t R = y.size(0), D = y.size(1);
    const at::Tensor &like = r ? *r : o ? *o : y;
    gdn_norm_problem p{};
    p.rows = R;
    p.dim = narrow(D);
    p.dtype = dtype_code(y, "y");
    p.residual_dtype = dtype_code(like, r ? "residual" : "out");
    p.activation = integer(a[5]);
    p.gate_first = flag(a[6]);
    p.scale = number(a[7]);
    p.eps = number(a[8]);
    p.y_stride = rows(y, "y", type, {R, D}, y);
    if (g) p.gate_stride = rows(*g, "gate", type, {R, D}, y);
    if (r) p.residual_stride = rows(*r, "residual", like.scalar_type(), {R, D}, y);
    const void *weight = data(w, "weight", at::kFloat, {D}, y);
    const void *next_weight = data(nw, "next_weight", at::kFloat, {D}, y);
    if (no && !nw) value_error("next_out without next_weight");
    const Call call(y);
    const at::Tensor out = result(a[9], "out", like.scalar_type(), {R, D}, y, &p.out_stride);
    at::Tensor next;
    if (nw) next = result(a[10], "next_out", type, {R, D}, y, &p.next_stride);
    if (!fine(norm_entry(&p, y.data_ptr(), static_cast<const float *>(weight),
                         g ? g->data_ptr() : nullptr, r ? r->data_ptr() : nullptr,
                         static_cast<const float *>(next_weight), out.data_ptr(),
                         nw ? next.data_ptr() : nullptr, call.stream),
              "gdn_norm_gate_residual"))
        return nullptr;
    return wrap_pair(out, next);
    END_HANDLE_TH_ERRORS
}

// GDNError, then the six entry points' addresses in the order below.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) type_error("wrong number of arguments");
    void *at[6];
    for (int i = 0; i < 6; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (PyErr_Occurred()) throw python_error();
        if (!at[i]) value_error("an entry point's address is null");
    }
    short_conv_entry = reinterpret_cast<decltype(short_conv_entry)>(at[0]);
    short_conv_step_entry = reinterpret_cast<decltype(short_conv_step_entry)>(at[1]);
    scan_entry = reinterpret_cast<decltype(scan_entry)>(at[2]);
    scan_step_entry = reinterpret_cast<decltype(scan_step_entry)>(at[3]);
    scan_workspace_entry = reinterpret_cast<decltype(scan_workspace_entry)>(at[4]);
    norm_entry = reinterpret_cast<decltype(norm_entry)>(at[5]);
    Py_XSETREF(error_class, Py_NewRef(a[0]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"short_conv", (PyCFunction)(void (*)(void))short_conv, METH_FASTCALL, nullptr},
    {"short_conv_step", (PyCFunction)(void (*)(void))short_conv_step, METH_FASTCALL, nullptr},
    {"selective_scan", (PyCFunction)(void (*)(void))selective_scan, METH_FASTCALL, nullptr},
    {"selective_scan_step", (PyCFunction)(void (*)(void))selective_scan_step, METH_FASTCALL,
     nullptr},
    {"norm_gate_residual", (PyCFunction)(void (*)(void))norm_gate_residual, METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_block_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_block_binding() { return PyModule_Create(&module); }
