// block_binding.cpp -- Python binding of the block operators (the C ABI of
// include/gdn_block.h) for PyTorch tensors.
//
// A single token's operator runs for a few microseconds, less than an
// interpreter takes to look over ten tensors: this module checks the tensors'
// types, shapes, strides and devices, allocates results, and calls the C entry
// points on the current stream.  It holds no kernel and no state but the entry
// points' addresses, which the Python module takes from libgdn and hands to
// bind() with its error class.
#include "binding.hpp"
#include "gdn_block.h"

using namespace gdn_binding;

extern PyMethodDef attention_methods[];  // attention_binding.cpp

namespace {

decltype(&gdn_short_conv) short_conv_entry = nullptr;
decltype(&gdn_short_conv_step) short_conv_step_entry = nullptr;
decltype(&gdn_selective_scan) scan_entry = nullptr;
decltype(&gdn_selective_scan_step) scan_step_entry = nullptr;
decltype(&gdn_selective_scan_workspace_size) scan_workspace_entry = nullptr;
decltype(&gdn_norm_gate_residual) norm_entry = nullptr;

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

PyMODINIT_FUNC PyInit_gdn_block_binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, attention_methods) < 0) Py_CLEAR(m);
    return m;
}
