// attention_binding.cpp -- Python binding of the attention operators (the C ABI
// of include/gdn_attention.h), functions of block_binding.cpp's module.
#include "binding.hpp"
#include "gdn_attention.h"

using namespace gdn_binding;

namespace {

decltype(&gdn_qk_norm_rope) rope_entry = nullptr;
decltype(&gdn_paged_append) append_entry = nullptr;
decltype(&gdn_paged_attention) attention_entry = nullptr;
decltype(&gdn_paged_attention_workspace_size) attention_workspace_entry = nullptr;

constexpr int kMostPairs = 256;  // of rotated elements in a head

struct Strides {
    int64_t token = 0, head = 0;
};

// Checks a tensor [..., heads, D] whose heads are contiguous.
void heads(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
           const at::Tensor &first) {
    check_type_and_shape(t, name, type, shape);
    if (t.numel() > 0 && t.size(-1) > 1 && t.stride(-1) != 1)
        value_error(std::string(name) + " must be contiguous within its heads (shape " +
                    shape_text(t.sizes()) + ", strides " + shape_text(t.strides()) + ")");
    check_device(t, name, first);
}
Strides heads3(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
               const at::Tensor &first) {
    heads(t, name, type, shape, first);
    return {t.stride(0), t.stride(1)};
}
// [N, L, heads, D] or [N, heads, D] as tokens one after the other.
Strides heads4(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
               const at::Tensor &first) {
    heads(t, name, type, shape, first);
    if (t.dim() == 3) return {t.stride(0), t.stride(1)};
    if (t.size(1) == 1) return {t.stride(0), t.stride(2)};
    if (t.size(0) > 1 && t.stride(0) != t.size(1) * t.stride(1))
        value_error(std::string(name) + " must have its sequences' tokens one after the other "
                    "(shape " + shape_text(t.sizes()) + ", strides " + shape_text(t.strides()) + ")");
    return {t.stride(1), t.stride(2)};
}

const float *floats(PyObject *o, const char *name, int64_t n, const at::Tensor &first) {
    return static_cast<const float *>(data(tensor(o, name, true), name, at::kFloat, {n}, first));
}

// positions, inv_freq, axes, interleaved, eps of a[0 .. 4].
struct Rotation {
    const int32_t *positions = nullptr;
    const float *inv_freq = nullptr;
    uint8_t axis[kMostPairs];
    Rotation(PyObject *const *a, gdn_rope_problem &p, const at::Tensor &first) {
        const at::Tensor *f = tensor(a[1], "inv_freq", true);
        const at::Tensor *pos = tensor(a[0], "positions", true);
        p.num_axes = 1;
        p.interleaved = flag(a[3]);
        p.eps = number(a[4]);
        if (f) {
            const int64_t pairs = with_dims(*f, "inv_freq", 1).size(0);
            inv_freq = floats(a[1], "inv_freq", pairs, first);
            p.rotary_dim = narrow(2 * std::min<int64_t>(pairs, INT32_MAX / 4));
            if (p.rotary_dim > p.head_dim) value_error("inv_freq has more pairs than a head");
            if (pairs == 0) inv_freq = nullptr;
        }
        if (pos) {
            if (pos->dim() == 2)
                p.num_axes = narrow(pos->size(0));
            else if (pos->dim() != 1)
                value_error("positions must have 1 or 2 dimensions, got shape " +
                            shape_text(pos->sizes()));
            if (pos->dim() == 2)
                check_type_and_shape(*pos, "positions", at::kInt, {pos->size(0), p.total_tokens});
            else
                check_type_and_shape(*pos, "positions", at::kInt, {p.total_tokens});
            if (pos->numel() > 1 && pos->size(-1) > 1 && pos->stride(-1) != 1)
                value_error("positions must be contiguous within its axes");
            check_device(*pos, "positions", first);
            p.axis_stride = pos->dim() == 2 ? pos->stride(0) : p.total_tokens;
            positions = static_cast<const int32_t *>(pos->data_ptr());
        }
        if (a[2] == Py_None) {
            if (p.num_axes > 1) value_error("positions of several axes need axes");
            return;
        }
        PyObject *seq = PySequence_Fast(a[2], "axes must be a sequence of integers");
        if (!seq) throw python_error();
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        bool good = n == p.rotary_dim / 2 && n <= kMostPairs, error = false;
        for (Py_ssize_t i = 0; good && i < n; ++i) {
            const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
            error = v == -1 && PyErr_Occurred();
            good = !error && v >= 0 && v < p.num_axes && v < 256;
            if (good) axis[i] = (uint8_t)v;
        }
        Py_DECREF(seq);
        if (error) throw python_error();
        if (!good) value_error("axes must name one of positions' axes for each pair of inv_freq");
        p.freq_axis = axis;
    }
};

// q, k, positions, inv_freq, axes, interleaved, eps, q_weight, k_weight, q_out, k_out
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 11);
    const at::Tensor *q = tensor(a[0], "q", true), *k = tensor(a[1], "k", true);
    if (!q && !k) value_error("q or k must be given");
    const at::Tensor &first = q ? with_dims(*q, "q", 3) : with_dims(*k, "k", 3);
    if (k) with_dims(*k, "k", 3);
    const auto type = first.scalar_type();
    const int64_t T = first.size(0), D = first.size(2), Hq = q ? q->size(1) : 0,
                  Hk = k ? k->size(1) : 0;
    gdn_rope_problem p{};
    p.total_tokens = T;
    p.q_heads = narrow(Hq);
    p.kv_heads = narrow(Hk);
    p.head_dim = narrow(D);
    p.dtype = dtype_code(first, q ? "q" : "k");
    Strides s;
    if (q) {
        s = heads3(*q, "q", type, {T, Hq, D}, first);
        p.q_stride = s.token, p.q_head_stride = s.head;
    }
    if (k) {
        s = heads3(*k, "k", type, {T, Hk, D}, first);
        p.k_stride = s.token, p.k_head_stride = s.head;
    }
    const Rotation turn(a + 2, p, first);
    const float *qw = floats(a[7], "q_weight", D, first), *kw = floats(a[8], "k_weight", D, first);
    const at::Tensor *qo = tensor(a[9], "q_out", true), *ko = tensor(a[10], "k_out", true);
    if ((qo && !q) || (ko && !k)) value_error("a result without its input");
    const Call call(first);
    at::Tensor q_out, k_out;
    if (q) {
        q_out = qo ? *qo : make({T, Hq, D}, type, first);
        s = heads3(q_out, "q_out", type, {T, Hq, D}, first);
        p.q_out_stride = s.token, p.q_out_head_stride = s.head;
    }
    if (k) {
        k_out = ko ? *ko : make({T, Hk, D}, type, first);
        s = heads3(k_out, "k_out", type, {T, Hk, D}, first);
        p.k_out_stride = s.token, p.k_out_head_stride = s.head;
    }
    if (!fine(rope_entry(&p, q && Hq ? q->data_ptr() : nullptr, k && Hk ? k->data_ptr() : nullptr, qw,
                         kw, turn.positions, turn.inv_freq, q && Hq ? q_out.data_ptr() : nullptr,
                         k && Hk ? k_out.data_ptr() : nullptr, call.stream),
              "gdn_qk_norm_rope"))
        return nullptr;
    PyObject *x = q ? wrap(q_out) : Py_NewRef(Py_None), *y = k ? wrap(k_out) : Py_NewRef(Py_None);
    PyObject *pair = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return pair;
    END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, page_table, seq_lens, k_scale, v_scale of a[0 .. 5].
struct Cache {
    gdn_paged_cache c{};
    int64_t N;
    Cache(PyObject *const *a, int64_t Hkv, int64_t D, const at::Tensor &first) {
        const at::Tensor &k = with_dims(*tensor(a[0], "k_cache"), "k_cache", 4),
                         &v = *tensor(a[1], "v_cache"),
                         &table = with_dims(*tensor(a[2], "page_table"), "page_table", 2);
        const auto type = k.scalar_type();
        if (type == at::kFloat8_e4m3fn)
            c.dtype = GDN_E4M3;
        else if (type == at::kBFloat16 || type == at::kFloat)
            c.dtype = dtype_code(k, "k_cache");
        else
            type_error(std::string("k_cache must be bfloat16, float32 or float8_e4m3fn, got ") +
                       c10::toString(type));
        if (c.dtype != GDN_E4M3 && type != first.scalar_type())
            type_error(std::string("k_cache must have the inputs' type or be float8_e4m3fn, got ") +
                       c10::toString(type));
        const int64_t P = k.size(0), S = k.size(1);
        heads(k, "k_cache", type, {P, S, Hkv, D}, first);
        heads(v, "v_cache", type, {P, S, Hkv, D}, first);
        N = table.size(0);
        check_type_and_shape(table, "page_table", at::kInt, {N, table.size(1)});
        if (table.numel() > 0 && table.size(1) > 1 && table.stride(1) != 1)
            value_error("page_table must be contiguous within its rows");
        check_device(table, "page_table", first);
        c.k = k.data_ptr(), c.v = v.data_ptr();
        c.num_pages = P;
        c.page_size = narrow(S);
        c.k_page_stride = k.stride(0), c.k_token_stride = k.stride(1), c.k_head_stride = k.stride(2);
        c.v_page_stride = v.stride(0), c.v_token_stride = v.stride(1), c.v_head_stride = v.stride(2);
        c.num_seqs = narrow(N);
        c.max_pages = narrow(table.size(1));
        c.page_table = static_cast<const int32_t *>(table.data_ptr());
        c.table_stride = table.stride(0);
        c.seq_lens = static_cast<const int32_t *>(
            data(tensor(a[3], "seq_lens"), "seq_lens", at::kInt, {N}, first));
        c.k_scale = floats(a[4], "k_scale", Hkv, first);
        c.v_scale = floats(a[5], "v_scale", Hkv, first);
        if ((c.dtype == GDN_E4M3) != (c.k_scale && c.v_scale) ||
            (c.k_scale != nullptr) != (c.v_scale != nullptr))
            value_error("k_scale and v_scale belong to a float8_e4m3fn cache");
    }
};

// k, v, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, positions,
// inv_freq, axes, interleaved, eps, cu_seqlens, q, q_weight, k_weight, q_out
PyObject *paged_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 18);
    const at::Tensor &k = with_dims(*tensor(a[0], "k"), "k", 3), &v = *tensor(a[1], "v");
    const at::Tensor *q = tensor(a[14], "q", true), *qo = tensor(a[17], "q_out", true),
                     *cu = tensor(a[13], "cu_seqlens", true);
    const auto type = k.scalar_type();
    const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2),
                  Hq = q ? with_dims(*q, "q", 3).size(1) : 0;
    gdn_rope_problem p{};
    p.total_tokens = T;
    p.q_heads = narrow(Hq);
    p.kv_heads = narrow(Hkv);
    p.head_dim = narrow(D);
    p.dtype = dtype_code(k, "k");
    Strides s = heads3(k, "k", type, {T, Hkv, D}, k);
    p.k_stride = s.token, p.k_head_stride = s.head;
    s = heads3(v, "v", type, {T, Hkv, D}, k);
    p.v_stride = s.token, p.v_head_stride = s.head;
    if (q) {
        s = heads3(*q, "q", type, {T, Hq, D}, k);
        p.q_stride = s.token, p.q_head_stride = s.head;
    } else if (qo) {
        value_error("q_out without q");
    }
    const Cache cache(a + 2, Hkv, D, k);
    const Rotation turn(a + 8, p, k);
    const float *qw = floats(a[15], "q_weight", D, k), *kw = floats(a[16], "k_weight", D, k);
    const void *lens = data(cu, "cu_seqlens", at::kInt, {cache.N + 1}, k);
    const Call call(k);
    at::Tensor q_out;
    if (q) {
        q_out = qo ? *qo : make({T, Hq, D}, type, k);
        s = heads3(q_out, "q_out", type, {T, Hq, D}, k);
        p.q_out_stride = s.token, p.q_out_head_stride = s.head;
    }
    if (!fine(append_entry(&p, &cache.c, q && Hq ? q->data_ptr() : nullptr, k.data_ptr(),
                           v.data_ptr(), qw, kw, turn.positions, turn.inv_freq,
                           static_cast<const int32_t *>(lens),
                           q && Hq ? q_out.data_ptr() : nullptr, call.stream),
              "gdn_paged_append"))
        return nullptr;
    return q ? wrap(q_out) : Py_NewRef(Py_None);
    END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, scale, gate,
// out, lse, want_lse, workspace
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 13);
    const at::Tensor &q = *tensor(a[0], "q");
    if (q.dim() != 3 && q.dim() != 4)
        value_error("q must have 3 or 4 dimensions, got shape " + shape_text(q.sizes()));
    const at::Tensor &k = with_dims(*tensor(a[1], "k_cache"), "k_cache", 4);
    const at::Tensor *gate = tensor(a[8], "gate", true), *given = tensor(a[9], "out", true),
                     *stats = tensor(a[10], "lse", true), *scratch = tensor(a[12], "workspace", true);
    const auto type = q.scalar_type();
    const int64_t D = q.size(-1), L = q.dim() == 4 ? q.size(1) : 1;
    gdn_attention_problem p{};
    p.new_tokens = narrow(L);
    p.q_heads = narrow(q.size(-2));
    p.kv_heads = narrow(k.size(2));
    p.head_dim = narrow(D);
    p.dtype = dtype_code(q, "q");
    p.scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(D, 1))) : number(a[7]);
    Strides s = heads4(q, "q", type, q.sizes(), q);
    p.q_stride = s.token, p.q_head_stride = s.head;
    const Cache cache(a + 1, k.size(2), D, q);
    if (q.size(0) != cache.N)
        value_error("page_table must have a row for each sequence of q");
    if (gate) {
        s = heads4(*gate, "gate", type, q.sizes(), q);
        p.gate_stride = s.token, p.gate_head_stride = s.head;
    }
    const Call call(q);
    const at::Tensor out = given ? *given : make(q.sizes(), type, q);
    s = heads4(out, "out", type, q.sizes(), q);
    p.out_stride = s.token, p.out_head_stride = s.head;
    at::Tensor lse;
    const at::IntArrayRef rows_shape = q.sizes().slice(0, q.dim() - 1);
    if (stats) {
        data(stats, "lse", at::kFloat, rows_shape, q);
        lse = *stats;
    } else if (flag(a[11])) {
        lse = make(rows_shape, at::kFloat, q);
    }
    at::Tensor own;
    if (scratch) {
        if (!scratch->is_contiguous()) value_error("workspace must be contiguous");
        check_device(*scratch, "workspace", q);
        p.workspace = scratch->data_ptr();
        p.workspace_bytes = scratch->nbytes();
    } else if (const size_t need = attention_workspace_entry(&p, &cache.c)) {
        own = make({(int64_t)need}, at::kByte, q);  // from the caching allocator, for this stream
        p.workspace = own.data_ptr();
        p.workspace_bytes = need;
    }
    if (!fine(attention_entry(&p, &cache.c, q.data_ptr(), gate ? gate->data_ptr() : nullptr,
                              out.data_ptr(),
                              lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr,
                              call.stream),
              "gdn_paged_attention"))
        return nullptr;
    return lse.defined() ? wrap_pair(out, lse) : wrap(out);
    END_HANDLE_TH_ERRORS
}

// The four entry points' addresses in the order below.
PyObject *bind_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 4) type_error("wrong number of arguments");
    void *at[4];
    for (int i = 0; i < 4; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) throw python_error();
        if (!at[i]) value_error("an entry point's address is null");
    }
    rope_entry = reinterpret_cast<decltype(rope_entry)>(at[0]);
    append_entry = reinterpret_cast<decltype(append_entry)>(at[1]);
    attention_entry = reinterpret_cast<decltype(attention_entry)>(at[2]);
    attention_workspace_entry = reinterpret_cast<decltype(attention_workspace_entry)>(at[3]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

}  // namespace

PyMethodDef attention_methods[] = {
    {"bind_attention", (PyCFunction)(void (*)(void))bind_attention, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, nullptr},
    {"paged_append", (PyCFunction)(void (*)(void))paged_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
