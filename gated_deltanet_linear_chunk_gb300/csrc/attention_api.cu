// attention_api.cu -- the C ABI of include/gdn_attention.h: argument checks and
// dispatch.  Every argument error is caught here, before any launch.
#include <initializer_list>

#include "attention.cuh"

namespace {

using namespace gdn;

constexpr int kMostTokens = INT32_MAX / 2, kMostHeads = 4096;

size_t size_of(int32_t dtype) { return dtype == GDN_F32 ? 4 : dtype == GDN_E4M3 ? 1 : 2; }

bool misaligned(size_t size, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0) return true;
    return false;
}

bool any_null(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!p) return true;
    return false;
}

bool over(const void *result, std::initializer_list<const void *> others) {
    for (const void *p : others)
        if (result && result == p) return true;
    return false;
}

// The outer dimensions of a tensor of rows of D elements: how many, how far
// apart.
struct Dim {
    int64_t size, stride;
};
// Whether no two rows share an element (dimensions of one, or of none, do not
// matter): each stride, from the shortest, passes all that lies within it.
bool apart(int64_t row, std::initializer_list<Dim> dims) {
    Dim d[3];
    int n = 0;
    for (const Dim &x : dims) {
        if (x.size == 0) return true;
        if (x.size > 1) d[n++] = x;
    }
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
            const Dim t = d[j];
            d[j] = d[j - 1];
            d[j - 1] = t;
        }
    int64_t span = row;
    for (int i = 0; i < n; ++i) {
        if (d[i].stride < span) return false;
        if (d[i].stride > (INT64_MAX - span) / d[i].size) return false;
        span += d[i].stride * (d[i].size - 1);
    }
    return true;
}

gdn_status check_rope(const gdn_rope_problem &p, int most_heads = kMostHeads) {
    if (p.total_tokens < 0 || p.total_tokens > kMostTokens || p.q_heads < 0 || p.kv_heads < 0 ||
        p.q_heads > most_heads || p.kv_heads > most_heads || p.head_dim < 1 || p.rotary_dim < 0 ||
        p.rotary_dim > p.head_dim || p.num_axes < 1 || !(p.eps >= 0.f))
        return GDN_ERR_INVALID_ARG;
    if (p.head_dim > 512 || p.rotary_dim % 2 != 0 || p.num_axes > 8 ||
        (p.dtype != GDN_BF16 && p.dtype != GDN_F32))
        return GDN_ERR_UNSUPPORTED;
    if (p.freq_axis)
        for (int i = 0; i < p.rotary_dim / 2; ++i)
            if (p.freq_axis[i] >= p.num_axes) return GDN_ERR_INVALID_ARG;
    if (p.num_axes > 1 && p.axis_stride < p.total_tokens) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// The queries and, in place, their results.
gdn_status check_rows(int64_t T, int heads, int D, size_t size, const void *x, int64_t stride,
                      int64_t head_stride, const void *out, int64_t out_stride,
                      int64_t out_head_stride) {
    if (heads == 0) return x || out ? GDN_ERR_INVALID_ARG : GDN_OK;
    if (T == 0) return GDN_OK;
    if (any_null({x, out}) || !apart(D, {{T, stride}, {heads, head_stride}}) ||
        !apart(D, {{T, out_stride}, {heads, out_head_stride}}))
        return GDN_ERR_INVALID_ARG;
    if (misaligned(size, {x, out})) return GDN_ERR_MISALIGNED;
    if (x == out && ((T > 1 && stride != out_stride) || (heads > 1 && head_stride != out_head_stride)))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status check_angles(const gdn_rope_problem &p, const int32_t *positions, const float *inv_freq,
                        const float *q_weight, const float *k_weight) {
    if ((q_weight && p.q_heads == 0) || (k_weight && p.kv_heads == 0)) return GDN_ERR_INVALID_ARG;
    if (p.rotary_dim > 0 ? !inv_freq : positions || inv_freq) return GDN_ERR_INVALID_ARG;
    return misaligned(4, {positions, inv_freq, q_weight, k_weight}) ? GDN_ERR_MISALIGNED : GDN_OK;
}

bool cache_type(int32_t cache, int32_t dtype) {
    return cache == dtype || (cache == GDN_E4M3 && dtype == GDN_BF16);
}

// 16-byte rows: what the attention reads.
gdn_status check_cache(const gdn_paged_cache &c, int32_t dtype, int heads, int D, bool words) {
    if (c.num_pages < 1 || c.num_pages > INT32_MAX || c.page_size < 1 || c.page_size > 1 << 20 ||
        c.num_seqs < 0 || c.num_seqs > kMostTokens || c.max_pages < 0 ||
        (int64_t)c.max_pages * c.page_size > kMaxCached)
        return GDN_ERR_INVALID_ARG;
    if (!cache_type(c.dtype, dtype)) return GDN_ERR_UNSUPPORTED;
    if (c.num_seqs > 1 && c.table_stride < c.max_pages) return GDN_ERR_INVALID_ARG;
    if (c.num_seqs > 0 && (!c.seq_lens || (c.max_pages > 0 && !c.page_table)))
        return GDN_ERR_INVALID_ARG;
    if (any_null({c.k, c.v})) return GDN_ERR_INVALID_ARG;
    if ((c.k_scale != nullptr) != (c.dtype == GDN_E4M3) ||
        (c.v_scale != nullptr) != (c.dtype == GDN_E4M3))
        return GDN_ERR_INVALID_ARG;
    auto fits = [&](int64_t ps, int64_t ts, int64_t hs) {
        return apart(D, {{c.num_pages, ps}, {c.page_size, ts}, {heads, hs}});
    };
    if (!fits(c.k_page_stride, c.k_token_stride, c.k_head_stride) ||
        !fits(c.v_page_stride, c.v_token_stride, c.v_head_stride))
        return GDN_ERR_INVALID_ARG;
    const size_t size = size_of(c.dtype);
    if (misaligned(size, {c.k, c.v}) || misaligned(4, {c.k_scale, c.v_scale, c.page_table, c.seq_lens}))
        return GDN_ERR_MISALIGNED;
    if (words) {
        auto whole = [&](const void *p, int64_t ps, int64_t ts, int64_t hs) {
            const uint64_t all = (c.num_pages > 1 ? (uint64_t)ps : 0) |
                                 (c.page_size > 1 ? (uint64_t)ts : 0) |
                                 (heads > 1 ? (uint64_t)hs : 0);
            return aligned16(p) && (all * size) % 16 == 0;
        };
        if (!whole(c.k, c.k_page_stride, c.k_token_stride, c.k_head_stride) ||
            !whole(c.v, c.v_page_stride, c.v_token_stride, c.v_head_stride))
            return GDN_ERR_MISALIGNED;
    }
    return GDN_OK;
}

gdn_status check_attention(const gdn_attention_problem &p, const gdn_paged_cache &c) {
    if (p.new_tokens < 1 || p.q_heads < 1 || p.kv_heads < 1 || p.q_heads > kMostHeads ||
        p.head_dim < 1)
        return GDN_ERR_INVALID_ARG;
    // Rows of q: a grid has as many blocks at most.
    if (c.num_seqs < 0 || (int64_t)c.num_seqs * p.new_tokens > INT32_MAX / p.q_heads)
        return GDN_ERR_INVALID_ARG;
    if (p.new_tokens > kMaxNewTokens || p.q_heads % p.kv_heads != 0 ||
        (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) ||
        (p.dtype != GDN_BF16 && p.dtype != GDN_F32))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

GDN_API gdn_status gdn_qk_norm_rope(const gdn_rope_problem *problem, const void *q, const void *k,
                                    const float *q_weight, const float *k_weight,
                                    const int32_t *positions, const float *inv_freq, void *q_out,
                                    void *k_out, gdn_stream_t stream) {
    if (!problem) return GDN_ERR_INVALID_ARG;
    const gdn_rope_problem &p = *problem;
    gdn_status st = check_rope(p);
    if (st != GDN_OK) return st;
    const size_t size = size_of(p.dtype);
    st = check_rows(p.total_tokens, p.q_heads, p.head_dim, size, q, p.q_stride, p.q_head_stride,
                    q_out, p.q_out_stride, p.q_out_head_stride);
    if (st != GDN_OK) return st;
    st = check_rows(p.total_tokens, p.kv_heads, p.head_dim, size, k, p.k_stride, p.k_head_stride,
                    k_out, p.k_out_stride, p.k_out_head_stride);
    if (st != GDN_OK) return st;
    st = check_angles(p, positions, inv_freq, q_weight, k_weight);
    if (st != GDN_OK) return st;
    if (p.total_tokens > 0 && p.rotary_dim > 0 && !positions) return GDN_ERR_INVALID_ARG;
    if (over(q_out, {k, k_out}) || over(k_out, {q})) return GDN_ERR_INVALID_ARG;
    if (p.total_tokens == 0 || p.q_heads + p.kv_heads == 0) return GDN_OK;
    return launch_qk_rope(p, nullptr, q, k, nullptr, q_weight, k_weight, positions, inv_freq,
                          nullptr, q_out, k_out, reinterpret_cast<cudaStream_t>(stream));
}

GDN_API gdn_status gdn_paged_append(const gdn_rope_problem *problem, const gdn_paged_cache *cache,
                                    const void *q, const void *k, const void *v,
                                    const float *q_weight, const float *k_weight,
                                    const int32_t *positions, const float *inv_freq,
                                    const int32_t *cu_seqlens, void *q_out, gdn_stream_t stream) {
    if (!problem || !cache) return GDN_ERR_INVALID_ARG;
    const gdn_rope_problem &p = *problem;
    const gdn_paged_cache &c = *cache;
    gdn_status st = check_rope(p);
    if (st != GDN_OK) return st;
    if (p.kv_heads < 1) return GDN_ERR_INVALID_ARG;
    st = check_cache(c, p.dtype, p.kv_heads, p.head_dim, false);
    if (st != GDN_OK) return st;
    const int64_t T = p.total_tokens;
    if (c.num_seqs == 0 ? T > 0 && !cu_seqlens : !cu_seqlens && T % c.num_seqs != 0)
        return GDN_ERR_INVALID_ARG;
    if (p.num_axes > 1 && !positions) return GDN_ERR_INVALID_ARG;
    const size_t size = size_of(p.dtype);
    st = check_rows(T, p.q_heads, p.head_dim, size, q, p.q_stride, p.q_head_stride, q_out,
                    p.q_out_stride, p.q_out_head_stride);
    if (st != GDN_OK) return st;
    st = check_angles(p, positions, inv_freq, q_weight, k_weight);
    if (st != GDN_OK) return st;
    if (T > 0) {
        if (any_null({k, v}) || !apart(p.head_dim, {{T, p.k_stride}, {p.kv_heads, p.k_head_stride}}) ||
            !apart(p.head_dim, {{T, p.v_stride}, {p.kv_heads, p.v_head_stride}}))
            return GDN_ERR_INVALID_ARG;
        if (misaligned(size, {k, v}) || misaligned(4, {cu_seqlens})) return GDN_ERR_MISALIGNED;
        if (over(q_out, {k, v, c.k, c.v}) || over(c.k, {q, k, v, c.v}) || over(c.v, {q, k, v}))
            return GDN_ERR_INVALID_ARG;
    }
    if (T == 0 || c.num_seqs == 0) return GDN_OK;
    return launch_qk_rope(p, &c, q, k, v, q_weight, k_weight, positions, inv_freq, cu_seqlens,
                          q_out, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

GDN_API size_t gdn_paged_attention_workspace_size(const gdn_attention_problem *problem,
                                                  const gdn_paged_cache *cache) {
    if (!problem || !cache || check_attention(*problem, *cache) != GDN_OK) return 0;
    const gdn_paged_cache &c = *cache;
    if (!cache_type(c.dtype, problem->dtype) || c.max_pages < 0 || c.page_size < 1 || c.page_size > 1 << 20 ||
        (int64_t)c.max_pages * c.page_size > kMaxCached)
        return 0;
    return paged_attention_workspace(*problem, c);
}

GDN_API gdn_status gdn_paged_attention(const gdn_attention_problem *problem,
                                       const gdn_paged_cache *cache, const void *q,
                                       const void *gate, void *out, float *lse,
                                       gdn_stream_t stream) {
    if (!problem || !cache) return GDN_ERR_INVALID_ARG;
    const gdn_attention_problem &p = *problem;
    const gdn_paged_cache &c = *cache;
    gdn_status st = check_attention(p, c);
    if (st != GDN_OK) return st;
    st = check_cache(c, p.dtype, p.kv_heads, p.head_dim, true);
    if (st != GDN_OK) return st;
    const int64_t T = (int64_t)c.num_seqs * p.new_tokens;
    const size_t size = size_of(p.dtype);
    st = check_rows(T, p.q_heads, p.head_dim, size, q, p.q_stride, p.q_head_stride, out,
                    p.out_stride, p.out_head_stride);
    if (st != GDN_OK) return st;
    if (gate) {
        st = check_rows(T, p.q_heads, p.head_dim, size, gate, p.gate_stride, p.gate_head_stride, out,
                        p.out_stride, p.out_head_stride);
        if (st != GDN_OK) return st;
    }
    if (misaligned(4, {lse})) return GDN_ERR_MISALIGNED;
    if (T == 0) return GDN_OK;
    if (over(out, {c.k, c.v, lse}) || over(lse, {q, gate, c.k, c.v})) return GDN_ERR_INVALID_ARG;
    const size_t need = paged_attention_workspace(p, c);
    if (need > 0 && (!p.workspace || p.workspace_bytes < need || !aligned16(p.workspace)))
        return GDN_ERR_WORKSPACE;
    return launch_paged_attention(p, c, q, gate, out, lse, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
