// block_api.cu -- the C ABI of include/gdn_block.h: argument checks and
// dispatch.  Every argument error is caught here, before any launch.
#include <initializer_list>

#include "block.cuh"

namespace {

using namespace gdn;

size_t size_of(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

bool dtype_ok(int32_t dtype) { return dtype == GDN_BF16 || dtype == GDN_F32; }

// Element alignment of the given (non-null) pointers.
bool misaligned(size_t size, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0) return true;
    return false;
}

// Whether the (non-null) result lies over one of the others.
bool over(const void *result, std::initializer_list<const void *> others) {
    for (const void *p : others)
        if (result && result == p) return true;
    return false;
}

bool any_null(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!p) return true;
    return false;
}

// Sequence and token counts and channels that the kernels' 32-bit indices hold
// (the search of a token's sequence adds two of them).
bool sizes_ok(int32_t seqs, int64_t tokens, int32_t channels) {
    constexpr int64_t most = INT32_MAX / 2;
    return seqs >= 0 && seqs <= most && tokens >= 0 && tokens <= most && channels >= 1 &&
           channels <= 1 << 20;
}

// A row stride matters from the second row on.
bool stride_ok(int64_t rows, int64_t stride, int64_t width) { return rows <= 1 || stride >= width; }

gdn_status check_conv(const gdn_conv_problem *pp) {
    if (!pp) return GDN_ERR_INVALID_ARG;
    const gdn_conv_problem &p = *pp;
    if (!sizes_ok(p.num_seqs, p.total_tokens, p.channels) || p.width < 1)
        return GDN_ERR_INVALID_ARG;
    if (!stride_ok(p.total_tokens, p.x_stride, p.channels) ||
        !stride_ok(p.total_tokens, p.out_stride, p.channels))
        return GDN_ERR_INVALID_ARG;
    if (p.width < 2 || p.width > 8 || !dtype_ok(p.dtype) ||
        (p.activation != GDN_ACT_NONE && p.activation != GDN_ACT_SILU))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_ssm(const gdn_ssm_problem *pp, bool gated) {
    if (!pp) return GDN_ERR_INVALID_ARG;
    const gdn_ssm_problem &p = *pp;
    if (!sizes_ok(p.num_seqs, p.total_tokens, p.channels) || p.state_dim < 1 || p.num_groups < 1)
        return GDN_ERR_INVALID_ARG;
    if (p.state_dim > 64 || p.channels % p.num_groups != 0 || !dtype_ok(p.dtype))
        return GDN_ERR_UNSUPPORTED;
    const int64_t T = p.total_tokens, D = p.channels, GS = (int64_t)p.num_groups * p.state_dim;
    if (!stride_ok(T, p.x_stride, D) || !stride_ok(T, p.dt_stride, D) ||
        !stride_ok(T, p.out_stride, D) || !stride_ok(T, p.b_stride, GS) ||
        !stride_ok(T, p.c_stride, GS) || (gated && !stride_ok(T, p.z_stride, D)))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

GDN_API gdn_status gdn_short_conv(const gdn_conv_problem *problem, const void *x,
                                  const float *weight, const float *bias,
                                  const int32_t *cu_seqlens, const void *initial_state, void *out,
                                  void *final_state, gdn_stream_t stream) {
    const gdn_status st = check_conv(problem);
    if (st != GDN_OK) return st;
    const gdn_conv_problem &p = *problem;
    if (p.num_seqs == 0) return p.total_tokens == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (any_null({weight, cu_seqlens})) return GDN_ERR_INVALID_ARG;
    if (p.total_tokens > 0 && any_null({x, out})) return GDN_ERR_INVALID_ARG;
    if (misaligned(size_of(p.dtype), {x, initial_state, out, final_state}) ||
        misaligned(4, {weight, bias, cu_seqlens}))
        return GDN_ERR_MISALIGNED;
    if (over(out, {x, initial_state, final_state}) || over(final_state, {x}))
        return GDN_ERR_INVALID_ARG;
    return launch_short_conv(p, x, weight, bias, cu_seqlens, initial_state, out, final_state,
                             reinterpret_cast<cudaStream_t>(stream));
}

GDN_API gdn_status gdn_short_conv_step(const gdn_conv_problem *problem, const void *x,
                                       const float *weight, const float *bias, const void *state,
                                       void *out, void *new_state, gdn_stream_t stream) {
    const gdn_status st = check_conv(problem);
    if (st != GDN_OK) return st;
    const gdn_conv_problem &p = *problem;
    if (p.total_tokens != p.num_seqs) return GDN_ERR_INVALID_ARG;
    if (p.num_seqs == 0) return GDN_OK;
    if (any_null({x, weight, state, out, new_state})) return GDN_ERR_INVALID_ARG;
    if (misaligned(size_of(p.dtype), {x, state, out, new_state}) || misaligned(4, {weight, bias}))
        return GDN_ERR_MISALIGNED;
    if (out == x || out == state || out == new_state) return GDN_ERR_INVALID_ARG;
    return launch_short_conv_step(p, x, weight, bias, state, out, new_state,
                                  reinterpret_cast<cudaStream_t>(stream));
}

GDN_API size_t gdn_selective_scan_workspace_size(const gdn_ssm_problem *problem) {
    if (!problem) return 0;
    gdn_ssm_problem p = *problem;  // the strides do not matter here
    p.x_stride = p.dt_stride = p.z_stride = p.out_stride = p.b_stride = p.c_stride = INT64_MAX;
    return check_ssm(&p, true) == GDN_OK ? scan_workspace_size(p) : 0;
}

GDN_API gdn_status gdn_selective_scan(const gdn_ssm_problem *problem, const void *x,
                                      const void *dt, const float *A, const void *B,
                                      const void *C, const float *skip, const void *z,
                                      const float *dt_bias, const int32_t *cu_seqlens,
                                      const float *initial_state, void *out, float *final_state,
                                      gdn_stream_t stream) {
    const gdn_status st = check_ssm(problem, z != nullptr);
    if (st != GDN_OK) return st;
    const gdn_ssm_problem &p = *problem;
    if (p.num_seqs == 0) return p.total_tokens == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (any_null({A, cu_seqlens})) return GDN_ERR_INVALID_ARG;
    if (p.total_tokens > 0 && any_null({x, dt, B, C, out})) return GDN_ERR_INVALID_ARG;
    if (misaligned(size_of(p.dtype), {x, dt, B, C, z, out}) ||
        misaligned(4, {A, skip, dt_bias, cu_seqlens, initial_state, final_state}))
        return GDN_ERR_MISALIGNED;
    if (over(out, {x, dt, z, B, C, initial_state, final_state}) ||
        over(final_state, {x, dt, z, A, B, C}))
        return GDN_ERR_INVALID_ARG;
    const size_t need = scan_workspace_size(p);
    if (need > 0 && (!p.workspace || p.workspace_bytes < need || !aligned16(p.workspace)))
        return GDN_ERR_WORKSPACE;
    const auto launch =
        p.dtype == GDN_BF16 ? launch_selective_scan_bf16 : launch_selective_scan_f32;
    return launch(p, x, dt, A, B, C, skip, z, dt_bias, cu_seqlens, initial_state, out, final_state,
                  reinterpret_cast<cudaStream_t>(stream));
}

GDN_API gdn_status gdn_selective_scan_step(const gdn_ssm_problem *problem, const void *x,
                                           const void *dt, const float *A, const void *B,
                                           const void *C, const float *skip, const void *z,
                                           const float *dt_bias, const float *state, void *out,
                                           float *new_state, gdn_stream_t stream) {
    const gdn_status st = check_ssm(problem, z != nullptr);
    if (st != GDN_OK) return st;
    const gdn_ssm_problem &p = *problem;
    if (p.total_tokens != p.num_seqs) return GDN_ERR_INVALID_ARG;
    if (p.num_seqs == 0) return GDN_OK;
    if (any_null({x, dt, A, B, C, state, out, new_state})) return GDN_ERR_INVALID_ARG;
    if (misaligned(size_of(p.dtype), {x, dt, B, C, z, out}) ||
        misaligned(4, {A, skip, dt_bias, state, new_state}))
        return GDN_ERR_MISALIGNED;
    if (out == x || out == dt || out == z || out == B || out == C || out == state ||
        out == new_state)
        return GDN_ERR_INVALID_ARG;
    const auto launch =
        p.dtype == GDN_BF16 ? launch_selective_scan_step_bf16 : launch_selective_scan_step_f32;
    return launch(p, x, dt, A, B, C, skip, z, dt_bias, state, out, new_state,
                  reinterpret_cast<cudaStream_t>(stream));
}

GDN_API gdn_status gdn_norm_gate_residual(const gdn_norm_problem *problem, const void *y,
                                          const float *weight, const void *gate,
                                          const void *residual, const float *next_weight,
                                          void *out, void *next, gdn_stream_t stream) {
    if (!problem) return GDN_ERR_INVALID_ARG;
    const gdn_norm_problem &p = *problem;
    if (p.rows < 0 || p.dim < 1 || !(p.eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (p.dim > 16384 || !dtype_ok(p.dtype) || !dtype_ok(p.residual_dtype) ||
        (p.dtype == GDN_F32 && p.residual_dtype != GDN_F32) || p.activation < GDN_ACT_NONE ||
        p.activation > GDN_ACT_SIGMOID)
        return GDN_ERR_UNSUPPORTED;
    if (!stride_ok(p.rows, p.y_stride, p.dim) || !stride_ok(p.rows, p.out_stride, p.dim) ||
        (gate && !stride_ok(p.rows, p.gate_stride, p.dim)) ||
        (residual && !stride_ok(p.rows, p.residual_stride, p.dim)) ||
        (next && !stride_ok(p.rows, p.next_stride, p.dim)))
        return GDN_ERR_INVALID_ARG;
    if (p.rows == 0) return GDN_OK;
    if (any_null({y, out}) || (next == nullptr) != (next_weight == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (misaligned(size_of(p.dtype), {y, gate, next}) ||
        misaligned(size_of(p.residual_dtype), {residual, out}) ||
        misaligned(4, {weight, next_weight}))
        return GDN_ERR_MISALIGNED;
    // In place only element by element: the same element size and, of several
    // rows, the same stride.
    const bool same_type = p.dtype == p.residual_dtype;
    auto same_rows = [&](int64_t stride, int64_t other) { return p.rows == 1 || stride == other; };
    if (out == gate || out == next || (next && next == residual)) return GDN_ERR_INVALID_ARG;
    if (out == y && !(same_type && same_rows(p.out_stride, p.y_stride))) return GDN_ERR_INVALID_ARG;
    if (out == residual && !same_rows(p.out_stride, p.residual_stride)) return GDN_ERR_INVALID_ARG;
    if (next && next == y && !same_rows(p.next_stride, p.y_stride)) return GDN_ERR_INVALID_ARG;
    if (next && next == gate && !same_rows(p.next_stride, p.gate_stride))
        return GDN_ERR_INVALID_ARG;
    return launch_norm_gate_residual(p, y, weight, gate, residual, next_weight, out, next,
                                     reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
