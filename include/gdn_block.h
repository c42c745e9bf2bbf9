/*
 * gdn_block.h -- C ABI of the operators that stand beside the Gated DeltaNet
 * layer in a hybrid model's block: the short causal convolution of its
 * projections, a selective state space scan (the other fixed-state layer),
 * and the norms around a block fused with its gate and residual.
 *
 * Conventions are those of gdn.h: device pointers, caller-owned buffers, no
 * allocation or synchronisation, launches on the given stream only, argument
 * errors reported before any launch with every output untouched.  Where they
 * differ:
 *   - rows of the token-major tensors may be strided (a slice of a wider
 *     projection): strides are given in elements, the elements of a row are
 *     contiguous.  Rows of an output must not overlap.
 *   - pointers need only the alignment of their elements.  Whole 16-byte
 *     words are loaded and stored where the rows allow it (pointer, stride and
 *     channel count); other alignments take narrower accesses.  A strided
 *     input's words between its first row and its last may be read (and are
 *     not used) where they lie between rows; nothing before its first element
 *     or after its last one is.
 * dtype is GDN_BF16 or GDN_F32.  Sums, states and statistics are fp32;
 * results are rounded once, to nearest even.
 *
 * cu_seqlens is as in gdn_chunk_prefill: device int32 [N + 1], cu[0] = 0,
 * nondecreasing, cu[N] = T, zero-length sequences allowed.  It is not checked
 * on the host; a malformed one gives unspecified values, and no access
 * outside the tensors.
 *
 * These operators have no device-side waits and no device status.  The only
 * process-wide state they add is, per device and variant of a kernel, whether
 * its shared-memory limit has been raised (set once).
 */
#ifndef GDN_BLOCK_H
#define GDN_BLOCK_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_ACT_NONE = 0,
    GDN_ACT_SILU = 1,    /* v sigmoid(v) */
    GDN_ACT_SIGMOID = 2  /* gates only   */
} gdn_activation;

/*
 * Short causal depthwise convolution.
 *   num_seqs      N;  total_tokens T (step: must equal N), each 0 to 2^30 - 1
 *   channels      C, 1 to 2^20;  width K, 2 to 8
 *   activation    GDN_ACT_NONE or GDN_ACT_SILU
 *   x_stride, out_stride   elements between rows, >= C
 */
typedef struct {
    int32_t num_seqs;
    int64_t total_tokens;
    int32_t channels;
    int32_t width;
    int32_t dtype;
    int32_t activation;
    int64_t x_stride;
    int64_t out_stride;
} gdn_conv_problem;

/*
 * out[t, c] = act(bias[c] + sum_{j < K} weight[c, j] x[t - K + 1 + j, c]),
 * where the K - 1 inputs before a sequence's first come from its state.
 *   x, out         [T, C]
 *   weight         fp32 [C, K]; bias fp32 [C] or NULL
 *   initial_state  [N, K - 1, C] in dtype, oldest input first, or NULL
 *                  (zeros)
 *   final_state    [N, K - 1, C] or NULL (not written): the last K - 1 inputs
 *                  of each sequence, the initial state's among them where it
 *                  is shorter.  May equal initial_state (in-place resume).
 * Nothing else may overlap.
 */
GDN_API gdn_status gdn_short_conv(const gdn_conv_problem *problem, const void *x,
                                  const float *weight, const float *bias,
                                  const int32_t *cu_seqlens, const void *initial_state,
                                  void *out, void *final_state, gdn_stream_t stream);

/*
 * The same for one token of each sequence: x, out [N, C]; state [N, K - 1, C]
 * is read, new_state written (it may equal state: update in place).
 */
GDN_API gdn_status gdn_short_conv_step(const gdn_conv_problem *problem, const void *x,
                                       const float *weight, const float *bias,
                                       const void *state, void *out, void *new_state,
                                       gdn_stream_t stream);

/*
 * Selective state space scan.
 *   num_seqs      N;  total_tokens T (step: must equal N), each 0 to 2^30 - 1
 *   channels      D, 1 to 2^20;  state_dim S, 1 to 64
 *   num_groups    G >= 1, dividing D: channels d D/G .. share B and C
 *   dt_softplus   nonzero: the step is softplus(dt + dt_bias)
 *   strides       elements between rows: x, dt, z, out >= D, B, C >= G S
 *   workspace     device scratch (see the size query), 16-byte aligned;
 *                 ignored by the step
 */
typedef struct {
    int32_t num_seqs;
    int64_t total_tokens;
    int32_t channels;
    int32_t state_dim;
    int32_t num_groups;
    int32_t dtype;
    int32_t dt_softplus;
    int64_t x_stride;
    int64_t dt_stride;
    int64_t b_stride;
    int64_t c_stride;
    int64_t z_stride;
    int64_t out_stride;
    void *workspace;
    size_t workspace_bytes;
} gdn_ssm_problem;

/*
 * Bytes of device workspace gdn_selective_scan needs (it depends on every
 * size of the descriptor, not on the strides); 0 when the descriptor is
 * invalid or no workspace is needed.
 */
GDN_API size_t gdn_selective_scan_workspace_size(const gdn_ssm_problem *problem);

/*
 * For every sequence and channel d (group g = d / (D / G)) a state h[S]:
 *   s_t = softplus(dt[t, d] + dt_bias[d])
 *   h_t = exp(s_t A[d, :]) h_{t-1} + s_t x[t, d] B[t, g, :]
 *   out[t, d] = (sum C[t, g, :] h_t + skip[d] x[t, d]) z[t, d] sigmoid(z[t, d])
 *   x, dt, z, out  [T, D]; z may be NULL (no gate)
 *   A              fp32 [D, S], finite, of any sign (negative for a decaying
 *                  state)
 *   B, C           [T, G, S]
 *   skip, dt_bias  fp32 [D] or NULL (no such term)
 *   initial_state  fp32 [N, D, S] or NULL (zeros)
 *   final_state    fp32 [N, D, S] or NULL (not written); may equal
 *                  initial_state (in-place resume)
 * Neither out nor final_state may overlap anything else.  Infinities and NaN
 * among the inputs give what the formula gives in fp32, in their own sequence
 * only.
 *
 * The packed tokens are cut into windows of equal length (at least 8 tokens),
 * as many as make one wave of blocks.  With more than one, three launches
 * run: the state that each window adds on its own (from a zero state, or from
 * the sequence's start inside it), the states entering the windows, and the
 * outputs of all windows; the later ones may start while the one before ends
 * (programmatic launches on `stream`).  Where final_state equals
 * initial_state, a fourth launch writes the final states that other windows
 * had to read as initial ones until then.  Few tokens run as one window, with
 * the launch of the outputs alone and no workspace.  The order of the fp32 sums depends
 * on the sizes alone, so a call gives the same bits every time.
 */
GDN_API gdn_status gdn_selective_scan(const gdn_ssm_problem *problem, const void *x,
                                      const void *dt, const float *A, const void *B,
                                      const void *C, const float *skip, const void *z,
                                      const float *dt_bias, const int32_t *cu_seqlens,
                                      const float *initial_state, void *out,
                                      float *final_state, gdn_stream_t stream);

/*
 * The same for one token of each sequence: row n of x, dt, B, C, z and out
 * belongs to sequence n; state fp32 [N, D, S] is read, new_state written (it
 * may equal state: update in place).
 */
GDN_API gdn_status gdn_selective_scan_step(const gdn_ssm_problem *problem, const void *x,
                                           const void *dt, const float *A, const void *B,
                                           const void *C, const float *skip, const void *z,
                                           const float *dt_bias, const float *state, void *out,
                                           float *new_state, gdn_stream_t stream);

/*
 * The norm after a block with its gate and scaled residual, and the norm
 * before the next block.
 *   rows, dim       R >= 0, D 1 to 16384
 *   dtype           of y, gate and next
 *   residual_dtype  of residual and out: dtype, or GDN_F32 for a residual
 *                   stream kept in fp32
 *   activation      of the gate (any gdn_activation)
 *   gate_first      nonzero: the gate multiplies y before the norm
 *   eps             >= 0;  scale: of the gated, normed y
 *   strides         elements between rows, >= D
 */
typedef struct {
    int64_t rows;
    int32_t dim;
    int32_t dtype;
    int32_t residual_dtype;
    int32_t activation;
    int32_t gate_first;
    float eps;
    float scale;
    int64_t y_stride;
    int64_t gate_stride;
    int64_t residual_stride;
    int64_t out_stride;
    int64_t next_stride;
} gdn_norm_problem;

/*
 * Row by row, with rms(v) = v / sqrt(mean(v^2) + eps):
 *   m    = weight rms(y) act(gate)          (gate_first: weight rms(y act(gate)))
 *   out  = residual + scale m
 *   next = next_weight rms(out)             (of out before its rounding)
 *   y               [R, D]
 *   weight          fp32 [D], or NULL: no norm of y
 *   gate            [R, D] or NULL (no gate)
 *   residual        [R, D] or NULL (zeros)
 *   next_weight     fp32 [D], or NULL: next is not computed
 *   out, next       [R, D]; next is NULL exactly when next_weight is
 * out may equal y or residual, and next may equal y or gate, where pointer,
 * element type and, of several rows, stride are the same; nothing else may
 * overlap.
 */
GDN_API gdn_status gdn_norm_gate_residual(const gdn_norm_problem *problem, const void *y,
                                          const float *weight, const void *gate,
                                          const void *residual, const float *next_weight,
                                          void *out, void *next, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_BLOCK_H */
