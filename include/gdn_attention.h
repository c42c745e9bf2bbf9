/*
 * gdn_attention.h -- C ABI of what a hybrid model's attention layers need
 * beside its fixed-state ones: norms of queries and keys for each head with
 * their rotation by position, a paged cache that new keys and values are
 * appended to on the way, and the attention of a sequence's newest tokens over
 * it.
 *
 * Conventions are those of gdn_block.h: device pointers, caller-owned
 * buffers, no allocation or synchronisation, launches on the given stream
 * only, argument errors reported before any launch with every output
 * untouched.  Where they differ:
 *   - token-major tensors [T, H, D] may be strided between tokens and between
 *     heads (queries that lie beside their gates, head by head, in one
 *     projection); strides are given in elements, and the D elements of a head
 *     are contiguous.  Neither heads nor tokens of a tensor may overlap, an
 *     input's no more than an output's (one key for all heads is kv_heads = 1),
 *     nor pages, places and heads of a cache: such strides are refused.
 *   - tokens behind the last sequence are allowed (a batch padded to a fixed
 *     size): their outputs are left as they were.
 * Sums, statistics, angles' sines and cosines and the softmax's maxima, weights
 * and sums are fp32; results are rounded once, to nearest even.  (What bf16
 * attention rounds on the way to its products is said there.)
 */
#ifndef GDN_ATTENTION_H
#define GDN_ATTENTION_H

#include "gdn_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm and rotation of queries and keys.
 *   total_tokens   T, 0 to 2^30 - 1
 *   q_heads        Hq, 0 (no queries) to 4096;  kv_heads Hk, likewise, of the keys
 *   head_dim       D, 1 to 512
 *   dtype          GDN_BF16 or GDN_F32
 *   rotary_dim     R, even, 0 (no rotation) to D: the first R elements of each
 *                  head are rotated in pairs
 *   interleaved    zero: element i is paired with i + R / 2; nonzero: 2 i with
 *                  2 i + 1  (i < R / 2)
 *   num_axes       axes of the positions, 1 to 8
 *   freq_axis      HOST array [R / 2] of the axis (below num_axes) that each
 *                  pair's angle goes by; NULL: axis 0
 *   eps            >= 0
 *   axis_stride    elements between the axes of positions, >= T
 *   *_stride       elements between tokens; *_head_stride between heads
 */
typedef struct {
    int64_t total_tokens;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t dtype;
    int32_t rotary_dim;
    int32_t interleaved;
    int32_t num_axes;
    const uint8_t *freq_axis;
    float eps;
    int64_t axis_stride;
    int64_t q_stride, q_head_stride;
    int64_t k_stride, k_head_stride;
    int64_t v_stride, v_head_stride;
    int64_t q_out_stride, q_out_head_stride;
    int64_t k_out_stride, k_out_head_stride;
} gdn_rope_problem;

/*
 * For every token t and head, with w the queries' or the keys' weight:
 *   y = w x / sqrt(mean(x^2) + eps)                      (no weight: y = x)
 *   (a, b) of pair i  ->  (a cos - b sin, b cos + a sin)  of the angle
 *                         positions[freq_axis[i], t] inv_freq[i]
 *   q, q_out            [T, Hq, D], or NULL with Hq = 0
 *   k, k_out            [T, Hk, D], or NULL with Hk = 0
 *   q_weight, k_weight  fp32 [D] or NULL
 *   positions           int32 [axes, T], any values; NULL with R = 0
 *   inv_freq            fp32 [R / 2], radians per position; NULL with R = 0
 * Angles are reduced exactly: far positions lose nothing.  q_out may equal q,
 * and k_out k, with the same strides; nothing else may overlap.
 */
GDN_API gdn_status gdn_qk_norm_rope(const gdn_rope_problem *problem, const void *q,
                                    const void *k, const float *q_weight, const float *k_weight,
                                    const int32_t *positions, const float *inv_freq, void *q_out,
                                    void *k_out, gdn_stream_t stream);

/*
 * A paged cache of keys and values, and what its N sequences hold of it.
 * Token j of sequence n lies in page page_table[n, j / page_size] at place
 * j % page_size.
 *   k, v         keys and values: head h of place s of page p begins at element
 *                p page_stride + s token_stride + h head_stride
 *   dtype        GDN_BF16, GDN_F32, or GDN_E4M3: 8-bit floating point (4 bits of
 *                exponent, 3 of mantissa, no infinities) times a scale
 *   num_pages    P, 1 to 2^31 - 1;  page_size 1 to 2^20
 *   k_scale, v_scale   fp32 [kv heads] of GDN_E4M3, positive; NULL otherwise
 *   num_seqs     N;  max_pages: columns of page_table; max_pages page_size at
 *                most 2^30 - 1
 *   page_table   int32 [N, max_pages], rows table_stride elements apart
 *   seq_lens     int32 [N]: tokens that each sequence holds, the new ones among
 *                them
 * Pages may be shared by sequences (a common prefix).  Entries of page_table
 * behind a sequence's last token are not used.  Neither array is checked on
 * the host.  Lengths outside 0 .. max_pages page_size count as the nearest
 * one.  A page outside 0 .. P - 1 is never accessed: nothing is appended there,
 * and the attention of a sequence that holds tokens in one is NaN.
 */
typedef struct {
    void *k;
    void *v;
    int32_t dtype;
    int64_t num_pages;
    int32_t page_size;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    const float *k_scale;
    const float *v_scale;
    int32_t num_seqs;
    int32_t max_pages;
    const int32_t *page_table;
    int64_t table_stride;
    const int32_t *seq_lens;
} gdn_paged_cache;

/*
 * Appends new keys and values: the last cu[n + 1] - cu[n] of the seq_lens[n]
 * tokens of each sequence.  Keys are normed and rotated as by
 * gdn_qk_norm_rope on the way (in fp32, rounded once, to the cache's type),
 * values only rounded; queries, where given, come out normed and rotated too.
 *   dtype         of q, k, v and q_out; the cache has the same, or is
 *                 GDN_E4M3 beside GDN_BF16: what is stored is x / scale, rounded
 *                 to nearest even, values beyond 448 as 448
 *   k, v          [T, kv heads, D]; k_out of the descriptor is not used
 *   q, q_out      [T, q heads, D]; NULL with q_heads = 0; q_out may equal q
 *   positions     int32 [axes, T]; NULL (one axis): a token's index in its
 *                 sequence
 *   cu_seqlens    int32 [N + 1]; NULL: T / N tokens of each sequence.  Tokens
 *                 from cu[N] on (and before cu[0]) are left out.
 * A token whose place in the cache does not exist (a length shorter than its
 * new tokens, or a page outside the cache) is not stored.  Two tokens for one
 * place leave either's key, and either's value.
 */
GDN_API gdn_status gdn_paged_append(const gdn_rope_problem *problem, const gdn_paged_cache *cache,
                                    const void *q, const void *k, const void *v,
                                    const float *q_weight, const float *k_weight,
                                    const int32_t *positions, const float *inv_freq,
                                    const int32_t *cu_seqlens, void *q_out, gdn_stream_t stream);

/*
 * Attention of each sequence's newest tokens over its paged cache.
 *   new_tokens    L, 1 to 8 of each sequence: token t of sequence n is row
 *                 n L + t of q, gate and out, and index seq_lens[n] - L + t of
 *                 the sequence
 *   q_heads       Hq, a multiple of kv_heads: query heads h Hq / Hkv .. share
 *                 key head h; 1 to 4096, and N L Hq at most 2^31 - 1
 *   head_dim      D: 64, 128 or 256
 *   dtype         GDN_BF16 or GDN_F32; the cache has the same, or is GDN_E4M3
 *                 beside GDN_BF16
 *   scale         of the scores
 *   workspace     device scratch (see the size query), 16-byte aligned
 */
typedef struct {
    int32_t new_tokens;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t dtype;
    float scale;
    int64_t q_stride, q_head_stride;
    int64_t gate_stride, gate_head_stride;
    int64_t out_stride, out_head_stride;
    void *workspace;
    size_t workspace_bytes;
} gdn_attention_problem;

/*
 * Bytes of device workspace gdn_paged_attention needs (from the descriptor's
 * sizes and the cache's type, page_size and max_pages); 0 when either is
 * invalid or there are no sequences.  A workspace needs no initial value and
 * belongs to one call at a time.
 */
GDN_API size_t gdn_paged_attention_workspace_size(const gdn_attention_problem *problem,
                                                  const gdn_paged_cache *cache);

/*
 * For row (n, t) and query head h, over the tokens j that it sees,
 * j <= seq_lens[n] - L + t:
 *   s_j = scale q . k_j
 *   out = sum_j e^s_j v_j / sum_j e^s_j, times sigmoid(gate) where given
 *   lse = log sum_j e^s_j                        (fp32 [N L, Hq] or NULL)
 * A row that sees no token, or only scores of -infinity, gets zeros and
 * -infinity.  What a row does not see has no effect on it, whatever it holds.
 * With bf16 queries the products take their operands in 16 bits.  Where up to 16
 * rows share a key head (L Hq / Hkv), a weight e^s_j goes in as the sum of two
 * parts, off by 2^-16 of itself; of more rows it is rounded to bf16, or to fp16
 * beside a GDN_E4M3 cache (where either way up to 2^-32 of a row's largest weight
 * is lost of each other one).  The sum that divides is that of the fp32 weights, and
 * so is lse.  Beside a GDN_E4M3 cache an element of a query is fp16 over a power
 * of two of its row's largest: exact, unless it is below 2^-14 of that.
 * k and v of the cache start on 16-byte boundaries, as do all their rows (the
 * strides): others are refused.  out may equal q or gate, with the same
 * strides; nothing else may overlap.
 *
 * Every group of warps takes an equal share of the cache's tokens, over the
 * sequences' ends; where a share ends inside a sequence, its sums go through the
 * workspace to a second launch, which joins them.  All launches of this header
 * are programmatic ones on `stream`: they may be set up, but read and write
 * nothing, before what is ahead of them has ended.  The order of the sums depends
 * on the sizes and lengths alone, so a call gives the same bits every time.
 */
GDN_API gdn_status gdn_paged_attention(const gdn_attention_problem *problem,
                                       const gdn_paged_cache *cache, const void *q,
                                       const void *gate, void *out, float *lse,
                                       gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H */
