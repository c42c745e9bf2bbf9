// attention.cuh -- shared pieces of the operators of include/gdn_attention.h
// (not part of the ABI).
#pragma once

#include <cuda_fp8.h>

#include "block.cuh"
#include "gdn_attention.h"
#include "sm103.cuh"

namespace gdn {

constexpr int kMaxRotary = 512;     // elements of a head that are rotated, at most
constexpr int kMaxNewTokens = 8;    // of a sequence, in one attention call
constexpr int kMaxCached = (1 << 30) - 1;  // tokens of a sequence

// Launches a kernel that waits itself for what is before it on the stream: its
// blocks may be set up while that ends.
template <typename... Params, typename... Args>
gdn_status launch_programmatic(void (*kernel)(Params...), dim3 grid, int threads, size_t bytes,
                               cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// ------------------------------------------------------------------ launchers
// v, cache and cu belong to the append (cache null: gdn_qk_norm_rope).
gdn_status launch_qk_rope(const gdn_rope_problem &p, const gdn_paged_cache *cache, const void *q,
                          const void *k, const void *v, const float *q_weight,
                          const float *k_weight, const int32_t *positions, const float *inv_freq,
                          const int32_t *cu, void *q_out, void *k_out, cudaStream_t stream);
size_t paged_attention_workspace(const gdn_attention_problem &p, const gdn_paged_cache &c);
gdn_status launch_paged_attention(const gdn_attention_problem &p, const gdn_paged_cache &c,
                                  const void *q, const void *gate, void *out, float *lse,
                                  cudaStream_t stream);

}  // namespace gdn
