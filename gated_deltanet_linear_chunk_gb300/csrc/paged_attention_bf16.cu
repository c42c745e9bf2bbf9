// paged_attention_bf16.cu -- attention of bf16 (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_simt.cuh"

namespace gdn {

AttentionShape shape_bf16(int R, int) { return simt_shape(R); }

gdn_status attention_bf16(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    return simt_attention<__nv_bfloat16, __nv_bfloat16>(D, blocks, a, stream);
}

}  // namespace gdn
