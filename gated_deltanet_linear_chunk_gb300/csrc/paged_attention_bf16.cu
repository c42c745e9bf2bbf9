// paged_attention_bf16.cu -- attention of bf16 (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_mma.cuh"

namespace gdn {

AttentionShape shape_bf16(int R, int D) { return mma_shape(false, R, D); }

gdn_status attention_bf16(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    return mma_attention<false>(D, blocks, a, stream);
}

}  // namespace gdn
