// paged_attention_e4m3.cu -- attention of bf16 over an 8-bit cache (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_mma.cuh"

namespace gdn {

AttentionShape shape_e4m3(int R, int D) { return mma_shape(true, R, D); }

gdn_status attention_e4m3(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    return mma_attention<true>(D, blocks, a, stream);
}

}  // namespace gdn
