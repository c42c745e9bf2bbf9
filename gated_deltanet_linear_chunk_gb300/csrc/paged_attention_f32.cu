// paged_attention_f32.cu -- attention of fp32 (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_simt.cuh"

namespace gdn {

AttentionShape shape_f32(int R, int) { return simt_shape(R); }

gdn_status attention_f32(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    return simt_attention<float, float>(D, blocks, a, stream);
}

}  // namespace gdn
