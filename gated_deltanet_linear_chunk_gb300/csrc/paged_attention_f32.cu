// paged_attention_f32.cu -- attention of fp32 (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_simt.cuh"

namespace gdn {

AttentionShape shape_f32(int R, int D) { return simt_shape(R, D); }

gdn_status attention_f32(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (D == 64) return simt_rows<64>(blocks, a, stream);
    if (D == 128) return simt_rows<128>(blocks, a, stream);
    return simt_rows<256>(blocks, a, stream);
}

}  // namespace gdn
