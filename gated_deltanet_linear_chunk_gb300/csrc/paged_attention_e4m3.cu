// paged_attention_e4m3.cu -- attention of bf16 over an 8-bit cache (a translation unit of its own,
// compiled beside the others).
#include "paged_attention_simt.cuh"

namespace gdn {

AttentionShape shape_e4m3(int R, int) { return simt_shape(R); }

gdn_status attention_e4m3(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    return simt_attention<__nv_bfloat16, __nv_fp8_e4m3>(D, blocks, a, stream);
}

}  // namespace gdn
