// selective_scan_f32.cu -- the selective scan and its step for fp32 inputs
// (selective_scan.cuh), in a translation unit of their own so that the two
// types compile side by side.
#include "selective_scan.cuh"

namespace gdn {

gdn_status launch_selective_scan_f32(const gdn_ssm_problem &p, const void *x, const void *dt,
                                      const float *A, const void *B, const void *C,
                                      const float *skip, const void *z, const float *bias,
                                      const int32_t *cu, const float *init, void *out, float *fin,
                                      cudaStream_t stream) {
    return scan_typed<float>(p, x, dt, A, B, C, skip, z, bias, cu, init, out, fin, stream);
}

gdn_status launch_selective_scan_step_f32(const gdn_ssm_problem &p, const void *x,
                                           const void *dt, const float *A, const void *B,
                                           const void *C, const float *skip, const void *z,
                                           const float *bias, const float *state, void *out,
                                           float *next, cudaStream_t stream) {
    return scan_step_typed<float>(p, x, dt, A, B, C, skip, z, bias, state, out, next, stream);
}

size_t scan_workspace_size(const gdn_ssm_problem &p) {
    const ScanPlan pl = scan_plan(p);
    if (pl.W <= 1) return 0;
    return (size_t)(pl.W - 1) * p.channels * (p.state_dim + 1) * sizeof(float);
}

}  // namespace gdn
