// ew_norm_f32.cu -- the RMS norm kernels for binary32.
#include "ew_norm.cuh"

namespace ew {

cudaError_t norm_f32(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return norm_dispatch<DT_F32>(quant, a, sms, s, info);
}
cudaError_t norm_grad_f32(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                         int *launches) {
    return norm_grad_dispatch<DT_F32>(a, most_writers, sms, s, info, launches);
}

}  // namespace ew
