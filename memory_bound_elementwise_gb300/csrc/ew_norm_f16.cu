// ew_norm_f16.cu -- the RMS norm kernels for binary16.
#include "ew_norm.cuh"

namespace ew {

cudaError_t norm_f16(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return norm_dispatch<DT_F16>(quant, a, sms, s, info);
}
cudaError_t norm_grad_f16(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                         int *launches) {
    return norm_grad_dispatch<DT_F16>(a, most_writers, sms, s, info, launches);
}

}  // namespace ew
