// ew_norm_bf16.cu -- the RMS norm kernels for bfloat16.
#include "ew_norm.cuh"

namespace ew {

cudaError_t norm_bf16(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return norm_dispatch<DT_BF16>(quant, a, sms, s, info);
}
cudaError_t norm_grad_bf16(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                         int *launches) {
    return norm_grad_dispatch<DT_BF16>(a, most_writers, sms, s, info, launches);
}

}  // namespace ew
