// ew_layernorm_bf16.cu -- the layer norm kernels for bfloat16.
#include "ew_layernorm.cuh"

namespace ew {

cudaError_t layernorm_bf16(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return layernorm_dispatch<DT_BF16>(a, sms, s, info);
}
cudaError_t layernorm_grad_bf16(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                              int *launches) {
    return layernorm_grad_dispatch<DT_BF16>(a, most_writers, sms, s, info, launches);
}

}  // namespace ew
