// ew_layernorm_f32.cu -- the layer norm kernels for binary32.
#include "ew_layernorm.cuh"

namespace ew {

cudaError_t layernorm_f32(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return layernorm_dispatch<DT_F32>(a, sms, s, info);
}
cudaError_t layernorm_grad_f32(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                              int *launches) {
    return layernorm_grad_dispatch<DT_F32>(a, most_writers, sms, s, info, launches);
}

}  // namespace ew
