// ew_logits_f32.cu -- the kernels on rows of logits for binary32.
#include "ew_logits.cuh"

namespace ew {

cudaError_t logprob_f32(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return logprob_launch<DT_F32>(a, sms, s, info);
}
cudaError_t logprob_grad_f32(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info) {
    return logprob_grad_launch<DT_F32>(a, s, info);
}

}  // namespace ew
