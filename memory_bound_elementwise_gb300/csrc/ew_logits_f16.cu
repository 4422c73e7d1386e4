// ew_logits_f16.cu -- the kernels on rows of logits for binary16.
#include "ew_logits.cuh"

namespace ew {

cudaError_t logprob_f16(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return logprob_launch<DT_F16>(a, sms, s, info);
}
cudaError_t logprob_grad_f16(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info) {
    return logprob_grad_launch<DT_F16>(a, s, info);
}

}  // namespace ew
