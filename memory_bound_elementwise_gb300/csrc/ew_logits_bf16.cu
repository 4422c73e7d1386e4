// ew_logits_bf16.cu -- the kernels on rows of logits for bfloat16.
#include "ew_logits.cuh"

namespace ew {

cudaError_t logprob_bf16(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return logprob_launch<DT_BF16>(a, sms, s, info);
}
cudaError_t logprob_grad_bf16(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info) {
    return logprob_grad_launch<DT_BF16>(a, s, info);
}

}  // namespace ew
