// ew_policy_bf16.cu -- the policy loss's kernels for bfloat16.
#include "ew_policy.cuh"

namespace ew {

cudaError_t policy_bf16(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return policy_launch<DT_BF16>(a, sums, grad, sms, s, info);
}

}  // namespace ew
