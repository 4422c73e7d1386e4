// ew_policy_f16.cu -- the policy loss's kernels for binary16.
#include "ew_policy.cuh"

namespace ew {

cudaError_t policy_f16(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return policy_launch<DT_F16>(a, sums, grad, sms, s, info);
}

}  // namespace ew
