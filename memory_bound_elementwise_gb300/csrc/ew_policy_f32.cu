// ew_policy_f32.cu -- the policy loss's kernels for binary32.
#include "ew_policy.cuh"

namespace ew {

cudaError_t policy_f32(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return policy_launch<DT_F32>(a, sums, grad, sms, s, info);
}

}  // namespace ew
