// ew_distill_f16.cu -- the distillation kernels for binary16.
#include "ew_distill.cuh"

namespace ew {

cudaError_t distill_f16(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return distill_launch<DT_F16>(a, sums, grad, sms, s, info);
}

}  // namespace ew
