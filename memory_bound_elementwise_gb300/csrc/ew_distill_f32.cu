// ew_distill_f32.cu -- the distillation kernels for binary32.
#include "ew_distill.cuh"

namespace ew {

cudaError_t distill_f32(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return distill_launch<DT_F32>(a, sums, grad, sms, s, info);
}

}  // namespace ew
