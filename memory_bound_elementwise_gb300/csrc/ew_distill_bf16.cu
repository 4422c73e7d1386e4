// ew_distill_bf16.cu -- the distillation kernels for bfloat16.
#include "ew_distill.cuh"

namespace ew {

cudaError_t distill_bf16(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    return distill_launch<DT_BF16>(a, sums, grad, sms, s, info);
}

}  // namespace ew
