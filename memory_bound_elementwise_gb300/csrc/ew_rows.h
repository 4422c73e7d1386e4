// ew_rows.h -- interface between the host side of the row operators
// (ew_rows_api.cu) and their kernels.  Not installed.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ew.h"
#include "ew_internal.h"

namespace ew {

// From ew_api.cu: state that all calls of the library share.
ew_status report_cuda(cudaError_t e);     // EW_ERR_CUDA, and keeps e for ew_last_cuda_error
ew_launch_record &launch_record();        // this thread's record of its last call
ew_status check_pointers(const void *const *p, int np);  // the optional pointer check; null entries pass
cudaError_t current_sms(int *sms);        // multiprocessors of the current device

// What a launch wrapper did, for the launch record.
struct LaunchInfo {
    int grid = 0, block = 0, smem = 0, vec_bytes = 0;
};

// launch_kernel with grids and blocks of up to three dimensions and, from two
// on, a thread-block cluster of `cluster` blocks along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned cluster,
                        cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (programmatic_launch()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) (void)cudaGetLastError();  // the failure is returned; do not leave it pending too
    return e;
}

// Lets a kernel use up to `bytes` of dynamic shared memory: once per kernel and
// device, of which `done` keeps a bit each (devices past 63 are asked every time).
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
    return e;
}

// Adds `n` rows of `cols` binary32 values in order into out[cols] (zeros where
// n is 0); with `two`, the n rows after those into out2[cols] in the same launch.
// Null outputs are left out.
cudaError_t launch_column_sums(const float *rows, int64_t n, int32_t cols, float *out, cudaStream_t s, bool two = false,
                               float *out2 = nullptr);

// ---------------------------------------------------------------- norm

struct NormArgs {
    const void *x, *residual, *weight;
    void *out;        // y, or q of the 8-bit forms
    void *h;          // null where not wanted
    float *rstd;      // null where not wanted
    float *scales;
    int64_t x_stride, residual_stride, out_stride, h_stride, scales_stride;
    int64_t rows;
    int32_t cols;
    int32_t group_shift;  // log2 of the columns a scale; 0: the row
    float eps, per_col;   // per_col: 1 / cols
    int32_t weight_f32;
    int32_t i8;       // 8-bit forms: int8 instead of e4m3
};
cudaError_t norm_f32(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t norm_f16(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t norm_bf16(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);

struct NormGradArgs {
    const void *dy, *h, *weight, *dh;
    const float *rstd;
    void *dx;
    float *dweight;
    float *partial;   // workspace: partial sums of dweight, one row of cols per writer
    int64_t dy_stride, h_stride, dh_stride, dx_stride;
    int64_t rows;
    int32_t cols;
    int32_t weight_f32;
};
// most_writers: rows of cols that the workspace holds.
cudaError_t norm_grad_f32(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                          int *launches);
cudaError_t norm_grad_f16(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                          int *launches);
cudaError_t norm_grad_bf16(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                           int *launches);

struct LayerNormArgs {
    const void *x, *residual, *weight, *bias;
    void *y, *h;          // h null where not wanted
    float *mean, *rstd;   // null where not wanted
    int64_t x_stride, residual_stride, y_stride, h_stride;
    int64_t rows;
    int32_t cols;
    float eps, per_col;   // per_col: 1 / cols
    int32_t weight_f32;   // the weight's and the bias's type
};
cudaError_t layernorm_f32(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t layernorm_f16(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t layernorm_bf16(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info);

struct LayerNormGradArgs {
    const void *dy, *h, *weight, *dh;
    const float *mean, *rstd;
    void *dx;
    float *dweight, *dbias;  // null where not wanted
    float *partial;          // workspace: each writer's sums of dweight, then each writer's of dbias
    int64_t dy_stride, h_stride, dh_stride, dx_stride;
    int64_t rows;
    int32_t cols;
    int32_t weight_f32;
};
// most_writers: twice as many rows of cols fit the workspace.
cudaError_t layernorm_grad_f32(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                               int *launches);
cudaError_t layernorm_grad_f16(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                               int *launches);
cudaError_t layernorm_grad_bf16(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                                int *launches);

// ---------------------------------------------------------------- embedding

struct EmbedArgs {
    const void *table, *tokens;
    void *out;
    int64_t table_rows, table_stride, out_stride, rows;
    int32_t cols;
    int32_t i64;  // tokens are 64-bit integers
    float scale;
};
cudaError_t launch_embed(int dtype, const EmbedArgs &a, int sms, cudaStream_t s, LaunchInfo *info);

struct EmbedGradArgs {
    const void *dout, *tokens;
    void *dtable;
    int64_t dout_stride, table_rows, table_stride, rows;
    int32_t cols;
    int32_t i64;
    int32_t accumulate;
    float scale;
    // workspace
    uint2 *items0, *items1;  // (token, position) between passes of the sort
    uint32_t *keys, *order;  // sorted tokens (table_rows: none) and their positions
    uint32_t *present;       // a bit for each table row that a token names; null with accumulate
    float *partial;          // sums of the runs that cross chunks
    // set by the launch
    int64_t blind;           // rows that are cleared beside the sort
    int32_t chunk;           // sorted positions a warp adds
};
int64_t embed_partial_bytes(int64_t rows, int64_t cols);
cudaError_t launch_embed_grad(int dtype, int gtype, const EmbedGradArgs &a, int sms, cudaStream_t s,
                              LaunchInfo *info, int *launches);

// ---------------------------------------------------------------- experts

constexpr int kMostExperts = 1024;
constexpr int kMostChoices = 64;  // experts a token

struct ExpertSortArgs {
    const void *experts;  // rows x k
    int32_t *positions, *offsets, *counts, *slots;
    uint32_t *partial;    // workspace: the blocks' counts
    int64_t stride, rows, capacity;
    int32_t k, n_experts, align, i64;
};
int64_t expert_sort_bytes(int64_t slots, int n_experts);
cudaError_t launch_expert_sort(const ExpertSortArgs &a, cudaStream_t s, LaunchInfo *info, int *launches);

// Dispatch: x by tokens, out by sorted rows.  Combine: x by sorted rows, residual
// and out by tokens.  Combine's gradient: x is combine's (null where dweights is),
// residual its output's gradient, out x's.
struct ExpertRowsArgs {
    const void *x, *residual, *weights;
    const int32_t *positions, *slots;
    void *out;
    float *dweights;
    int64_t x_stride, residual_stride, out_stride;
    int64_t rows, sorted;  // tokens, and sorted rows
    int32_t cols, k, wtype;
};
enum ExpertRows : int { EXPERT_DISPATCH = 0, EXPERT_COMBINE = 1, EXPERT_COMBINE_GRAD = 2 };
cudaError_t launch_expert_rows(int what, int dtype, const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info);

// ---------------------------------------------------------------- logits

constexpr int kMostTop = 64;        // alternatives a row
constexpr int kMostTeacher = 1024;  // teacher entries a row

struct LogprobArgs {
    const void *logits, *tokens;
    float *logp, *entropy, *lse;  // null where not wanted
    float *top_logp;
    int32_t *top_ids;
    int64_t stride, rows;
    int32_t cols, i64, top;
    float scale;
};
struct LogprobGradArgs {
    const void *logits, *tokens;
    const float *lse, *entropy, *dlogp, *dentropy;
    void *dlogits;
    int64_t stride, dstride, rows;
    int32_t cols, i64;
    float scale;
};
struct DistillArgs {
    const void *logits, *ids, *teacher;
    const float *dloss;
    float *loss, *lse;  // lse: an input of the gradient alone
    void *dlogits;
    int64_t stride, ids_stride, teacher_stride, dstride, rows;
    int32_t cols, i64, teacher_f32, k;
    float scale;
};
struct PolicyArgs {
    const void *logits, *tokens;
    const float *advantage, *old_logp, *ref_logp;  // the last two null where not given
    const float *logp, *lse;                       // inputs of the gradient alone
    const float *dloss;
    float *loss, *logp_out, *lse_out;              // the last two null where not wanted
    void *dlogits;
    int64_t stride, dstride, rows;
    int32_t cols, i64;
    float least, most;  // of the ratio, where it is clipped
    float kl, scale;
};
cudaError_t policy_f32(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t policy_f16(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t policy_bf16(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);
// sums: the loss and lse are computed; grad: dlogits is.
cudaError_t logprob_f32(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t logprob_grad_f32(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info);
cudaError_t distill_f32(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t logprob_f16(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t logprob_grad_f16(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info);
cudaError_t distill_f16(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t logprob_bf16(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info);
cudaError_t logprob_grad_bf16(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info);
cudaError_t distill_bf16(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info);

}  // namespace ew
