// ew_rows.cu -- kernels that several row operators share.
#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// out[c] = sum over r of rows[r][c], in a fixed order: 32 warps each add every
// 32nd row, then the 32 sums are added in order.  A block takes 32 columns, so
// a warp reads whole lines; the rows come from L2, where the kernel before
// left them, and what counts is how many loads are under way at once.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float *rows, int64_t n, int32_t cols, float *out) {
    enter_grid();
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < cols) {
        int64_t r = strip;
        for (; r + 7 * 32 < n; r += 8 * 32) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = rows[(r + k * 32) * cols + col];
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += v[k];
        }
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = r + k * 32 < n ? rows[(r + k * 32) * cols + col] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += v[k];
    }
    part[strip][lane] = sum;
    __syncthreads();
    // warp w finishes column w: lane k takes strip k
    sum = warp_sum(part[lane][strip]);
    if (lane == 0 && blockIdx.x * 32 + strip < cols) out[blockIdx.x * 32 + strip] = sum;
}

}  // namespace

cudaError_t launch_column_sums(const float *rows, int64_t n, int32_t cols, float *out, cudaStream_t s) {
    return launch_rows(column_sums_kernel, dim3((cols + 31) / 32), dim3(1024), 0, 1, s, rows, n, cols, out);
}

}  // namespace ew
