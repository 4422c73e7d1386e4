// ew_rows.cu -- kernels that several row operators share.
#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// out[c] = sum over r of rows[r][c], in a fixed order: 8 lanes of rows each add
// every eighth row, then the 8 sums are added.  A block takes 32 columns.
__global__ void __launch_bounds__(256) column_sums_kernel(const float *rows, int64_t n, int32_t cols, float *out) {
    enter_grid();
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int64_t r = strip; r < n; r += 8) sum += rows[r * cols + col];
    }
    part[strip][lane] = sum;
    __syncthreads();
    if (strip == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) sum += part[k][lane];
        out[col] = sum;
    }
}

}  // namespace

cudaError_t launch_column_sums(const float *rows, int64_t n, int32_t cols, float *out, cudaStream_t s) {
    return launch_rows(column_sums_kernel, dim3((cols + 31) / 32), dim3(256), 0, 1, s, rows, n, cols, out);
}

}  // namespace ew
