// ew_rows.cu -- kernels that several row operators share.
#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// out[c] = sum over r of rows[r][c], in a fixed order: 32 warps each add every
// 32nd row, then the 32 sums are added in order.  A block takes 32 columns, so
// a warp reads whole lines; the rows come from L2, where the kernel before
// left them, and what counts is how many loads are under way at once.
// TWO: the second row of blocks adds the n rows after the first n, into out2.  A kernel of
// its own: with the choice in the one for both, the norm's backward of 9 rows of 12000
// binary32 took 11.7 us, without 10.1.
template <bool TWO>
__global__ void __launch_bounds__(1024) column_sums_kernel(const float *rows, int64_t n, int32_t cols, float *out,
                                                           float *out2) {
    enter_grid();
    if constexpr (TWO) {
        if (blockIdx.y > 0) {
            rows += n * cols;
            out = out2;
        }
        if (out == nullptr) return;
    }
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

cudaError_t launch_column_sums(const float *rows, int64_t n, int32_t cols, float *out, cudaStream_t s, bool two,
                               float *out2) {
    return launch_rows(two ? column_sums_kernel<true> : column_sums_kernel<false>, dim3((cols + 31) / 32, two ? 2 : 1),
                       dim3(1024), 0, 1, s, rows, n, cols, out, out2);
}

}  // namespace ew
