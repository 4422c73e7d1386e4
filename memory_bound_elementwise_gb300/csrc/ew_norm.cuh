// ew_norm.cuh -- root-mean-square norm with the residual's addition, its 8-bit
// output, and its backward.  Compiled once per element type.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * w
//
// Each row is read once: a block holds it in registers (KT tiles of 8 elements
// a thread) between the sum of squares and the outputs.  The bound is memory:
// x, residual, h and y of 16-bit elements move 8 bytes an element for about 5
// operations.
#pragma once

#include <algorithm>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100: a scale is never zero

__device__ __forceinline__ uint32_t quant_pair(float hi, float lo, bool i8) {
    if (i8) {
        int32_t a, b;
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(lo));
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(hi));
        return (a & 0xff) | ((b & 0xff) << 8);
    }
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Scale of a group whose largest absolute value is amax, and the factor that
// takes y to q.  One division a group instead of one an element: the product
// is within a rounding of y / scale.
__device__ __forceinline__ float quant_factor(float amax, float qmax, float *scale) {
    amax = max_nan(amax, kAmaxFloor);
    *scale = amax / qmax;
    return qmax / amax;
}

// Quantises the lane's 8 values of y of one tile and stores them, with the
// group's scales.  Every lane of the warp takes part.
template <bool VEC>
__device__ __forceinline__ void quant_tile(const float (&y)[8], const NormArgs &a, int64_t row, int base, int lane,
                                           float row_factor) {
    const float qmax = a.i8 ? 127.0f : 448.0f;
    uint8_t *q = static_cast<uint8_t *>(a.out) + row * a.out_stride;
    float f[8];
    if (a.group == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = row_factor;
    } else {
        float *scales = a.scales + row * a.scales_stride;
        if (VEC) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(y[j]));
            const int lanes = a.group / 8;
            m = lanes_max_nan(m, lanes);
            float scale;
            const float factor = quant_factor(m, qmax, &scale);
            const int c0 = base + lane * 8;
            if (lane % lanes == 0 && c0 < a.cols) scales[c0 / a.group] = scale;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = factor;
        } else {
            const int per = a.group / 32;  // steps of 32 columns a group
            float m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = lanes_max_nan(fabsf(y[j]), 32);
            for (int d = 1; d < per; d <<= 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (((j & d) == 0)) {
                        const float v = max_nan(m[j], m[(j + d) & 7]);
                        m[j] = v;
                    }
                }
            }
            // after log2(per) rounds the first step of each group holds its largest value
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float first = m[0];
#pragma unroll
                for (int k = 1; k < 8; ++k) first = (j / per) * per == k ? m[k] : first;
                float scale;
                f[j] = quant_factor(first, qmax, &scale);
                const int c = base + j * 32;
                if (lane == 0 && j % per == 0 && c < a.cols) scales[c / a.group] = scale;
            }
        }
    }
    const int c0 = tile_col<VEC>(base, lane, 0);
    if (VEC && c0 + 8 <= a.cols) {
        Vec<8> v;
        v.w[0] = quant_pair(y[1] * f[1], y[0] * f[0], a.i8) | (quant_pair(y[3] * f[3], y[2] * f[2], a.i8) << 16);
        v.w[1] = quant_pair(y[5] * f[5], y[4] * f[4], a.i8) | (quant_pair(y[7] * f[7], y[6] * f[6], a.i8) << 16);
        st<8>(q + c0, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tile_col<VEC>(base, lane, j);
            if (c < a.cols) q[c] = static_cast<uint8_t>(quant_pair(0.0f, y[j] * f[j], a.i8));
        }
    }
}

// One row to a block of `warps` warps (blockDim.x), tile t of the row to warp
// t mod warps; with one warp a row, blockDim.y rows to a block.  HELD: the
// warps x KT tiles cover the row, which stays in registers.  Otherwise (rows
// beyond 16 warps x 4 tiles) the passes read the row again, each thread its
// own elements, and h is written by the last pass, so in-place forms hold.
template <int DT, bool VEC, int KT, bool QUANT, bool HELD>
__global__ void __launch_bounds__(HELD ? 512 : 1024) norm_kernel(NormArgs a) {
    enter_grid();
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;  // whole warps: blockDim.y > 1 only with one warp a row
    const void *x = row_of<DT>(a.x, row, a.x_stride);
    const void *res = a.residual ? row_of<DT>(a.residual, row, a.residual_stride) : nullptr;
    void *h = a.h ? row_of<DT>(a.h, row, a.h_stride) : nullptr;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    const float qmax = a.i8 ? 127.0f : 448.0f;

    auto sum_of = [&](int base, float (&f)[8]) {
        unpack8<DT>(load_tile<DT, VEC>(x, base, a.cols, lane), f);
        if (res) {
            float g[8];
            unpack8<DT>(load_tile<DT, VEC>(res, base, a.cols, lane), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
        }
    };
    auto scaled = [&](int base, float r, const float (&f)[8], float (&y)[8]) {
        load_weight<DT, VEC>(a.weight, a.weight_f32, base, a.cols, lane, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= f[j] * r;
    };
    auto put = [&](int base, const float (&y)[8], float row_factor) {
        if constexpr (QUANT) quant_tile<VEC>(y, a, row, base, lane, row_factor);
        else store_tile<DT, VEC>(row_of<DT>(a.out, row, a.out_stride), base, a.cols, lane, pack8<DT>(y));
    };
    auto rstd_of = [&](float ss) {
        const float r = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
        return r;
    };
    auto row_scale = [&](float amax) {
        float scale;
        const float factor = quant_factor(amax, qmax, &scale);
        if (threadIdx.x == 0) a.scales[row * a.scales_stride] = scale;
        return factor;
    };

    float ss = 0.0f;
    if constexpr (HELD) {
        float f[KT][8];
        Raw8<DT> rx[KT], rr[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) rx[k] = load_tile<DT, VEC>(x, (warp + k * warps) * kTileCols, a.cols, lane);
        if (res) {
#pragma unroll
            for (int k = 0; k < KT; ++k) rr[k] = load_tile<DT, VEC>(res, (warp + k * warps) * kTileCols, a.cols, lane);
        }
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            unpack8<DT>(rx[k], f[k]);
            if (res) {
                float g[8];
                unpack8<DT>(rr[k], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[k][j] += g[j];
            }
            if (h) store_tile<DT, VEC>(h, (warp + k * warps) * kTileCols, a.cols, lane, pack8<DT>(f[k]));
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[k][j], f[k][j], ss);
        }
        const float r = rstd_of(block_sum(ss, warps, part[0]));
        float amax = 0.0f, factor = 0.0f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float y[8];
            scaled((warp + k * warps) * kTileCols, r, f[k], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[k][j] = y[j];
        }
        if (QUANT && a.group == 0) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(f[k][j]));
            factor = row_scale(block_max_nan(amax, warps, part[1]));
        }
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const int base = (warp + k * warps) * kTileCols;
            if (base < a.cols) put(base, f[k], factor);
        }
    } else {
        for (int t = warp; t < tiles; t += warps) {
            float f[8];
            sum_of(t * kTileCols, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
        }
        const float r = rstd_of(block_sum(ss, warps, part[0]));
        float factor = 0.0f;
        if (QUANT && a.group == 0) {
            float amax = 0.0f;
            for (int t = warp; t < tiles; t += warps) {
                float f[8], y[8];
                sum_of(t * kTileCols, f);
                scaled(t * kTileCols, r, f, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(y[j]));
            }
            factor = row_scale(block_max_nan(amax, warps, part[1]));
        }
        for (int t = warp; t < tiles; t += warps) {
            float f[8], y[8];
            sum_of(t * kTileCols, f);
            if (h) store_tile<DT, VEC>(h, t * kTileCols, a.cols, lane, pack8<DT>(f));
            scaled(t * kTileCols, r, f, y);
            put(t * kTileCols, y, factor);
        }
    }
}

// Backward.  Per row: c = mean(g * n) with n = h * r, g = dy * w; then
// dx = r * (g - n * c) + dh.  Blocks walk over rows (row, row + writers, ..)
// and keep their columns' sums of dy * n in registers; each writes them once,
// to its own row of `partial`, and dweight_kernel adds those rows in order.
template <int DT, bool VEC, int KT>
__global__ void __launch_bounds__(512) norm_grad_kernel(NormGradArgs a) {
    enter_grid();
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t writer = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t writers = static_cast<int64_t>(gridDim.x) * blockDim.y;
    float dw[KT][8];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
    int turn = 0;
    for (int64_t row = writer; row < a.rows; row += writers, turn ^= 1) {
        const void *dy = row_of<DT>(a.dy, row, a.dy_stride), *h = row_of<DT>(a.h, row, a.h_stride);
        const float r = a.rstd[row];
        Raw8<DT> rdy[KT], rh[KT], rdh[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            rdy[k] = load_tile<DT, VEC>(dy, (warp + k * warps) * kTileCols, a.cols, lane);
            rh[k] = load_tile<DT, VEC>(h, (warp + k * warps) * kTileCols, a.cols, lane);
        }
        if (a.dh) {
            const void *dh = row_of<DT>(a.dh, row, a.dh_stride);
#pragma unroll
            for (int k = 0; k < KT; ++k) rdh[k] = load_tile<DT, VEC>(dh, (warp + k * warps) * kTileCols, a.cols, lane);
        }
        // dy and n of a tile, and its weights, read again from L1 rather than held
        auto products = [&](int k, float (&g)[8], float (&n)[8]) {
            float w[8];
            load_weight<DT, VEC>(a.weight, a.weight_f32, (warp + k * warps) * kTileCols, a.cols, lane, w);
            unpack8<DT>(rdy[k], g);
            unpack8<DT>(rh[k], n);
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] *= r;
            return [&, w](int j) { return w[j]; };
        };
        float c = 0.0f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float g[8], n[8];
            auto w = products(k, g, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[k][j] = fmaf(g[j], n[j], dw[k][j]);
                c = fmaf(g[j] * w(j), n[j], c);
            }
        }
        c = block_sum(c, warps, part[turn]) / static_cast<float>(a.cols);
        void *dx = row_of<DT>(a.dx, row, a.dx_stride);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float g[8], n[8], d[8];
            auto w = products(k, g, n);
            if (a.dh) unpack8<DT>(rdh[k], d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fmaf(-c, n[j], g[j] * w(j));
                d[j] = a.dh ? fmaf(r, v, d[j]) : r * v;
            }
            store_tile<DT, VEC>(dx, (warp + k * warps) * kTileCols, a.cols, lane, pack8<DT>(d));
        }
    }
    if (a.dweight == nullptr) return;
    float *out = a.partial + writer * a.cols;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = tile_col<VEC>((warp + k * warps) * kTileCols, lane, j);
            if (col < a.cols) out[col] = dw[k][j];
        }
}

// Rows too wide to hold: the row's two passes read it twice.  dweight has its
// own kernel (norm_dweight_wide_kernel), which runs first: dx may be dy.
template <int DT, bool VEC>
__global__ void __launch_bounds__(1024) norm_grad_wide_kernel(NormGradArgs a) {
    enter_grid();
    __shared__ float part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    const void *dy = row_of<DT>(a.dy, row, a.dy_stride), *h = row_of<DT>(a.h, row, a.h_stride);
    const float r = a.rstd[row];
    auto products = [&](int base, float (&g)[8], float (&n)[8]) {
        float w[8];
        load_weight<DT, VEC>(a.weight, a.weight_f32, base, a.cols, lane, w);
        unpack8<DT>(load_tile<DT, VEC>(dy, base, a.cols, lane), g);
        unpack8<DT>(load_tile<DT, VEC>(h, base, a.cols, lane), n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            n[j] *= r;
            g[j] *= w[j];
        }
    };
    float c = 0.0f, g[8], n[8];
    for (int t = warp; t < tiles; t += warps) {
        products(t * kTileCols, g, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) c = fmaf(g[j], n[j], c);
    }
    c = block_sum(c, warps, part) / static_cast<float>(a.cols);
    void *dx = row_of<DT>(a.dx, row, a.dx_stride);
    for (int t = warp; t < tiles; t += warps) {
        products(t * kTileCols, g, n);
        float d[8];
        if (a.dh) unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.dh, row, a.dh_stride), t * kTileCols, a.cols, lane), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fmaf(-c, n[j], g[j]);
            d[j] = a.dh ? fmaf(r, v, d[j]) : r * v;
        }
        store_tile<DT, VEC>(dx, t * kTileCols, a.cols, lane, pack8<DT>(d));
    }
}

// dweight of wide rows: one warp takes a tile of columns over the rows
// blockIdx.y, blockIdx.y + gridDim.y, ..
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) norm_dweight_wide_kernel(NormGradArgs a) {
    enter_grid();
    const int lane = threadIdx.x & 31;
    const int base = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kTileCols;
    if (base >= a.cols) return;
    float dw[8] = {};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float g[8], n[8];
        const float r = a.rstd[row];
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.dy, row, a.dy_stride), base, a.cols, lane), g);
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.h, row, a.h_stride), base, a.cols, lane), n);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = fmaf(g[j], n[j] * r, dw[j]);
    }
    float *out = a.partial + static_cast<int64_t>(blockIdx.y) * a.cols;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = tile_col<VEC>(base, lane, j);
        if (col < a.cols) out[col] = dw[j];
    }
}

// ---------------------------------------------------------------- launches

constexpr int kHeldWarps = 16;

// Smallest number of tiles a thread (1, 2 or 4) with which `warps` warps hold a
// row of `tiles` tiles; 0 where none does.
inline int tiles_per_thread(int tiles, int warps, int most) {
    for (int kt = 1; kt <= most; kt *= 2)
        if ((tiles + kt - 1) / kt <= warps) return kt;
    return 0;
}

template <int DT> bool wide_weight(const void *w, bool f32) {
    return reinterpret_cast<uintptr_t>(w) % (f32 || DT == DT_F32 ? 32 : 16) == 0;
}

template <int DT, bool VEC, bool QUANT>
cudaError_t norm_launch(const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    // One tile a thread where rows are few (the row's latency counts), up to
    // four where they are many.
    const bool many = a.rows >= 4 * static_cast<int64_t>(sms);
    const int kt = tiles_per_thread(tiles, many ? std::min(kHeldWarps, std::max(1, (tiles + 1) / 2)) : kHeldWarps, 4);
    int warps = 32, per_block = 1;
    if (kt != 0) {
        warps = (tiles + kt - 1) / kt;
        if (warps == 1 && many) per_block = 8;
    }
    const int64_t grid = (a.rows + per_block - 1) / per_block;
    const dim3 block(32 * warps, per_block);
    info->grid = static_cast<int>(grid);
    info->block = 32 * warps * per_block;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    switch (kt) {
        case 1: return launch_rows(norm_kernel<DT, VEC, 1, QUANT, true>, dim3(grid), block, 0, 1, s, a);
        case 2: return launch_rows(norm_kernel<DT, VEC, 2, QUANT, true>, dim3(grid), block, 0, 1, s, a);
        case 4: return launch_rows(norm_kernel<DT, VEC, 4, QUANT, true>, dim3(grid), block, 0, 1, s, a);
        default: return launch_rows(norm_kernel<DT, VEC, 1, QUANT, false>, dim3(grid), block, 0, 1, s, a);
    }
}

template <int DT> cudaError_t norm_dispatch(bool quant, const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const bool out_wide = quant ? reinterpret_cast<uintptr_t>(a.out) % 8 == 0 && a.out_stride % 8 == 0
                                : wide_rows<DT>(a.out, a.out_stride);
    const bool vec = out_wide && wide_rows<DT>(a.x, a.x_stride) && wide_rows<DT>(a.residual, a.residual_stride) &&
                     wide_rows<DT>(a.h, a.h_stride) && wide_weight<DT>(a.weight, a.weight_f32);
    if (quant) return vec ? norm_launch<DT, true, true>(a, sms, s, info) : norm_launch<DT, false, true>(a, sms, s, info);
    return vec ? norm_launch<DT, true, false>(a, sms, s, info) : norm_launch<DT, false, false>(a, sms, s, info);
}

template <int DT, bool VEC>
cudaError_t norm_grad_launch(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                             int *launches) {
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int kt = tiles_per_thread(tiles, kHeldWarps, DT == DT_F32 ? 2 : 4);
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    int64_t writers = 0;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && kt != 0) {
        const int warps = (tiles + kt - 1) / kt;
        const int per_block = warps == 1 && a.rows >= 4 * static_cast<int64_t>(sms) ? 4 : 1;
        const int resident = std::max(1, 16 / (warps * per_block));  // blocks that 512 threads of an SM make
        const int64_t grid = std::min<int64_t>({(a.rows + per_block - 1) / per_block,
                                                static_cast<int64_t>(sms) * resident, most_writers / per_block});
        writers = grid * per_block;
        const dim3 block(32 * warps, per_block);
        info->grid = static_cast<int>(grid);
        info->block = 32 * warps * per_block;
        e = kt == 1   ? launch_rows(norm_grad_kernel<DT, VEC, 1>, dim3(grid), block, 0, 1, s, a)
            : kt == 2 ? launch_rows(norm_grad_kernel<DT, VEC, 2>, dim3(grid), block, 0, 1, s, a)
                      : launch_rows(norm_grad_kernel<DT, VEC, 4>, dim3(grid), block, 0, 1, s, a);
        ++*launches;
    } else if (a.rows > 0) {
        if (a.dweight) {
            writers = std::min<int64_t>({a.rows, most_writers, std::max(1, 8 * sms * 8 / tiles)});
            e = launch_rows(norm_dweight_wide_kernel<DT, VEC>, dim3((tiles + 7) / 8, static_cast<unsigned>(writers)),
                            dim3(256), 0, 1, s, a);
            ++*launches;
        }
        if (e == cudaSuccess)
            e = launch_rows(norm_grad_wide_kernel<DT, VEC>, dim3(static_cast<unsigned>(a.rows)), dim3(1024), 0, 1, s, a);
        ++*launches;
        info->grid = static_cast<int>(a.rows);
        info->block = 1024;
    }
    if (e != cudaSuccess || a.dweight == nullptr) return e;
    ++*launches;
    return launch_column_sums(a.partial, writers, a.cols, a.dweight, s);
}

template <int DT>
cudaError_t norm_grad_dispatch(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                               int *launches) {
    const bool vec = wide_rows<DT>(a.dy, a.dy_stride) && wide_rows<DT>(a.h, a.h_stride) &&
                     wide_rows<DT>(a.dh, a.dh_stride) && wide_rows<DT>(a.dx, a.dx_stride) &&
                     wide_weight<DT>(a.weight, a.weight_f32);
    return vec ? norm_grad_launch<DT, true>(a, most_writers, sms, s, info, launches)
               : norm_grad_launch<DT, false>(a, most_writers, sms, s, info, launches);
}

}  // namespace
}  // namespace ew
