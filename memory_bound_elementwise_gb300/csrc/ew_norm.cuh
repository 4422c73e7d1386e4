// ew_norm.cuh -- root-mean-square norm with the residual's addition, its 8-bit
// output, and its backward.  Compiled once per element type.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * w
//
// Each row is read once: a block holds it in registers (KT tiles of 8 elements
// a thread) between the sum of squares and the outputs.  The bound is memory:
// x, residual, h and y of 16-bit elements move 8 bytes an element for about 5
// operations.  16384 rows of 8192 bf16 with residual, h and e4m3 outputs take 151
// us (6.2 TB/s, floor 139); 7 rows of 5120 take 2.4 us, one load's and one
// reduction's latency.  Rows that start anywhere are bounded by their loads and
// stores of single elements: 7390 rows of 9081 bf16 take 307 us (floor 70).
#pragma once

#include <algorithm>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

constexpr int kGradWarps = 16;  // most warps that hold a row in the backward
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100: a scale is never zero

enum Quant : int { kPlain = 0, kE4m3 = 1, kI8 = 2 };  // what a norm kernel writes

template <int QUANT> __device__ __forceinline__ uint32_t quant_pair(float2 v) {
    if constexpr (QUANT == kI8) {
        int32_t a, b;
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(v.x));
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(v.y));
        return (a & 0xff) | ((b & 0xff) << 8);
    } else {
        uint16_t d;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v.y), "f"(v.x));
        return d;
    }
}

// Scale of a group whose largest absolute value is amax, and the factor that
// takes y to q.  Products with reciprocals: within two roundings of the
// quotients, which moves a q only where y / scale all but ties.
template <int QUANT> __device__ __forceinline__ float quant_factor(float amax, float *scale) {
    amax = max_nan(amax, kAmaxFloor);
    *scale = amax * (QUANT == kI8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(amax));
    return r * (QUANT == kI8 ? 127.0f : 448.0f);
}

// Quantises the lane's 8 values of y of one tile and stores them, with the
// group's scales.  Every lane of the warp takes part.
template <int QUANT, bool VEC>
__device__ __forceinline__ void quant_tile(const float2 (&y)[4], const NormArgs &a, int64_t row, int base, int lane,
                                           float row_factor) {
    uint8_t *q = static_cast<uint8_t *>(a.out) + row * a.out_stride;
    const int shift = a.group_shift;  // log2 of the group, 0: the row
    const int c0 = tile_col<VEC>(base, lane, 0);
    if constexpr (VEC) {
        float factor = row_factor;
        if (shift != 0) {
            float m = largest_of(y);
            m = max_nan(m, __shfl_xor_sync(kAllLanes, m, 1));
            m = max_nan(m, __shfl_xor_sync(kAllLanes, m, 2));
            if (shift > 5) m = max_nan(m, __shfl_xor_sync(kAllLanes, m, 4));
            if (shift > 6) m = max_nan(m, __shfl_xor_sync(kAllLanes, m, 8));
            if (shift > 7) m = max_nan(m, __shfl_xor_sync(kAllLanes, m, 16));
            float scale;
            factor = quant_factor<QUANT>(m, &scale);
            if ((lane << 3 & ((1 << shift) - 1)) == 0 && c0 < a.cols)
                a.scales[row * a.scales_stride + (c0 >> shift)] = scale;
        }
        const float2 f = both(factor);
        const uint32_t q0 = quant_pair<QUANT>(mul2(y[0], f)), q1 = quant_pair<QUANT>(mul2(y[1], f));
        const uint32_t q2 = quant_pair<QUANT>(mul2(y[2], f)), q3 = quant_pair<QUANT>(mul2(y[3], f));
        Vec<8> v;
        v.w[0] = q0 | (q1 << 16);
        v.w[1] = q2 | (q3 << 16);
        if (c0 + 8 <= a.cols) {
            st<8>(q + c0, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < a.cols) q[c0 + j] = static_cast<uint8_t>(v.w[j / 4] >> (8 * (j & 3)));
        }
    } else {
        // step j of the tile is columns base + 32 j .. + 31; a group is 1, 2, 4 or 8 steps
        float v[8], f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = y[j].x;
            v[2 * j + 1] = y[j].y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = row_factor;
        if (shift != 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = lanes_max_nan(fabsf(v[j]), 32);
            // butterflies over the steps of a group: every step has its group's largest value
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                if ((32 << 1) * d > (1 << shift)) break;
                float g[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = max_nan(f[j], f[j ^ d]);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float scale;
                f[j] = quant_factor<QUANT>(f[j], &scale);
                const int c = base + j * 32;
                if (lane == 0 && (c & ((1 << shift) - 1)) == 0 && c < a.cols)
                    a.scales[row * a.scales_stride + (c >> shift)] = scale;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * 32;
            if (c < a.cols) q[c] = static_cast<uint8_t>(quant_pair<QUANT>(both(v[j] * f[j])));
        }
    }
}

// One row to a block of `warps` warps (blockDim.x), tile t of the row to warp
// t mod warps; with one warp a row, blockDim.y rows to a block.  HELD: the
// warps x KT tiles cover the row, which stays in registers.  Otherwise (rows
// beyond 16 warps x 4 tiles) the passes read the row again, each thread its
// own elements, and h is written by the last pass, so in-place forms hold.
template <int DT, bool VEC, int KT, int QUANT, bool HELD>
__global__ void __launch_bounds__(HELD ? 512 : 1024, HELD && VEC && KT * ElemOf<DT>::kBytes <= 8 ? 2 : 1)
    norm_kernel(NormArgs a) {
    enter_grid();
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;  // whole warps: blockDim.y > 1 only with one warp a row
    const void *x = row_of<DT>(a.x, row, a.x_stride);
    const void *res = a.residual ? row_of<DT>(a.residual, row, a.residual_stride) : nullptr;
    void *h = a.h ? row_of<DT>(a.h, row, a.h_stride) : nullptr;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;

    auto scaled = [&](int base, float r, const float2 (&f)[4], float2 (&y)[4]) {
        load_weight<DT, VEC>(a.weight, a.weight_f32, base, a.cols, lane, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], mul2(f[j], both(r)));
    };
    auto put = [&](int base, const float2 (&y)[4], float row_factor) {
        if constexpr (QUANT != kPlain) quant_tile<QUANT, VEC>(y, a, row, base, lane, row_factor);
        else store_tile<DT, VEC>(row_of<DT>(a.out, row, a.out_stride), base, a.cols, lane, pack8<DT>(y));
    };
    auto rstd_of = [&](float2 ss) {
        const float r = rsqrtf(fmaf(block_sum(ss.x + ss.y, warps, part[0]), a.per_col, a.eps));
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
        return r;
    };
    auto row_scale = [&](float amax) {
        float scale;
        const float factor = quant_factor<QUANT>(block_max_nan(amax, warps, part[1]), &scale);
        if (threadIdx.x == 0) a.scales[row * a.scales_stride] = scale;
        return factor;
    };

    float2 ss = both(0.0f);
    float amax = 0.0f, factor = 0.0f;
    if constexpr (HELD) {
        float2 f[KT][4];
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
                float2 g[4];
                unpack8<DT>(rr[k], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[k][j] = add2(f[k][j], g[j]);
            }
            if (h) store_tile<DT, VEC>(h, (warp + k * warps) * kTileCols, a.cols, lane, pack8<DT>(f[k]));
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma2(f[k][j], f[k][j], ss);
        }
        const float r = rstd_of(ss);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 y[4];
            const int base = (warp + k * warps) * kTileCols;
            scaled(base, r, f[k], y);
            if (QUANT != kPlain && a.group_shift == 0) {
                amax = max_nan(amax, largest_of(y));
#pragma unroll
                for (int j = 0; j < 4; ++j) f[k][j] = y[j];
            } else if (base < a.cols) {
                put(base, y, 0.0f);
            }
        }
        if (QUANT != kPlain && a.group_shift == 0) {
            factor = row_scale(amax);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const int base = (warp + k * warps) * kTileCols;
                if (base < a.cols) put(base, f[k], factor);
            }
        }
    } else {
        auto sum_of = [&](int base, float2 (&f)[4]) {
            unpack8<DT>(load_tile<DT, VEC>(x, base, a.cols, lane), f);
            if (res) {
                float2 g[4];
                unpack8<DT>(load_tile<DT, VEC>(res, base, a.cols, lane), g);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = add2(f[j], g[j]);
            }
        };
        for (int t = warp; t < tiles; t += warps) {
            float2 f[4];
            sum_of(t * kTileCols, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma2(f[j], f[j], ss);
        }
        const float r = rstd_of(ss);
        if (QUANT != kPlain && a.group_shift == 0) {
            for (int t = warp; t < tiles; t += warps) {
                float2 f[4], y[4];
                sum_of(t * kTileCols, f);
                scaled(t * kTileCols, r, f, y);
                amax = max_nan(amax, largest_of(y));
            }
            factor = row_scale(amax);
        }
        for (int t = warp; t < tiles; t += warps) {
            float2 f[4], y[4];
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
// to its own row of `partial`, and column_sums_kernel adds those rows in order.
//
// This kernel takes rows that start anywhere, element by element, which bounds
// it: 3075 rows of 8011 f16 take 148 us (floor 29), 1023 of 1001 binary32 6.6 us,
// the latency of two kernels.  AHEAD, for
// rows that 8 warps hold: a row's loads are issued while the row before is
// worked on, and the weights stay in registers; wider rows have no registers
// left for either.
template <int DT, int KT, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 256 : 512, AHEAD && KT * ElemOf<DT>::kBytes <= 4 ? 2 : 1)
    norm_grad_kernel(NormGradArgs a) {
    enter_grid();
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t writer = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t writers = static_cast<int64_t>(gridDim.x) * blockDim.y;
    float2 dw[KT][4], held[AHEAD ? KT : 1][4];
    auto weight = [&](int k, float2 (&w)[4]) {
        load_weight<DT, false>(a.weight, a.weight_f32, (warp + k * warps) * kTileCols, a.cols, lane, w);
    };
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        if constexpr (AHEAD) weight(k, held[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = both(0.0f);
    }
    const float per_col = 1.0f / static_cast<float>(a.cols);
    Raw8<DT> rdy[KT], rh[KT], rdh[KT];
    float r = 0.0f;
    auto fetch = [&](int64_t row) {
        const void *dy = row_of<DT>(a.dy, row, a.dy_stride), *h = row_of<DT>(a.h, row, a.h_stride);
        r = a.rstd[row];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            rdy[k] = load_tile<DT, false>(dy, (warp + k * warps) * kTileCols, a.cols, lane);
            rh[k] = load_tile<DT, false>(h, (warp + k * warps) * kTileCols, a.cols, lane);
        }
        if (a.dh) {
            const void *dh = row_of<DT>(a.dh, row, a.dh_stride);
#pragma unroll
            for (int k = 0; k < KT; ++k) rdh[k] = load_tile<DT, false>(dh, (warp + k * warps) * kTileCols, a.cols, lane);
        }
    };
    int turn = 0;
    if (AHEAD && writer < a.rows) fetch(writer);
    for (int64_t row = writer; row < a.rows; row += writers, turn ^= 1) {
        Raw8<DT> cdy[KT], ch[KT], cdh[KT];
        if constexpr (!AHEAD) fetch(row);
        const float cr = r;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            cdy[k] = rdy[k];
            ch[k] = rh[k];
            cdh[k] = rdh[k];
        }
        if (AHEAD && row + writers < a.rows) fetch(row + writers);
        float2 c2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4], w[4];
            if constexpr (!AHEAD) weight(k, w);
            unpack8<DT>(cdy[k], g);
            unpack8<DT>(ch[k], n);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (AHEAD) w[j] = held[k][j];
                n[j] = mul2(n[j], both(cr));
                dw[k][j] = fma2(g[j], n[j], dw[k][j]);
                c2 = fma2(mul2(g[j], w[j]), n[j], c2);
            }
        }
        const float c = block_sum(c2.x + c2.y, warps, part[turn]) * per_col;
        const float2 minus_c = both(-c), r2 = both(cr);
        void *dx = row_of<DT>(a.dx, row, a.dx_stride);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4], w[4], d[4];
            if constexpr (!AHEAD) weight(k, w);
            unpack8<DT>(cdy[k], g);
            unpack8<DT>(ch[k], n);
            if (a.dh) {
                unpack8<DT>(cdh[k], d);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = both(0.0f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (AHEAD) w[j] = held[k][j];
                d[j] = fma2(r2, fma2(minus_c, mul2(n[j], r2), mul2(g[j], w[j])), d[j]);
            }
            store_tile<DT, false>(dx, (warp + k * warps) * kTileCols, a.cols, lane, pack8<DT>(d));
        }
    }
    if (a.dweight == nullptr) return;
    float *out = a.partial + writer * a.cols;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        const int base = (warp + k * warps) * kTileCols;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = tile_col<false>(base, lane, j);
            if (col < a.cols) out[col] = (j & 1) ? dw[k][j / 2].y : dw[k][j / 2].x;
        }
    }
}

// The same for rows that start at multiples of 8 elements, their loads as
// asynchronous copies into a ring of `depth` rows in shared memory: rows on
// their way take no registers, so that an SM has two to four rows of each block
// in flight whatever their width.  Each thread copies and reads its own elements
// alone, waits for its own copies and needs no barrier for them.  The bound is
// memory: 12000 rows of 5056 bf16 take 81 us (floor 72; with the rows ahead held
// in registers, 156), of 12288 bf16 175 us (174), of 4096 binary32 120 us (116).
template <int DT, int KT> __global__ void __launch_bounds__(512, 1) norm_grad_ring_kernel(NormGradArgs a, int depth) {
    enter_grid();
    // P pieces of 16 bytes hold a lane's 8 elements: of binary32 the two are 128
    // columns apart, so that a copy of the warp takes whole sectors
    constexpr int B = ElemOf<DT>::kBytes, P = B / 2, E = 16 / B;
    extern __shared__ uint4 ring[];                   // [row][dy, h, dh][tile][piece][thread]
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int threads = blockDim.x * blockDim.y, slot_size = 3 * KT * P * threads;
    uint4 *const mine = ring + threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t writer = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t writers = static_cast<int64_t>(gridDim.x) * blockDim.y;
    auto col = [&](int k, int piece) { return (warp + k * warps) * kTileCols + piece * 128 + lane * E; };
    auto place = [&](int slot, int matrix, int k, int piece) {
        return mine + slot * slot_size + ((matrix * KT + k) * P + piece) * threads;
    };
    float2 dw[KT][4], w[KT][4];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col(k, j / 4) + j % 4;
                const float v = a.weight == nullptr ? 1.0f : c < a.cols ? static_cast<const float *>(a.weight)[c] : 0.0f;
                (j & 1 ? w[k][j / 2].y : w[k][j / 2].x) = v;
            }
        } else {
            load_weight<DT, true>(a.weight, a.weight_f32, (warp + k * warps) * kTileCols, a.cols, lane, w[k]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = both(0.0f);
    }
    // pieces past the row stay zero: nothing is copied there
    for (int slot = 0; slot < depth; ++slot)
#pragma unroll
        for (int matrix = 0; matrix < 3; ++matrix)
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int piece = 0; piece < P; ++piece)
                    if (col(k, piece) >= a.cols || (matrix == 2 && a.dh == nullptr))
                        *place(slot, matrix, k, piece) = make_uint4(0u, 0u, 0u, 0u);
    auto copy = [&](const void *row, int slot, int matrix) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int piece = 0; piece < P; ++piece) {
                const int c = col(k, piece);
                if (c < a.cols) {
                    const int bytes = min(16, (a.cols - c) * B);  // zeros after them
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(place(slot, matrix, k, piece)))),
                                    "l"(static_cast<const char *>(row) + static_cast<int64_t>(c) * B), "r"(bytes) : "memory");
                }
            }
    };
    auto start = [&](int64_t row, int slot) {
        if (row < a.rows) {
            copy(row_of<DT>(a.dy, row, a.dy_stride), slot, 0);
            copy(row_of<DT>(a.h, row, a.h_stride), slot, 1);
            if (a.dh) copy(row_of<DT>(a.dh, row, a.dh_stride), slot, 2);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto held = [&](int slot, int matrix, int k, float2 (&f)[4]) {
        Raw8<DT> r;
#pragma unroll
        for (int piece = 0; piece < P; ++piece) {
            const uint4 v = *place(slot, matrix, k, piece);
            r.w[piece * 4] = v.x;
            r.w[piece * 4 + 1] = v.y;
            r.w[piece * 4 + 2] = v.z;
            r.w[piece * 4 + 3] = v.w;
        }
        unpack8<DT>(r, f);
    };
    const float per_col = 1.0f / static_cast<float>(a.cols);
#pragma unroll 1
    for (int q = 0; q < depth; ++q) start(writer + q * writers, q);
    float next_r = writer < a.rows ? a.rstd[writer] : 0.0f;
    int turn = 0, slot = 0;
#pragma unroll 1
    for (int64_t row = writer; row < a.rows; row += writers, turn ^= 1) {
        if (depth == 2) copies_left<1>();
        else if (depth == 3) copies_left<2>();
        else copies_left<3>();
        const float r = next_r;
        if (row + writers < a.rows) next_r = a.rstd[row + writers];
        float2 c2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4];
            held(slot, 0, k, g);
            held(slot, 1, k, n);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n[j] = mul2(n[j], both(r));
                dw[k][j] = fma2(g[j], n[j], dw[k][j]);
                c2 = fma2(mul2(g[j], w[k][j]), n[j], c2);
            }
        }
        const float c = block_sum(c2.x + c2.y, warps, part[turn]) * per_col;
        const float2 minus_c = both(-c), r2 = both(r);
        void *dx = row_of<DT>(a.dx, row, a.dx_stride);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4], d[4];
            held(slot, 0, k, g);
            held(slot, 1, k, n);
            held(slot, 2, k, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = fma2(r2, fma2(minus_c, mul2(n[j], r2), mul2(g[j], w[k][j])), d[j]);
            const Raw8<DT> o = pack8<DT>(d);
#pragma unroll
            for (int piece = 0; piece < P; ++piece) {
                const int c = col(k, piece);
                typename ElemOf<DT>::type *to = static_cast<typename ElemOf<DT>::type *>(dx) + c;
                if (c + E <= a.cols) {
                    Vec<16> v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v.w[i] = o.w[piece * 4 + i];
                    st<16>(to, v);
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        if (c + j < a.cols)
                            to[j] = static_cast<typename ElemOf<DT>::type>(o.w[piece * 4 + j * B / 4] >> (j * B % 4 * 8));
                }
            }
        }
        start(row + depth * writers, slot);
        if (++slot == depth) slot = 0;
    }
    copies_left<0>();
    if (a.dweight == nullptr) return;
    float *out = a.partial + writer * a.cols;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const int c = col(k, P == 2 ? j / 2 : 0) + (P == 2 ? 0 : 2 * j);
            if (c + 4 <= a.cols && a.cols % 4 == 0) {
                *reinterpret_cast<float4 *>(out + c) = make_float4(dw[k][j].x, dw[k][j].y, dw[k][j + 1].x, dw[k][j + 1].y);
            } else {
                const float f[4] = {dw[k][j].x, dw[k][j].y, dw[k][j + 1].x, dw[k][j + 1].y};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < a.cols) out[c + i] = f[i];
            }
        }
    }
}

// Rows too wide to hold: the row's two passes read it twice.  12000 rows of
// 12288 binary32 take 678 us (floor 348), three passes over them.  dweight has its
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
    auto products = [&](int base, float2 (&g)[4], float2 (&n)[4]) {
        float2 w[4];
        load_weight<DT, VEC>(a.weight, a.weight_f32, base, a.cols, lane, w);
        unpack8<DT>(load_tile<DT, VEC>(dy, base, a.cols, lane), g);
        unpack8<DT>(load_tile<DT, VEC>(h, base, a.cols, lane), n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = mul2(n[j], both(r));
            g[j] = mul2(g[j], w[j]);
        }
    };
    float2 c2 = both(0.0f), g[4], n[4];
    for (int t = warp; t < tiles; t += warps) {
        products(t * kTileCols, g, n);
#pragma unroll
        for (int j = 0; j < 4; ++j) c2 = fma2(g[j], n[j], c2);
    }
    const float c = block_sum(c2.x + c2.y, warps, part) / static_cast<float>(a.cols);
    void *dx = row_of<DT>(a.dx, row, a.dx_stride);
    for (int t = warp; t < tiles; t += warps) {
        products(t * kTileCols, g, n);
        float2 d[4] = {};
        if (a.dh) unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.dh, row, a.dh_stride), t * kTileCols, a.cols, lane), d);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = fma2(both(r), fma2(both(-c), n[j], g[j]), d[j]);
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
    float2 dw[4] = {};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float2 g[4], n[4];
        const float r = a.rstd[row];
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.dy, row, a.dy_stride), base, a.cols, lane), g);
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.h, row, a.h_stride), base, a.cols, lane), n);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[j] = fma2(g[j], mul2(n[j], both(r)), dw[j]);
    }
    float *out = a.partial + static_cast<int64_t>(blockIdx.y) * a.cols;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = tile_col<VEC>(base, lane, j);
        if (col < a.cols) out[col] = (j & 1) ? dw[j / 2].y : dw[j / 2].x;
    }
}

// ---------------------------------------------------------------- launches

constexpr int kHeldWarps = 16;

template <int DT, bool VEC, int QUANT>
cudaError_t norm_launch(const NormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    // Few rows: as few tiles a thread as 16 warps allow, for the row's latency.
    // Many: two tiles a thread, and four for 16-bit rows past 2048 columns,
    // where blocks are small enough that four of them share an SM and cover
    // one another's waits.  e4m3 of 2^26 bf16 at 8192 columns: 4 tiles 79 us,
    // 2 tiles 88 us; at 1024: 77 and 75 us, 1 tile 92 us.  binary32 at 4096:
    // 4, 2 and 1 tiles 126, 125 and 123 us.
    const bool many = a.rows >= 4 * static_cast<int64_t>(sms);
    int kt = tiles_per_thread(tiles, kHeldWarps, 4);
    if (many && kt != 0) kt = std::max(kt, tiles == 1 ? 1 : DT != DT_F32 && tiles > 8 ? 4 : 2);
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
    if (!quant) return vec ? norm_launch<DT, true, kPlain>(a, sms, s, info) : norm_launch<DT, false, kPlain>(a, sms, s, info);
    if (a.i8) return vec ? norm_launch<DT, true, kI8>(a, sms, s, info) : norm_launch<DT, false, kI8>(a, sms, s, info);
    return vec ? norm_launch<DT, true, kE4m3>(a, sms, s, info) : norm_launch<DT, false, kE4m3>(a, sms, s, info);
}

// Of an SM's shared memory.  A row of the 16 warps that an SM holds (512 threads
// of up to 128 registers) takes up to 96 KiB, so at least two fit.
constexpr int kRingBytes = 200 * 1024;

template <int DT, bool VEC>
cudaError_t norm_grad_launch(const NormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                             int *launches) {
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    constexpr int most = DT == DT_F32 ? 2 : 4;
    int kt = tiles_per_thread(tiles, 8, most);
    const bool ahead = kt != 0;
    // 12000 rows of 1984 bf16: 41 us with one tile a thread, 37 us with two; of 1000: 25 and 27 us.
    if (VEC && DT != DT_F32 && kt == 1 && tiles > 6 && a.rows >= 4 * static_cast<int64_t>(sms)) kt = 2;
    if (!ahead) kt = tiles_per_thread(tiles, kGradWarps, most);
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    int64_t writers = 0;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && kt != 0) {
        const int warps = (tiles + kt - 1) / kt;
        const int per_block = warps == 1 && a.rows >= 4 * static_cast<int64_t>(sms) ? 4 : 1;
        const int resident = std::max(1, 16 / (warps * per_block));  // blocks that make 512 threads an SM
        const int64_t grid = std::min<int64_t>({(a.rows + per_block - 1) / per_block,
                                                static_cast<int64_t>(sms) * resident, most_writers / per_block});
        writers = grid * per_block;
        const dim3 block(32 * warps, per_block);
        info->grid = static_cast<int>(grid);
        info->block = 32 * warps * per_block;
        if constexpr (VEC) {
            auto kernel = kt == 1 ? norm_grad_ring_kernel<DT, 1> : norm_grad_ring_kernel<DT, 2>;
            if constexpr (most == 4)
                if (kt == 4) kernel = norm_grad_ring_kernel<DT, 4>;
            const int row_bytes = 3 * kt * info->block * 8 * ElemOf<DT>::kBytes;  // of a row of each of the block's writers
            const int depth = std::max(2, std::min(4, kRingBytes / (resident * row_bytes)));
            static std::atomic<uint64_t> allowed[3];
            e = allow_smem(reinterpret_cast<const void *>(kernel), kRingBytes, &allowed[kt / 2]);
            if (e != cudaSuccess) return e;
            info->smem = depth * row_bytes;
            e = launch_rows(kernel, dim3(grid), block, depth * row_bytes, 1, s, a, depth);
        } else {
            auto kernel = norm_grad_kernel<DT, 1, true>;
            if (kt == 2) kernel = ahead ? norm_grad_kernel<DT, 2, true> : norm_grad_kernel<DT, 2, false>;
            if constexpr (most == 4)
                if (kt == 4) kernel = ahead ? norm_grad_kernel<DT, 4, true> : norm_grad_kernel<DT, 4, false>;
            e = launch_rows(kernel, dim3(grid), block, 0, 1, s, a);
        }
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
