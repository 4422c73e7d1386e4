// ew_layernorm.cuh -- layer norm with the residual's addition, and its backward.
// Compiled once per element type.
//
//   h = x + residual,  m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps),  y = (h - m) r w + b
//
// Both directions move their matrices once and are bounded by memory.  Rows may
// start anywhere: where all matrices of a call have their rows at the same place
// between multiples of 8 elements, a row is taken in runs of 8 that start at such
// a multiple, `past` elements before the row, and the runs at its two ends are
// moved element by element (RUNS).  Other matrices are moved an element at a time.
//
// The mean is subtracted in two steps, so that y does not lose what its rounding to
// binary32 would cost.  First a number L near the mean: one of the row's elements where it
// is within a factor of two of the mean, which makes the differences of elements near it
// exact and those of a row of one value 0; otherwise the mean as a plain sum gives it.  Then
// the mean d of the differences.  With those, v = h - L - d, the squares are summed, and the
// v, whose mean e is what rounding took from d:
//     m = L + (d + e),  sum (h - m)^2 = sum v^2 - n e^2,
// where e^2 is next to nothing beside the squares.  Rows that share a warp, whose time is
// that of instructions, take zero for L where their elements have both signs, and e only
// where L is a mean (65536 x 201 bf16 35.2 us; always 36.1).
#pragma once

#include <algorithm>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// ---------------------------------------------------------------- columns

// How the rows of a call's matrices lie: all at multiples of 8 elements; all alike,
// but anywhere; or apart.
enum Rows : int { kApart = 0, kAligned = 1, kShifted = 2 };
// 16-bit elements one by one, zero outside the row; those of a whole tile without a
// comparison, after which they would be waited for one by one (of views of stride cols + 1:
// 9 rows of 5120 bf16 3.7 us, in the other way 5.4; 16384 of 4096 133 and 153 us).
template <int DT> __device__ __forceinline__ Raw8<DT> load_elements(const void *row, int tile, int cols, int lane) {
    const uint16_t *p = static_cast<const uint16_t *>(row);
    const int c0 = tile * kTileCols + lane;
    uint32_t v[8];
    if (tile * kTileCols + kTileCols <= cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ld<2>(p + c0 + j * 32).h;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c0 + j * 32 < cols ? ld<2>(p + c0 + j * 32).h : 0u;
    }
    Raw8<DT> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = v[2 * j] | v[2 * j + 1] << 16;
    return r;
}
template <int DT, int ROWS>
__device__ __forceinline__ Raw8<DT> load_row(const void *row, int tile, int past, int cols, int lane, bool inner) {
    if constexpr (ROWS == kShifted) return load_run<DT>(row, tile, past, cols, lane, inner);
    else if constexpr (ROWS == kApart && DT != DT_F32) return load_elements<DT>(row, tile, cols, lane);
    else return load_tile<DT, ROWS == kAligned>(row, tile * kTileCols, cols, lane);
}
template <int DT, int ROWS>
__device__ __forceinline__ void store_row(void *row, int tile, int past, int cols, int lane, const Raw8<DT> &r) {
    if constexpr (ROWS == kShifted) store_run<DT>(row, tile, past, cols, lane, r);
    else store_tile<DT, ROWS == kAligned>(row, tile * kTileCols, cols, lane, r);
}
// The columns of a vector, in binary32; null stands for `other`, columns
// outside for zero.  Beside shifted rows a run of it starts anywhere.
template <int DT, int ROWS>
__device__ __forceinline__ void load_columns(const void *w, bool f32, float other, int tile, int past, int cols, int lane,
                                             float2 (&f)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = both(other);
    } else if constexpr (ROWS != kShifted) {
        load_weight<DT, ROWS == kAligned>(w, f32, tile * kTileCols, cols, lane, f);
    } else {
        const int c0 = col_of<true>(tile, past, lane, 0);
        if (c0 >= 8 && c0 + 16 <= cols) {
            if (DT == DT_F32 || f32) unpack8<DT_F32>(cut_run<DT_F32>(w, c0), f);
            else unpack8<DT>(cut_run<DT>(w, c0), f);
            return;
        }
        // at its ends element by element, all under way together
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float e = 0.0f;
            if (c0 + j >= 0 && c0 + j < cols) {
                if (DT == DT_F32 || f32) e = static_cast<const float *>(w)[c0 + j];
                else e = elem_to_f32<DT>(static_cast<const typename ElemOf<DT>::type *>(w)[c0 + j]);
            }
            (j & 1 ? f[j / 2].y : f[j / 2].x) = e;
        }
    }
}
// Columns of the row in tile `tile`.
__device__ __forceinline__ int columns_in(int tile, int past, int cols) {
    const int first = max(tile * kTileCols - past, 0), end = min(static_cast<int64_t>(tile + 1) * kTileCols - past, static_cast<int64_t>(cols));
    return max(end - first, 0);
}

// Sums over the LANES lanes around this one.
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAllLanes, v, d);
    return v;
}
template <int LANES> __device__ __forceinline__ float2 lanes_sum(float2 v) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(kAllLanes, v.x, d), __shfl_xor_sync(kAllLanes, v.y, d)));
    return v;
}
// Two sums over a block of `warps` warps at once; `part` as in block_sum.
__device__ __forceinline__ float2 warp_sum2(float2 v) { return lanes_sum<32>(v); }
__device__ __forceinline__ float2 block_sum2(float2 v, int warps, float2 *part) {
    v = warp_sum2(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum2(lane < warps ? part[lane] : both(0.0f));
}

// ---------------------------------------------------------------- forward

// What the elements are first compared with: of samples (`mine`, where `given`), one to
// each of the LANES lanes that share a row, the first where all have one sign, and so may lie
// far from zero, else zero.
template <int LANES = 32> __device__ __forceinline__ float landmark(float mine, bool given) {
    unsigned all = __ballot_sync(kAllLanes, given), negative = __ballot_sync(kAllLanes, given && mine < 0.0f);
    const int from = threadIdx.x & 31 & ~(LANES - 1);
    if constexpr (LANES < 32) {
        const unsigned peers = (kAllLanes >> (32 - LANES)) << from;
        all &= peers, negative &= peers;
    }
    const float first = __shfl_sync(kAllLanes, mine, from);
    return negative == 0 || negative == all ? first : 0.0f;
}
// The landmark and the mean `beyond` it, where they lie apart, as where the landmark stands
// out of its row: differences to it hold fewer of the elements' bits then, and the mean
// takes its place.  Apart: more than the mean's size over `times`; with 1, zero never is.
__device__ __forceinline__ bool to_mean(float &at, float &beyond, float times) {
    const float mean = at + beyond;
    const bool apart = times * fabsf(beyond) > fabsf(mean);
    at = apart ? mean : at;
    beyond = apart ? 0.0f : beyond;
    return apart;
}
// What `beyond` lacks, from the sum of what n elements have beyond it; the squares become
// those around the mean.  Squares past binary32 stay.
__device__ __forceinline__ void finish_mean(float &beyond, float &squares, float sum, float n, float per) {
    const bool finite = squares < __int_as_float(0x7f800000);
    const float e = finite ? sum * per : 0.0f;
    squares = finite ? fmaxf(fmaf(-n * e, e, squares), 0.0f) : squares;
    beyond += e;
}

// One row to a block of `warps` warps, tile t of the row to warp t mod warps;
// with one warp a row, blockDim.y rows to a block.  HELD: the warps x KT tiles
// cover the row, which stays in registers.  Each warp takes the mean of its own
// columns, beyond one of them, and the squares around that; the parts are joined by
//     sum (v - m)^2 = sum over warps of (squares + n (mean - m)^2),
// so that both statistics cost one barrier and no cancellation.  Otherwise the
// passes read the row again.  Bounded by memory: 16384 rows of 8192 bf16 with a residual
// 171 us at a floor of 161; by latency where there are few rows (9 of 5120 3.0 us) and
// by the issue rate where rows are narrow (65536 of 201 bf16 35 us at 16).
//
// Weights beside shifted rows have to be cut to their phase, which takes as long
// as all else, and those of rows of more than 32 tiles of 16 bits are read from the
// L2 as often as the rows.  Blocks therefore walk over such rows, in steps of a
// multiple of 8, after which the phase is the same: each thread keeps its weights in
// shared memory, and the next row is on its way while one is worked on.
//
// PAIR: the row goes to a cluster of two blocks, which read each other's parts.
__host__ __device__ constexpr bool layernorm_walks(int dt, int rows, int kt, int warps) {
    return rows == kShifted || (rows == kAligned && dt != DT_F32 && kt == 4 && warps == 16);
}
__host__ __device__ constexpr int layernorm_resident(int dt, int rows, int kt, bool held, int warps) {  // blocks to an SM
    if (!held || rows == kApart) return 1;
    if (warps == 8) return 3;
    return kt == 1 || (rows == kAligned && kt == 2) ? 2 : 1;
}
template <int DT, int ROWS, int KT, bool HELD, int WARPS, bool PAIR>
__global__ void __launch_bounds__(WARPS * 32, layernorm_resident(DT, ROWS, KT, HELD, WARPS))
    layernorm_kernel(const __grid_constant__ LayerNormArgs a) {
    enter_grid();
    constexpr bool kWalks = HELD && layernorm_walks(DT, ROWS, KT, WARPS);
    extern __shared__ float4 cut[];  // of walkers, [tile][weight's 4 and 4, bias' 4 and 4][thread]
    __shared__ float4 parts[2][32];  // of a warp's columns: an element, mean beyond that, squares, number
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    // the row's warps, of this block and its neighbour
    const int half = PAIR ? blockIdx.x & 1 : 0, row_warps = PAIR ? 2 * warps : warps, row_warp = half * warps + warp;
    int64_t row = static_cast<int64_t>(PAIR ? blockIdx.x >> 1 : blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;  // whole warps: blockDim.y > 1 only with one warp a row
    const int past = ROWS == kShifted ? past_of<DT>(row_of<DT>(a.x, row, a.x_stride)) : 0;
    const float per_col = a.per_col;
    auto statistics = [&](int64_t row, float at, float mean, float squares) {
        const float r = rsqrtf(fmaf(squares, per_col, a.eps));
        if (threadIdx.x == 0 && half == 0) {
            if (a.mean) a.mean[row] = at + mean;
            if (a.rstd) a.rstd[row] = r;
        }
        return r;
    };
    auto weights = [&](int tile, float2 (&w)[4], float2 (&b)[4]) {
        load_columns<DT, ROWS>(a.weight, a.weight_f32, 1.0f, tile, past, a.cols, lane, w);
        load_columns<DT, ROWS>(a.bias, a.weight_f32, 0.0f, tile, past, a.cols, lane, b);
    };
    // y of one tile from h, the element `at` and the mean beyond it
    auto put = [&](void *out, int tile, const float2 (&f)[4], float at, float mean, float r, const float2 (&w)[4], const float2 (&b)[4]) {
        float2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            y[j] = fma2(fma2(add2(f[j], both(-at)), both(r), both(-mean * r)), w[j], b[j]);
        store_row<DT, ROWS>(out, tile, past, a.cols, lane, pack8<DT>(y));
    };

    if constexpr (HELD) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < KT; ++k) n += columns_in(row_warp + k * row_warps, past, a.cols);
        const float per_own = 1.0f / static_cast<float>(max(n, 1));
        const int threads = blockDim.x * blockDim.y;
        float4 *const mine = cut + threadIdx.y * blockDim.x + threadIdx.x;
        int turn = 0;
        Raw8<DT> rx[KT], rr[KT];
        auto load = [&] {
            const void *x = row_of<DT>(a.x, row, a.x_stride);
            const bool inner = row > 0 && row + 1 < a.rows;  // strides are at least 8
#pragma unroll
            for (int k = 0; k < KT; ++k) rx[k] = load_row<DT, ROWS>(x, row_warp + k * row_warps, past, a.cols, lane, inner);
            if (a.residual) {
                const void *res = row_of<DT>(a.residual, row, a.residual_stride);
#pragma unroll
                for (int k = 0; k < KT; ++k) rr[k] = load_row<DT, ROWS>(res, row_warp + k * row_warps, past, a.cols, lane, inner);
            }
        };
        load();
        if constexpr (kWalks) {
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                float2 w[4], b[4];
                weights(row_warp + k * row_warps, w, b);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mine[(4 * k + i) * threads] = make_float4(w[2 * i].x, w[2 * i].y, w[2 * i + 1].x, w[2 * i + 1].y);
                    mine[(4 * k + 2 + i) * threads] = make_float4(b[2 * i].x, b[2 * i].y, b[2 * i + 1].x, b[2 * i + 1].y);
                }
            }
        }
        do {
            void *h = a.h ? row_of<DT>(a.h, row, a.h_stride) : nullptr;
            void *out = row_of<DT>(a.y, row, a.y_stride);
            const int64_t here = row;
            float2 f[KT][4];
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                unpack8<DT>(rx[k], f[k]);
                if (a.residual) {
                    float2 g[4];
                    unpack8<DT>(rr[k], g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[k][j] = add2(f[k][j], g[j]);
                }
                if (h) store_row<DT, ROWS>(h, row_warp + k * row_warps, past, a.cols, lane, pack8<DT>(f[k]));
            }
            row += static_cast<int64_t>(PAIR ? gridDim.x >> 1 : gridDim.x) * blockDim.y;
            if (kWalks && row < a.rows) load();  // on its way while this row is worked on
            // lane 0's lies in the row, if any of the warp's first tile does (a shifted row has 8)
            const int j = ROWS == kShifted && row_warp == 0 ? 7 : 0;
            float at = landmark(j == 0 ? f[0][0].x : f[0][3].y, col_of<ROWS != kApart>(row_warp, past, lane, j) < a.cols);
            float2 s2 = both(0.0f), e2 = both(0.0f), q2 = both(0.0f);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                float2 d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = add2(f[k][j], both(-at));
                clip_columns<ROWS != kApart>(row_warp + k * row_warps, past, a.cols, lane, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = add2(s2, d[j]);
            }
            float mean = warp_sum(s2.x + s2.y) * per_own;
            to_mean(at, mean, 2.0f);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                float2 d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = add2(add2(f[k][j], both(-at)), both(-mean));
                clip_columns<ROWS != kApart>(row_warp + k * row_warps, past, a.cols, lane, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e2 = add2(e2, d[j]);
                    q2 = fma2(d[j], d[j], q2);
                }
            }
            float squares = warp_sum(q2.x + q2.y);
            finish_mean(mean, squares, warp_sum(e2.x + e2.y), static_cast<float>(n), per_own);
            if (warps > 1) {
                float4 *part = parts[turn];
                turn ^= 1;  // read by all before it is written again: a barrier lies between
                if (lane == 0) part[warp] = make_float4(at, mean, squares, static_cast<float>(n));
                if (PAIR) cluster_sync();
                else __syncthreads();
                // a part to each lane, twice where half the warp has enough
                constexpr int kLanes = PAIR ? 32 : 16;
                static_assert(WARPS <= 16, "a lane for each part");
                const int peer = lane % kLanes, other = peer < row_warps ? peer : 0;
                const float4 v = PAIR ? *in_block(&part[other % warps], other / warps) : part[other];
                const float count = peer < row_warps ? v.w : 0.0f;
                at = __shfl_sync(kAllLanes, v.x, 0);
                mean = lanes_sum<kLanes>(count > 0.0f ? count * (v.x - at + v.y) : 0.0f) * per_col;
                to_mean(at, mean, 2.0f);
                const float off = v.x - at + v.y - mean;
                // together: one after the other, 16384 shifted rows of 2001 binary32 take 58 us, not 52
                const float2 sums = lanes_sum<kLanes>(count > 0.0f ? make_float2(count * off, fmaf(count * off, off, v.z)) : both(0.0f));
                squares = sums.y;
                finish_mean(mean, squares, sums.x, static_cast<float>(a.cols), per_col);
            }
            const float r = statistics(here, at, mean, squares);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const int tile = row_warp + k * row_warps;
                if (tile * kTileCols - past >= a.cols) continue;
                float2 w[4], b[4];
                if constexpr (kWalks) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 u = mine[(4 * k + i) * threads], v = mine[(4 * k + 2 + i) * threads];
                        w[2 * i] = make_float2(u.x, u.y), w[2 * i + 1] = make_float2(u.z, u.w);
                        b[2 * i] = make_float2(v.x, v.y), b[2 * i + 1] = make_float2(v.z, v.w);
                    }
                } else {
                    weights(tile, w, b);
                }
                put(out, tile, f[k], at, mean, r, w, b);
            }
        } while (kWalks && row < a.rows);
        if (PAIR) cluster_sync();  // the neighbour has read this block's parts
    } else {
        __shared__ float part[32];
        __shared__ float2 part2[32];
        const int tiles = (a.cols + past + kTileCols - 1) / kTileCols;
        const void *x = row_of<DT>(a.x, row, a.x_stride);
        const void *res = a.residual ? row_of<DT>(a.residual, row, a.residual_stride) : nullptr;
        void *h = a.h ? row_of<DT>(a.h, row, a.h_stride) : nullptr;
        const bool inner = row > 0 && row + 1 < a.rows;
        auto sum_of = [&](int tile, float2 (&f)[4]) {
            unpack8<DT>(load_row<DT, ROWS>(x, tile, past, a.cols, lane, inner), f);
            if (res) {
                float2 g[4];
                unpack8<DT>(load_row<DT, ROWS>(res, tile, past, a.cols, lane, inner), g);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = add2(f[j], g[j]);
            }
        };
        // the row's first 32 elements, to every warp: read before h or y may take their place
        auto element = [&](const void *p) {
            using T = typename ElemOf<DT>::type;
            return elem_to_f32<DT>(static_cast<const T *>(p)[min(lane, a.cols - 1)]);
        };
        float at = landmark(res ? element(x) + element(res) : element(x), lane < a.cols);
        float2 s2 = both(0.0f), e2 = both(0.0f), q2 = both(0.0f), f[4];
        for (int t = warp; t < tiles; t += warps) {
            sum_of(t, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = add2(f[j], both(-at));
            clip_columns<ROWS != kApart>(t, past, a.cols, lane, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) s2 = add2(s2, f[j]);
        }
        float mean = block_sum(s2.x + s2.y, warps, part) * per_col;
        to_mean(at, mean, 2.0f);
        for (int t = warp; t < tiles; t += warps) {
            sum_of(t, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = add2(add2(f[j], both(-at)), both(-mean));
            clip_columns<ROWS != kApart>(t, past, a.cols, lane, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e2 = add2(e2, f[j]);
                q2 = fma2(f[j], f[j], q2);
            }
        }
        float2 sums = block_sum2(make_float2(e2.x + e2.y, q2.x + q2.y), warps, part2);
        finish_mean(mean, sums.y, sums.x, static_cast<float>(a.cols), per_col);
        const float r = statistics(row, at, mean, sums.y);
        for (int t = warp; t < tiles; t += warps) {
            float2 w[4], b[4];
            sum_of(t, f);
            weights(t, w, b);
            if (h) store_row<DT, ROWS>(h, t, past, a.cols, lane, pack8<DT>(f));
            put(row_of<DT>(a.y, row, a.y_stride), t, f, at, mean, r, w, b);
        }
    }
}

// Aligned rows of up to 128 columns, such as the heads of a query: LANES lanes (8 or
// 16) to a row, 8 elements each, so that the steps of the reductions are shared by 4 or
// 2 rows of a warp.  131072 rows of 64 bf16 take 12 us (floor 10; a warp a row 60),
// 65536 of 128 12 us (10; 31), of 128 binary32 21 us (20; 33).  TURNS rows of a lane
// are under way together: two where there are many rows of 16 bits (262144 of 128 bf16
// 47 us, 52 with one), one otherwise (2464 of 64 1.7 us, 2.2 with two; 65536 of 128
// binary32 22 and 24).  Many 16-bit rows of up to 256 columns go this way, too, a
// warp to two rows: 65536 of 192 24 us (33), of 256 23 us (26).
constexpr int kNarrowWarps = 8;
constexpr int kNarrowWalkers = 3;  // blocks to an SM
template <int DT, int LANES, int TURNS>
__global__ void __launch_bounds__(32 * kNarrowWarps, 4) layernorm_narrow_kernel(const __grid_constant__ LayerNormArgs a) {
    enter_grid();
    constexpr int kRows = 32 / LANES;  // of a warp at a time
    const int lane = threadIdx.x & (LANES - 1), group = (threadIdx.x & 31) / LANES;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * kNarrowWarps + (threadIdx.x >> 5);
    const int64_t first = warp * kRows * TURNS + group;
    Raw8<DT> rx[TURNS], rr[TURNS];
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        const int64_t row = min(first + t * kRows, a.rows - 1);  // behind the last one it again
        rx[t] = load_tile<DT, true>(row_of<DT>(a.x, row, a.x_stride), 0, a.cols, lane);
        if (a.residual) rr[t] = load_tile<DT, true>(row_of<DT>(a.residual, row, a.residual_stride), 0, a.cols, lane);
    }
    float2 w[4], b[4];
    load_columns<DT, kAligned>(a.weight, a.weight_f32, 1.0f, 0, 0, a.cols, lane, w);
    load_columns<DT, kAligned>(a.bias, a.weight_f32, 0.0f, 0, 0, a.cols, lane, b);
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        const int64_t row = first + t * kRows;
        const bool given = row < a.rows;
        float2 f[4], d[4];
        unpack8<DT>(rx[t], f);
        if (a.residual) {
            float2 g[4];
            unpack8<DT>(rr[t], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = add2(f[j], g[j]);
        }
        // lane 0 of a row has its first element
        float at = landmark<LANES>(f[0].x, lane * 8 < a.cols);
        float2 s2 = both(0.0f), q2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = add2(f[j], both(-at));
        clip_columns<true>(0, 0, a.cols, lane, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = add2(s2, d[j]);
        float mean = lanes_sum<LANES>(s2.x + s2.y) * a.per_col;
        const bool moved = to_mean(at, mean, 1.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = d[j] = add2(add2(f[j], both(-at)), both(-mean));
        clip_columns<true>(0, 0, a.cols, lane, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) q2 = fma2(d[j], d[j], q2);
        float squares = lanes_sum<LANES>(q2.x + q2.y), off = 0.0f;  // off: what f has beyond the mean
        if (__any_sync(kAllLanes, moved)) {
            float2 e2 = both(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) e2 = add2(e2, d[j]);
            const float lacks = lanes_sum<LANES>(e2.x + e2.y);  // not of the rows beside: each has its own bits
            finish_mean(off, squares, moved ? lacks : 0.0f, static_cast<float>(a.cols), a.per_col);
            mean += off;
        }
        const float r = rsqrtf(fmaf(squares, a.per_col, a.eps));
        if (!given) continue;
        if (lane == 0) {
            if (a.mean) a.mean[row] = at + mean;
            if (a.rstd) a.rstd[row] = r;
        }
        if (a.h) {
            float2 h[4];
            unpack8<DT>(rx[t], h);
            if (a.residual) {
                float2 g[4];
                unpack8<DT>(rr[t], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = add2(h[j], g[j]);
            }
            store_tile<DT, true>(row_of<DT>(a.h, row, a.h_stride), 0, a.cols, lane, pack8<DT>(h));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = fma2(fma2(f[j], both(r), both(-off * r)), w[j], b[j]);
        store_tile<DT, true>(row_of<DT>(a.y, row, a.y_stride), 0, a.cols, lane, pack8<DT>(f));
    }
}

// Shifted narrow rows, which share a warp in the same way.  A lane's rows are a multiple of
// 8 apart, so that its weights, cut once, stay in registers; the next row is on its way
// while one is worked on.  65536 rows of 101 bf16 take 22 us (floor 8; a warp a row 37),
// 131072 of 51 22 us (8; 70), 65536 of 201, a warp each, 35 us (16; 37), of 51 binary32
// 14 us (8; 36).  Four blocks an SM have to spill: 22 us for 101 bf16.
template <int DT, int LANES>
__global__ void __launch_bounds__(32 * kNarrowWarps, kNarrowWalkers) layernorm_narrow_walk_kernel(const __grid_constant__ LayerNormArgs a) {
    enter_grid();
    constexpr int kRows = 32 / LANES;  // of a warp at a time
    const int lane = threadIdx.x & (LANES - 1), group = (threadIdx.x & 31) / LANES;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kNarrowWarps * kRows;  // a multiple of 8
    int64_t base = (static_cast<int64_t>(blockIdx.x) * kNarrowWarps + (threadIdx.x >> 5)) * kRows;  // of the warp's rows the first
    const int past = past_of<DT>(row_of<DT>(a.x, base + group, a.x_stride));
    Raw8<DT> rx, rr;
    auto load = [&] {
        const int64_t row = base + group;
        const bool inner = row > 0 && row + 1 < a.rows;  // strides are at least 8
        const int cols = row < a.rows ? a.cols : 0;      // nothing behind the last row
        rx = load_run<DT>(row_of<DT>(a.x, row, a.x_stride), 0, past, cols, lane, inner);
        if (a.residual) rr = load_run<DT>(row_of<DT>(a.residual, row, a.residual_stride), 0, past, cols, lane, inner);
    };
    if (base < a.rows) load();
    float2 w[4], b[4];
    load_columns<DT, kShifted>(a.weight, a.weight_f32, 1.0f, 0, past, a.cols, lane, w);
    load_columns<DT, kShifted>(a.bias, a.weight_f32, 0.0f, 0, past, a.cols, lane, b);
    while (base < a.rows) {
        const int64_t row = base + group;
        float2 f[4], d[4];
        unpack8<DT>(rx, f);
        if (a.residual) {
            float2 g[4];
            unpack8<DT>(rr, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = add2(f[j], g[j]);
        }
        base += step;
        if (base < a.rows) load();
        if (a.h && row < a.rows) store_run<DT>(row_of<DT>(a.h, row, a.h_stride), 0, past, a.cols, lane, pack8<DT>(f));
        // element 7 of lane 0, element 0 of the others, where the row has it
        float at = landmark<LANES>(lane == 0 ? f[3].y : f[0].x, lane == 0 || lane * 8 - past < a.cols);
        float2 s2 = both(0.0f), q2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = add2(f[j], both(-at));
        clip_columns<true>(0, past, a.cols, lane, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = add2(s2, d[j]);
        float mean = lanes_sum<LANES>(s2.x + s2.y) * a.per_col;
        const bool moved = to_mean(at, mean, 1.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = d[j] = add2(add2(f[j], both(-at)), both(-mean));
        clip_columns<true>(0, past, a.cols, lane, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) q2 = fma2(d[j], d[j], q2);
        float squares = lanes_sum<LANES>(q2.x + q2.y), off = 0.0f;  // off: what f has beyond the mean
        if (__any_sync(kAllLanes, moved)) {
            float2 e2 = both(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) e2 = add2(e2, d[j]);
            const float lacks = lanes_sum<LANES>(e2.x + e2.y);  // not of the rows beside: each has its own bits
            finish_mean(off, squares, moved ? lacks : 0.0f, static_cast<float>(a.cols), a.per_col);
            mean += off;
        }
        const float r = rsqrtf(fmaf(squares, a.per_col, a.eps));
        if (row >= a.rows) continue;
        if (lane == 0) {
            if (a.mean) a.mean[row] = at + mean;
            if (a.rstd) a.rstd[row] = r;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = fma2(fma2(f[j], both(r), both(-off * r)), w[j], b[j]);
        store_run<DT>(row_of<DT>(a.y, row, a.y_stride), 0, past, a.cols, lane, pack8<DT>(f));
    }
}

// ---------------------------------------------------------------- backward
//
// With n = (h - m) r and g = dy w:  dx = r (g - mean(g) - n mean(g n)) + dh.
// Blocks walk over rows (row, row + writers, ..) and keep their columns' sums of
// dy n and dy in registers; each writes them once, to its own row of `partial`,
// and column_sums_kernel adds those rows in order.

// Matrices whose rows lie apart, element by element: slower, for the views that
// need it.
template <int DT, int KT> __global__ void __launch_bounds__(512) layernorm_grad_kernel(LayerNormGradArgs a) {
    enter_grid();
    __shared__ float2 part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t writer = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t writers = static_cast<int64_t>(gridDim.x) * blockDim.y;
    float2 dw[KT][4], db[KT][4];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = both(0.0f);
    const float per_col = 1.0f / static_cast<float>(a.cols);
    int turn = 0;
    for (int64_t row = writer; row < a.rows; row += writers, turn ^= 1) {
        const void *dy = row_of<DT>(a.dy, row, a.dy_stride), *h = row_of<DT>(a.h, row, a.h_stride);
        const float2 m = both(-a.mean[row]), r = both(a.rstd[row]);
        Raw8<DT> cdy[KT], ch[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            cdy[k] = load_tile<DT, false>(dy, (warp + k * warps) * kTileCols, a.cols, lane);
            ch[k] = load_tile<DT, false>(h, (warp + k * warps) * kTileCols, a.cols, lane);
        }
        float2 c1 = both(0.0f), c2 = both(0.0f);
        auto products = [&](int k, float2 (&g)[4], float2 (&n)[4], bool add) {
            float2 w[4];
            load_columns<DT, kApart>(a.weight, a.weight_f32, 1.0f, warp + k * warps, 0, a.cols, lane, w);
            unpack8<DT>(cdy[k], g);
            unpack8<DT>(ch[k], n);
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = mul2(add2(n[j], m), r);
            clip_columns<false>(warp + k * warps, 0, a.cols, lane, n);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (add) {
                    dw[k][j] = fma2(g[j], n[j], dw[k][j]);
                    db[k][j] = add2(g[j], db[k][j]);
                }
                g[j] = mul2(g[j], w[j]);
            }
        };
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4];
            products(k, g, n, true);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c1 = add2(c1, g[j]);
                c2 = fma2(g[j], n[j], c2);
            }
        }
        const float2 c = block_sum2(make_float2(c1.x + c1.y, c2.x + c2.y), warps, part[turn]);
        const float2 m1 = both(-c.x * per_col), m2 = both(-c.y * per_col);
        void *dx = row_of<DT>(a.dx, row, a.dx_stride);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4], d[4];
            products(k, g, n, false);
            if (a.dh) {
                unpack8<DT>(load_tile<DT, false>(row_of<DT>(a.dh, row, a.dh_stride), (warp + k * warps) * kTileCols, a.cols, lane), d);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = both(0.0f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = fma2(r, fma2(m2, n[j], add2(g[j], m1)), d[j]);
            store_tile<DT, false>(dx, (warp + k * warps) * kTileCols, a.cols, lane, pack8<DT>(d));
        }
    }
    if (a.partial == nullptr) return;
    float *out = a.partial + writer * a.cols, *out_b = a.partial + (writers + writer) * a.cols;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = col_of<false>(warp + k * warps, 0, lane, j);
            if (col < a.cols) {
                out[col] = (j & 1) ? dw[k][j / 2].y : dw[k][j / 2].x;
                out_b[col] = (j & 1) ? db[k][j / 2].y : db[k][j / 2].x;
            }
        }
}

// Matrices whose rows lie alike, their loads as asynchronous copies of 16 bytes
// into a ring of `depth` rows in shared memory: rows on their way take no
// registers.  Each thread copies and reads its own elements alone, waits for its
// own copies and needs no barrier for them.  P pieces of 16 bytes hold a lane's 8
// elements of a tile: of binary32 the two are 128 columns apart, so that a copy of
// the warp takes whole sectors.  Rows that start anywhere: a writer's rows are a
// multiple of 8 apart and so start at one place between multiples of 16 bytes, and
// the columns that a thread holds, and sums, stay the same.  A row's first piece
// begins `past` elements before the row, in the row before it or the gap there, and
// what it brings along is cleared; only before the first row nothing is read.
//
// PAIR: rows of more than 16 warps x 2 tiles go to clusters of two blocks, a half of
// the warps' tiles each, which write their sums into each other's shared memory.  The
// barrier between a row's two passes is the cluster's then; what its wait takes passes
// while the row before is finished.
//
// Bounded by memory where rows are many and wide (8192 of 4096 bf16 50 us at a floor of
// 40, of 16384 210 at 161, 4096 of 12288 binary32 146 at 121), by the latency of a
// row after the other where they are few (3001 of 2001 f16 20 us at 7).  512 threads
// an SM: more blocks write more sums of columns, and fit fewer rows ahead (768 threads
// took 24 us there).
template <int DT, int KT, bool ALIGNED, bool PAIR>
__global__ void __launch_bounds__(512, 1) layernorm_grad_ring_kernel(const __grid_constant__ LayerNormGradArgs a, int depth) {
    enter_grid();
    using T = typename ElemOf<DT>::type;
    constexpr int B = ElemOf<DT>::kBytes, P = B / 2, E = 16 / B;
    extern __shared__ uint4 ring[];  // [row][dy, h, dh][tile][piece][thread]
    __shared__ alignas(16) float2 parts[4][2][16];  // of a row and the next: the warps' sums, zeros beyond
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int threads = blockDim.x * blockDim.y, slot_size = 3 * KT * P * threads;
    uint4 *const mine = ring + threadIdx.y * blockDim.x + threadIdx.x;
    // the row's warps, of this block and its neighbour
    const int half = PAIR ? blockIdx.x & 1 : 0, row_warps = PAIR ? 2 * warps : warps, row_warp = half * warps + warp;
    const int64_t team = PAIR ? blockIdx.x >> 1 : blockIdx.x, teams = PAIR ? gridDim.x >> 1 : gridDim.x;
    const int64_t writer = team * blockDim.y + threadIdx.y, writers = teams * blockDim.y;
    const int past = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row_of<DT>(a.dy, writer, a.dy_stride)) % 16) / B;
    auto col = [&](int k, int piece) { return (row_warp + k * row_warps) * kTileCols + piece * 128 + lane * E - past; };
    auto place = [&](int slot, int matrix, int k, int piece) {
        return mine + slot * slot_size + ((matrix * KT + k) * P + piece) * threads;
    };
    // columns of the weight, in the layout of the pieces
    auto weights = [&](int k, float2 (&w)[4]) {
        if constexpr (P == 1) {
            load_columns<DT, ALIGNED ? kAligned : kShifted>(a.weight, a.weight_f32, 1.0f, row_warp + k * row_warps, past, a.cols, lane, w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col(k, j / 4) + j % 4;
                float v = a.weight == nullptr ? 1.0f : 0.0f;
                if (a.weight != nullptr && c >= 0 && c < a.cols) v = static_cast<const float *>(a.weight)[c];
                (j & 1 ? w[j / 2].y : w[j / 2].x) = v;
            }
        }
    };
    float2 dw[KT][4], db[KT][4], w[KT][4];
    int bytes[KT][P];  // that a piece has up to the row's end, 0 to 16; zeros after them
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        weights(k, w[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = both(0.0f);
#pragma unroll
        for (int piece = 0; piece < P; ++piece) bytes[k][piece] = max(0, min(16, (a.cols - col(k, piece)) * B));
    }
    // pieces outside the row stay zero: nothing is copied there
    for (int slot = 0; slot < depth; ++slot)
#pragma unroll
        for (int matrix = 0; matrix < 3; ++matrix)
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int piece = 0; piece < P; ++piece)
                    if (bytes[k][piece] == 0 || (matrix == 2 && a.dh == nullptr))
                        *place(slot, matrix, k, piece) = make_uint4(0u, 0u, 0u, 0u);
    const int tile_bytes = row_warps * kTileCols * B;  // from one of a thread's tiles to the next
    auto copy = [&](const char *from, bool first, uint4 *to) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int piece = 0; piece < P; ++piece) {
                uint4 *at = to + (k * P + piece) * threads;
                if (!ALIGNED && k == 0 && piece == 0 && first && col(0, 0) < 0) {  // nothing before this row is the matrix's
                    const T *elements = reinterpret_cast<const T *>(from);
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        reinterpret_cast<T *>(at)[j] = j >= past && j - past < a.cols ? elements[j] : T(0);
                } else if (bytes[k][piece] > 0) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))),
                                    "l"(from + k * tile_bytes + piece * 128 * B), "r"(bytes[k][piece]) : "memory");
                }
            }
    };
    // the next row to be copied, from this thread's first piece on
    int64_t copy_row = writer;
    const int64_t first_byte = static_cast<int64_t>(col(0, 0)) * B;
    const char *from_dy = static_cast<const char *>(row_of<DT>(a.dy, writer, a.dy_stride)) + first_byte;
    const char *from_h = static_cast<const char *>(row_of<DT>(a.h, writer, a.h_stride)) + first_byte;
    const char *from_dh = a.dh ? static_cast<const char *>(row_of<DT>(a.dh, writer, a.dh_stride)) + first_byte : nullptr;
    auto copy_next = [&](int slot) {
        if (copy_row < a.rows) {
            uint4 *to = mine + slot * slot_size;
            copy(from_dy, copy_row * a.dy_stride < past, to);
            copy(from_h, copy_row * a.h_stride < past, to + KT * P * threads);
            if (a.dh) copy(from_dh, copy_row * a.dh_stride < past, to + 2 * KT * P * threads);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        copy_row += writers;
        from_dy += writers * a.dy_stride * B;
        from_h += writers * a.h_stride * B;
        if (a.dh) from_dh += writers * a.dh_stride * B;
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
    // zeros in what the row's first piece brought along
    auto clear_first = [&](int slot, int matrix) {
        uint4 *at = place(slot, matrix, 0, 0);
        uint4 v = *at;
        const int words = past * B / 4;
        const uint32_t half = past * B % 4 ? 0xffff0000u : 0xffffffffu;  // of the word in which the row begins
        v.x &= words > 0 ? 0u : half;
        v.y &= words > 1 ? 0u : words == 1 ? half : 0xffffffffu;
        v.z &= words > 2 ? 0u : words == 2 ? half : 0xffffffffu;
        v.w &= words == 3 ? half : 0xffffffffu;
        *at = v;
    };
    const float per_col = 1.0f / static_cast<float>(a.cols);
    // A row's first pass: its columns' sums, and its own two to `sums`.  The second is of
    // g (h - m), whose r comes later: columns outside the row have g 0 and h 0, and -m r
    // might be infinite.
    auto add_row = [&](int slot, float mean, float rstd, float2 *sums) {
        const float2 m = both(-mean), r = both(rstd);
        if (!ALIGNED && col(0, 0) < 0) {
            clear_first(slot, 0);
            clear_first(slot, 1);
        }
        float2 c1 = both(0.0f), c2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4];
            held(slot, 0, k, g);
            held(slot, 1, k, n);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n[j] = add2(n[j], m);
                dw[k][j] = fma2(g[j], mul2(n[j], r), dw[k][j]);
                db[k][j] = add2(g[j], db[k][j]);
                g[j] = mul2(g[j], w[k][j]);
                c1 = add2(c1, g[j]);
                c2 = fma2(g[j], n[j], c2);
            }
        }
        const float2 c = warp_sum2(make_float2(c1.x + c1.y, c2.x + c2.y));
        if (lane == 0) {
            sums[PAIR ? half * 16 + warp : warp] = c;
            if (PAIR) *const_cast<float2 *>(in_block(&sums[half * 16 + warp], half ^ 1)) = c;
        }
    };
    // read two rows ahead, and not touched before it is needed
    auto statistics = [&](int64_t row, float &m, float &r) {
        if (row < a.rows) m = a.mean[row], r = a.rstd[row];
    };
    constexpr int kParts = PAIR ? 32 : 16;  // of a row
    float2 *const part = &parts[threadIdx.y][0][0];
    for (int i = threadIdx.x; i < 2 * kParts; i += blockDim.x) part[i] = both(0.0f);
    if (PAIR) cluster_sync();  // before the neighbour writes here
    else __syncthreads();
#pragma unroll 1
    for (int q = 0; q < depth; ++q) copy_next(q);
    float mean = 0.0f, rstd = 0.0f, next_mean = 0.0f, next_rstd = 0.0f;
    statistics(writer, mean, rstd);
    statistics(writer + writers, next_mean, next_rstd);
    if (depth == 2) copies_left<1>();
    else if (depth == 3) copies_left<2>();
    else copies_left<3>();
    if (writer < a.rows) add_row(0, mean, rstd, part);
    if (PAIR) cluster_arrive();
    int turn = 0, slot = 0;
#pragma unroll 1
    for (int64_t row = writer; row < a.rows; row += writers, turn ^= 1) {
        const int next_slot = slot + 1 == depth ? 0 : slot + 1;
        float2 c = both(0.0f);
        if constexpr (PAIR) {
            cluster_wait();
            c = warp_sum2(part[turn * kParts + lane]);
        } else {
            if (warps > 1) __syncthreads();
            else __syncwarp();
            const float4 *all = reinterpret_cast<const float4 *>(part + turn * kParts);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if (2 * i >= warps) break;
                const float4 p = all[i], q = all[i + 1];
                c = add2(add2(c, add2(make_float2(p.x, p.y), make_float2(p.z, p.w))), add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
            }
        }
        if (depth == 2) copies_left<0>();
        else if (depth == 3) copies_left<1>();
        else copies_left<2>();
        float after_mean = 0.0f, after_rstd = 0.0f;
        statistics(row + 2 * writers, after_mean, after_rstd);
        if (row + writers < a.rows) add_row(next_slot, next_mean, next_rstd, part + (turn ^ 1) * kParts);
        if (PAIR) cluster_arrive();
        const float2 m = both(-mean), r = both(rstd);
        const float2 m1 = both(-c.x * per_col), m2 = both(-c.y * rstd * per_col * rstd);
        T *dx = static_cast<T *>(row_of<DT>(a.dx, row, a.dx_stride));
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float2 g[4], n[4], d[4];
            held(slot, 0, k, g);
            held(slot, 1, k, n);
            held(slot, 2, k, d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d[j] = fma2(r, fma2(g[j], w[k][j], fma2(m2, add2(n[j], m), m1)), d[j]);
            const Raw8<DT> o = pack8<DT>(d);
#pragma unroll
            for (int piece = 0; piece < P; ++piece) {
                const int c = col(k, piece);
                if ((ALIGNED || c >= 0) && bytes[k][piece] == 16) {
                    Vec<16> v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v.w[i] = o.w[piece * 4 + i];
                    st<16>(dx + c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        if ((ALIGNED || c + j >= 0) && c + j < a.cols)
                            dx[c + j] = static_cast<T>(o.w[piece * 4 + j * B / 4] >> (j * B % 4 * 8));
                }
            }
        }
        copy_next(slot);
        slot = next_slot;
        mean = next_mean, rstd = next_rstd, next_mean = after_mean, next_rstd = after_rstd;
    }
    copies_left<0>();
    if (PAIR) cluster_wait();  // the neighbour has written its last sums here
    if (a.partial == nullptr) return;
    // The block's sums: of one writer straight from the registers, where whole runs
    // can be written; otherwise by columns through the ring's place, the writers' in order.
    float *out = a.partial + team * a.cols, *out_b = out + teams * a.cols;
    if (ALIGNED && blockDim.y == 1 && a.cols % 4 == 0) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int c = col(k, P == 2 ? j / 2 : 0) + (P == 2 ? 0 : 2 * j);
                if (c >= a.cols) continue;
                *reinterpret_cast<float4 *>(out + c) = make_float4(dw[k][j].x, dw[k][j].y, dw[k][j + 1].x, dw[k][j + 1].y);
                *reinterpret_cast<float4 *>(out_b + c) = make_float4(db[k][j].x, db[k][j].y, db[k][j + 1].x, db[k][j + 1].y);
            }
        return;
    }
    __syncthreads();
    float *sums = reinterpret_cast<float *>(ring) + static_cast<int64_t>(threadIdx.y) * 2 * a.cols;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = P == 2 ? col(k, j / 4) + j % 4 : col(k, 0) + j;
            if (c < 0 || c >= a.cols) continue;
            sums[c] = j & 1 ? dw[k][j / 2].y : dw[k][j / 2].x;
            sums[a.cols + c] = j & 1 ? db[k][j / 2].y : db[k][j / 2].x;
        }
    if (blockDim.y == 1) {  // a warp's own columns
        __syncwarp();
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (row_warp + k * row_warps) * kTileCols - past + j * 32 + lane;
                if (c < 0 || c >= a.cols) continue;
                out[c] = sums[c];
                out_b[c] = sums[a.cols + c];
            }
        return;
    }
    __syncthreads();
    sums = reinterpret_cast<float *>(ring);
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * a.cols; i += threads) {
        float sum = sums[i];
        for (int y = 1; y < static_cast<int>(blockDim.y); ++y) sum += sums[y * 2 * a.cols + i];
        if (i < a.cols) out[i] = sum;
        else out_b[i - a.cols] = sum;
    }
}

// Narrow rows, several to a warp as in layernorm_narrow_kernel: each lane holds its 8
// columns' sums over its rows, which are a multiple of 8 apart, and the next row is on its
// way, in registers, while one is worked on.  131072 rows of 64 bf16 16 us (floor 10; by
// the ring 50), 65536 of 128 16 us (10; 29), of 256 24 us (20; 32), of 128 binary32 24 us
// (20; 31); shifted ones, where there are many, 131072 of 51 bf16 21 us (8; 70), 65536 of
// 101 22 us (8; 39), of 201 36 us (16; 41).  As many blocks as an SM holds at once: two,
// with three at fewer registers 17 us for 65536 of 128 bf16; three where an aligned row
// takes a warp, with two 28 us for 256 columns.
__host__ __device__ constexpr int narrow_resident(int dt, int rows, int lanes) {
    return dt != DT_F32 && rows == kAligned && lanes == 32 ? 3 : 2;
}
template <int DT, int ROWS, int LANES>
__global__ void __launch_bounds__(32 * kNarrowWarps, narrow_resident(DT, ROWS, LANES)) layernorm_grad_narrow_kernel(const __grid_constant__ LayerNormGradArgs a) {
    enter_grid();
    constexpr int kRows = 32 / LANES;  // of a warp at a time
    // sums of a warp, or of each of its groups, whose columns lie apart by `past`
    constexpr int kSums = kNarrowWarps * (ROWS == kShifted ? kRows : 1);
    __shared__ alignas(8) float sums[kSums][2][8 * LANES];
    const int lane = threadIdx.x & (LANES - 1), group = (threadIdx.x & 31) / LANES, warp = threadIdx.x >> 5;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kNarrowWarps * kRows;
    int64_t base = (static_cast<int64_t>(blockIdx.x) * kNarrowWarps + warp) * kRows;  // of the warp's rows the first
    const int past = ROWS == kShifted ? past_of<DT>(row_of<DT>(a.dy, base + group, a.dy_stride)) : 0;
    const float per_col = 1.0f / static_cast<float>(a.cols);
    float2 w[4], dw[4], db[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = db[j] = both(0.0f);
    Raw8<DT> rdy, rh, rdh;
    float mean = 0.0f, rstd = 0.0f;
    auto load = [&] {
        // behind the last row: of aligned ones it again, of shifted ones nothing
        const int64_t row = ROWS == kAligned ? min(base + group, a.rows - 1) : base + group;
        const bool inner = row > 0 && row + 1 < a.rows;
        const int cols = ROWS == kAligned || row < a.rows ? a.cols : 0;
        rdy = load_row<DT, ROWS>(row_of<DT>(a.dy, row, a.dy_stride), 0, past, cols, lane, inner);
        rh = load_row<DT, ROWS>(row_of<DT>(a.h, row, a.h_stride), 0, past, cols, lane, inner);
        if (a.dh) rdh = load_row<DT, ROWS>(row_of<DT>(a.dh, row, a.dh_stride), 0, past, cols, lane, inner);
        const int64_t at = ROWS == kAligned ? row : min(row, a.rows - 1);
        mean = a.mean[at], rstd = a.rstd[at];
    };
    if (base < a.rows) load();
    load_columns<DT, ROWS>(a.weight, a.weight_f32, 1.0f, 0, past, a.cols, lane, w);
    while (base < a.rows) {
        const int64_t row = base + group;
        const bool given = row < a.rows;
        float2 g[4], n[4], d[4];
        unpack8<DT>(rdy, g);
        unpack8<DT>(rh, n);
        if (a.dh) unpack8<DT>(rdh, d);
        const float2 m = both(-mean), r = both(rstd);
        base += step;
        if (base < a.rows) load();
        float2 c = both(0.0f), c2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = add2(n[j], m);
        if constexpr (ROWS == kShifted) {  // what runs have of the rows beside
            clip_columns<true>(0, past, a.cols, lane, g);
            clip_columns<true>(0, past, a.cols, lane, n);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!given) g[j] = both(0.0f);
            if (!a.dh) d[j] = both(0.0f);
            if (given) dw[j] = fma2(g[j], mul2(n[j], r), dw[j]);
            db[j] = add2(g[j], db[j]);
            g[j] = mul2(g[j], w[j]);
            c = add2(c, g[j]);
            c2 = fma2(g[j], n[j], c2);
        }
        c = make_float2(c.x + c.y, c2.x + c2.y);
#pragma unroll
        for (int i = LANES / 2; i > 0; i >>= 1)
            c = add2(c, make_float2(__shfl_xor_sync(kAllLanes, c.x, i), __shfl_xor_sync(kAllLanes, c.y, i)));
        if (row >= a.rows) continue;
        const float2 m1 = both(-c.x * per_col), m2 = both(-c.y * r.x * per_col * r.x);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = fma2(r, add2(g[j], fma2(m2, n[j], m1)), d[j]);
        store_row<DT, ROWS>(row_of<DT>(a.dx, row, a.dx_stride), 0, past, a.cols, lane, pack8<DT>(d));
    }
    if (a.partial == nullptr) return;
    if constexpr (ROWS == kAligned) {
#pragma unroll
        for (int i = LANES; i < 32; i *= 2)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dw[j] = add2(dw[j], make_float2(__shfl_xor_sync(kAllLanes, dw[j].x, i), __shfl_xor_sync(kAllLanes, dw[j].y, i)));
                db[j] = add2(db[j], make_float2(__shfl_xor_sync(kAllLanes, db[j].x, i), __shfl_xor_sync(kAllLanes, db[j].y, i)));
            }
        if (group == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                *reinterpret_cast<float2 *>(&sums[warp][0][lane * 8 + 2 * j]) = dw[j];
                *reinterpret_cast<float2 *>(&sums[warp][1][lane * 8 + 2 * j]) = db[j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = lane * 8 + j - past;
            if (col < 0 || col >= a.cols) continue;
            sums[warp * kRows + group][0][col] = j & 1 ? dw[j / 2].y : dw[j / 2].x;
            sums[warp * kRows + group][1][col] = j & 1 ? db[j / 2].y : db[j / 2].x;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * 8 * LANES; i += 32 * kNarrowWarps) {
        const int which = i / (8 * LANES), col = i % (8 * LANES);
        if (col >= a.cols) continue;
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kSums; ++v) sum += sums[v][which][col];
        a.partial[(which * static_cast<int64_t>(gridDim.x) + blockIdx.x) * a.cols + col] = sum;
    }
}

// Rows too wide to hold are read twice, a block of 32 warps a row, after
// layernorm_columns_kernel has taken the columns' sums (dx may be dy).
template <int DT, int ROWS> __global__ void __launch_bounds__(1024) layernorm_grad_wide_kernel(LayerNormGradArgs a) {
    enter_grid();
    __shared__ float2 part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const void *dy = row_of<DT>(a.dy, row, a.dy_stride), *h = row_of<DT>(a.h, row, a.h_stride);
    const int past = ROWS == kShifted ? past_of<DT>(dy) : 0, tiles = (a.cols + past + kTileCols - 1) / kTileCols;
    const bool inner = row > 0 && row + 1 < a.rows;
    const float2 m = both(-a.mean[row]), r = both(a.rstd[row]);
    auto products = [&](int tile, float2 (&g)[4], float2 (&n)[4]) {
        float2 w[4];
        load_columns<DT, ROWS>(a.weight, a.weight_f32, 1.0f, tile, past, a.cols, lane, w);
        unpack8<DT>(load_row<DT, ROWS>(dy, tile, past, a.cols, lane, inner), g);
        unpack8<DT>(load_row<DT, ROWS>(h, tile, past, a.cols, lane, inner), n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = mul2(add2(n[j], m), r);
            g[j] = mul2(g[j], w[j]);
        }
        clip_columns<ROWS != kApart>(tile, past, a.cols, lane, n);
        clip_columns<ROWS != kApart>(tile, past, a.cols, lane, g);
    };
    float2 c1 = both(0.0f), c2 = both(0.0f), g[4], n[4];
    for (int t = warp; t < tiles; t += warps) {
        products(t, g, n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c1 = add2(c1, g[j]);
            c2 = fma2(g[j], n[j], c2);
        }
    }
    const float2 c = block_sum2(make_float2(c1.x + c1.y, c2.x + c2.y), warps, part);
    const float per_col = 1.0f / static_cast<float>(a.cols);
    const float2 m1 = both(-c.x * per_col), m2 = both(-c.y * per_col);
    void *dx = row_of<DT>(a.dx, row, a.dx_stride);
    for (int t = warp; t < tiles; t += warps) {
        products(t, g, n);
        float2 d[4] = {};
        if (a.dh) unpack8<DT>(load_row<DT, ROWS>(row_of<DT>(a.dh, row, a.dh_stride), t, past, a.cols, lane, inner), d);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = fma2(r, fma2(m2, n[j], add2(g[j], m1)), d[j]);
        store_row<DT, ROWS>(dx, t, past, a.cols, lane, pack8<DT>(d));
    }
}

// dweight and dbias of wide rows: one warp takes a tile of columns over the rows
// blockIdx.y, blockIdx.y + gridDim.y, ..
template <int DT, bool VEC> __global__ void __launch_bounds__(256) layernorm_columns_kernel(LayerNormGradArgs a) {
    enter_grid();
    const int lane = threadIdx.x & 31;
    const int base = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kTileCols;
    if (base >= a.cols) return;
    float2 dw[4] = {}, db[4] = {};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float2 g[4], n[4];
        const float2 m = both(-a.mean[row]), r = both(a.rstd[row]);
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.dy, row, a.dy_stride), base, a.cols, lane), g);
        unpack8<DT>(load_tile<DT, VEC>(row_of<DT>(a.h, row, a.h_stride), base, a.cols, lane), n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dw[j] = fma2(g[j], mul2(add2(n[j], m), r), dw[j]);
            db[j] = add2(g[j], db[j]);
        }
    }
    float *out = a.partial + static_cast<int64_t>(blockIdx.y) * a.cols;
    float *out_b = out + static_cast<int64_t>(gridDim.y) * a.cols;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = tile_col<VEC>(base, lane, j);
        if (col < a.cols) {
            out[col] = (j & 1) ? dw[j / 2].y : dw[j / 2].x;
            out_b[col] = (j & 1) ? db[j / 2].y : db[j / 2].x;
        }
    }
}

// ---------------------------------------------------------------- launches

constexpr int kLayerNormWarps = 16;  // that hold a row
constexpr int kRingBytes = 200 * 1024;  // of an SM's shared memory

// Whether two matrices have their rows at the same place between multiples of 8 elements.
template <int DT> bool same_runs(const void *p, int64_t stride, const void *q, int64_t other) {
    return q == nullptr || (past_of<DT>(p) == past_of<DT>(q) && (stride - other) % 8 == 0);
}

// Tiles a thread: as few as hold the row in 16 warps, which is the shortest way for
// few rows.  Where there are many, two keep more loads on their way, and four pay for
// the statistics of wide 16-bit rows: 16384 rows of 4096 bf16 take 83 us with four, 94 with
// two, 16384 of 4001 94 us with four and 119 with one; of 2001 binary32 93 us with one,
// 90 with two.  But walkers hold weights as well, fewer of them fit, and what matters is
// how many columns an SM works on: 6392 rows of 2135 bf16 take 35 us with four (45 of
// 64 tiles), 30 with one (27 of 32); of less than 8 tiles the barrier is short and one
// is as good or better (7897 x 777 f16 17.5 us, 18.7 with four).
//
// Rows of more than 32 tiles: up to a row an SM go to clusters of two blocks (30 of 12480
// bf16 4.4 us, by one block of four tiles a thread 5.3; 600 of 16384 22.8 and 14.7 us),
// of shifted rows half as many.  More go to one block each: 8192 of 16384 bf16 163 us by
// walkers, 224 by a block a row, 288 by clusters; 4096 of 16384 binary32 169 us by a
// block a row, 218 by walkers, 190 by clusters; but shifted rows of binary32, for which
// the registers do not suffice, to clusters, 231 and 256 us.
template <int DT, int ROWS> cudaError_t layernorm_launch(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    constexpr bool kNarrow = DT != DT_F32;
    const int tiles = static_cast<int>((static_cast<int64_t>(a.cols) + (ROWS == kShifted ? 7 : 0) + kTileCols - 1) / kTileCols);
    const bool many = a.rows >= 4 * static_cast<int64_t>(sms);
    info->vec_bytes = ROWS != kApart ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    int kt = tiles_per_thread(tiles, kLayerNormWarps, 4);
    const bool pair = ROWS != kApart && kt == 4 && (a.rows <= (ROWS == kShifted ? sms / 2 : sms) || (ROWS == kShifted && !kNarrow));
    if (pair) {
        kt = 2;
    } else if (kt != 0 && ROWS == kShifted && kNarrow && tiles >= 8) {
        // tiles of the rows that an SM holds, of 32 by ones and of 64 by fours
        const int one = kt == 1 ? tiles * (32 / tiles) : 0, four = tiles * (16 / ((tiles + 3) / 4));
        if (many ? 4 * four >= 7 * one : kt == 2 && a.rows > sms) kt = 4;
    } else if (kt != 0 && many) {
        const bool spread = ROWS == kShifted && tiles > 2 && (kNarrow || a.rows < 32 * static_cast<int64_t>(sms));
        kt = std::max(kt, tiles == 1 || spread ? 1 : kNarrow && tiles > 8 ? 4 : 2);
    }
    const int blocks = pair ? 2 : 1;  // to a row
    int warps = 32, per_block = 1;
    if (kt != 0) {
        warps = (tiles + blocks * kt - 1) / (blocks * kt);
        if (warps == 1 && many) per_block = 8;
    }
    const bool small = kNarrow && ROWS != kShifted && kt == 4 && warps <= 8;
    int64_t teams = (a.rows + per_block - 1) / per_block;
    size_t smem = 0;
    if (kt != 0 && layernorm_walks(DT, ROWS, kt, small ? 8 : 16)) {
        smem = static_cast<size_t>(kt) * warps * per_block * 32 * 4 * sizeof(float4);
        // as many walkers as an SM holds at 64 or 128 registers
        const int resident = std::max(1, (kt == 1 ? 32 : 16) / (warps * per_block));
        const int64_t most = static_cast<int64_t>(sms) * resident / (8 * blocks) * 8;
        if (most > 0) teams = std::min(teams, most);
    }
    info->grid = static_cast<int>(blocks * teams);
    info->block = 32 * warps * per_block;
    auto kernel = kt == 0   ? layernorm_kernel<DT, ROWS, 1, false, 32, false>
                  : kt == 1 ? layernorm_kernel<DT, ROWS, 1, true, 16, false>
                            : layernorm_kernel<DT, ROWS, 2, true, 16, false>;
    if constexpr (kNarrow || ROWS != kShifted)
        if (kt == 4) kernel = layernorm_kernel<DT, ROWS, 4, true, 16, false>;
    if constexpr (kNarrow && ROWS != kShifted)
        if (small) kernel = layernorm_kernel<DT, ROWS, 4, true, 8, false>;
    if constexpr (ROWS != kApart)
        if (pair) kernel = layernorm_kernel<DT, ROWS, 2, true, 16, true>;
    if (smem > 32 * 1024) {  // up to 48 KiB less the kernel's own variables go without asking
        static std::atomic<uint64_t> ready[5];
        constexpr int kMost = 4 * kLayerNormWarps * 32 * 4 * sizeof(float4);
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), kMost, &ready[pair ? 3 : kt]);
        if (e != cudaSuccess) return e;
    }
    return launch_rows(kernel, dim3(info->grid), dim3(32 * warps, per_block), smem, blocks, s, a);
}

template <int DT, int LANES, int TURNS> cudaError_t layernorm_narrow(const LayerNormArgs &a, cudaStream_t s, LaunchInfo *info) {
    constexpr int kRows = kNarrowWarps * 32 / LANES * TURNS;
    info->grid = static_cast<int>((a.rows + kRows - 1) / kRows);
    info->block = 32 * kNarrowWarps;
    info->vec_bytes = 8 * ElemOf<DT>::kBytes;
    return launch_rows(layernorm_narrow_kernel<DT, LANES, TURNS>, dim3(info->grid), dim3(info->block), 0, 1, s, a);
}

template <int DT, int LANES> cudaError_t layernorm_narrow_walk(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    constexpr int kRows = kNarrowWarps * 32 / LANES;
    info->grid = static_cast<int>(std::min<int64_t>((a.rows + kRows - 1) / kRows, static_cast<int64_t>(sms) * kNarrowWalkers));
    info->block = 32 * kNarrowWarps;
    info->vec_bytes = 8 * ElemOf<DT>::kBytes;
    return launch_rows(layernorm_narrow_walk_kernel<DT, LANES>, dim3(info->grid), dim3(info->block), 0, 1, s, a);
}

template <int DT> cudaError_t layernorm_dispatch(const LayerNormArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const bool alike = a.cols >= 8 && same_runs<DT>(a.x, a.x_stride, a.residual, a.residual_stride) &&
                       same_runs<DT>(a.x, a.x_stride, a.y, a.y_stride) && same_runs<DT>(a.x, a.x_stride, a.h, a.h_stride);
    if (!alike) return layernorm_launch<DT, kApart>(a, sms, s, info);
    if (!wide_rows<DT>(a.x, a.x_stride) || !wide_weight<DT>(a.weight, a.weight_f32) || !wide_weight<DT>(a.bias, a.weight_f32)) {
        if (a.cols + 7 <= 64) return layernorm_narrow_walk<DT, 8>(a, sms, s, info);
        if (a.cols + 7 <= 128) return layernorm_narrow_walk<DT, 16>(a, sms, s, info);
        if (a.cols + 7 <= 256) return layernorm_narrow_walk<DT, 32>(a, sms, s, info);
        return layernorm_launch<DT, kShifted>(a, sms, s, info);
    }
    const bool two = DT != DT_F32 && a.rows >= 64 * static_cast<int64_t>(sms);
    if constexpr (DT != DT_F32) {
        if (two && a.cols <= 64) return layernorm_narrow<DT, 8, 2>(a, s, info);
        if (two && a.cols <= 128) return layernorm_narrow<DT, 16, 2>(a, s, info);
        if (two && a.cols <= 256) return layernorm_narrow<DT, 32, 2>(a, s, info);
    }
    if (a.cols <= 64) return layernorm_narrow<DT, 8, 1>(a, s, info);
    if (a.cols <= 128) return layernorm_narrow<DT, 16, 1>(a, s, info);
    return layernorm_launch<DT, kAligned>(a, sms, s, info);
}

template <int DT>
cudaError_t layernorm_grad_dispatch(const LayerNormGradArgs &a, int64_t most_writers, int sms, cudaStream_t s, LaunchInfo *info,
                                    int *launches) {
    const bool runs = a.cols >= 8 && same_runs<DT>(a.dy, a.dy_stride, a.h, a.h_stride) &&
                      same_runs<DT>(a.dy, a.dy_stride, a.dh, a.dh_stride) && same_runs<DT>(a.dy, a.dy_stride, a.dx, a.dx_stride);
    const bool aligned = runs && wide_rows<DT>(a.dy, a.dy_stride) && wide_weight<DT>(a.weight, a.weight_f32);
    const int tiles = static_cast<int>((static_cast<int64_t>(a.cols) + (aligned ? 0 : 7) + kTileCols - 1) / kTileCols);
    const bool many = a.rows >= 4 * static_cast<int64_t>(sms);
    int kt = tiles_per_thread(tiles, 8, 2);
    // One tile a thread spreads a row over more warps; two save the barrier of rows of
    // two tiles, and instructions of wide 16-bit rows, where there are many.  16384 rows
    // of 2048 bf16: 50 us with two, 57 with one; 3000 rows: 17 and 16 us.
    if (kt == 1 && many && tiles == 2) kt = 2;
    if (DT != DT_F32 && kt == 1 && tiles > 5 && a.rows >= 32 * static_cast<int64_t>(sms)) kt = 2;
    if (kt == 0) kt = tiles_per_thread(tiles, kLayerNormWarps, 2);
    const bool pair = kt == 0 && runs && tiles <= 4 * kLayerNormWarps && (aligned || sms >= 16);  // 8 pairs of blocks
    if (pair) kt = 2;
    const bool sums = a.dweight != nullptr || a.dbias != nullptr;
    int64_t writers = 0;
    cudaError_t e = cudaSuccess;
    info->vec_bytes = runs ? 16 : ElemOf<DT>::kBytes;
    if (a.rows > 0 && tiles == 1 && (aligned || (runs && many))) {
        const int width = a.cols + (aligned ? 0 : 7), lanes = width <= 64 ? 8 : width <= 128 ? 16 : 32;
        const int rows = kNarrowWarps * 32 / lanes;  // of a block at a time
        const int resident = narrow_resident(DT, aligned ? kAligned : kShifted, lanes);
        writers = std::min<int64_t>({(a.rows + rows - 1) / rows, static_cast<int64_t>(sms) * resident, most_writers});
        info->grid = static_cast<int>(writers);
        info->block = 32 * kNarrowWarps;
        info->vec_bytes = 8 * ElemOf<DT>::kBytes;
        auto kernel = lanes == 8    ? layernorm_grad_narrow_kernel<DT, kAligned, 8>
                      : lanes == 16 ? layernorm_grad_narrow_kernel<DT, kAligned, 16>
                                    : layernorm_grad_narrow_kernel<DT, kAligned, 32>;
        if (!aligned)
            kernel = lanes == 8    ? layernorm_grad_narrow_kernel<DT, kShifted, 8>
                     : lanes == 16 ? layernorm_grad_narrow_kernel<DT, kShifted, 16>
                                   : layernorm_grad_narrow_kernel<DT, kShifted, 32>;
        e = launch_rows(kernel, dim3(info->grid), dim3(info->block), 0, 1, s, a);
        ++*launches;
    } else if (a.rows > 0 && kt != 0) {
        const int blocks = pair ? 2 : 1, warps = (tiles + kt * blocks - 1) / (kt * blocks);
        // a row for each of 4 warps, where one holds it: their sums leave the block as one
        const int per_block = runs && warps == 1 && many ? 4 : 1;
        const int resident = std::max(1, 16 / (warps * per_block));  // blocks that make 512 threads an SM
        int64_t grid = std::min<int64_t>({(a.rows + per_block - 1) / per_block, static_cast<int64_t>(sms) * resident / blocks, most_writers});
        // a writer's rows start alike: a multiple of 8 apart, where it has more than one
        if (!aligned && grid * per_block < a.rows && grid > 8) grid = grid / 8 * 8;
        grid = std::max<int64_t>(grid, 1);
        writers = grid;
        const dim3 block(32 * warps, per_block);
        info->grid = static_cast<int>(grid * blocks);
        info->block = 32 * warps * per_block;
        if (runs && (aligned || grid * per_block % 8 == 0 || grid * per_block >= a.rows)) {
            auto kernel = aligned ? kt == 1 ? layernorm_grad_ring_kernel<DT, 1, true, false> : layernorm_grad_ring_kernel<DT, 2, true, false>
                                  : kt == 1 ? layernorm_grad_ring_kernel<DT, 1, false, false> : layernorm_grad_ring_kernel<DT, 2, false, false>;
            if (pair) kernel = aligned ? layernorm_grad_ring_kernel<DT, 2, true, true> : layernorm_grad_ring_kernel<DT, 2, false, true>;
            const int row_bytes = 3 * kt * info->block * 8 * ElemOf<DT>::kBytes;  // of a row of each of the block's writers
            const int depth = std::max(2, std::min(4, kRingBytes / (resident * row_bytes)));
            static std::atomic<uint64_t> allowed[2][3];
            e = allow_smem(reinterpret_cast<const void *>(kernel), kRingBytes, &allowed[aligned][pair ? 2 : kt - 1]);
            if (e != cudaSuccess) return e;
            info->smem = depth * row_bytes;
            e = launch_rows(kernel, dim3(grid * blocks), block, depth * row_bytes, blocks, s, a, depth);
        } else {
            info->vec_bytes = ElemOf<DT>::kBytes;
            e = launch_rows(kt == 1 ? layernorm_grad_kernel<DT, 1> : layernorm_grad_kernel<DT, 2>, dim3(grid), block, 0, 1, s, a);
        }
        ++*launches;
    } else if (a.rows > 0) {
        if (sums) {
            const bool vec = aligned && wide_rows<DT>(a.h, a.h_stride);
            writers = std::min<int64_t>({a.rows, most_writers, std::max(1, 8 * sms * 8 / tiles)});
            e = launch_rows(vec ? layernorm_columns_kernel<DT, true> : layernorm_columns_kernel<DT, false>,
                            dim3((tiles + 7) / 8, static_cast<unsigned>(writers)), dim3(256), 0, 1, s, a);
            ++*launches;
        }
        if (e == cudaSuccess)
            e = launch_rows(aligned ? layernorm_grad_wide_kernel<DT, kAligned> : runs ? layernorm_grad_wide_kernel<DT, kShifted>
                                                                               : layernorm_grad_wide_kernel<DT, kApart>,
                            dim3(static_cast<unsigned>(a.rows)), dim3(1024), 0, 1, s, a);
        ++*launches;
        info->grid = static_cast<int>(a.rows);
        info->block = 1024;
    }
    if (e != cudaSuccess || !sums) return e;
    ++*launches;
    return launch_column_sums(a.partial, writers, a.cols, a.dweight, s, true, a.dbias);
}

}  // namespace
}  // namespace ew
