// ew_rows.cuh -- device-side building blocks of the row operators: 8-element
// tiles of a row in registers, reductions over warps and blocks.
//
// A warp takes 256 consecutive columns of a row at a time, 8 of them per lane:
// lane l holds columns 8l .. 8l+7 (one 16-byte access for 16-bit elements, one
// 32-byte access for binary32) where the row starts on such a boundary, and
// columns l, l+32, .., l+224 (eight coalesced single-element accesses) where it
// does not.  Both hold the same 256 columns, so a group of up to 256 columns
// that starts at a multiple of its size always lies within one warp.
#pragma once

#include <type_traits>

#include "ew_device.cuh"
#include "ew_internal.h"

namespace ew {

constexpr int kTileCols = 256;  // columns a warp holds at a time
constexpr unsigned kAllLanes = 0xffffffffu;

template <int DT> struct ElemOf { using type = uint16_t; static constexpr int kBytes = 2, kWords = 4; };
template <> struct ElemOf<DT_F32> { using type = uint32_t; static constexpr int kBytes = 4, kWords = 8; };

template <int DT> __device__ __forceinline__ float elem_to_f32(typename ElemOf<DT>::type v) {
    if constexpr (DT == DT_F32) return __uint_as_float(v);
    else if constexpr (DT == DT_F16) return f16_to_f32(v);
    else return bf16_to_f32(v);
}
template <int DT> __device__ __forceinline__ typename ElemOf<DT>::type f32_to_elem(float f) {
    if constexpr (DT == DT_F32) return __float_as_uint(f);
    else if constexpr (DT == DT_F16) return f32_to_f16(f);
    else return f32_to_bf16(f);
}

// Two binary32 values in one instruction each (the sm_100 family's f32x2 forms).
__device__ __forceinline__ uint64_t pair_bits(float2 a) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a.x), "f"(a.y));
    return d;
}
__device__ __forceinline__ float2 pair_of(uint64_t d) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
    return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
    return pair_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
    return pair_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
    return pair_of(d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// The two 16-bit elements of a word, and back, rounded.
template <int DT> __device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (DT == DT_F16)
        return make_float2(f16_to_f32(static_cast<uint16_t>(w)), f16_to_f32(static_cast<uint16_t>(w >> 16)));
    else
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int DT> __device__ __forceinline__ uint32_t narrow(float2 a) {
    if constexpr (DT == DT_F16) return f32x2_to_f16x2(a.y, a.x);
    else return f32x2_to_bf16x2(a.y, a.x);
}

// 8 elements as they lie in memory (16-bit elements two to a word).
template <int DT> struct Raw8 { uint32_t w[ElemOf<DT>::kWords]; };

// The same as 4 pairs.
template <int DT> __device__ __forceinline__ void unpack8(const Raw8<DT> &r, float2 (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == DT_F32) f[j] = make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
        else f[j] = widen<DT>(r.w[j]);
    }
}
template <int DT> __device__ __forceinline__ Raw8<DT> pack8(const float2 (&f)[4]) {
    Raw8<DT> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == DT_F32) {
            r.w[2 * j] = __float_as_uint(f[j].x);
            r.w[2 * j + 1] = __float_as_uint(f[j].y);
        } else {
            r.w[j] = narrow<DT>(f[j]);
        }
    }
    return r;
}

// Column of element j of this lane in the tile that starts at column `base`.
template <bool VEC> __device__ __forceinline__ int tile_col(int base, int lane, int j) {
    return VEC ? base + lane * 8 + j : base + j * 32 + lane;
}

// The lane's 8 elements of the tile at `base`; columns from `cols` on are zero.
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load_tile(const void *row, int base, int cols, int lane) {
    using T = typename ElemOf<DT>::type;
    const T *p = static_cast<const T *>(row);
    Raw8<DT> r;
    const int c0 = tile_col<VEC>(base, lane, 0);
    if (VEC && c0 + 8 <= cols) {
        const Vec<8 * ElemOf<DT>::kBytes> v = ld<8 * ElemOf<DT>::kBytes>(p + c0);
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) r.w[k] = v.w[k];
    } else {
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) r.w[k] = 0u;
        // A lane without a column.  Not of binary32, where four tiles a thread would then be
        // waited for one by one (4096 rows of 12288: layer norm 192 us, 130 without), nor of
        // single elements, for the same reason (the norm's backward of 33520 x 1001 bf16 79 us
        // and 66).
        if (VEC && DT != DT_F32 && c0 >= cols) return r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tile_col<VEC>(base, lane, j);
            if (c < cols) {
                if constexpr (DT == DT_F32) r.w[j] = ld<4>(p + c).w[0];
                else r.w[j / 2] |= static_cast<uint32_t>(ld<2>(p + c).h) << (16 * (j & 1));
            }
        }
    }
    return r;
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_tile(void *row, int base, int cols, int lane, const Raw8<DT> &r) {
    using T = typename ElemOf<DT>::type;
    T *p = static_cast<T *>(row);
    const int c0 = tile_col<VEC>(base, lane, 0);
    if (VEC && c0 + 8 <= cols) {
        Vec<8 * ElemOf<DT>::kBytes> v;
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) v.w[k] = r.w[k];
        st<8 * ElemOf<DT>::kBytes>(p + c0, v);
    } else if (!VEC || c0 < cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tile_col<VEC>(base, lane, j);
            if (c < cols) {
                if constexpr (DT == DT_F32) { Vec<4> v; v.w[0] = r.w[j]; st<4>(p + c, v); }
                else { Vec<2> v; v.h = static_cast<uint16_t>(r.w[j / 2] >> (16 * (j & 1))); st<2>(p + c, v); }
            }
        }
    }
}

// The same 8 columns of a vector that every row reads again (cached in L1), in
// binary32; its type is the matrix's or binary32, one for the whole launch.
// Null stands for ones; columns from `cols` on are zero.
template <int DT, bool VEC>
__device__ __forceinline__ void load_weight(const void *w, bool f32, int base, int cols, int lane, float2 (&f)[4]) {
    const int c0 = tile_col<VEC>(base, lane, 0);
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = both(1.0f);
    } else if (VEC && c0 + 8 <= cols) {
        if (DT == DT_F32 || f32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c0);
            const float4 a = q[0], b = q[1];
            f[0] = make_float2(a.x, a.y);
            f[1] = make_float2(a.z, a.w);
            f[2] = make_float2(b.x, b.y);
            f[3] = make_float2(b.z, b.w);
        } else if constexpr (DT != DT_F32) {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + c0);
            f[0] = widen<DT>(a.x);
            f[1] = widen<DT>(a.y);
            f[2] = widen<DT>(a.z);
            f[3] = widen<DT>(a.w);
        }
    } else {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tile_col<VEC>(base, lane, j);
            e[j] = 0.0f;
            if (c < cols) {
                if (DT == DT_F32 || f32) e[j] = static_cast<const float *>(w)[c];
                else e[j] = elem_to_f32<DT>(static_cast<const typename ElemOf<DT>::type *>(w)[c]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = make_float2(e[2 * j], e[2 * j + 1]);
    }
}

// ---------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAllLanes, v, d);
    return v;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float largest_of(const float2 (&y)[4]) {  // by absolute value
    const float m = max_nan(fabsf(y[0].x), fabsf(y[0].y), fabsf(y[1].x));
    const float n = max_nan(fabsf(y[1].y), fabsf(y[2].x), fabsf(y[2].y));
    return max_nan(max_nan(m, fabsf(y[3].x), fabsf(y[3].y)), n);
}
// Largest over the `width` lanes (a power of two) around this one.
__device__ __forceinline__ float lanes_max_nan(float v, int width) {
    for (int d = width >> 1; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(kAllLanes, v, d));
    return v;
}

// Sum over a block of `warps` warps, to every thread; `part` has a slot per
// warp and is free again when the call after the next __syncthreads begins.
// The order of the additions is fixed.
__device__ __forceinline__ float block_sum(float v, int warps, float *part) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}
__device__ __forceinline__ float block_max_nan(float v, int warps, float *part, float least = 0.0f) {
    v = lanes_max_nan(v, 32);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return lanes_max_nan(lane < warps ? part[lane] : least, 32);
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of a shared variable of this block as block `rank` of the cluster has it.
template <typename T> __device__ __forceinline__ const T *in_block(const T *mine, uint32_t rank) {
    uint64_t at;
    asm("mapa.u64 %0, %1, %2;" : "=l"(at) : "l"(reinterpret_cast<uint64_t>(mine)), "r"(rank));
    return reinterpret_cast<const T *>(at);
}

__device__ __forceinline__ int64_t token_at(const void *tokens, bool i64, int64_t t) {
    return i64 ? static_cast<const int64_t *>(tokens)[t] : static_cast<const int32_t *>(tokens)[t];
}

// Waits until at most LEFT of this thread's latest groups of asynchronous copies are under way.
template <int LEFT> __device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

// base + row * stride elements, in 64 bits
template <int DT> __device__ __forceinline__ const void *row_of(const void *base, int64_t row, int64_t stride) {
    return static_cast<const char *>(base) + row * stride * ElemOf<DT>::kBytes;
}
template <int DT> __device__ __forceinline__ void *row_of(void *base, int64_t row, int64_t stride) {
    return static_cast<char *>(base) + row * stride * ElemOf<DT>::kBytes;
}

// ---------------------------------------------------------------- runs of 8 elements
//
// Rows that start anywhere, in runs of 8 elements that start at multiples of 8
// in memory: the first begins `past` elements before the row.  Nothing outside
// the row is written.  Reading, a run at a row's end may bring elements of the
// rows beside it along, whatever they hold, so that all lanes load alike: loads of
// single elements in a branch are waited for there, one matrix after another.

// Elements of a row's first run that lie before the row.
template <int DT> __host__ __device__ __forceinline__ int past_of(const void *row) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(row) % (8 * ElemOf<DT>::kBytes)) / ElemOf<DT>::kBytes;
}
// Column of element j of this lane in tile `tile` of a row.
template <bool RUNS> __device__ __forceinline__ int col_of(int tile, int past, int lane, int j) {
    return RUNS ? tile * kTileCols - past + lane * 8 + j : tile * kTileCols + j * 32 + lane;
}
// Elements c0 .. c0 + 7 one by one, zero outside the row: for a matrix's first and
// last rows, and so in few registers rather than fast.
template <int DT> __device__ __forceinline__ Raw8<DT> load_single(const void *row, int c0, int cols) {
    constexpr int B = ElemOf<DT>::kBytes;
    const auto *p = static_cast<const typename ElemOf<DT>::type *>(row);
    Raw8<DT> r;
#pragma unroll
    for (int k = 0; k < ElemOf<DT>::kWords; ++k) r.w[k] = 0u;
#pragma unroll 1
    for (int j = max(-c0, 0); j < min(cols - c0, 8); ++j) {
        const uint32_t v = static_cast<uint32_t>(p[c0 + j]) << (j * B % 4 * 8);
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) r.w[k] |= j * B / 4 == k ? v : 0u;
    }
    return r;
}
// The lane's run.  `inner`: the 7 elements before the row and after it may be
// read; otherwise, and in lanes without a column of the row, those outside are zero.
template <int DT> __device__ __forceinline__ Raw8<DT> load_run(const void *row, int tile, int past, int cols, int lane, bool inner) {
    const int c0 = col_of<true>(tile, past, lane, 0);
    if (inner ? c0 > -8 && c0 < cols : c0 >= 0 && c0 + 8 <= cols) {
        const Vec<8 * ElemOf<DT>::kBytes> v = ld<8 * ElemOf<DT>::kBytes>(static_cast<const typename ElemOf<DT>::type *>(row) + c0);
        Raw8<DT> r;
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) r.w[k] = v.w[k];
        return r;
    }
    return load_single<DT>(row, c0, cols);
}
// Elements `from` to 7 of a run, or 0 to `to` - 1, where the row begins or ends in
// it: one, two and four at a time, as they are aligned.
template <int DT> __device__ __forceinline__ void store_part(typename ElemOf<DT>::type *run, const Raw8<DT> &r, int from, int to) {
    constexpr int B = ElemOf<DT>::kBytes;
    auto put = [&](int at, auto n) {  // elements at .. at + n - 1, `at` a multiple of n
        constexpr int N = decltype(n)::value, W = N * B / 4;
        if constexpr (W == 0) {
            const uint32_t w = at & 4 ? (at & 2 ? r.w[3] : r.w[2]) : (at & 2 ? r.w[1] : r.w[0]);
            run[at] = static_cast<typename ElemOf<DT>::type>(at & 1 ? w >> 16 : w);
        } else {
            Vec<N * B> v;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v.w[i] = r.w[i];
#pragma unroll
                for (int k = 1; k < 8 / N; ++k)
                    if (at == k * N) v.w[i] = r.w[k * W + i];
            }
            st<N * B>(run + at, v);
        }
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    if (to == 8) {
        if (from & 1) put(from, One());
        from += from & 1;
        if (from & 2) put(from, Two());
        from += from & 2;
        if (from & 4) put(4, Four());
    } else {
        if (to & 4) put(0, Four());
        if (to & 2) put(to & 4, Two());
        if (to & 1) put(to & 6, One());
    }
}
template <int DT> __device__ __forceinline__ void store_run(void *row, int tile, int past, int cols, int lane, const Raw8<DT> &r) {
    using T = typename ElemOf<DT>::type;
    const int c0 = col_of<true>(tile, past, lane, 0);
    T *p = static_cast<T *>(row) + c0;
    if (c0 >= 0 && c0 + 8 <= cols) {
        Vec<8 * ElemOf<DT>::kBytes> v;
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) v.w[k] = r.w[k];
        st<8 * ElemOf<DT>::kBytes>(p, v);
    } else if (c0 > -8 && c0 < cols) {
        if (c0 >= 0 || c0 + 8 <= cols) {
            store_part<DT>(p, r, max(-c0, 0), min(cols - c0, 8));
        } else {  // a row within one run
#pragma unroll 1
            for (int j = -c0; j < cols - c0; ++j) {
                uint32_t w = 0;
#pragma unroll
                for (int k = 0; k < ElemOf<DT>::kWords; ++k) w |= j * ElemOf<DT>::kBytes / 4 == k ? r.w[k] : 0u;
                p[j] = static_cast<T>(w >> (j * ElemOf<DT>::kBytes % 4 * 8));
            }
        }
    }
}

// The 8 elements from column c0 on, wherever they start, cut out of the 16-byte
// pieces around them, which may reach up to 7 elements out of the run.
template <int DT> __device__ __forceinline__ Raw8<DT> cut_run(const void *row, int c0) {
    constexpr int B = ElemOf<DT>::kBytes, W = ElemOf<DT>::kWords;
    const char *at = static_cast<const char *>(row) + static_cast<int64_t>(c0) * B;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    const uint4 *q = reinterpret_cast<const uint4 *>(at - shift);
    uint32_t v[W + 4] = {};
#pragma unroll
    for (int k = 0; k < W / 4 + 1; ++k)
        if (k < W / 4 || shift != 0) {
            const uint4 a = q[k];
            v[4 * k] = a.x, v[4 * k + 1] = a.y, v[4 * k + 2] = a.z, v[4 * k + 3] = a.w;
        }
#pragma unroll
    for (int j = 0; j < W + 2; ++j) v[j] = shift & 8 ? v[j + 2] : v[j];
#pragma unroll
    for (int j = 0; j < W + 1; ++j) v[j] = shift & 4 ? v[j + 1] : v[j];
    Raw8<DT> r;
#pragma unroll
    for (int j = 0; j < W; ++j) r.w[j] = B == 4 ? v[j] : __funnelshift_r(v[j], v[j + 1], (shift & 3) * 8);
    return r;
}
// Zeros in columns outside the row.
template <bool RUNS> __device__ __forceinline__ void clip_columns(int tile, int past, int cols, int lane, float2 (&f)[4]) {
    const int first = tile * kTileCols - (RUNS ? past : 0);
    if (first >= 0 && first + kTileCols <= cols) return;
    if constexpr (RUNS) {
        const int c0 = col_of<true>(tile, past, lane, 0);
        if (past == 0 && cols % 8 == 0) {  // whole lanes: 16384 rows of 4000 bf16 82 us, element by element 93
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = c0 < cols ? f[j] : both(0.0f);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int a = col_of<RUNS>(tile, past, lane, 2 * j), b = col_of<RUNS>(tile, past, lane, 2 * j + 1);
        if (a < 0 || a >= cols) f[j].x = 0.0f;
        if (b < 0 || b >= cols) f[j].y = 0.0f;
    }
}

// ---------------------------------------------------------------- pairs
//
// Rows that lie apart, by what lies at multiples of 4 bytes in the row that is
// written: lane l of a warp has the pairs of 16-bit elements l, l + 32, .. of its
// 256 columns, the first pair of a row beginning `odd` elements (0 or 1) before it;
// of binary32 the elements l, l + 32, ...  A row that is read may lie half a word
// off: then its elements are read one by one, and put together when they are needed,
// so that loads of several rows are under way together.
template <int DT> __host__ __device__ __forceinline__ int odd_of(const void *row) {
    return DT == DT_F32 ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 1);
}
template <int DT> struct Pairs8 {
    uint32_t a[8];  // words, then what belongs into their upper halves; of binary32 elements
    __device__ __forceinline__ Raw8<DT> whole() const {
        Raw8<DT> r;
#pragma unroll
        for (int j = 0; j < ElemOf<DT>::kWords; ++j) r.w[j] = DT == DT_F32 ? a[j] : a[j] | a[(j + 4) & 7] << 16;
        return r;
    }
};
template <int DT> __device__ __forceinline__ Pairs8<DT> load_pairs(const void *row, int tile, int odd, int cols, int lane) {
    Pairs8<DT> r;
    const int first = tile * kTileCols - odd;
    if constexpr (DT == DT_F32) {
        const uint32_t *p = static_cast<const uint32_t *>(row) + first + lane;
        if (first + kTileCols <= cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.a[j] = p[j * 32];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.a[j] = first + j * 32 + lane < cols ? p[j * 32] : 0u;
        }
    } else {
        const int c0 = first + 2 * lane;
        const uint16_t *p = static_cast<const uint16_t *>(row) + c0;
        const bool words = (reinterpret_cast<uintptr_t>(p) & 3) == 0;
        if (words && first >= 0 && first + kTileCols <= cols) {
#pragma unroll
            for (int j = 0; j < 4; ++j) r.a[j] = *reinterpret_cast<const uint32_t *>(p + j * 64);
#pragma unroll
            for (int j = 4; j < 8; ++j) r.a[j] = 0u;
        } else if (first >= 0 && first + kTileCols <= cols) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r.a[j] = p[j * 64];
                r.a[j + 4] = p[j * 64 + 1];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + j * 64;
                r.a[j] = c >= 0 && c < cols ? p[j * 64] : 0u;
                r.a[j + 4] = c + 1 < cols ? p[j * 64 + 1] : 0u;
            }
        }
    }
    return r;
}
template <int DT> __device__ __forceinline__ void store_pairs(void *row, int tile, int odd, int cols, int lane, const Raw8<DT> &r) {
    const int first = tile * kTileCols - odd;
    const bool whole = first >= 0 && first + kTileCols <= cols;
    if constexpr (DT == DT_F32) {
        uint32_t *p = static_cast<uint32_t *>(row) + first + lane;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (whole || first + j * 32 + lane < cols) p[j * 32] = r.w[j];
    } else {
        const int c0 = first + 2 * lane;
        uint16_t *p = static_cast<uint16_t *>(row) + c0;
        if (whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t *>(p + j * 64) = r.w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + j * 64;
                if (c >= 0 && c < cols) p[j * 64] = static_cast<uint16_t>(r.w[j]);
                if (c + 1 < cols) p[j * 64 + 1] = static_cast<uint16_t>(r.w[j] >> 16);
            }
        }
    }
}

// One row of zeros, by a warp: whole runs of 8 elements wherever the row starts,
// and the elements before the first and after the last of them.
template <int GT> __device__ __forceinline__ void clear_row(void *row, int cols, int lane) {
    using T = typename ElemOf<GT>::type;
    constexpr int B = ElemOf<GT>::kBytes;
    T *p = static_cast<T *>(row);
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(row) % (8 * B)) / B;
    const int head = min((8 - past) % 8, cols), runs = (cols - head) / 8;
    const Vec<8 * B> zero = {};
#pragma unroll 4
    for (int k = lane; k < runs; k += 32) st<8 * B>(p + head + k * 8, zero);
    if (lane < head) p[lane] = 0;
    if (head + runs * 8 + lane < cols) p[head + runs * 8 + lane] = 0;
}

// ---------------------------------------------------------------- sorts

// Inclusive prefix sum over the block's threads; `scan` has a slot a warp.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t *scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(kAllLanes, v, d);
        v += lane >= d ? u : 0u;
    }
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    uint32_t before = lane < warp ? scan[lane] : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(kAllLanes, before, d);
    return v + before;
}

// The lanes of `active` whose digit is this lane's: a ballot for each bit.  (A
// match instruction takes about 64 cycles of the SM for 32 different digits,
// ten ballots a quarter of that.)
__device__ __forceinline__ unsigned lanes_alike(uint32_t digit, int bits, unsigned active) {
    unsigned same = active;
#pragma unroll 2
    for (int b = 0; b < bits; ++b) {
        const bool one = digit >> b & 1;
        const unsigned ones = __ballot_sync(kAllLanes, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// ---------------------------------------------------------------- host

// 16-byte accesses (32-byte ones for binary32): the base and the stride of a
// matrix are multiples of 8 elements.  Null matrices allow anything.
template <int DT> inline bool wide_rows(const void *p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % (8 * ElemOf<DT>::kBytes) == 0 && (p == nullptr || stride % 8 == 0);
}
template <int DT> inline bool wide_weight(const void *w, bool f32) {
    return reinterpret_cast<uintptr_t>(w) % (f32 || DT == DT_F32 ? 32 : 16) == 0;
}

// Smallest number of tiles a thread (1, 2 or 4) with which `warps` warps hold a
// row of `tiles` tiles; 0 where none does.
inline int tiles_per_thread(int tiles, int warps, int most) {
    for (int kt = 1; kt <= most; kt *= 2)
        if ((tiles + kt - 1) / kt <= warps) return kt;
    return 0;
}

}  // namespace ew
