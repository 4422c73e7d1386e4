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
    } else {
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

// base + row * stride elements, in 64 bits
template <int DT> __device__ __forceinline__ const void *row_of(const void *base, int64_t row, int64_t stride) {
    return static_cast<const char *>(base) + row * stride * ElemOf<DT>::kBytes;
}
template <int DT> __device__ __forceinline__ void *row_of(void *base, int64_t row, int64_t stride) {
    return static_cast<char *>(base) + row * stride * ElemOf<DT>::kBytes;
}

// 16-byte accesses (32-byte ones for binary32): the base and the stride of a
// matrix are multiples of 8 elements.  Null matrices allow anything.
template <int DT> inline bool wide_rows(const void *p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % (8 * ElemOf<DT>::kBytes) == 0 && (p == nullptr || stride % 8 == 0);
}

}  // namespace ew
