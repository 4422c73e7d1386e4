// ew_embed.cu -- embedding lookup with scaling, and its gradient by sorted
// tokens.
//
//   out[t,:]    = scale * table[token_t,:]
//   dtable[v,:] = scale * sum over t with token_t == v of dout[t,:]
//
// Both move memory and compute next to nothing.  The gradient sorts the
// positions by token (stable), so that each table row's terms lie in one run,
// in the order of their positions.  Warps take 32 sorted positions by 256
// columns each and add run by run in binary32; a run that ends within the
// chunk goes straight to its table row, one that crosses a chunk's edge leaves
// a partial sum, and embed_join_kernel adds those in order.  The split depends
// on the tokens alone, so the result does too.
#include <algorithm>
#include <atomic>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// ---------------------------------------------------------------- lookup

// A warp takes U consecutive (row, tile of 256 columns) items.
template <int DT, bool VEC, int U> __global__ void __launch_bounds__(256) embed_kernel(EmbedArgs a) {
    enter_grid();
    const int lane = threadIdx.x & 31;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int64_t items = a.rows * tiles;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * U;
    int64_t row = first / tiles;
    int tile = static_cast<int>(first - row * tiles);
    Raw8<DT> r[U];
    int64_t rows[U];
    int bases[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        rows[u] = row;
        bases[u] = tile * kTileCols;
#pragma unroll
        for (int k = 0; k < ElemOf<DT>::kWords; ++k) r[u].w[k] = 0u;
        if (first + u < items) {
            const int64_t v = token_at(a.tokens, a.i64, row);
            if (v >= 0 && v < a.table_rows)
                r[u] = load_tile<DT, VEC>(row_of<DT>(a.table, v, a.table_stride), bases[u], a.cols, lane);
        }
        if (++tile == tiles) { tile = 0; ++row; }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (first + u >= items) break;
        float2 f[4];
        unpack8<DT>(r[u], f);
        const int64_t v = token_at(a.tokens, a.i64, rows[u]);
        // a row of no token is zeros whatever the scale is
        const bool given = v >= 0 && v < a.table_rows;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = given ? mul2(f[j], both(a.scale)) : both(0.0f);
        store_tile<DT, VEC>(row_of<DT>(a.out, rows[u], a.out_stride), bases[u], a.cols, lane, pack8<DT>(f));
    }
}

template <int DT, bool VEC> cudaError_t embed_launch(const EmbedArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int64_t items = a.rows * ((a.cols + kTileCols - 1) / kTileCols);
    // Four items a warp keep 2 KiB (16-bit) in flight each; few items are
    // spread over as many warps as there are.
    const bool many = items >= static_cast<int64_t>(sms) * 64;
    const int64_t per_block = 8 * (many ? 4 : 1);
    const int64_t grid = (items + per_block - 1) / per_block;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    info->grid = static_cast<int>(grid);
    info->block = 256;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    return many ? launch_rows(embed_kernel<DT, VEC, 4>, dim3(grid), dim3(256), 0, 1, s, a)
                : launch_rows(embed_kernel<DT, VEC, 1>, dim3(grid), dim3(256), 0, 1, s, a);
}

template <int DT> cudaError_t embed_dispatch(const EmbedArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return wide_rows<DT>(a.table, a.table_stride) && wide_rows<DT>(a.out, a.out_stride)
               ? embed_launch<DT, true>(a, sms, s, info)
               : embed_launch<DT, false>(a, sms, s, info);
}

// ---------------------------------------------------------------- sort
//
// Stable radix sort of the positions by token, by one cluster of 8 blocks:
// each block takes an eighth of the positions, each of its 32 warps a
// consecutive part of that.  A pass counts its digits per warp in shared
// memory, turns the counts into places by a prefix over (digit, block, warp),
// the other blocks' totals read from their shared memory, and moves the items;
// lanes with equal digits are ranked by a match.  Passes are separated by
// cluster barriers.  Digits have at most 10 bits, so tables of less than 2^20
// rows take two passes.

constexpr int kSortBlocks = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 10;

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(EmbedGradArgs a, int passes, int bits) {
    enter_grid();
    extern __shared__ uint32_t count[];  // [warp][digit]
    __shared__ uint32_t total[1 << kDigitBits];
    __shared__ uint32_t scan[kSortWarps];
    const uint32_t rank = cluster_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bins = 1 << bits;
    uint32_t *mine = count + warp * bins;
    // this warp's consecutive part of the positions
    const int64_t parts = kSortBlocks * kSortWarps, part = rank * kSortWarps + warp;
    const int64_t each = ((a.rows + parts - 1) / parts + 31) / 32 * 32;
    const int64_t begin = min(part * each, a.rows), end = min(begin + each, a.rows);
    const uint32_t nowhere = static_cast<uint32_t>(a.table_rows);  // the key of positions without a token
    if (a.present != nullptr) {
        const int64_t words = (a.table_rows + 31) / 32;
        for (int64_t w = rank * kSortThreads + threadIdx.x; w < words; w += kSortBlocks * kSortThreads) a.present[w] = 0u;
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * bits;
        const uint2 *src = (pass & 1) ? a.items1 : a.items0;  // unused in pass 0
        uint2 *dst = (pass & 1) ? a.items0 : a.items1;
        auto item = [&](int64_t t) {
            if (pass > 0) return __ldcg(src + t);  // written by other blocks: not from L1
            const int64_t v = token_at(a.tokens, a.i64, t);
            return make_uint2(v >= 0 && v < a.table_rows ? static_cast<uint32_t>(v) : nowhere, static_cast<uint32_t>(t));
        };
        for (int k = threadIdx.x; k < kSortWarps * bins; k += kSortThreads) count[k] = 0u;
        __syncthreads();
        for (int64_t t = begin + lane; t < end; t += 32) atomicAdd(mine + ((item(t).x >> shift) & (bins - 1)), 1u);
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < bins) {  // counts become places within the block's digit
            uint32_t sum = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = count[w * bins + threadIdx.x];
                count[w * bins + threadIdx.x] = sum;
                sum += c;
            }
            total[threadIdx.x] = sum;
        }
        cluster_sync();
        uint32_t all = 0, lower = 0;
        if (static_cast<int>(threadIdx.x) < bins) {
#pragma unroll
            for (uint32_t b = 0; b < kSortBlocks; ++b) {
                const uint32_t c = load_of_block(total + threadIdx.x, b);
                all += c;
                lower += b < rank ? c : 0u;
            }
        }
        uint32_t before = all;  // inclusive prefix over the digits of a warp, then of the block
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(kAllLanes, before, d);
            before += lane >= d ? v : 0u;
        }
        if (lane == 31) scan[warp] = before;
        __syncthreads();
        uint32_t warps_before = lane < warp ? scan[lane] : 0u;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) warps_before += __shfl_xor_sync(kAllLanes, warps_before, d);
        const uint32_t base = before - all + warps_before + lower;
        if (static_cast<int>(threadIdx.x) < bins)
            for (int w = 0; w < kSortWarps; ++w) count[w * bins + threadIdx.x] += base;
        __syncthreads();
        for (int64_t t0 = begin; t0 < end; t0 += 32) {
            const bool valid = t0 + lane < end;
            const unsigned active = __ballot_sync(kAllLanes, valid);
            if (valid) {
                const uint2 it = item(t0 + lane);
                const uint32_t digit = (it.x >> shift) & (bins - 1);
                const unsigned same = __match_any_sync(active, digit);
                const uint32_t place = mine[digit] + __popc(same & ((1u << lane) - 1u));
                __syncwarp(active);
                if (lane == __ffs(same) - 1) mine[digit] += __popc(same);
                __syncwarp(active);
                if (pass + 1 < passes) {
                    dst[place] = it;
                } else {
                    a.keys[place] = it.x;
                    a.order[place] = it.y;
                }
                if (pass == 0 && a.present != nullptr && it.x != nowhere)
                    atomicOr(a.present + (it.x >> 5), 1u << (it.x & 31));
            }
        }
        __threadfence();
        cluster_sync();  // the next pass reads what all blocks moved, and reuses `total`
    }
}

// ---------------------------------------------------------------- sums

constexpr int kChunk = 32;  // sorted positions a warp takes, one to a lane

template <int GT, bool VEC>
__device__ __forceinline__ void write_sum(const EmbedGradArgs &a, uint32_t v, int base, int lane, const float2 (&sum)[4]) {
    void *row = row_of<GT>(a.dtable, v, a.table_stride);
    float2 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = mul2(sum[j], both(a.scale));
    if (a.accumulate) {
        float2 old[4];
        unpack8<GT>(load_tile<GT, VEC>(row, base, a.cols, lane), old);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = add2(f[j], old[j]);
    }
    store_tile<GT, VEC>(row, base, a.cols, lane, pack8<GT>(f));
}

// Partial sums: for each chunk its first run where that began before the chunk
// (slot 0), and its last run where it began in the chunk and goes on (slot 1).
// A lane's 8 columns lie together, whatever the matrix's access width.
__device__ __forceinline__ float4 *partial_at(const EmbedGradArgs &a, int64_t chunk, int slot, int tile, int lane) {
    const int64_t tiles = (a.cols + kTileCols - 1) / kTileCols;
    return reinterpret_cast<float4 *>(a.partial) + (((chunk * 2 + slot) * tiles + tile) * 32 + lane) * 2;
}

template <int DT, int GT, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(EmbedGradArgs a, int64_t sum_blocks) {
    enter_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    if (static_cast<int64_t>(blockIdx.x) >= sum_blocks) {  // rows that no token names become zero
        const int64_t w = (static_cast<int64_t>(blockIdx.x) - sum_blocks) * 8 + warp;
        if (w * 32 >= a.table_rows) return;
        uint32_t absent = ~a.present[w];
        if (a.table_rows - w * 32 < 32) absent &= (1u << (a.table_rows - w * 32)) - 1u;
        Raw8<GT> zero;
#pragma unroll
        for (int k = 0; k < ElemOf<GT>::kWords; ++k) zero.w[k] = 0u;
        while (absent) {
            const int64_t v = w * 32 + __ffs(absent) - 1;
            absent &= absent - 1;
            void *row = row_of<GT>(a.dtable, v, a.table_stride);
#pragma unroll 4
            for (int t = 0; t < tiles; ++t) store_tile<GT, VEC>(row, t * kTileCols, a.cols, lane, zero);
        }
        return;
    }
    const int64_t chunks = (a.rows + kChunk - 1) / kChunk;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    const int64_t chunk = item / tiles;
    const int tile = static_cast<int>(item - chunk * tiles), base = tile * kTileCols;
    if (chunk >= chunks) return;
    const uint32_t nowhere = static_cast<uint32_t>(a.table_rows);
    const int64_t at = chunk * kChunk + lane;
    const uint32_t key = at < a.rows ? a.keys[at] : nowhere;
    const uint32_t pos = at < a.rows ? a.order[at] : 0u;
    const uint32_t key_before = chunk > 0 ? a.keys[chunk * kChunk - 1] : nowhere;
    const uint32_t key_after = (chunk + 1) * kChunk < a.rows ? a.keys[(chunk + 1) * kChunk] : nowhere;
    const int count = __popc(__ballot_sync(kAllLanes, key != nowhere));  // positions without a token come last
    if (count == 0) return;

    float2 sum[4] = {};
    uint32_t current = __shfl_sync(kAllLanes, key, 0);
    bool from_before = chunk > 0 && key_before == current;
    auto put = [&](bool goes_on) {
        if (!from_before && !goes_on) {
            write_sum<GT, VEC>(a, current, base, lane, sum);
        } else {
            float4 *p = partial_at(a, chunk, from_before ? 0 : 1, tile, lane);
            p[0] = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
            p[1] = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
        }
    };
    constexpr int U = 8;  // rows in flight
    for (int i0 = 0; i0 < count; i0 += U) {
        Raw8<DT> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t t = __shfl_sync(kAllLanes, pos, i0 + u);
            if (i0 + u < count) r[u] = load_tile<DT, VEC>(row_of<DT>(a.dout, t, a.dout_stride), base, a.cols, lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = __shfl_sync(kAllLanes, key, i0 + u);
            if (i0 + u >= count) break;
            if (k != current) {
                put(false);
                current = k;
                from_before = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = both(0.0f);
            }
            float2 f[4];
            unpack8<DT>(r[u], f);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], f[j]);
        }
    }
    put(count == kChunk && key_after == current);
}

// Runs that cross chunks: the block of the chunk where a run begins adds its
// slot 1 and the slots 0 of the chunks after it, its 8 warps every eighth.
template <int GT, bool VEC> __global__ void __launch_bounds__(256) embed_join_kernel(EmbedGradArgs a) {
    enter_grid();
    __shared__ float2 part[8][4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = blockIdx.y, base = tile * kTileCols;
    const int64_t chunk = blockIdx.x, chunks = (a.rows + kChunk - 1) / kChunk;
    const int64_t last = chunk * kChunk + kChunk - 1;
    if (last + 1 >= a.rows) return;
    const uint32_t v = a.keys[last];
    if (v == static_cast<uint32_t>(a.table_rows) || a.keys[last + 1] != v) return;  // no run goes on from here
    if (chunk > 0 && a.keys[chunk * kChunk - 1] == v) return;                       // or it began earlier
    // chunks after this one that the run reaches: heads[chunk + 1 .. chunk + reach] == v
    int64_t reach = 0;
    while (true) {
        const int64_t c = chunk + 1 + reach + lane;
        const unsigned in = __ballot_sync(kAllLanes, c < chunks && a.keys[c * kChunk] == v);
        reach += in == kAllLanes ? 32 : __ffs(~in) - 1;
        if (in != kAllLanes) break;
    }
    float2 sum[4] = {};
    auto add = [&](int64_t c, int slot) {
        const float4 *p = partial_at(a, c, slot, tile, lane);
        const float4 x = p[0], y = p[1];
        sum[0] = add2(sum[0], make_float2(x.x, x.y));
        sum[1] = add2(sum[1], make_float2(x.z, x.w));
        sum[2] = add2(sum[2], make_float2(y.x, y.y));
        sum[3] = add2(sum[3], make_float2(y.z, y.w));
    };
    if (warp == 0) add(chunk, 1);
#pragma unroll 4
    for (int64_t k = warp; k < reach; k += 8) add(chunk + 1 + k, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][j][lane] = sum[j];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], part[w][j][lane]);
    write_sum<GT, VEC>(a, v, base, lane, sum);
}

template <int DT, int GT, bool VEC>
cudaError_t embed_grad_launch(const EmbedGradArgs &a, cudaStream_t s, LaunchInfo *info, int *launches) {
    const int64_t tiles = (a.cols + kTileCols - 1) / kTileCols, chunks = (a.rows + kChunk - 1) / kChunk;
    const int64_t sums = (chunks * tiles + 7) / 8;
    const int64_t fills = a.accumulate ? 0 : (a.table_rows + 255) / 256;
    if (sums + fills > INT32_MAX || tiles > 65535) return cudaErrorInvalidConfiguration;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    info->grid = static_cast<int>(sums + fills);
    info->block = 256;
    cudaError_t e = cudaSuccess;
    if (sums + fills > 0) {
        e = launch_rows(embed_sum_kernel<DT, GT, VEC>, dim3(sums + fills), dim3(256), 0, 1, s, a, sums);
        ++*launches;
    }
    if (e != cudaSuccess || chunks < 2) return e;
    ++*launches;
    return launch_rows(embed_join_kernel<GT, VEC>, dim3(chunks, tiles), dim3(256), 0, 1, s, a);
}

template <int DT, int GT>
cudaError_t embed_grad_dispatch(const EmbedGradArgs &a, cudaStream_t s, LaunchInfo *info, int *launches) {
    return wide_rows<DT>(a.dout, a.dout_stride) && wide_rows<GT>(a.dtable, a.table_stride)
               ? embed_grad_launch<DT, GT, true>(a, s, info, launches)
               : embed_grad_launch<DT, GT, false>(a, s, info, launches);
}

}  // namespace

cudaError_t launch_embed(int dtype, const EmbedArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return dtype == DT_F32   ? embed_dispatch<DT_F32>(a, sms, s, info)
           : dtype == DT_F16 ? embed_dispatch<DT_F16>(a, sms, s, info)
                             : embed_dispatch<DT_BF16>(a, sms, s, info);
}

int64_t embed_partial_bytes(int64_t rows, int64_t cols) {
    return (rows + kChunk - 1) / kChunk * 2 * ((cols + kTileCols - 1) / kTileCols) * kTileCols * 4;
}

cudaError_t launch_embed_grad(int dtype, int gtype, const EmbedGradArgs &a, cudaStream_t s, LaunchInfo *info,
                              int *launches) {
    int width = 0;  // bits of a key: 0 .. table_rows
    while (width < 32 && (static_cast<uint64_t>(a.table_rows) >> width) != 0) ++width;
    const int passes = std::max(1, (width + kDigitBits - 1) / kDigitBits);
    const int bits = std::max(1, (width + passes - 1) / passes);
    const size_t smem = size_t(kSortWarps) * 4 << bits;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(embed_sort_kernel), (kSortWarps * 4) << kDigitBits, &allowed);
    if (e == cudaSuccess)
        e = launch_rows(embed_sort_kernel, dim3(kSortBlocks), dim3(kSortThreads), smem, kSortBlocks, s, a, passes, bits);
    if (e != cudaSuccess) return e;
    ++*launches;
    info->smem = static_cast<int>(smem);
    if (dtype == DT_F32) return embed_grad_dispatch<DT_F32, DT_F32>(a, s, info, launches);
    if (dtype == DT_F16)
        return gtype == DT_F32 ? embed_grad_dispatch<DT_F16, DT_F32>(a, s, info, launches)
                               : embed_grad_dispatch<DT_F16, DT_F16>(a, s, info, launches);
    return gtype == DT_F32 ? embed_grad_dispatch<DT_BF16, DT_F32>(a, s, info, launches)
                           : embed_grad_dispatch<DT_BF16, DT_BF16>(a, s, info, launches);
}

}  // namespace ew
