// ew_embed.cu -- embedding lookup with scaling, and its gradient by sorted
// tokens.
//
//   out[t,:]    = scale * table[token_t,:]
//   dtable[v,:] = scale * sum over t with token_t == v of dout[t,:]
//
// Both move memory and compute next to nothing.  The gradient sorts the
// positions by token (stable), so that each table row's terms lie in one run,
// in the order of their positions.  Warps take 32 (or 8) sorted positions by 256
// columns each and add run by run in binary32; a run that ends within the
// chunk goes straight to its table row, one that crosses a chunk's edge leaves
// a partial sum, and embed_join_kernel adds those in order.  The split depends
// on the tokens alone, so the result does too.  The gradient's bound is memory:
// 131072 rows of 2048 bf16 from 16384 tokens take 103 us (5.9 TB/s, floor 89);
// small ones the latency of three kernels, 9 to 20 us.
#include <algorithm>
#include <atomic>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// ---------------------------------------------------------------- lookup

// A warp takes U consecutive (row, tile of 256 columns) items.  The bound is
// memory: 16384 tokens of 4096 bf16 columns take 42 us (6.4 TB/s, floor 40), 64
// tokens 1.4 us.
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
// cluster barriers, which order the blocks' global stores too.  Digits have at
// most 10 bits, so tables of less than 2^20 rows take two passes.
//
// The other SMs meanwhile write zeros: the grid's further blocks clear the
// first `blind` rows of the table, which at the end of the sort need not be
// looked at again (a row that a token names is written once more, by its sum).

constexpr int kSortBlocks = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 10;

constexpr int kKept = 4;  // items a lane keeps between counting and moving them

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

template <int GT> __device__ __forceinline__ void clear_blind(const EmbedGradArgs &a, int sort_blocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t v = (static_cast<int64_t>(blockIdx.x) - sort_blocks) * kSortWarps + warp; v < a.blind;
         v += static_cast<int64_t>(gridDim.x - sort_blocks) * kSortWarps)
        clear_row<GT>(row_of<GT>(a.dtable, v, a.table_stride), a.cols, lane);
}

template <int GT>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(EmbedGradArgs a, int passes, int bits) {
    enter_grid();
    extern __shared__ uint32_t count[];  // [warp][digit]
    __shared__ uint32_t total[1 << kDigitBits], first_place[1 << kDigitBits];
    __shared__ uint32_t scan[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= kSortBlocks) {
        clear_blind<GT>(a, kSortBlocks);
        return;
    }
    const uint32_t rank = blockIdx.x;
    const int bins = 1 << bits;
    uint32_t *mine = count + warp * bins;
    // this warp's consecutive part of the positions
    const int64_t parts = kSortBlocks * kSortWarps, part = rank * kSortWarps + warp;
    const int64_t each = ((a.rows + parts - 1) / parts + 31) / 32 * 32;
    const int64_t begin = min(part * each, a.rows), end = min(begin + each, a.rows);
    const bool keep = each <= 32 * kKept;
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
        auto digit_of = [&](uint2 it) { return (it.x >> shift) & (bins - 1); };
        uint2 kept[kKept];
        if (keep) {
#pragma unroll
            for (int k = 0; k < kKept; ++k)
                if (begin + k * 32 + lane < end) kept[k] = item(begin + k * 32 + lane);
        }
        for (int k = threadIdx.x; k < kSortWarps * bins; k += kSortThreads) count[k] = 0u;
        __syncthreads();
        if (keep) {
#pragma unroll
            for (int k = 0; k < kKept; ++k)
                if (begin + k * 32 + lane < end) atomicAdd(mine + digit_of(kept[k]), 1u);
        } else {
            for (int64_t t = begin + lane; t < end; t += 32) atomicAdd(mine + digit_of(item(t)), 1u);
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < bins) {  // counts become places within the block's digit
            uint32_t c[kSortWarps], sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = count[w * bins + threadIdx.x];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                count[w * bins + threadIdx.x] = sum;
                sum += c[w];
            }
            total[threadIdx.x] = sum;
        }
        cluster_sync();
        uint32_t all = 0, lower = 0;
        if (static_cast<int>(threadIdx.x) < bins) {
            uint32_t c[kSortBlocks];
#pragma unroll
            for (uint32_t b = 0; b < kSortBlocks; ++b) c[b] = *in_block(total + threadIdx.x, b);
#pragma unroll
            for (uint32_t b = 0; b < kSortBlocks; ++b) {
                all += c[b];
                lower += b < rank ? c[b] : 0u;
            }
        }
        const uint32_t upto = block_prefix(all, scan);
        if (static_cast<int>(threadIdx.x) < bins) first_place[threadIdx.x] = upto - all + lower;
        __syncthreads();
        auto move = [&](uint2 it, bool valid) {  // the valid lanes' items, in the order of their lanes
            const unsigned active = __ballot_sync(kAllLanes, valid);
            const uint32_t digit = digit_of(it);
            const unsigned same = lanes_alike(digit, bits, active);
            const uint32_t in_digit = mine[digit];
            __syncwarp();
            if (valid) {
                if (lane == __ffs(same) - 1) mine[digit] = in_digit + __popc(same);
                const uint32_t place = first_place[digit] + in_digit + __popc(same & ((1u << lane) - 1u));
                if (pass + 1 < passes) {
                    dst[place] = it;
                } else {
                    a.keys[place] = it.x;
                    a.order[place] = it.y;
                }
                if (pass == 0 && a.present != nullptr && it.x != nowhere) atomicOr(a.present + (it.x >> 5), 1u << (it.x & 31));
            }
            __syncwarp();
        };
        if (keep) {
#pragma unroll
            for (int k = 0; k < kKept; ++k)
                if (begin + k * 32 < end) move(kept[k], begin + k * 32 + lane < end);
        } else {
            for (int64_t t0 = begin; t0 < end; t0 += 32) {
                const bool valid = t0 + lane < end;
                move(valid ? item(t0 + lane) : make_uint2(0u, 0u), valid);
            }
        }
        cluster_sync();  // the next pass reads what all blocks moved, and reuses `total`
    }
}

// Few positions: a bitonic sort of (token, position) by one block, one to a
// thread.  Steps within a warp exchange by shuffles, wider ones through shared
// memory with a barrier each.  The pairs differ, so the order is that of a
// stable sort.  The whole gradient of 4296 rows from 22 positions takes 8.7 us, of
// 5656 rows from 443 positions 12.4 us; with the cluster's sort 13.4 us each.
constexpr int kFew = 512;
template <int GT> __global__ void __launch_bounds__(kSortThreads) embed_sort_few_kernel(EmbedGradArgs a) {
    enter_grid();
    if (blockIdx.x > 0) {
        clear_blind<GT>(a, 1);
        return;
    }
    __shared__ uint64_t exchange[2][kFew];
    const int tid = static_cast<int>(threadIdx.x), n = static_cast<int>(a.rows);
    int padded = 32;
    while (padded < n) padded *= 2;
    uint64_t item = ~0ull;
    if (tid < n) {
        const int64_t v = token_at(a.tokens, a.i64, tid);
        item = static_cast<uint64_t>(v >= 0 && v < a.table_rows ? v : a.table_rows) << 32 | static_cast<uint32_t>(tid);
    }
    if (a.present != nullptr)
        for (int64_t w = tid; w < (a.table_rows + 31) / 32; w += kSortThreads) a.present[w] = 0u;
    __syncthreads();  // the bitmap is clear
    if (tid >= padded) return;  // whole warps; the barriers below are of those that stay
    int turn = 0;
    for (int size = 2; size <= padded; size *= 2) {
        for (int d = size / 2; d > 0; d /= 2) {
            uint64_t other;
            if (d >= 32) {
                exchange[turn][tid] = item;
                asm volatile("barrier.sync 1, %0;" :: "r"(padded) : "memory");
                other = exchange[turn][tid ^ d];
                turn ^= 1;  // read by all before it is written again: a barrier lies between
            } else {
                other = __shfl_xor_sync(kAllLanes, item, d);
            }
            const bool low = ((tid & d) == 0) == ((tid & size) == 0);
            item = low ? min(item, other) : max(item, other);
        }
    }
    if (tid >= n) return;
    const uint32_t v = static_cast<uint32_t>(item >> 32);
    a.keys[tid] = v;
    a.order[tid] = static_cast<uint32_t>(item);
    if (a.present != nullptr && v < a.table_rows) atomicOr(a.present + (v >> 5), 1u << (v & 31));
}

// ---------------------------------------------------------------- sums

// Sorted positions a warp takes, one to a lane: 32, or 8 where 32 leave fewer than
// kFewWarps warps, about 13 for each of the device's SMs, and positions are few.  A
// warp takes its positions some at a time, each time waiting for memory; more chunks
// cut more runs, which count the more the more positions share a table.  Whole
// gradients of 32000 rows in us, with 8 and with 32 a warp, and the warps of the latter
// (of 2000 rows, 40000 x 64 bf16: 45.7 and 42.8):
//     positions x columns         bf16          binary32      warps
//     2000 x 64                18.5   23.7     18.2   22.5       63
//     20000 x 64               26.7   32.3     27.0   30.4      625
//     40000 x 64               41.6   44.7     42.5   39.3     1250
//     10000 x 1000             30.5   36.4     41.1   41.7     1252
//     16384 x 1000             36.0   36.3     50.4   46.7     2048
//     20000 x 1000             39.9   38.9     56.4   52.6     2500
//     16384 x 2048             52.6   46.9     88.1   79.2     4096
// The workspace's size goes by it, so it asks no device.
constexpr int64_t kFewWarps = 2048, kFewPositions = 32768;
inline int chunk_of(int64_t rows, int64_t cols) {
    return rows <= kFewPositions && (rows + 31) / 32 * ((cols + kTileCols - 1) / kTileCols) < kFewWarps ? 8 : 32;
}

// The table's row of a sum, or what the sum is added to.
template <int GT, bool VEC>
__device__ __forceinline__ void write_sum(const EmbedGradArgs &a, uint32_t v, int base, int lane, const float2 (&sum)[4],
                                          const Raw8<GT> &old) {
    float2 f[4], o[4];
    unpack8<GT>(old, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = mul2(sum[j], both(a.scale));
        if (a.accumulate) f[j] = add2(f[j], o[j]);
    }
    store_tile<GT, VEC>(row_of<GT>(a.dtable, v, a.table_stride), base, a.cols, lane, pack8<GT>(f));
}
template <int GT, bool VEC>
__device__ __forceinline__ Raw8<GT> old_row(const EmbedGradArgs &a, uint32_t v, int base, int lane) {
    return load_tile<GT, VEC>(row_of<GT>(a.dtable, v, a.table_stride), base, a.cols, lane);
}

// Partial sums: for each chunk its first run where that began before the chunk
// (slot 0), and its last run where it began in the chunk and goes on (slot 1).
// A lane's 8 columns lie together, whatever the matrix's access width.
__device__ __forceinline__ float4 *partial_at(const EmbedGradArgs &a, int64_t chunk, int slot, int tile, int lane) {
    const int64_t tiles = (a.cols + kTileCols - 1) / kTileCols;
    return reinterpret_cast<float4 *>(a.partial) + (((chunk * 2 + slot) * tiles + tile) * 32 + lane) * 2;
}

// Blocks of two kinds, the sums spread evenly among the others: 8 warps that
// each add a chunk's tile, and 8 warps that write the zeros of 32 table rows.
template <int DT, int GT, bool VEC, bool ACCUMULATE>
__global__ void __launch_bounds__(256) embed_sum_kernel(EmbedGradArgs a, uint32_t sum_blocks, uint32_t every) {
    enter_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (a.cols + kTileCols - 1) / kTileCols;
    const uint32_t turn = blockIdx.x / every;
    if (blockIdx.x % every != 0 || turn >= sum_blocks) {  // rows that no token names become zero
        const int64_t w = a.blind / 32 + (blockIdx.x - min(turn + 1, sum_blocks));
        if (w * 32 >= a.table_rows) return;
        const uint32_t present = a.present[w];
#pragma unroll 1
        for (int k = warp; k < 32; k += 8)
            if (!((present >> k) & 1) && w * 32 + k < a.table_rows)
                clear_row<GT>(row_of<GT>(a.dtable, w * 32 + k, a.table_stride), a.cols, lane);
        return;
    }
    const int size = a.chunk;
    const int64_t chunks = (a.rows + size - 1) / size;
    const int64_t item = static_cast<int64_t>(turn) * 8 + warp;
    const int64_t chunk = item / tiles;
    const int tile = static_cast<int>(item - chunk * tiles), base = tile * kTileCols;
    if (chunk >= chunks) return;
    const uint32_t nowhere = static_cast<uint32_t>(a.table_rows);
    const int64_t at = chunk * size + lane;
    const bool mine = lane < size && at < a.rows;
    const uint32_t key = mine ? a.keys[at] : nowhere;
    const uint32_t pos = mine ? a.order[at] : 0u;
    const uint32_t key_before = chunk > 0 ? a.keys[chunk * size - 1] : nowhere;
    const uint32_t key_after = (chunk + 1) * size < a.rows ? a.keys[(chunk + 1) * size] : nowhere;
    const int count = __popc(__ballot_sync(kAllLanes, key != nowhere));  // positions without a token come last
    if (count == 0) return;
    // where a run ends: the next key is another (last lane: the next chunk's first)
    uint32_t key_next = __shfl_down_sync(kAllLanes, key, 1);
    if (lane == size - 1) key_next = key_after;
    const unsigned ends = __ballot_sync(kAllLanes, lane < count && (key_next != key || lane == count - 1));
    const bool goes_on = count == size && key_after == __shfl_sync(kAllLanes, key, size - 1);

    float2 sum[4] = {};
    bool from_before = chunk > 0 && key_before == __shfl_sync(kAllLanes, key, 0);
    constexpr int U = ACCUMULATE ? 4 : 8;  // rows in flight, with accumulate each with the row it is added to
    for (int i0 = 0; i0 < count; i0 += U) {
        Raw8<DT> r[U];
        Raw8<GT> old[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t t = __shfl_sync(kAllLanes, pos, i0 + u), k = __shfl_sync(kAllLanes, key, i0 + u);
            if (i0 + u < count) {
                r[u] = load_tile<DT, VEC>(row_of<DT>(a.dout, t, a.dout_stride), base, a.cols, lane);
                if (ACCUMULATE && (ends >> (i0 + u) & 1)) old[u] = old_row<GT, VEC>(a, k, base, lane);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = __shfl_sync(kAllLanes, key, i0 + u);
            if (i0 + u >= count) break;
            float2 f[4];
            unpack8<DT>(r[u], f);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], f[j]);
            if (!(ends >> (i0 + u) & 1)) continue;
            const bool crosses = from_before || (goes_on && i0 + u == count - 1);
            if (!crosses) {
                write_sum<GT, VEC>(a, k, base, lane, sum, old[u]);
            } else {
                float4 *p = partial_at(a, chunk, from_before ? 0 : 1, tile, lane);
                p[0] = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
                p[1] = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
            }
            from_before = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = both(0.0f);
        }
    }
}

// Runs that cross chunks: the warp of the chunk where a run begins adds its slot
// 1 and the slots 0 of the chunks after it; runs of more than kLongRun chunks
// are added by the whole block, each warp every eighth chunk.
constexpr int kLongRun = 16;

// Block blockIdx.x takes eight chunks of tile blockIdx.x / strips.
template <int GT, bool VEC> __global__ void __launch_bounds__(256) embed_join_kernel(EmbedGradArgs a, uint32_t strips) {
    enter_grid();
    __shared__ float2 part[8][4][32];
    __shared__ int64_t reaches[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = static_cast<int>(blockIdx.x / strips), base = tile * kTileCols;
    const int size = a.chunk;
    const int64_t first = static_cast<int64_t>(blockIdx.x % strips) * 8, chunk = first + warp, chunks = (a.rows + size - 1) / size;
    const int64_t last = chunk * size + size - 1;
    const uint32_t nowhere = static_cast<uint32_t>(a.table_rows);
    uint32_t v = nowhere, after = nowhere, ahead = nowhere;
    if (last + 1 < a.rows) {
        v = a.keys[last];
        after = a.keys[last + 1];
        ahead = chunk > 0 ? a.keys[last - size] : nowhere;
    }
    int64_t reach = 0;  // chunks after this one that a run reaches which begins here
    if (v != nowhere && after == v && ahead != v) {
        // the chunks' first keys rise, so those equal to v come first: 32 probes at a time
        int64_t lo = chunk + 1, hi = chunks;
        while (lo < hi) {
            const int64_t step = (hi - lo + 31) / 32, probe = lo + lane * step;
            const int found = __popc(__ballot_sync(kAllLanes, probe < hi && a.keys[probe * size] == v));
            hi = min(hi, lo + found * step);
            if (found > 0) lo += (found - 1) * step + 1;
        }
        reach = lo - (chunk + 1);
    }
    if (lane == 0) reaches[warp] = reach;
    auto add = [&](float2 (&sum)[4], int64_t c, int slot) {
        const float4 *p = partial_at(a, c, slot, tile, lane);
        const float4 x = p[0], y = p[1];
        sum[0] = add2(sum[0], make_float2(x.x, x.y));
        sum[1] = add2(sum[1], make_float2(x.z, x.w));
        sum[2] = add2(sum[2], make_float2(y.x, y.y));
        sum[3] = add2(sum[3], make_float2(y.z, y.w));
    };
    if (reach > 0 && reach <= kLongRun) {
        float2 sum[4] = {};
        Raw8<GT> old = {};
        if (a.accumulate) old = old_row<GT, VEC>(a, v, base, lane);
        add(sum, chunk, 1);
#pragma unroll 8
        for (int64_t k = 0; k < reach; ++k) add(sum, chunk + 1 + k, 0);
        write_sum<GT, VEC>(a, v, base, lane, sum, old);
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
        const int64_t far = reaches[w];
        if (far <= kLongRun) continue;
        const int64_t from = first + w;
        float2 sum[4] = {};
        if (warp == 0) add(sum, from, 1);
#pragma unroll 8
        for (int64_t k = warp; k < far; k += 8) add(sum, from + 1 + k, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[warp][j][lane] = sum[j];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int k = 1; k < 8; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], part[k][j][lane]);
            const uint32_t far_v = a.keys[from * size + size - 1];
            Raw8<GT> old = {};
            if (a.accumulate) old = old_row<GT, VEC>(a, far_v, base, lane);
            write_sum<GT, VEC>(a, far_v, base, lane, sum, old);
        }
        __syncthreads();
    }
}

template <int DT, int GT, bool VEC>
cudaError_t embed_grad_launch(EmbedGradArgs a, int sms, cudaStream_t s, LaunchInfo *info, int *launches) {
    const bool few = a.rows <= kFew;
    // Rows to clear meanwhile: what 6 TB/s write in the sort's time, 3 us of few
    // positions, otherwise about 9 us and 0.4 ns a position; whole words of the bitmap.
    // The blocks beside the sort write 4.2 to 4.5 TB/s and end after it; with the rows
    // that 4.4 TB/s write, calls took 9 % less to 7 % more time.
    a.chunk = chunk_of(a.rows, a.cols);
    a.blind = 0;
    int64_t clear_blocks = 0;
    if (!a.accumulate) {
        const double bytes = (few ? 3e-6 : 9e-6 + 0.4e-9 * static_cast<double>(a.rows)) * 6e12;
        const double rows = bytes / (static_cast<double>(a.cols) * ElemOf<GT>::kBytes);
        a.blind = rows >= static_cast<double>(a.table_rows) ? (a.table_rows + 31) / 32 * 32 : static_cast<int64_t>(rows) / 32 * 32;
        a.blind = std::min(a.blind, a.table_rows);
        // up to two blocks of 1024 threads an SM, in whole clusters
        clear_blocks = std::min<int64_t>((a.blind + kSortWarps - 1) / kSortWarps, 2 * sms);
        clear_blocks = (clear_blocks + kSortBlocks - 1) / kSortBlocks * kSortBlocks;
    }
    cudaError_t e = cudaSuccess;
    if (few) {
        e = launch_rows(embed_sort_few_kernel<GT>, dim3(1 + clear_blocks), dim3(kSortThreads), 0, 1, s, a);
    } else {
        int width = 0;  // bits of a key: 0 .. table_rows
        while (width < 32 && (static_cast<uint64_t>(a.table_rows) >> width) != 0) ++width;
        const int passes = std::max(1, (width + kDigitBits - 1) / kDigitBits);
        const int bits = std::max(1, (width + passes - 1) / passes);
        const size_t smem = size_t(kSortWarps) * 4 << bits;
        static std::atomic<uint64_t> allowed{0};
        auto sort = embed_sort_kernel<GT>;
        e = allow_smem(reinterpret_cast<const void *>(sort), (kSortWarps * 4) << kDigitBits, &allowed);
        if (e != cudaSuccess) return e;
        e = launch_rows(sort, dim3(kSortBlocks + clear_blocks), dim3(kSortThreads), smem, kSortBlocks, s, a, passes, bits);
    }
    if (e != cudaSuccess) return e;
    ++*launches;

    const int64_t tiles = (a.cols + kTileCols - 1) / kTileCols, chunks = (a.rows + a.chunk - 1) / a.chunk;
    const int64_t sums = (chunks * tiles + 7) / 8;
    const int64_t fills = a.accumulate ? 0 : (a.table_rows + 31) / 32 - a.blind / 32;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : ElemOf<DT>::kBytes;
    info->grid = static_cast<int>(sums + fills);
    info->block = 256;
    if (sums + fills > 0) {
        const uint32_t every = sums > 0 ? static_cast<uint32_t>((sums + fills) / sums) : 1;
        auto sum = a.accumulate ? embed_sum_kernel<DT, GT, VEC, true> : embed_sum_kernel<DT, GT, VEC, false>;
        e = launch_rows(sum, dim3(sums + fills), dim3(256), 0, 1, s, a, static_cast<uint32_t>(sums), every);
        ++*launches;
    }
    if (e != cudaSuccess || chunks < 2) return e;
    ++*launches;
    const int64_t strips = (chunks + 7) / 8;
    return launch_rows(embed_join_kernel<GT, VEC>, dim3(strips * tiles), dim3(256), 0, 1, s, a, static_cast<uint32_t>(strips));
}

template <int DT, int GT>
cudaError_t embed_grad_dispatch(const EmbedGradArgs &a, int sms, cudaStream_t s, LaunchInfo *info, int *launches) {
    return wide_rows<DT>(a.dout, a.dout_stride) && wide_rows<GT>(a.dtable, a.table_stride)
               ? embed_grad_launch<DT, GT, true>(a, sms, s, info, launches)
               : embed_grad_launch<DT, GT, false>(a, sms, s, info, launches);
}

}  // namespace

cudaError_t launch_embed(int dtype, const EmbedArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return dtype == DT_F32   ? embed_dispatch<DT_F32>(a, sms, s, info)
           : dtype == DT_F16 ? embed_dispatch<DT_F16>(a, sms, s, info)
                             : embed_dispatch<DT_BF16>(a, sms, s, info);
}

int64_t embed_partial_bytes(int64_t rows, int64_t cols) {
    const int size = chunk_of(rows, cols);
    return (rows + size - 1) / size * 2 * ((cols + kTileCols - 1) / kTileCols) * kTileCols * 4;
}

cudaError_t launch_embed_grad(int dtype, int gtype, const EmbedGradArgs &a, int sms, cudaStream_t s, LaunchInfo *info,
                              int *launches) {
    if (dtype == DT_F32) return embed_grad_dispatch<DT_F32, DT_F32>(a, sms, s, info, launches);
    if (dtype == DT_F16)
        return gtype == DT_F32 ? embed_grad_dispatch<DT_F16, DT_F32>(a, sms, s, info, launches)
                               : embed_grad_dispatch<DT_F16, DT_F16>(a, sms, s, info, launches);
    return gtype == DT_F32 ? embed_grad_dispatch<DT_BF16, DT_F32>(a, sms, s, info, launches)
                           : embed_grad_dispatch<DT_BF16, DT_BF16>(a, sms, s, info, launches);
}

}  // namespace ew
