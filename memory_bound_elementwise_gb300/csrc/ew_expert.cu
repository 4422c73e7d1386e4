// ew_expert.cu -- tokens sorted by expert and back, weights applied, and the gradients.
//
// Each of n tokens names k experts: n k slots, slot t k + j the j-th of token t.
//   sort      positions[slot]: the slot's row among the rows sorted by expert (stable), each
//             expert's rows beginning at a multiple of `align`
//   dispatch  out[positions[t,j],:] = x[t,:], zeros in rows of no slot
//   combine   out[t,:] = residual[t,:] + sum_j weights[t,j] y[positions[t,j],:]
//             (without weights and residual: the gradient of dispatch)
//   its gradient  dy[positions[t,j],:] = weights[t,j] dout[t,:], zeros in rows of no slot,
//             dweights[t,j] = dout[t,:] . y[positions[t,j],:]
//
// All but the sort move rows and compute next to nothing: the bound is memory.
// Everything goes by tokens, so that a token's row is read once for all its
// experts; by the sorted rows it would be read k times, from DRAM where the
// tokens do not fit L2.
#include <algorithm>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// ---------------------------------------------------------------- sort
//
// A counting sort.  A block takes kTileSlots consecutive slots at a time, a warp
// consecutive ones of those, 32 a step: lanes with the same expert are ranked by
// ballots, and a count for each warp and expert says how many came before.  Up to
// kTileSlots slots, one block does all of it in one launch; more take two, the
// first leaving each slot's rank within its block in `positions` and the blocks'
// counts in the workspace.  Latency bounds it: 512 slots of 128 experts take 3.8 us,
// 4000 6.3, 131072 9.0 in a graph.  Rows of no slot are marked before anything else;
// marked at the end, expert by expert, they took 10 to 37 us.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortSteps = 4;  // of 32 slots, at most, that a warp takes of a tile
constexpr int kTileSlots = kSortThreads * kSortSteps;
constexpr int kMostSortBlocks = 256;

struct SortShape {
    int blocks, tiles_each;  // tiles of a block
};
SortShape sort_shape(int64_t slots) {
    const int64_t tiles = std::max<int64_t>(1, (slots + kTileSlots - 1) / kTileSlots);
    const int64_t each = (tiles + kMostSortBlocks - 1) / kMostSortBlocks;
    return {static_cast<int>((tiles + each - 1) / each), static_cast<int>(each)};
}

// The expert of a slot, -1 for none.
__device__ __forceinline__ int expert_of(const ExpertSortArgs &a, int64_t slot) {
    const int64_t at = a.stride == a.k ? slot : slot / a.k * a.stride + slot % a.k;
    const int64_t e = token_at(a.experts, a.i64, at);
    return e >= 0 && e < a.n_experts ? static_cast<int>(e) : -1;
}

// Ranks of the block's slots among those of the same expert, into positions;
// `seen` has the block's counts at the end.
__device__ __forceinline__ void rank_slots(const ExpertSortArgs &a, int bits, int tiles_each, uint16_t *count, uint32_t *seen) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slots = a.rows * a.k, first = static_cast<int64_t>(blockIdx.x) * tiles_each * kTileSlots;
    uint16_t *mine = count + warp * a.n_experts;
    // a row is of no slot until one is placed there
    for (int64_t r = blockIdx.x * static_cast<int64_t>(kSortThreads) + threadIdx.x; r < a.capacity; r += static_cast<int64_t>(gridDim.x) * kSortThreads)
        a.slots[r] = -1;
    for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads) seen[e] = 0u;
    for (int tile = 0; tile < tiles_each; ++tile) {
        const int64_t begin = first + static_cast<int64_t>(tile) * kTileSlots;
        if (begin >= slots) break;
        const int here = static_cast<int>(min(slots - begin, static_cast<int64_t>(kTileSlots)));
        const int each = (here + kSortThreads - 1) / kSortThreads;  // steps of a warp
        int expert[kSortSteps], rank[kSortSteps];
#pragma unroll
        for (int i = 0; i < kSortSteps; ++i) {
            const int at = (warp * each + i) * 32 + lane;
            expert[i] = i < each && at < here ? expert_of(a, begin + at) : -1;
        }
        for (int e = threadIdx.x; e < kSortWarps * a.n_experts; e += kSortThreads) count[e] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortSteps; ++i) {
            const unsigned active = __ballot_sync(kAllLanes, expert[i] >= 0);
            const unsigned same = lanes_alike(static_cast<uint32_t>(expert[i]), bits, active);
            const int before = expert[i] >= 0 ? mine[expert[i]] : 0;
            __syncwarp();
            if (expert[i] >= 0 && lane == __ffs(same) - 1) mine[expert[i]] = static_cast<uint16_t>(before + __popc(same));
            rank[i] = before + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
        }
        __syncthreads();
        // counts become the ranks of the warps' first slots within the block
        uint32_t total[2] = {0u, 0u};
        int part = 0;
        for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads, ++part) {
            uint32_t sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = count[w * a.n_experts + e];
                count[w * a.n_experts + e] = static_cast<uint16_t>(sum);
                sum += c;
            }
            total[part] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortSteps; ++i) {
            const int at = (warp * each + i) * 32 + lane;
            if (i < each && at < here)
                a.positions[begin + at] = expert[i] >= 0 ? static_cast<int32_t>(seen[expert[i]] + mine[expert[i]] + rank[i]) : -1;
        }
        __syncthreads();
        part = 0;
        for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads, ++part) seen[e] += total[part];
    }
    __syncthreads();
}

// Positions from ranks: first[e] is the row of the block's first slot of expert e.
__device__ __forceinline__ void place_slots(const ExpertSortArgs &a, int tiles_each, const uint32_t *first, const uint32_t *total,
                                            const uint32_t *offset) {
    const int64_t slots = a.rows * a.k, each = static_cast<int64_t>(tiles_each) * kTileSlots;
    const int64_t begin = blockIdx.x * each, end = min(begin + each, slots);
    for (int64_t s = begin + threadIdx.x; s < end; s += kSortThreads) {
        const int e = expert_of(a, s);
        if (e < 0) continue;  // -1 already
        const int32_t at = a.positions[s] + static_cast<int32_t>(first[e]);
        a.positions[s] = at;
        a.slots[at] = static_cast<int32_t>(s);
    }
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads) a.counts[e] = static_cast<int32_t>(total[e]);
        for (int e = threadIdx.x; e <= a.n_experts; e += kSortThreads) a.offsets[e] = static_cast<int32_t>(offset[e]);
    }
}

// offset[e]: the first row of expert e, from the experts' totals.
__device__ __forceinline__ void experts_offsets(const ExpertSortArgs &a, const uint32_t *total, uint32_t *offset, uint32_t *scan) {
    static_assert(kMostExperts <= 2 * kSortThreads, "two experts a thread");
    const int e = 2 * static_cast<int>(threadIdx.x);
    const uint32_t align = static_cast<uint32_t>(a.align);
    const uint32_t x = e < a.n_experts ? (total[e] + align - 1) / align * align : 0u;
    const uint32_t y = e + 1 < a.n_experts ? (total[e + 1] + align - 1) / align * align : 0u;
    const uint32_t upto = block_prefix(x + y, scan);
    if (e < a.n_experts) offset[e + 1] = upto - y;
    if (e + 1 < a.n_experts) offset[e + 2] = upto;
    if (threadIdx.x == 0) offset[0] = 0u;
    __syncthreads();
}

// Shared memory: counts of the warps, then three numbers an expert.
int sort_smem(int n_experts) { return kSortWarps * n_experts * 2 + (3 * n_experts + 2) * 4; }

template <bool WHOLE> __global__ void __launch_bounds__(kSortThreads) expert_rank_kernel(ExpertSortArgs a, int bits, int tiles_each) {
    enter_grid();
    extern __shared__ uint32_t shared[];
    __shared__ uint32_t scan[kSortWarps];
    uint32_t *seen = shared, *offset = seen + a.n_experts, *first = offset + a.n_experts + 2;
    uint16_t *count = reinterpret_cast<uint16_t *>(first + a.n_experts);
    rank_slots(a, bits, tiles_each, count, seen);
    if constexpr (WHOLE) {
        experts_offsets(a, seen, offset, scan);
        place_slots(a, tiles_each, offset, seen, offset);
    } else {
        for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads) a.partial[static_cast<int64_t>(blockIdx.x) * a.n_experts + e] = seen[e];
    }
}

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(ExpertSortArgs a, int tiles_each) {
    enter_grid();
    extern __shared__ uint32_t shared[];
    __shared__ uint32_t scan[kSortWarps];
    uint32_t *total = shared, *offset = total + a.n_experts, *first = offset + a.n_experts + 2;
    const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
    for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads) {
        uint32_t before = 0, all = 0;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
            const uint32_t c = a.partial[static_cast<int64_t>(b) * a.n_experts + e];
            all += c;
            before += b < block ? c : 0u;
        }
        total[e] = all;
        first[e] = before;
    }
    __syncthreads();
    experts_offsets(a, total, offset, scan);
    for (int e = threadIdx.x; e < a.n_experts; e += kSortThreads) first[e] += offset[e];
    __syncthreads();
    place_slots(a, tiles_each, first, total, offset);
}

// ---------------------------------------------------------------- rows of no slot

constexpr int kWarpsABlock = 8;
constexpr int kMostZeroRows = 256;

// Zeros in the rows of no slot among the `each` rows of this block, a warp a row.
template <int DT> __device__ __forceinline__ void clear_rows(void *out, int64_t stride, const int32_t *slots, int64_t rows,
                                                             int cols, int each) {
    __shared__ int list[kMostZeroRows], found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * each, row = first + threadIdx.x;
    if (static_cast<int>(threadIdx.x) < each && row < rows && slots[row] < 0) list[atomicAdd(&found, 1)] = static_cast<int>(threadIdx.x);
    __syncthreads();
    for (int i = warp; i < found; i += kWarpsABlock) clear_row<DT>(row_of<DT>(out, first + list[i], stride), cols, lane);
}
// Rows a block looks at: few enough for two blocks an SM.
int zero_rows_each(int64_t rows, int sms) {
    int each = kMostZeroRows;
    while (each > 1 && rows < static_cast<int64_t>(each) * 2 * sms) each /= 2;
    return each;
}

// A warp's share of the positions (and weights) of a token's slots j0 .. j0 + 31.
__device__ __forceinline__ int64_t position_of(const int32_t *positions, int64_t at, bool mine, int64_t rows) {
    const int64_t p = mine ? positions[at] : -1;
    return p < rows ? p : -1;
}
__device__ __forceinline__ float weight_at(const void *w, int wtype, int64_t at) {
    if (wtype == DT_F32) return static_cast<const float *>(w)[at];
    const uint16_t v = static_cast<const uint16_t *>(w)[at];
    return wtype == DT_F16 ? f16_to_f32(v) : bf16_to_f32(v);
}

// How a warp moves 256 columns of a row.  VEC: all rows start at multiples of 8
// elements; otherwise by pairs, as they lie in the row that is written.
template <int DT, bool VEC> struct Mover {
    using Run = std::conditional_t<VEC, Raw8<DT>, Pairs8<DT>>;
    int cols, lane;
    __device__ __forceinline__ static int odd(const void *written) { return VEC ? 0 : odd_of<DT>(written); }
    __device__ __forceinline__ Run load(const void *row, int tile, int odd) const {
        if constexpr (VEC) return load_tile<DT, true>(row, tile * kTileCols, cols, lane);
        else return load_pairs<DT>(row, tile, odd, cols, lane);
    }
    __device__ __forceinline__ static Raw8<DT> whole(const Run &r) {
        if constexpr (VEC) return r;
        else return r.whole();
    }
    __device__ __forceinline__ void store(void *row, int tile, int odd, const Raw8<DT> &r) const {
        if constexpr (VEC) store_tile<DT, true>(row, tile * kTileCols, cols, lane, r);
        else store_pairs<DT>(row, tile, odd, cols, lane, r);
    }
};

// ---------------------------------------------------------------- dispatch

// A warp takes U consecutive tiles of a token.  VEC: a tile is read once;
// otherwise anew for each of the places, whose rows may start anywhere.  Bounded by
// what it writes: 16384 tokens of 4096 bf16 to 8 experts 199 us at a floor of 202 with
// the sort (0.96 of a plain copy's rate); of 2001 columns 108 us at 89.  Few
// tokens take a warp for each tile, so that all SMs have one.
template <int DT, bool VEC, int U>
__global__ void __launch_bounds__(32 * kWarpsABlock) expert_dispatch_kernel(ExpertRowsArgs a, uint32_t zero_blocks, int zero_each, int tiles) {
    enter_grid();
    if (blockIdx.x < zero_blocks) {
        clear_rows<DT>(a.out, a.out_stride, a.slots, a.sorted, a.cols, zero_each);
        return;
    }
    const int lane = threadIdx.x & 31, groups = (tiles + U - 1) / U;
    const int64_t item = static_cast<int64_t>(blockIdx.x - zero_blocks) * kWarpsABlock + (threadIdx.x >> 5);
    const int64_t token = item / groups;
    if (token >= a.rows) return;
    const int tile0 = static_cast<int>(item - token * groups) * U;
    const Mover<DT, VEC> mover = {a.cols, lane};
    const void *x = row_of<DT>(a.x, token, a.x_stride);
    typename Mover<DT, VEC>::Run r[U];
    if constexpr (VEC) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = mover.load(x, tile0 + u, 0);
    }
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int64_t p = position_of(a.positions, token * a.k + j0 + lane, j0 + lane < a.k, a.sorted);
        for (int j = 0; j < 32 && j0 + j < a.k; ++j) {
            const int64_t to = __shfl_sync(kAllLanes, p, j);
            if (to < 0) continue;
            void *out = row_of<DT>(a.out, to, a.out_stride);
            const int odd = mover.odd(out);
            if constexpr (!VEC) {
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = mover.load(x, tile0 + u, odd);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) mover.store(out, tile0 + u, odd, mover.whole(r[u]));
        }
    }
}

// ---------------------------------------------------------------- combine

// A warp takes U consecutive tiles of a token, and of its slots KB at a time, all
// of whose loads are under way together: in registers, so KB x U is what fits 80 of
// them.  Bounded by what it reads: 16384 tokens of 4096 bf16 from 8 experts each 206
// us at a floor of 202; of 2001 columns 150 us at 99, by 4-byte and 2-byte loads.
template <int DT, bool VEC, int KB, int U>
__global__ void __launch_bounds__(32 * kWarpsABlock, !VEC && (KB <= 2 || DT == DT_F32) ? 4 : DT != DT_F32 ? 3 : 2) expert_combine_kernel(ExpertRowsArgs a, int tiles) {
    enter_grid();
    const int lane = threadIdx.x & 31, groups = (tiles + U - 1) / U;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarpsABlock + (threadIdx.x >> 5);
    const int64_t token = item / groups;
    if (token >= a.rows) return;
    const int tile0 = static_cast<int>(item - token * groups) * U;
    const Mover<DT, VEC> mover = {a.cols, lane};
    using Run = typename Mover<DT, VEC>::Run;
    void *out = row_of<DT>(a.out, token, a.out_stride);
    const int odd = mover.odd(out);
    float2 sum[U][4] = {};
    for (int j0 = 0; j0 < a.k; j0 += KB) {
        const bool mine = lane < KB && j0 + lane < a.k;
        const int64_t at = token * a.k + j0 + lane, p = position_of(a.positions, at, mine, a.sorted);
        const float w = a.weights && mine ? weight_at(a.weights, a.wtype, at) : 1.0f;
        Run r[KB][U], first[U];
        int64_t from[KB];
        if (a.residual && j0 == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) first[u] = mover.load(row_of<DT>(a.residual, token, a.residual_stride), tile0 + u, odd);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            from[b] = __shfl_sync(kAllLanes, p, b);
            if (from[b] < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) r[b][u] = mover.load(row_of<DT>(a.x, from[b], a.x_stride), tile0 + u, odd);
        }
        if (a.residual && j0 == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) unpack8<DT>(mover.whole(first[u]), sum[u]);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const float2 wb = both(__shfl_sync(kAllLanes, w, b));
            if (from[b] < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 f[4];
                unpack8<DT>(mover.whole(r[b][u]), f);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[u][i] = fma2(f[i], wb, sum[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) mover.store(out, tile0 + u, odd, pack8<DT>(sum[u]));
}

// ---------------------------------------------------------------- the gradient of combine

// The sums over the warp of N values a lane (N a power of two up to 32): lane l
// returns the sum of value l / (32 / N).  Halves of the values change lanes at each
// step, so 8 values take 9 shuffles instead of 40.
template <int N> __device__ __forceinline__ float warp_sums_of(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int d = 16;
#pragma unroll
    for (int half = N / 2; half > 0; half /= 2, d /= 2) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
            v[i] = keep + __shfl_xor_sync(kAllLanes, give, d);
        }
    }
    for (; d > 0; d /= 2) v[0] += __shfl_xor_sync(kAllLanes, v[0], d);
    return v[0];
}

// `split` warps of a block (1, 2, 4 or 8) take a token, tile t warp t mod split, KB
// of its slots at a time: a tile of dout is read once and both used for the slots'
// rows and multiplied with theirs.  Bounded by memory: 16384 tokens of 4096 bf16 to 8
// experts 355 us at a floor of 343; 5003 of 1001 binary32 to 2 16.7 at 15.1; of 2001
// bf16 242 at 168, where dout is kept for rows at either half of a word.
template <int DT, bool VEC, int KB>
__global__ void __launch_bounds__(32 * kWarpsABlock) expert_combine_grad_kernel(ExpertRowsArgs a, uint32_t zero_blocks, int zero_each,
                                                                               int tiles, int split) {
    enter_grid();
    if (blockIdx.x < zero_blocks) {
        clear_rows<DT>(a.out, a.out_stride, a.slots, a.sorted, a.cols, zero_each);
        return;
    }
    constexpr int kPlaces = VEC || DT == DT_F32 ? 1 : 2;
    __shared__ float part[2][kWarpsABlock][KB];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp & (split - 1);
    const int64_t token = (static_cast<int64_t>(blockIdx.x - zero_blocks) * kWarpsABlock + warp) / split;
    const bool given = token < a.rows;  // all warps stay for the barriers
    const Mover<DT, VEC> mover = {a.cols, lane};
    using Run = typename Mover<DT, VEC>::Run;
    const void *dout = row_of<DT>(a.residual, token, a.residual_stride);  // not read unless the token is given
    int turn = 0;
    for (int j0 = 0; j0 < a.k; j0 += KB, turn ^= 1) {
        const bool mine = given && lane < KB && j0 + lane < a.k;
        const int64_t at = token * a.k + j0 + lane, p = position_of(a.positions, at, mine, a.sorted);
        const float w = a.weights && mine ? weight_at(a.weights, a.wtype, at) : 1.0f;
        int64_t row[KB];
        float wb[KB], dot[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            row[b] = __shfl_sync(kAllLanes, p, b);
            wb[b] = __shfl_sync(kAllLanes, w, b);
            dot[b] = 0.0f;
        }
        for (int tile = share; given && tile < tiles; tile += split) {
            // dout as it lies beside rows of either place, where there are two
            Run rd[kPlaces], ry[KB];
#pragma unroll
            for (int o = 0; o < kPlaces; ++o) rd[o] = mover.load(dout, tile, o);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                if (row[b] < 0) continue;
                const int odd = mover.odd(row_of<DT>(a.out, row[b], a.out_stride));
                if (a.x) ry[b] = mover.load(row_of<DT>(a.x, row[b], a.x_stride), tile, odd);
            }
            float2 d[kPlaces][4];
#pragma unroll
            for (int o = 0; o < kPlaces; ++o) unpack8<DT>(mover.whole(rd[o]), d[o]);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                if (row[b] < 0) continue;
                void *out = row_of<DT>(a.out, row[b], a.out_stride);
                const int odd = mover.odd(out);
                float2 own[4], o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) own[i] = kPlaces == 2 && odd ? d[kPlaces - 1][i] : d[0][i];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = mul2(own[i], both(wb[b]));
                mover.store(out, tile, odd, pack8<DT>(o));
                if (a.x) {
                    float2 f[4], s = both(0.0f);
                    unpack8<DT>(mover.whole(ry[b]), f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s = fma2(f[i], own[i], s);
                    dot[b] += s.x + s.y;
                }
            }
        }
        if (a.dweights == nullptr) continue;
        float sum = warp_sums_of<KB>(dot);
        const int b = lane / (32 / KB);  // the slot whose sum this lane has
        if (split > 1) {
            if (lane % (32 / KB) == 0) part[turn][warp][b] = sum;
            __syncthreads();
            sum = 0.0f;
            for (int s = 0; s < split; ++s) sum += part[turn][warp - share + s][b];
        }
        if (given && share == 0 && lane % (32 / KB) == 0 && j0 + b < a.k) a.dweights[token * a.k + j0 + b] = sum;
    }
}

// ---------------------------------------------------------------- launches

int tiles_of(int cols, bool vec) { return static_cast<int>((static_cast<int64_t>(cols) + (vec ? 0 : 1) + kTileCols - 1) / kTileCols); }
// Slots whose loads are under way together: as many as registers allow.
int slots_at_once(int k, int most) {
    int kb = 1;
    while (kb < most && kb < k) kb *= 2;
    return kb;
}

template <int DT, bool VEC> cudaError_t dispatch_launch(const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int tiles = tiles_of(a.cols, VEC);
    const bool many = a.rows * tiles >= static_cast<int64_t>(sms) * 64;
    const int u = many ? 4 : 1, each = zero_rows_each(a.sorted, sms);
    const int64_t zeros = (a.sorted + each - 1) / each, items = a.rows * ((tiles + u - 1) / u);
    const int64_t grid = zeros + (items + kWarpsABlock - 1) / kWarpsABlock;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    info->grid = static_cast<int>(grid);
    info->block = 32 * kWarpsABlock;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : 4;
    auto kernel = many ? expert_dispatch_kernel<DT, VEC, 4> : expert_dispatch_kernel<DT, VEC, 1>;
    return launch_rows(kernel, dim3(grid), dim3(32 * kWarpsABlock), 0, 1, s, a, static_cast<uint32_t>(zeros), each, tiles);
}

template <int DT, bool VEC, int KB> cudaError_t combine_launch(const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    constexpr int U = VEC && DT != DT_F32 ? (KB == 1 ? 4 : KB == 8 ? 1 : 2) : VEC ? (KB == 1 ? 4 : KB == 2 ? 2 : 1) : 1;
    const int tiles = tiles_of(a.cols, VEC);
    const bool many = a.rows * tiles >= static_cast<int64_t>(sms) * 64;
    const int u = many ? U : 1;
    const int64_t items = a.rows * ((tiles + u - 1) / u), grid = (items + kWarpsABlock - 1) / kWarpsABlock;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    info->grid = static_cast<int>(grid);
    info->block = 32 * kWarpsABlock;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : 4;
    auto kernel = many ? expert_combine_kernel<DT, VEC, KB, U> : expert_combine_kernel<DT, VEC, KB, 1>;
    return launch_rows(kernel, dim3(grid), dim3(32 * kWarpsABlock), 0, 1, s, a, tiles);
}

template <int DT, bool VEC, int KB> cudaError_t combine_grad_launch(const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int tiles = tiles_of(a.cols, VEC), each = zero_rows_each(a.sorted, sms);
    int split = 1;
    while (split < kWarpsABlock && split * 2 <= tiles && a.rows * split < static_cast<int64_t>(sms) * 16) split *= 2;
    const int64_t zeros = (a.sorted + each - 1) / each;
    const int64_t grid = zeros + (a.rows * split + kWarpsABlock - 1) / kWarpsABlock;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    info->grid = static_cast<int>(grid);
    info->block = 32 * kWarpsABlock;
    info->vec_bytes = VEC ? 8 * ElemOf<DT>::kBytes : 4;
    return launch_rows(expert_combine_grad_kernel<DT, VEC, KB>, dim3(grid), dim3(32 * kWarpsABlock), 0, 1, s, a,
                       static_cast<uint32_t>(zeros), each, tiles, split);
}

template <int DT, bool VEC> cudaError_t by_slots(int what, const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    constexpr int kCombine = VEC ? 8 : 4, kGrad = VEC ? 8 : DT != DT_F32 ? 4 : 2;
    if (what == EXPERT_COMBINE) {
        switch (slots_at_once(a.k, kCombine)) {
            case 1: return combine_launch<DT, VEC, 1>(a, sms, s, info);
            case 2: return combine_launch<DT, VEC, 2>(a, sms, s, info);
            case 4: return combine_launch<DT, VEC, 4>(a, sms, s, info);
            default: return combine_launch<DT, VEC, kCombine>(a, sms, s, info);
        }
    }
    switch (slots_at_once(a.k, kGrad)) {
        case 1: return combine_grad_launch<DT, VEC, 1>(a, sms, s, info);
        case 2: return combine_grad_launch<DT, VEC, 2>(a, sms, s, info);
        case 4: return combine_grad_launch<DT, VEC, std::min(kGrad, 4)>(a, sms, s, info);
        default: return combine_grad_launch<DT, VEC, kGrad>(a, sms, s, info);
    }
}
template <int DT> bool all_wide(const ExpertRowsArgs &a) {
    return wide_rows<DT>(a.x, a.x_stride) && wide_rows<DT>(a.residual, a.residual_stride) && wide_rows<DT>(a.out, a.out_stride);
}
template <int DT> cudaError_t by_alignment(int what, const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    return all_wide<DT>(a) ? by_slots<DT, true>(what, a, sms, s, info) : by_slots<DT, false>(what, a, sms, s, info);
}

}  // namespace

int64_t expert_sort_bytes(int64_t slots, int n_experts) {
    const SortShape shape = sort_shape(slots);
    return shape.blocks == 1 ? 0 : static_cast<int64_t>(shape.blocks) * n_experts * 4;
}

cudaError_t launch_expert_sort(const ExpertSortArgs &a, cudaStream_t s, LaunchInfo *info, int *launches) {
    const SortShape shape = sort_shape(a.rows * a.k);
    int bits = 0;
    while ((a.n_experts - 1) >> bits) ++bits;
    const int smem = sort_smem(a.n_experts);
    info->grid = shape.blocks;
    info->block = kSortThreads;
    info->vec_bytes = 4;
    info->smem = smem;
    ++*launches;
    if (shape.blocks == 1) return launch_rows(expert_rank_kernel<true>, dim3(1), dim3(kSortThreads), smem, 1, s, a, bits, shape.tiles_each);
    cudaError_t e = launch_rows(expert_rank_kernel<false>, dim3(shape.blocks), dim3(kSortThreads), smem, 1, s, a, bits, shape.tiles_each);
    if (e != cudaSuccess) return e;
    ++*launches;
    return launch_rows(expert_place_kernel, dim3(shape.blocks), dim3(kSortThreads), (3 * a.n_experts + 2) * 4, 1, s, a, shape.tiles_each);
}

cudaError_t launch_expert_rows(int what, int dtype, const ExpertRowsArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    if (what == EXPERT_DISPATCH) {  // moves bits: 16-bit types are alike
        if (dtype == DT_F32) return all_wide<DT_F32>(a) ? dispatch_launch<DT_F32, true>(a, sms, s, info) : dispatch_launch<DT_F32, false>(a, sms, s, info);
        return all_wide<DT_BF16>(a) ? dispatch_launch<DT_BF16, true>(a, sms, s, info) : dispatch_launch<DT_BF16, false>(a, sms, s, info);
    }
    return dtype == DT_F32   ? by_alignment<DT_F32>(what, a, sms, s, info)
           : dtype == DT_F16 ? by_alignment<DT_F16>(what, a, sms, s, info)
                             : by_alignment<DT_BF16>(what, a, sms, s, info);
}

}  // namespace ew
