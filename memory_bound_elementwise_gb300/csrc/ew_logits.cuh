// ew_logits.cuh -- operators on rows of logits: log probabilities of given
// tokens with entropy and top alternatives, and their gradient; and what
// distillation (ew_distill.cuh) shares with them.  Compiled once per element
// type.
//
// With a = scale * log2(e), a row is summed as
//     s = sum 2^(a x - c),   u = sum 2^(a x - c) (a x - c),
// c an integer at least as large as every a x so far, so that shifting c by
// an integer rescales s exactly.  From these
//     lse = ln2 c + ln s,  log p(x) = ln2 (a x - c) - ln s,
//     H = -sum p log p = ln s - ln2 u / s.
// Elements count as at least kLeast, which keeps masked ones (-inf, or the
// type's lowest value) finite: they add 2^-huge = 0 to both sums.  A row for
// which this does not hold a sum (only masked elements, NaN, infinities,
// values past +-1e6 / scale) is summed again by careful_row().
//
// What bounds these kernels is the rate at which instructions issue as much as
// memory: a bf16 element arrives in 1/8 ns an SM, in which four schedulers
// issue about 7 instructions for 32 of them.  So maxima and the bound by kLeast
// work on packed pairs, and products and sums on pairs of binary32.
#pragma once

#include <algorithm>
#include <type_traits>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

// Four blocks of 256 threads share an SM, each thread with 8 chunks of 16 bytes
// in flight: 128 KiB an SM when all of them wait, and blocks small enough that
// some load while others reduce.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFlight = 8;
constexpr int kResident = 4;
constexpr int kNarrow = 64;                // threads of a block where rows are many and short
constexpr float kLeast = -1e12f;
constexpr float kLeastExponent = -1048576.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DT> struct Chunk {  // 16 bytes of a row
    static constexpr int kElems = 16 / ElemOf<DT>::kBytes;
    uint32_t w[4];
};
template <int DT> __device__ __forceinline__ void unpack(const Chunk<DT> &r, float (&f)[Chunk<DT>::kElems]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == DT_F32) {
            f[j] = __uint_as_float(r.w[j]);
        } else {
            const float2 p = widen<DT>(r.w[j]);
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        }
    }
}
// A word of masked elements.
template <int DT> __device__ __forceinline__ uint32_t masked_word() {
    return DT == DT_F32 ? 0xff800000u : DT == DT_F16 ? 0xfc00fc00u : 0xff80ff80u;
}
template <int DT> __device__ __forceinline__ Chunk<DT> masked_chunk() {
    return Chunk<DT>{{masked_word<DT>(), masked_word<DT>(), masked_word<DT>(), masked_word<DT>()}};
}
// Largest of two words, element by element, NaN kept.
template <int DT> __device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (DT == DT_F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else if constexpr (DT == DT_F16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int DT> __device__ __forceinline__ float max_of_word(uint32_t w) {
    if constexpr (DT == DT_F32) return __uint_as_float(w);
    else {
        const float2 p = widen<DT>(w);
        return max_nan(p.x, p.y);
    }
}
// The pair of elements in words w (and v for binary32), at least kLeast each.
// bfloat16: the bound is applied to the packed pair, as -1e12 rounded to it.
template <int DT> __device__ __forceinline__ float2 bounded(uint32_t w, uint32_t v) {
    if constexpr (DT == DT_F32) {
        return make_float2(fmaxf(__uint_as_float(w), kLeast), fmaxf(__uint_as_float(v), kLeast));
    } else if constexpr (DT == DT_F16) {
        const float2 p = widen<DT>(w);
        return make_float2(fmaxf(p.x, kLeast), fmaxf(p.y, kLeast));
    } else {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0xd369d369u));
        return widen<DT>(d);
    }
}
// Pair j of a chunk: 4 pairs of 16-bit elements, 2 of binary32.  Unbounded
// masked elements have t = -inf and 2^t = 0; only a product with t needs the
// bound.
template <int DT> struct Pairs { static constexpr int kCount = DT == DT_F32 ? 2 : 4; };
template <int DT, bool BOUNDED> __device__ __forceinline__ float2 pair_at(const Chunk<DT> &r, int j) {
    if constexpr (DT == DT_F32) {
        if constexpr (BOUNDED) return bounded<DT>(r.w[2 * j], r.w[2 * j + 1]);
        else return make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
    } else {
        if constexpr (BOUNDED) return bounded<DT>(r.w[j], 0u);
        else return widen<DT>(r.w[j]);
    }
}

// How a launch splits its rows: 2^shift blocks a row, a cluster of them where
// they work together, each with `each` chunks (the last with the rest).
struct Split {
    int shift, each;
    __host__ __device__ __forceinline__ int blocks() const { return 1 << shift; }
};
// The whole row to one block.
__device__ __forceinline__ Split unsplit() { return {0, INT32_MAX}; }

// A block's share of a row: whole 16-byte chunks from element `head` on, and
// the single elements before the first (block 0) and after the last chunk
// (the last block).  Rows may start anywhere.
template <int DT> struct Share {
    using T = typename ElemOf<DT>::type;
    static constexpr int V = Chunk<DT>::kElems;
    const T *row;
    int cols, head;
    int first, end;        // chunks of this block
    int singles, tail0;    // single elements: [0, n_head) and [tail0, cols)
    int n_head;
    __device__ __forceinline__ Share(const void *p, int cols_, int block, Split split) {
        row = static_cast<const T *>(p);
        cols = cols_;
        const int past = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16) / ElemOf<DT>::kBytes;
        head = min((V - past) % V, cols);
        const int chunks = (cols - head) / V;
        // each * blocks may be past 2^31 only where each is at least chunks
        first = block == 0 ? 0 : min(static_cast<int>(min(static_cast<int64_t>(block) * split.each, int64_t(INT32_MAX))), chunks);
        end = split.each >= chunks - first ? chunks : first + split.each;
        n_head = block == 0 ? head : 0;
        tail0 = head + chunks * V;
        singles = n_head + (block == split.blocks() - 1 ? cols - tail0 : 0);
    }
    __device__ __forceinline__ int column(int chunk, int j) const { return head + chunk * V + j; }
    // the column of single element k < singles
    __device__ __forceinline__ int single(int k) const { return k < n_head ? k : tail0 + k - n_head; }
    __device__ __forceinline__ bool holds(int col) const {
        return (col >= head + first * V && col < head + end * V) || col < n_head ||
               (col >= tail0 && singles > n_head);
    }
    __device__ __forceinline__ Chunk<DT> chunk(int c) const {
        const Vec<16> v = ld<16>(row + head + static_cast<int64_t>(c) * V);
        return Chunk<DT>{{v.w[0], v.w[1], v.w[2], v.w[3]}};
    }
    __device__ __forceinline__ float at(int col) const {
        if constexpr (DT == DT_F32) return __uint_as_float(ld<4>(row + col).w[0]);
        else return elem_to_f32<DT>(ld<2>(row + col).h);
    }
};

// ---------------------------------------------------------------- sums

struct Sums {
    float c, s, u;  // u where the entropy is wanted, else 0
};
__device__ __forceinline__ Sums no_sums() { return {kLeastExponent, 0.0f, 0.0f}; }

template <bool ENTROPY> __device__ __forceinline__ void move_to(Sums &v, float c) {
    const float d = v.c - c;  // an integer <= 0
    const float f = ex2(d);
    if (ENTROPY) v.u = f * fmaf(v.s, d, v.u);
    v.s *= f;
    v.c = c;
}
// One element.
template <bool ENTROPY> __device__ __forceinline__ void add_element(Sums &v, float x, float a) {
    const float c = fmaxf(ceilf(x * a), kLeastExponent);
    if (c > v.c) move_to<ENTROPY>(v, c);
    const float t = x < kLeast ? kLeast * a - v.c : fmaf(x, a, -v.c), e = ex2(t);  // NaN stays
    v.s += e;
    if (ENTROPY) v.u = fmaf(e, t, v.u);
}
// A thread's chunks; sums in two lanes of a pair each.  Returns the largest element, or NaN.
struct PairSums {
    float c;
    float2 s, u;
};
template <int DT, bool ENTROPY, int N>
__device__ __forceinline__ float add_chunks(PairSums &v, const Chunk<DT> (&r)[N], float a) {
    uint32_t m = max_words<DT>(r[0].w[0], r[0].w[1]);
    m = max_words<DT>(m, max_words<DT>(r[0].w[2], r[0].w[3]));
#pragma unroll
    for (int k = 1; k < N; ++k)
        m = max_words<DT>(m, max_words<DT>(max_words<DT>(r[k].w[0], r[k].w[1]), max_words<DT>(r[k].w[2], r[k].w[3])));
    const float top = max_of_word<DT>(m);
    const float c = fmaxf(ceilf(top * a), kLeastExponent);
    if (ENTROPY && top != top) v.s = both(top);  // the bound of the pairs below would lose a NaN
    if (c > v.c) {
        const float d = v.c - c, f = ex2(d);
        if (ENTROPY) v.u = mul2(both(f), fma2(v.s, both(d), v.u));
        v.s = mul2(both(f), v.s);
        v.c = c;
    }
    const float2 scale = both(a), shift = both(-v.c);
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int j = 0; j < Pairs<DT>::kCount; ++j) {
            const float2 t = fma2(pair_at<DT, ENTROPY>(r[k], j), scale, shift);
            const float2 e = make_float2(ex2(t.x), ex2(t.y));
            v.s = add2(v.s, e);
            if (ENTROPY) v.u = fma2(e, t, v.u);
        }
    }
    return top;
}
// The sums of the first LANES lanes together (all others' are no_sums()), to
// all lanes: the largest exponent first, then plain sums.  Every lane adds the
// same pairs, so all get the same bits.
template <int LANES, bool ENTROPY> __device__ __forceinline__ Sums warp_sums(Sums v) {
    float c = v.c;
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) c = fmaxf(c, __shfl_xor_sync(kAllLanes, c, d));
    if (LANES < 32) c = __shfl_sync(kAllLanes, c, 0);
    move_to<ENTROPY>(v, c);
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) {
        v.s += __shfl_xor_sync(kAllLanes, v.s, d);
        if (ENTROPY) v.u += __shfl_xor_sync(kAllLanes, v.u, d);
    }
    if (LANES < 32) {
        v.s = __shfl_sync(kAllLanes, v.s, 0);
        if (ENTROPY) v.u = __shfl_sync(kAllLanes, v.u, 0);
    }
    return v;
}
// Sums of the block, to all its threads, from its WARPS warps' in `part`.
template <int WARPS, bool ENTROPY> __device__ __forceinline__ Sums sums_of_warps(const Sums *part) {
    const int lane = threadIdx.x & 31;
    return warp_sums<WARPS, ENTROPY>(lane < WARPS ? part[lane] : no_sums());
}
// The sums of all blocks of the cluster, to every thread: lane b reads block b's.
template <bool ENTROPY> __device__ __forceinline__ Sums cluster_sums(const Sums *mine, int blocks) {
    const int lane = threadIdx.x & 31;
    return warp_sums<8, ENTROPY>(lane < blocks ? *in_block(mine, lane) : no_sums());
}

// What a row's elements are compared with: log p(x) = ln2 (a x - c) - log_s,
// or, where `careful`, scale (x - top) - log_s.
struct RowSum {
    float c, log_s, inv_s, u_over_s, top;
    bool careful;
};
__device__ __forceinline__ float lse_of(const RowSum &r, float scale) {
    return r.careful ? fmaf(r.top, scale, r.log_s) : fmaf(r.c, kLn2, r.log_s);
}
// At most 0, where rounding would leave a little more; NaN stays.
__device__ __forceinline__ float logp_of(const RowSum &r, float x, float a, float scale) {
    float v;
    if (r.careful) v = x == kNegInf ? kNegInf : (x - r.top) * scale - r.log_s;
    else if (x < kLeast) v = fmaf(x, scale, -lse_of(r, scale));  // a x may be beyond binary32 where scale x is not
    else v = fmaf(kLn2, fmaf(x, a, -r.c), -r.log_s);
    return v > 0.0f ? 0.0f : v;
}
__device__ __forceinline__ float entropy_of(const RowSum &r) {
    const float h = fmaf(-kLn2, r.u_over_s, r.log_s);
    return h < 0.0f ? 0.0f : h;
}

// The sums of a whole row, relative to its largest element and without the
// shortcuts above: rows of masked elements alone, of NaN or infinity, or of
// huge values.  An empty row (no element above -inf) has lse -inf, entropy 0;
// NaN or +inf make everything NaN.  Every thread of the block takes part.
template <int DT> __device__ __noinline__ RowSum careful_row(const void *row, int cols, float a, float *part) {
    const Share<DT> all(row, cols, 0, unsplit());
    const int warps = blockDim.x >> 5;
    float top = kNegInf, s = 0.0f, u = 0.0f;
    for (int k = threadIdx.x; k < cols; k += blockDim.x) top = max_nan(top, all.at(k));
    __syncthreads();
    top = block_max_nan(top, warps, part, kNegInf);
    RowSum r = {0.0f, 0.0f, 0.0f, 0.0f, top, true};
    if (top == kNegInf) return r;
    for (int k = threadIdx.x; k < cols; k += blockDim.x) {
        const float t = fmaxf((all.at(k) - top) * a, -200.0f);
        const float e = ex2(t);
        s += e;
        u = fmaf(e, t, u);
    }
    if (!(top < -kNegInf)) s = top - top;  // NaN
    __syncthreads();
    s = block_sum(s, warps, part);
    __syncthreads();
    u = block_sum(u, warps, part);
    r.log_s = logf(s);
    r.inv_s = 1.0f / s;
    r.u_over_s = u / s;
    return r;
}
// A sum that is 0, infinite or NaN says that the shortcuts do not hold for the
// row: an infinity has c infinite and so a NaN, too.  The branch holds barriers,
// so it goes by sums that every thread of the block has the same bits of: u only
// where warp_sums() added it up.
template <int DT, bool ENTROPY>
__device__ __forceinline__ RowSum finish_row(const Sums &v, const void *row, int cols, float a, float *part) {
    if (v.s > 0.0f && v.s < 1e37f && (!ENTROPY || fabsf(v.u) < 1e37f)) {
        const float inv_s = 1.0f / v.s;
        return {v.c, logf(v.s), inv_s, ENTROPY ? v.u * inv_s : 0.0f, 0.0f, false};
    }
    return careful_row<DT>(row, cols, a, part);
}

// ---------------------------------------------------------------- top alternatives
//
// The largest `k` elements, equal ones by index.  Any k-th largest of disjoint
// groups' maxima is a bound that at least k elements reach, and not many more:
// of 32 groups, about 31 elements for k = 20.  The first turn gives a bound for
// the rest of the row, the first two and four turns better ones; elements that
// reach it are collected while the row streams past (a hundred or so of a row
// in no particular order).  At the end the groups' maxima over the whole row
// give the last bound, and the few that reach it are ranked.  Where more than
// kCandidates are collected, exact_top finds the k-th value by bisection
// instead.

constexpr int kCandidates = 2048;
constexpr int kFew = 512;
constexpr int kManyGroups = 128;    // of two lanes each, for k past kFewGroupsTop
constexpr int kFewGroups = 32;      // of eight
constexpr int kFewGroupsTop = 24;
constexpr int kBounds = 4;          // times that a bound is found
constexpr int kRankedAtOnce = 128;  // candidates that are compared with each other without a bound

struct alignas(8) Candidate {
    float x;
    int id;
};
__device__ __forceinline__ bool before(const Candidate &a, const Candidate &b) {
    return a.x > b.x || (a.x == b.x && a.id < b.id);
}

struct TopShared {  // every array at a multiple of 16 bytes
    alignas(16) float group[kManyGroups];
    alignas(16) Candidate list[kCandidates];
    alignas(16) Candidate few[kFew];
    alignas(16) Candidate best[kMostTop];  // ids of -1 at the end where there are fewer
    alignas(16) float bound;
    int count, few_count;
};

__device__ __forceinline__ void collect(TopShared &t, float x, int id) {
    const int at = atomicAdd(&t.count, 1);
    if (at < kCandidates) t.list[at] = {x, id};
}

// The elements of a chunk that reach the bound.  Out of line: it is rarely
// run, and 8 copies of it in the loop would crowd the instruction cache.
template <int DT>
__device__ __noinline__ void collect_chunk(TopShared &t, uint4 w, int col, float bound) {
    constexpr int V = Chunk<DT>::kElems;
    const Chunk<DT> r = {{w.x, w.y, w.z, w.w}};
    float f[V];
    unpack<DT>(r, f);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (f[j] >= bound && f[j] > kNegInf) collect(t, f[j], col + j);
}

// The k best of n entries into best[0 .. k): the rank of an entry is the
// number of entries before it.
template <int THREADS>
__device__ __forceinline__ void rank_list(const Candidate *list, int n, int k, Candidate *best) {
    for (int i = n + static_cast<int>(threadIdx.x); i < k; i += THREADS) best[i] = {kNegInf, -1};
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const Candidate mine = list[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += before(list[j], mine) ? 1 : 0;
        if (rank < k) best[rank] = mine;
    }
}

// The bound that the largest elements which the threads have seen give.  Every
// thread of the block takes part; what else was written to shared memory is
// visible after it.  The calls of a kernel use different slots: a warp may be in
// the next while another still reads for the last.
template <int THREADS> __device__ __forceinline__ float find_bound(TopShared &t, float mine, int k, int slot) {
    static_assert(kManyGroups * 2 == kThreads && kFewGroups * 8 == kThreads && kManyGroups >= kMostTop &&
                      kFewGroups >= kFewGroupsTop && kBounds * kFewGroups <= kManyGroups, "groups of lanes, and a k-th largest of them");
    static_assert(THREADS == kThreads || THREADS == kNarrow, "narrow blocks have few groups alone");
    const int lane = threadIdx.x & 31;
    mine = fmaxf(mine, __shfl_xor_sync(kAllLanes, mine, 1));
    if (THREADS == kNarrow || k <= kFewGroupsTop) {
        constexpr int kLanes = THREADS / kFewGroups;
#pragma unroll
        for (int d = 2; d < kLanes; d *= 2) mine = fmaxf(mine, __shfl_xor_sync(kAllLanes, mine, d));
        if (lane % kLanes == 0) t.group[slot * kFewGroups + threadIdx.x / kLanes] = mine;
        __syncthreads();
        float v = t.group[slot * kFewGroups + lane];  // each warp sorts them, the largest first
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int d = size / 2; d > 0; d /= 2) {
                const float o = __shfl_xor_sync(kAllLanes, v, d);
                v = ((lane & d) == 0) == ((lane & size) == 0) ? fmaxf(v, o) : fminf(v, o);
            }
        return __shfl_sync(kAllLanes, v, k - 1);
    }
    if ((lane & 1) == 0) t.group[threadIdx.x >> 1] = mine;
    __syncthreads();
    if (threadIdx.x < kManyGroups) {
        const float v = t.group[threadIdx.x];
        const int me = threadIdx.x;
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < kManyGroups; j += 4) {
            const float4 g = *reinterpret_cast<const float4 *>(t.group + j);
            rank += (g.x > v || (g.x == v && j < me)) + (g.y > v || (g.y == v && j + 1 < me)) +
                    (g.z > v || (g.z == v && j + 2 < me)) + (g.w > v || (g.w == v && j + 3 < me));
        }
        if (rank == k - 1) t.bound = v;
    }
    __syncthreads();
    return t.bound;
}

// The k best of the list's entries that reach the bound, into best.
template <int THREADS> __device__ __forceinline__ void rank_few(TopShared &t, float bound, int k) {
    const int n = t.count;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const Candidate c = t.list[i];
        if (c.x >= bound) {
            const int at = atomicAdd(&t.few_count, 1);
            if (at < kFew) t.few[at] = c;
        }
    }
    __syncthreads();
    const int few = t.few_count;
    if (few <= kFew) rank_list<THREADS>(t.few, few, k, t.best);
    else rank_list<THREADS>(t.list, n, k, t.best);
}

// Order of binary32 values as unsigned integers (-0 and +0 the same).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

// The exact k best of the block's share, however many elements tie.
template <int DT> __device__ __noinline__ void exact_top(TopShared &t, const Share<DT> &sh, int k, float bound) {
    constexpr int V = Chunk<DT>::kElems;
    auto count_from = [&](uint32_t least) {  // elements of the share from `least` on
        int n = 0;
        for (int c = sh.first + threadIdx.x; c < sh.end; c += static_cast<int>(blockDim.x)) {
            float f[V];
            unpack<DT>(sh.chunk(c), f);
#pragma unroll
            for (int j = 0; j < V; ++j) n += f[j] == f[j] && order_of(f[j]) >= least;
        }
        if (static_cast<int>(threadIdx.x) < sh.singles) {
            const float x = sh.at(sh.single(threadIdx.x));
            n += x == x && order_of(x) >= least;
        }
        __syncthreads();
        if (threadIdx.x == 0) t.count = 0;
        __syncthreads();
        n = __reduce_add_sync(kAllLanes, n);
        if ((threadIdx.x & 31) == 0) atomicAdd(&t.count, n);
        __syncthreads();
        return t.count;
    };
    // the k-th largest value: the largest `least` that k elements reach, which
    // the bound is known to be; often no more than that lie above it
    uint32_t lo = order_of(bound), hi = 0xffffffffu;
    for (uint32_t probe = lo + 1; lo < hi; probe = lo + (hi - lo) / 2 + 1) {
        if (count_from(probe) >= k) lo = probe;
        else hi = probe - 1;
    }
    // larger ones (fewer than k), then the first of those equal to it, in order
    __syncthreads();
    if (threadIdx.x == 0) t.count = 0;
    __syncthreads();
    for (int c = sh.first + threadIdx.x; c < sh.end; c += static_cast<int>(blockDim.x)) {
        float f[V];
        unpack<DT>(sh.chunk(c), f);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (f[j] == f[j] && order_of(f[j]) > lo) collect(t, f[j], sh.column(c, j));
    }
    if (static_cast<int>(threadIdx.x) < sh.singles) {
        const int col = sh.single(threadIdx.x);
        const float x = sh.at(col);
        if (x == x && order_of(x) > lo) collect(t, x, col);
    }
    __syncthreads();
    // A column order walk: the single elements before the chunks, the chunks, those after.
    const int begin = sh.n_head > 0 ? 0 : sh.column(sh.first, 0);
    const int stop = sh.singles > sh.n_head ? sh.cols : sh.column(sh.end, 0);
    for (int base = begin; base < stop; base += static_cast<int>(blockDim.x)) {
        const int taken = t.count;
        if (taken >= k) break;
        const int col = base + threadIdx.x;
        const float x = col < stop ? sh.at(col) : kNegInf;
        const bool equal = col < stop && x == x && order_of(x) == lo;
        const unsigned in_warp = __ballot_sync(kAllLanes, equal);
        int *warp_counts = reinterpret_cast<int *>(t.group);
        if ((threadIdx.x & 31) == 0) warp_counts[threadIdx.x >> 5] = __popc(in_warp);
        __syncthreads();
        int place = taken + __popc(in_warp & ((1u << (threadIdx.x & 31)) - 1u));
        for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) place += warp_counts[w];
        if (equal && place < k) t.list[place] = {x, col};
        __syncthreads();
        if (threadIdx.x == 0) {
            int n = taken;
            for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) n += warp_counts[w];
            t.count = min(n, k);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the pass over a row

// A thread's sums out of its pairs, and one of the single elements.
template <int DT, bool ENTROPY>
__device__ __forceinline__ Sums finished(const PairSums &v, bool single, float one, float a) {
    Sums sums = {v.c, v.s.x + v.s.y, ENTROPY ? v.u.x + v.u.y : 0.0f};
    if (single) add_element<ENTROPY>(sums, one, a);
    return sums;
}

// The thread's chunks of the turn that begins at its chunk c0; those past the share are masked.
template <int DT, int THREADS = kThreads>
__device__ __forceinline__ void load_turn(const Share<DT> &sh, int c0, Chunk<DT> (&r)[kFlight]) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
        r[u] = c0 + u * THREADS < sh.end ? sh.chunk(c0 + u * THREADS) : masked_chunk<DT>();
}

// A thread's sums over the block's share of a row; with TOP, the elements
// that may be among the k best are in t's list when the block next synchronises.
// r comes with the first turn loaded; largest is the thread's largest element,
// bound the last one found.
template <int DT, bool ENTROPY, bool TOP, int THREADS = kThreads>
__device__ __forceinline__ Sums pass_over(const Share<DT> &sh, float a, TopShared *t, int k, Chunk<DT> (&r)[kFlight],
                                          float &largest, float &bound) {
    PairSums v = {kLeastExponent, both(0.0f), both(0.0f)};
    const bool single = static_cast<int>(threadIdx.x) < sh.singles;
    const float one = single ? sh.at(sh.single(threadIdx.x)) : kNegInf;
    largest = one;
    bound = kNegInf;
    int c0 = sh.first + static_cast<int>(threadIdx.x);
    for (int turn = 0;; ++turn) {
        const float top = add_chunks<DT, ENTROPY>(v, r, a);
        if constexpr (TOP) {
            largest = fmaxf(largest, top);
            if (turn == 0 && threadIdx.x == 0) t->count = t->few_count = 0;
            if (turn == 0 || turn == 1 || turn == 3) {
                bound = find_bound<THREADS>(*t, largest, k, (turn + 1) / 2);
                if (turn == 0 && one >= bound && one > kNegInf) collect(*t, one, sh.single(threadIdx.x));
            }
            if (top >= bound && top > kNegInf) {
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    // few of the chunks that get here hold a candidate
                    const uint32_t m = max_words<DT>(max_words<DT>(r[u].w[0], r[u].w[1]), max_words<DT>(r[u].w[2], r[u].w[3]));
                    if (max_of_word<DT>(m) >= bound)
                        collect_chunk<DT>(*t, make_uint4(r[u].w[0], r[u].w[1], r[u].w[2], r[u].w[3]),
                                          sh.column(c0 + u * THREADS, 0), bound);
                }
            }
        }
        c0 += kFlight * THREADS;
        if (c0 - static_cast<int>(threadIdx.x) >= sh.end) break;
        load_turn<DT, THREADS>(sh, c0, r);
    }
    return finished<DT, ENTROPY>(v, single, one, a);
}

// ---------------------------------------------------------------- log probabilities

// A row to a cluster of `blocks` blocks (one block: no cluster); the first
// puts the parts together.  2048 rows of 131072 bf16 with the 5 best take 101 us
// (5.3 TB/s, floor 79), as much for the instructions as for memory; 5 rows with
// the 20 best 11 us, all latency (3.3 us without alternatives).
template <int DT, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, kResident * kThreads / THREADS) logprob_kernel(LogprobArgs a, Split split) {
    enter_grid();
    __shared__ Sums part[THREADS / 32];
    __shared__ Sums mine;
    __shared__ float fpart[32];
    __shared__ typename std::conditional<TOP, TopShared, int>::type top_store;
    TopShared *t = nullptr;
    if constexpr (TOP) t = &top_store;
    const int blocks = split.blocks(), block = blockIdx.x & (blocks - 1);
    const int64_t row = blockIdx.x >> split.shift;
    const void *logits = row_of<DT>(a.logits, row, a.stride);
    const Share<DT> sh(logits, a.cols, block, split);
    const float ax = a.scale * kLog2e;
    Chunk<DT> r_chunks[kFlight];
    load_turn<DT, THREADS>(sh, sh.first + static_cast<int>(threadIdx.x), r_chunks);
    // the token's logit, on its way while the row is
    int64_t token = -1;
    typename ElemOf<DT>::type chosen = 0;
    if (threadIdx.x == 0 && a.logp && block == 0) token = token_at(a.tokens, a.i64, row);
    const bool given = token >= 0 && token < a.cols;
    if (given) chosen = sh.row[token];
    float largest, bound;
    Sums v = warp_sums<32, true>(pass_over<DT, true, TOP, THREADS>(sh, ax, t, a.top, r_chunks, largest, bound));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    // After a single turn the bound is of the whole share already, and all candidates reach it.
    const bool once = sh.end - sh.first <= kFlight * THREADS;
    if (TOP && !once) bound = find_bound<THREADS>(*t, largest, a.top, kBounds - 1);
    else __syncthreads();
    // every candidate is in the list now
    v = sums_of_warps<THREADS / 32, true>(part);
    if constexpr (TOP) {
        const int n = t->count;
        bool all_reach = once;
        if (n > kCandidates) {
            exact_top<DT>(*t, sh, a.top, bound);
        } else if (bound == kNegInf && n > kRankedAtOnce) {
            // fewer groups than k have an element (a short row, or one masked but for a short part): the same
            // bound over the list, spread over all threads
            float most = kNegInf;
            for (int i = threadIdx.x; i < n; i += THREADS) most = fmaxf(most, t->list[i].x);
            bound = find_bound<THREADS>(*t, most, a.top, 0);
            all_reach = false;
        }
        if (all_reach) rank_list<THREADS>(t->list, t->count, a.top, t->best);
        else rank_few<THREADS>(*t, bound, a.top);
    }
    if (blocks > 1) {
        if (threadIdx.x == 0) mine = v;
        if constexpr (TOP) {
            __syncthreads();
            if (threadIdx.x == 0) t->count = 0;
        }
        cluster_sync();
        if (block == 0) {
            v = cluster_sums<true>(&mine, blocks);
            if constexpr (TOP) {
                // Of every block's best ceil(k / blocks) are at least k, all of which reach the least of them; and
                // every block's k-th best is reached by k.
                const int lane = threadIdx.x & 31, each = (a.top + blocks - 1) / blocks;
                float low = -kNegInf, high = kNegInf;
                if (lane < blocks) {
                    const Candidate *its = in_block(t->best, lane);
                    low = its[each - 1].x;
                    high = its[a.top - 1].x;
                }
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) {
                    low = fminf(low, __shfl_xor_sync(kAllLanes, low, d));
                    high = fmaxf(high, __shfl_xor_sync(kAllLanes, high, d));
                }
                bound = fmaxf(__shfl_sync(kAllLanes, low, 0), __shfl_sync(kAllLanes, high, 0));
                for (int i = threadIdx.x; i < blocks * a.top; i += THREADS) {
                    const Candidate c = in_block(t->best, i / a.top)[i % a.top];
                    if (c.id >= 0 && c.x >= bound) collect(*t, c.x, c.id);
                }
                __syncthreads();
                rank_list<THREADS>(t->list, t->count, a.top, t->best);
            }
        }
        cluster_sync();  // no block leaves while its shared memory is read
        if (block != 0) return;
    }
    if (TOP) __syncthreads();  // best is written
    const RowSum r = finish_row<DT, true>(v, logits, a.cols, ax, fpart);
    if (threadIdx.x == 0) {
        const bool empty = r.careful && r.top == kNegInf;
        if (a.lse) a.lse[row] = empty ? kNegInf : lse_of(r, a.scale);
        if (a.entropy) a.entropy[row] = empty ? 0.0f : entropy_of(r);
        if (a.logp) a.logp[row] = !given ? 0.0f : empty ? kNegInf : logp_of(r, elem_to_f32<DT>(chosen), ax, a.scale);
    }
    if constexpr (TOP) {
        for (int i = threadIdx.x; i < a.top; i += THREADS) {
            const Candidate b = t->best[i];
            const float logp = b.id < 0 ? kNegInf : logp_of(r, b.x, ax, a.scale);
            a.top_ids[row * a.top + i] = r.log_s == r.log_s ? b.id : -1;  // a row with NaN has no order
            a.top_logp[row * a.top + i] = r.log_s == r.log_s ? logp : r.log_s;
        }
    }
}

// ---------------------------------------------------------------- gradients

// p(x) = weight * 2^(a x - c) with an integer c, or, careful, weight * 2^(a (x - top)).
struct Weights {
    float c, weight, top;
    bool careful;
};
__device__ __forceinline__ float p_of(const Weights &w, float x, float a) {
    if (w.careful) return w.weight * ex2(fmaxf((x - w.top) * a, -200.0f));
    return w.weight * ex2(fmaf(fmaxf(x, kLeast), a, -w.c));
}
// A saved lse, rounded to binary32, keeps a row's normalisation to half of its
// own last place, which at 4096 makes p off by up to 2.4e-4 of itself, at 5e5 by 1.5e-2, and
// from about 1e7 on the log of the number of elements that share the row is lost.
// Rows from kMostLse on are summed again (careful_row).
constexpr float kMostLse = 4096.0f;
__device__ __forceinline__ bool lse_holds(float lse) { return fabsf(lse) < kMostLse || lse != lse; }
// From a saved lse that holds: c is lse * log2(e) rounded to an integer, weight 2^ of
// what is left, formed with the two parts of log2(e) (Cody and Waite's reduction: a
// constant as the binary32 next to it and what that leaves).
__device__ __forceinline__ Weights weights_of(float lse) {
    const float c = rintf(lse * kLog2e);
    const float left = fmaf(lse, kLog2e, -c) + lse * 1.9259629911266175e-8f;
    if (lse == lse) return {c, ex2(-left), 0.0f, false};
    return {0.0f, lse, 0.0f, true};  // NaN everywhere
}

// A row's gradient but for single places: d(x) = p(x) (g - dent (log p(x) + H)).
// With e = 2^t, t = a x - c, and log p = ln2 t + (ln2 c - lse):
//     d = e (A + B t),  A = weight (g - dent (H + ln2 c - lse)),  B = -weight dent ln2.
// Without an entropy term (lse and H 0 there) d = e A.  Careful: lse is relative to top.
struct RowGrad {
    Weights w;
    float g, dent, lse, entropy, A, B;
};
__device__ __forceinline__ RowGrad row_grad(const Weights &w, float g, float dent, float lse, float entropy) {
    const float offset = fmaf(w.c, kLn2, w.c * -1.9046543e-9f) - lse;  // ln2 in two parts, after Cody and Waite
    return {w, g, dent, lse, entropy, w.weight * fmaf(-dent, entropy + offset, g), w.weight * -dent * kLn2};
}
template <bool ENTROPY> __device__ __forceinline__ float grad_of(const RowGrad &r, float x, float a, float scale) {
    if (r.w.careful) {
        const float p = p_of(r.w, x, a);
        if constexpr (!ENTROPY) return p * r.g;
        const float logp = fmaf(x - r.w.top, scale, -r.lse);
        return p * fmaf(-r.dent, p > 0.0f ? logp + r.entropy : 0.0f, r.g);
    }
    const float t = fmaf(fmaxf(x, kLeast), a, -r.w.c);
    return ex2(t) * (ENTROPY ? fmaf(r.B, t, r.A) : r.A);
}
template <int DT> __device__ __forceinline__ void store_one(void *row, int col, float x) {
    using T = typename ElemOf<DT>::type;
    static_cast<T *>(row)[col] = f32_to_elem<DT>(x);
}

// Rows whose p is formed the careful way.
template <int DT, bool ENTROPY>
__device__ __noinline__ void write_grad_slowly(const Share<DT> &sh, void *out, const RowGrad &r, float a, float scale,
                                               int threads = kThreads) {
    constexpr int V = Chunk<DT>::kElems;
    for (int c = sh.first * V + static_cast<int>(threadIdx.x); c < sh.end * V; c += threads)
        store_one<DT>(out, sh.head + c, grad_of<ENTROPY>(r, sh.at(sh.head + c), a, scale));
    if (static_cast<int>(threadIdx.x) < sh.singles) {
        const int col = sh.single(threadIdx.x);
        store_one<DT>(out, col, grad_of<ENTROPY>(r, sh.at(col), a, scale));
    }
}

// Zeros for the block's share, whatever the logits are.
template <int DT> __device__ __forceinline__ void write_zeros(void *out_row, int cols, int block, Split split,
                                                               int threads = kThreads) {
    const Share<DT> sh(out_row, cols, block, split);
    typename ElemOf<DT>::type *out = static_cast<typename ElemOf<DT>::type *>(out_row);
    const Vec<16> zero = {};
    for (int c = sh.first + static_cast<int>(threadIdx.x); c < sh.end; c += threads) st<16>(out + sh.column(c, 0), zero);
    if (static_cast<int>(threadIdx.x) < sh.singles) store_one<DT>(out, sh.single(threadIdx.x), 0.0f);
}

// The gradient of a chunk, by the formula above.
template <int DT, bool ENTROPY> struct ChunkGrad {
    float2 slope, shift, A, B;
    __device__ __forceinline__ ChunkGrad(const RowGrad &g, float a)
        : slope(both(a)), shift(both(-g.w.c)), A(both(g.A)), B(both(g.B)) {}
    __device__ __forceinline__ Vec<16> operator()(const Chunk<DT> &r) const {
        Vec<16> o;
#pragma unroll
        for (int j = 0; j < Pairs<DT>::kCount; ++j) {
            const float2 t = fma2(pair_at<DT, ENTROPY>(r, j), slope, shift);
            float2 d = make_float2(ex2(t.x), ex2(t.y));
            d = mul2(d, ENTROPY ? fma2(B, t, A) : A);
            if constexpr (DT == DT_F32) {
                o.w[2 * j] = __float_as_uint(d.x);
                o.w[2 * j + 1] = __float_as_uint(d.y);
            } else {
                o.w[j] = narrow<DT>(d);
            }
        }
        return o;
    }
};
// Bytes that an output row lies past the input row's place between multiples
// of 16 bytes: chunks of both are 16-byte aligned where it is 0.
template <int DT> __device__ __forceinline__ int bytes_apart(const void *out, const Share<DT> &sh) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(sh.row)) % 16);
}
// Stores a chunk's gradient.  Where the rows lie apart, a warp that stores 32
// chunks in a row (`whole`, the same in all its lanes) shifts them by `apart`
// bytes: a lane stores the end of the chunk of the lane before and the start of
// its own to the aligned 16 bytes that they share, and the first and the last
// lane the two ends left over, element by element.  Where a warp has fewer
// chunks it stores elements.  1565 rows of 50605 f16, 2 bytes apart, take 69 us
// (floor 47); with elements alone 200.
template <int DT>
__device__ __forceinline__ void store_chunk(typename ElemOf<DT>::type *to, const Vec<16> &d, int apart, bool whole) {
    constexpr int B = ElemOf<DT>::kBytes;
    if (apart == 0) {
        st<16>(to, d);
        return;
    }
    int first = 0, last = 16;  // bytes that go as elements
    if (whole) {
        const int lane = threadIdx.x & 31, from = 16 - apart;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = __shfl_up_sync(kAllLanes, d.w[j], 1);
            w[j + 4] = d.w[j];
        }
#pragma unroll
        for (int j = 0; j < 6; ++j) w[j] = from & 8 ? w[j + 2] : w[j];
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = from & 4 ? w[j + 1] : w[j];
        Vec<16> o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[j] = __funnelshift_r(w[j], w[j + 1], (from & 3) * 8);
        if (lane != 0) st<16>(reinterpret_cast<char *>(to) - apart, o);
        first = lane == 31 ? from : 0;
        last = lane == 0 ? from : lane == 31 ? 16 : 0;
    }
#pragma unroll
    for (int j = 0; j < 16 / B; ++j)
        if (j * B >= first && j * B < last) to[j] = static_cast<typename ElemOf<DT>::type>(d.w[j * B / 4] >> (j * B % 4 * 8));
}

// Writes the gradient of the block's share, which it reads (again).
template <int DT, bool ENTROPY, int THREADS = kThreads>
__device__ __forceinline__ void write_grad(const Share<DT> &sh, void *out_row, const RowGrad &g, float a, float scale) {
    using T = typename ElemOf<DT>::type;
    T *out = static_cast<T *>(out_row);
    const int apart = bytes_apart(out, sh), last_lane = 31 - static_cast<int>(threadIdx.x & 31);
    if (g.w.careful) {
        write_grad_slowly<DT, ENTROPY>(sh, out_row, g, a, scale, THREADS);
        return;
    }
    const ChunkGrad<DT, ENTROPY> grad(g, a);
    for (int c0 = sh.first + static_cast<int>(threadIdx.x); c0 < sh.end; c0 += kFlight * THREADS) {
        Chunk<DT> r[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (c0 + u * THREADS < sh.end) r[u] = sh.chunk(c0 + u * THREADS);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int c = c0 + u * THREADS;
            if (c >= sh.end) break;
            store_chunk<DT>(out + sh.column(c, 0), grad(r[u]), apart, c + last_lane < sh.end);
        }
    }
    if (static_cast<int>(threadIdx.x) < sh.singles) {
        const int col = sh.single(threadIdx.x);
        store_one<DT>(out, col, grad_of<ENTROPY>(g, sh.at(col), a, scale));
    }
}

// The block's share of dlogits = scale (dlogp (1_token - p) - dentropy p (log p + H)).
// lse: the row's, in careful form relative to its largest element.
template <int DT, bool ENTROPY>
__device__ __forceinline__ void write_logprob_grad(const LogprobGradArgs &a, const Split split, int64_t row, int block,
                                                   const Weights &w, float lse, int64_t token) {
    const Share<DT> sh(row_of<DT>(a.logits, row, a.stride), a.cols, block, split);
    void *out = row_of<DT>(a.dlogits, row, a.dstride);
    const float ax = a.scale * kLog2e;
    if (token >= a.cols) token = -1;
    const float dlogp = token >= 0 ? a.dlogp[row] : 0.0f;
    const RowGrad r = row_grad(w, -a.scale * dlogp, ENTROPY ? a.scale * a.dentropy[row] : 0.0f, ENTROPY ? lse : 0.0f,
                               ENTROPY ? a.entropy[row] : 0.0f);
    const bool here = token >= 0 && sh.holds(static_cast<int>(token));
    const float x = here ? sh.at(static_cast<int>(token)) : 0.0f;  // read before it may be overwritten
    if (here) __syncthreads();                                     // uniform: all threads have the same token
    write_grad<DT, ENTROPY>(sh, out, r, ax, a.scale);
    if (!here) return;
    __syncthreads();
    if (threadIdx.x == 0)
        store_one<DT>(out, static_cast<int>(token), grad_of<ENTROPY>(r, x, ax, a.scale) + a.scale * dlogp);
}

// Rows whose lse does not hold.  Out of line, all of it, so that nothing is kept
// in registers for it.
template <int DT, bool ENTROPY>
__device__ __noinline__ void resummed_grad(const LogprobGradArgs &a, Split split, int64_t row, int block, int64_t token,
                                           float *part) {
    const RowSum sum = careful_row<DT>(row_of<DT>(a.logits, row, a.stride), a.cols, a.scale * kLog2e, part);
    // in place: all blocks have read the row before any writes to it
    if (split.shift > 0 && a.dlogits == a.logits) cluster_sync();
    if (sum.top == kNegInf) write_zeros<DT>(row_of<DT>(a.dlogits, row, a.dstride), a.cols, block, split);
    else write_logprob_grad<DT, ENTROPY>(a, split, row, block, {0.0f, sum.inv_s, sum.top, true}, sum.log_s, token);
}

// The bound is memory: 1500 rows of 50001 f16 take 48 us (6.2 TB/s, floor 44).
template <int DT, bool ENTROPY>
__global__ void __launch_bounds__(kThreads, kResident)
    logprob_grad_kernel(const __grid_constant__ LogprobGradArgs a, Split split) {
    enter_grid();
    __shared__ float part[32];
    const int block = blockIdx.x & (split.blocks() - 1);
    const int64_t row = blockIdx.x >> split.shift;
    const int64_t token = a.dlogp ? token_at(a.tokens, a.i64, row) : -1;
    const float lse = a.lse[row];
    if (lse == kNegInf && a.scale <= 1.0f)  // an empty row: nothing depends on its logits
        write_zeros<DT>(row_of<DT>(a.dlogits, row, a.dstride), a.cols, block, split);
    else if (lse_holds(lse))
        write_logprob_grad<DT, ENTROPY>(a, split, row, block, weights_of(lse), lse, token);
    else  // past a scale of 1 the lse of a row of the type's lowest values may be -inf, too
        resummed_grad<DT, ENTROPY>(a, split, row, block, token, part);
}

// ---------------------------------------------------------------- launches

// Blocks a row: one where the rows alone fill the device or have up to 16384
// elements, up to a cluster of 8 where they are few; each with 4096 elements at
// least while SMs are idle, and with 16384 after that.  Splitting costs two cluster
// barriers and the joining of the parts: with the 5 best, 152 rows of 16384 bf16
// take 5.9 us whole and 8.2 us by 2 blocks, 5 rows of 32768 7.5 us by 8 blocks and
// 8.3 us by 2.  And no more blocks than fit at a time: clusters of 4 and 8 do not
// fill every SM of a partition of the device, so a tenth is left.  Of 65536
// elements, 134 rows by 4 blocks 11 us, by 8 (two waves) 20 us; 340 rows by 1 block
// 19 us, by 2 23 us; 76 rows by 8, which all but fill the device, 16 us.
inline int split_shift(int64_t rows, int cols, int sms) {
    const int64_t fit = kResident * static_cast<int64_t>(sms);
    int shift = 0;
    if (cols <= 16384) return 0;
    while (shift < 3 && (rows << (shift + 1)) <= (shift == 0 ? fit : fit * 9 / 10) &&
           (cols >> (shift + 1)) >= (rows << shift >= sms ? 16384 : 4096))
        ++shift;
    return shift;
}
template <int DT> Split split_of(int cols, int shift) {
    const int chunks = cols / Chunk<DT>::kElems;
    return {shift, (chunks >> shift) + ((chunks & ((1 << shift) - 1)) != 0)};
}
inline void describe(LaunchInfo *info, int64_t grid) {
    info->grid = static_cast<int>(grid);
    info->block = kThreads;
    info->vec_bytes = 16;
}

template <int DT> cudaError_t logprob_launch(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    // Many short rows: blocks of 64 threads, sixteen to an SM, or ten with
    // alternatives, whose lists take 21 KiB of shared memory each.  600 rows of 2000
    // bf16 with the 5 best: 5.3 us, with 256 threads a row 6.9; 300 rows: the
    // same; 5 rows: 4.5 and 4.2.
    if (a.rows > 2 * sms && a.cols <= kNarrow * kFlight * Chunk<DT>::kElems && a.top <= kFewGroupsTop) {
        info->grid = static_cast<int>(a.rows);
        info->block = kNarrow;
        info->vec_bytes = 16;
        auto kernel = a.top > 0 ? logprob_kernel<DT, true, kNarrow> : logprob_kernel<DT, false, kNarrow>;
        return launch_rows(kernel, dim3(a.rows), dim3(kNarrow), 0, 1, s, a, split_of<DT>(a.cols, 0));
    }
    const Split split = split_of<DT>(a.cols, split_shift(a.rows, a.cols, sms));
    const int64_t grid = a.rows << split.shift;
    describe(info, grid);
    auto kernel = a.top > 0 ? logprob_kernel<DT, true, kThreads> : logprob_kernel<DT, false, kThreads>;
    return launch_rows(kernel, dim3(grid), dim3(kThreads), 0, split.blocks(), s, a, split);
}
template <int DT> cudaError_t logprob_grad_launch(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info) {
    // blocks of 16384 to 32768 elements; in place a cluster of up to 8 a row, for the
    // rows that are summed again before any block writes
    const bool in_place = a.dlogits == a.logits;
    int shift = 0;
    while ((a.cols >> (shift + 1)) >= 16384 && a.rows << (shift + 1) <= INT32_MAX && !(in_place && shift == 3)) ++shift;
    const Split split = split_of<DT>(a.cols, shift);
    const int64_t grid = a.rows << shift;
    describe(info, grid);
    auto kernel = a.dentropy ? logprob_grad_kernel<DT, true> : logprob_grad_kernel<DT, false>;
    return launch_rows(kernel, dim3(grid), dim3(kThreads), 0, in_place ? split.blocks() : 1, s, a, split);
}
}  // namespace
}  // namespace ew
