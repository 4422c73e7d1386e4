// ew_logits.cuh -- operators on rows of logits: log probabilities of given
// tokens with entropy and top alternatives, distillation from a teacher's top
// logits, and their gradients.  Compiled once per element type.
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
#pragma once

#include <algorithm>
#include <type_traits>

#include "ew_rows.cuh"
#include "ew_rows.h"

namespace ew {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kFlight = 4;             // 16-byte chunks a thread has in flight
constexpr float kLeast = -1e30f;
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
    for (int j = 0; j < Chunk<DT>::kElems; ++j) {
        if constexpr (DT == DT_F32) f[j] = __uint_as_float(r.w[j]);
        else if constexpr (DT == DT_F16) f[j] = f16_to_f32(static_cast<uint16_t>(r.w[j / 2] >> (16 * (j & 1))));
        else f[j] = __uint_as_float((j & 1) ? (r.w[j / 2] & 0xffff0000u) : (r.w[j / 2] << 16));
    }
}

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
    __device__ __forceinline__ Share(const void *p, int cols_, int block, int blocks) {
        row = static_cast<const T *>(p);
        cols = cols_;
        const int past = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16) / ElemOf<DT>::kBytes;
        head = min((V - past) % V, cols);
        const int chunks = (cols - head) / V;
        first = static_cast<int>(static_cast<int64_t>(chunks) * block / blocks);
        end = static_cast<int>(static_cast<int64_t>(chunks) * (block + 1) / blocks);
        n_head = block == 0 ? head : 0;
        tail0 = head + chunks * V;
        singles = n_head + (block == blocks - 1 ? cols - tail0 : 0);
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
    float c, s, u;
    float top;  // largest element, NaN kept
};
__device__ __forceinline__ Sums no_sums() { return {kLeastExponent, 0.0f, 0.0f, kNegInf}; }

__device__ __forceinline__ void move_to(Sums &v, float c) {
    const float d = v.c - c;  // an integer <= 0
    const float f = ex2(d);
    v.u = f * fmaf(v.s, d, v.u);
    v.s *= f;
    v.c = c;
}
// Both sums at the larger exponent; symmetric, so that a butterfly gives every lane the same bits.
__device__ __forceinline__ Sums merged(Sums a, Sums b) {
    const float c = fmaxf(a.c, b.c);
    move_to(a, c);
    move_to(b, c);
    return {c, a.s + b.s, a.u + b.u, max_nan(a.top, b.top)};
}
template <int N> __device__ __forceinline__ void add_elements(Sums &v, const float (&x)[N], float a) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = max_nan(top, x[j]);
    v.top = max_nan(v.top, top);
    const float c = fmaxf(ceilf(top * a), kLeastExponent);
    if (c > v.c) move_to(v, c);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float t = fmaf(fmaxf(x[j], kLeast), a, -v.c);
        const float e = ex2(t);
        v.s += e;
        v.u = fmaf(e, t, v.u);
    }
}
__device__ __forceinline__ Sums warp_sums(Sums v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const Sums o = {__shfl_xor_sync(kAllLanes, v.c, d), __shfl_xor_sync(kAllLanes, v.s, d),
                        __shfl_xor_sync(kAllLanes, v.u, d), __shfl_xor_sync(kAllLanes, v.top, d)};
        v = merged(v, o);
    }
    return v;
}
// Sums of the block, to all its threads.
__device__ __forceinline__ Sums block_sums(Sums v, Sums *part) {
    v = warp_sums(v);
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sums(lane < kWarps ? part[lane] : no_sums());
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
template <int DT> __device__ __noinline__ RowSum careful_row(const void *row, int cols, float a, float top, float *part) {
    RowSum r = {0.0f, 0.0f, 0.0f, 0.0f, top, true};
    if (top == kNegInf) return r;
    const Share<DT> all(row, cols, 0, 1);
    float s = 0.0f, u = 0.0f;
    for (int k = threadIdx.x; k < cols; k += kThreads) {
        const float t = fmaxf((all.at(k) - top) * a, -200.0f);
        const float e = ex2(t);
        s += e;
        u = fmaf(e, t, u);
    }
    if (!(top < -kNegInf)) s = top - top;  // NaN
    __syncthreads();
    s = block_sum(s, kWarps, part);
    __syncthreads();
    u = block_sum(u, kWarps, part);
    r.log_s = logf(s);
    r.inv_s = 1.0f / s;
    r.u_over_s = u / s;
    return r;
}
template <int DT>
__device__ __forceinline__ RowSum finish_row(const Sums &v, const void *row, int cols, float a, float *part) {
    if (v.s > 0.0f && v.s < 1e37f && fabsf(v.u) < 1e37f && v.top < -kNegInf)
        return {v.c, logf(v.s), 1.0f / v.s, v.u / v.s, v.top, false};
    return careful_row<DT>(row, cols, a, v.top, part);
}

// ---------------------------------------------------------------- top alternatives
//
// The largest `k` elements, equal ones by index.  The first elements that the
// block reads give a bound: of 128 groups of lanes, the k-th largest group
// maximum; at least k elements reach it.  Elements that reach it are collected
// while the row streams past (a few hundred of a row in no particular order)
// and ranked at the end.  Where more than kCandidates are collected, exact_top
// finds the k-th value by bisection instead.

constexpr int kCandidates = 2048;
constexpr int kGroups = kThreads / 4;

struct Candidate {
    float x;
    int id;
};
__device__ __forceinline__ bool before(const Candidate &a, const Candidate &b) {
    return a.x > b.x || (a.x == b.x && a.id < b.id);
}

struct TopShared {
    float group[kGroups];
    float bound;
    int count;
    Candidate list[kCandidates];
    Candidate best[kMostTop];  // ids of -1 at the end where there are fewer
};

__device__ __forceinline__ void collect(TopShared &t, float x, int id) {
    const int at = atomicAdd(&t.count, 1);
    if (at < kCandidates) t.list[at] = {x, id};
}

// The k best of n entries into best[0 .. k): the rank of an entry is the
// number of entries before it.
__device__ __forceinline__ void rank_list(const Candidate *list, int n, int k, Candidate *best) {
    for (int i = n + static_cast<int>(threadIdx.x); i < k; i += kThreads) best[i] = {kNegInf, -1};
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const Candidate mine = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += before(list[j], mine) ? 1 : 0;
        if (rank < k) best[rank] = mine;
    }
}

// Bound from the largest element that each thread has seen.
__device__ __forceinline__ void find_bound(TopShared &t, float mine, int k) {
    mine = fmaxf(mine, __shfl_xor_sync(kAllLanes, mine, 1));
    mine = fmaxf(mine, __shfl_xor_sync(kAllLanes, mine, 2));
    if ((threadIdx.x & 3) == 0) t.group[threadIdx.x >> 2] = mine;
    if (threadIdx.x == 0) t.count = 0;
    __syncthreads();
    if (threadIdx.x < kGroups) {
        const float v = t.group[threadIdx.x];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < kGroups; ++j) rank += t.group[j] > v || (t.group[j] == v && j < static_cast<int>(threadIdx.x));
        if (rank == k - 1) t.bound = v;
    }
    __syncthreads();
}

// Order of binary32 values as unsigned integers (-0 and +0 the same).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

// The exact k best of the block's share, however many elements tie.
template <int DT> __device__ __noinline__ void exact_top(TopShared &t, const Share<DT> &sh, int k) {
    constexpr int V = Chunk<DT>::kElems;
    auto count_from = [&](uint32_t least) {  // elements of the share from `least` on
        int n = 0;
        for (int c = sh.first + threadIdx.x; c < sh.end; c += kThreads) {
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
    // the k-th largest value: the largest `least` that k elements reach.  The
    // collected elements say that k reach the bound; often no more lie above.
    uint32_t lo = order_of(t.bound), hi = 0xffffffffu;
    for (uint32_t probe = lo + 1; lo < hi; probe = lo + (hi - lo) / 2 + 1) {
        if (count_from(probe) >= k) lo = probe;
        else hi = probe - 1;
    }
    // larger ones (fewer than k), then the first of those equal to it, in order
    __syncthreads();
    if (threadIdx.x == 0) t.count = 0;
    __syncthreads();
    for (int c = sh.first + threadIdx.x; c < sh.end; c += kThreads) {
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
    for (int base = begin; base < stop; base += kThreads) {
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
            for (int w = 0; w < kWarps; ++w) n += warp_counts[w];
            t.count = min(n, k);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the pass over a row

// Sums of the block's share of a row and, where k > 0, its k best elements in
// t.best, sorted.
template <int DT, bool TOP>
__device__ __forceinline__ Sums pass_over(const Share<DT> &sh, float a, TopShared *t, int k, Sums *part) {
    constexpr int V = Chunk<DT>::kElems;
    Sums v = no_sums();
    Chunk<DT> r[kFlight];
    float bound = kNegInf;
    auto take = [&](int c0) {  // up to kFlight chunks of this thread from c0 on
        float top = kNegInf;
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (c0 + u * kThreads < sh.end) r[u] = sh.chunk(c0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (c0 + u * kThreads < sh.end) {
                float f[V];
                unpack<DT>(r[u], f);
                const float seen = v.top;
                v.top = kNegInf;
                add_elements(v, f, a);
                top = fmaxf(top, v.top);
                v.top = max_nan(v.top, seen);
            }
        }
        return top;
    };
    auto offer = [&](int c0, float top) {  // those that reach the bound become candidates
        if (!(top >= bound)) return;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (c0 + u * kThreads < sh.end) {
                float f[V];
                unpack<DT>(r[u], f);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (f[j] >= bound && f[j] > kNegInf) collect(*t, f[j], sh.column(c0 + u * kThreads, j));
            }
        }
    };
    int c0 = sh.first + threadIdx.x;
    float top = take(c0);
    float one = kNegInf;
    if (static_cast<int>(threadIdx.x) < sh.singles) {
        one = sh.at(sh.single(threadIdx.x));
        const float f[1] = {one};
        add_elements(v, f, a);
    }
    if constexpr (TOP) {
        find_bound(*t, fmaxf(top, one), k);
        bound = t->bound;
        offer(c0, top);
        if (one >= bound && one > kNegInf) collect(*t, one, sh.single(threadIdx.x));
    }
    for (c0 += kFlight * kThreads; c0 < sh.end; c0 += kFlight * kThreads) {
        top = take(c0);
        if constexpr (TOP) offer(c0, top);
    }
    v = block_sums(v, part);  // and every candidate is in the list
    if constexpr (TOP) {
        if (t->count > kCandidates) exact_top<DT>(*t, sh, k);
        rank_list(t->list, t->count, k, t->best);
        __syncthreads();
    }
    return v;
}

// ---------------------------------------------------------------- log probabilities

// A row to a cluster of `blocks` blocks (one block: no cluster); the first
// puts the parts together.
template <int DT, bool TOP> __global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobArgs a, int blocks) {
    enter_grid();
    __shared__ Sums part[kWarps];
    __shared__ Sums mine;
    __shared__ float fpart[32];
    __shared__ typename std::conditional<TOP, TopShared, int>::type top_store;
    TopShared *t = nullptr;
    if constexpr (TOP) t = &top_store;
    const int block = static_cast<int>(blockIdx.x % blocks);
    const int64_t row = blockIdx.x / blocks;
    const void *logits = row_of<DT>(a.logits, row, a.stride);
    const Share<DT> sh(logits, a.cols, block, blocks);
    const float ax = a.scale * kLog2e;
    Sums v = pass_over<DT, TOP>(sh, ax, t, a.top, part);
    if (blocks > 1) {
        if (threadIdx.x == 0) mine = v;
        cluster_sync();
        if (block == 0) {
            for (int b = 1; b < blocks; ++b) v = merged(v, *in_block(&mine, b));
            if constexpr (TOP) {
                for (int i = threadIdx.x; i < blocks * a.top; i += kThreads)
                    t->list[i] = in_block(t->best, i / a.top)[i % a.top];
                __syncthreads();
                // entries that are not there (-inf, -1) rank behind all others; drop them
                if (threadIdx.x == 0) t->count = 0;
                __syncthreads();
                Candidate keep[2];
                int n = 0;
                for (int i = threadIdx.x; i < blocks * a.top; i += kThreads) keep[n++] = t->list[i];
                __syncthreads();
                for (int i = 0; i < n; ++i)
                    if (keep[i].id >= 0) collect(*t, keep[i].x, keep[i].id);
                __syncthreads();
                rank_list(t->list, t->count, a.top, t->best);
            }
        }
        cluster_sync();  // no block leaves while its shared memory is read
        if (block != 0) return;
    }
    const RowSum r = finish_row<DT>(v, logits, a.cols, ax, fpart);
    if (threadIdx.x == 0) {
        const bool empty = r.careful && r.top == kNegInf;
        if (a.lse) a.lse[row] = empty ? kNegInf : lse_of(r, a.scale);
        if (a.entropy) a.entropy[row] = empty ? 0.0f : entropy_of(r);
        if (a.logp) {
            const int64_t token = token_at(a.tokens, a.i64, row);
            const bool given = token >= 0 && token < a.cols;
            a.logp[row] = !given ? 0.0f : empty ? kNegInf : logp_of(r, sh.at(static_cast<int>(given ? token : 0)), ax, a.scale);
        }
    }
    if constexpr (TOP) {
        for (int i = threadIdx.x; i < a.top; i += kThreads) {
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
// p = 0 whatever x is.
__device__ __forceinline__ Weights no_weights() { return {0.0f, 0.0f, -kNegInf, true}; }
// From a saved lse: c is lse * log2(e) rounded to an integer, weight 2^ of what
// is left, formed with the two parts of log2(e).
__device__ __forceinline__ Weights weights_of(float lse, float scale) {
    const float c = rintf(lse * kLog2e);
    const float left = fmaf(lse, kLog2e, -c) + lse * 1.9259629911266175e-8f;
    if (fabsf(lse) < 1e6f) return {c, ex2(-left), 0.0f, false};
    if (lse == kNegInf) return no_weights();  // an empty row
    return {0.0f, lse == lse ? 1.0f : lse, lse / scale, true};  // huge values; NaN stays NaN
}

// d(x) = g p(x), or with entropy g p(x) - dH p(x) (log p(x) + H), into dlogits.
struct RowGrad {
    Weights w;
    float g, dent, lse, entropy;
};
template <bool ENTROPY> __device__ __forceinline__ float grad_of(const RowGrad &r, float x, float a, float scale) {
    const float p = p_of(r.w, x, a);
    if constexpr (ENTROPY) {
        const float logp = fmaf(fmaxf(x, kLeast), scale, -r.lse);
        return p * fmaf(-r.dent, p > 0.0f ? logp + r.entropy : 0.0f, r.g);
    } else {
        return p * r.g;
    }
}

// Writes the gradient of the block's share.  The output row may start at
// another offset from 16 bytes than the input's: then element by element.
template <int DT, bool ENTROPY>
__device__ __forceinline__ void write_grad(const Share<DT> &sh, void *out_row, const RowGrad &r, float a, float scale) {
    using T = typename ElemOf<DT>::type;
    constexpr int V = Chunk<DT>::kElems;
    T *out = static_cast<T *>(out_row);
    const bool alike = (reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(sh.row)) % 16 == 0;
    auto put_one = [&](int col, float x) {
        const T d = f32_to_elem<DT>(grad_of<ENTROPY>(r, x, a, scale));
        if constexpr (DT == DT_F32) { Vec<4> v; v.w[0] = d; st<4>(out + col, v); }
        else { Vec<2> v; v.h = d; st<2>(out + col, v); }
    };
    for (int c0 = sh.first + static_cast<int>(threadIdx.x); c0 < sh.end; c0 += kFlight * kThreads) {
        Chunk<DT> raw[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (c0 + u * kThreads < sh.end) raw[u] = sh.chunk(c0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (c0 + u * kThreads >= sh.end) break;
            float f[V];
            unpack<DT>(raw[u], f);
            if (alike) {
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] = grad_of<ENTROPY>(r, f[j], a, scale);
                Vec<16> o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (DT == DT_F32) o.w[j] = __float_as_uint(f[j]);
                    else if constexpr (DT == DT_F16) o.w[j] = f32x2_to_f16x2(f[2 * j + 1], f[2 * j]);
                    else o.w[j] = f32x2_to_bf16x2(f[2 * j + 1], f[2 * j]);
                }
                st<16>(out + sh.column(c0 + u * kThreads, 0), o);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) put_one(sh.column(c0 + u * kThreads, j), f[j]);
            }
        }
    }
    if (static_cast<int>(threadIdx.x) < sh.singles) {
        const int col = sh.single(threadIdx.x);
        put_one(col, sh.at(col));
    }
}
template <int DT> __device__ __forceinline__ void store_one(void *row, int col, float x) {
    using T = typename ElemOf<DT>::type;
    static_cast<T *>(row)[col] = f32_to_elem<DT>(x);
}

// dlogits = scale (dlogp (1_token - p) - dentropy p (log p + H)).
template <int DT, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) logprob_grad_kernel(LogprobGradArgs a, int blocks) {
    enter_grid();
    const int block = static_cast<int>(blockIdx.x % blocks);
    const int64_t row = blockIdx.x / blocks;
    const Share<DT> sh(row_of<DT>(a.logits, row, a.stride), a.cols, block, blocks);
    void *out = row_of<DT>(a.dlogits, row, a.dstride);
    const float ax = a.scale * kLog2e;
    int64_t token = a.dlogp ? token_at(a.tokens, a.i64, row) : -1;
    if (token >= a.cols) token = -1;
    const float dlogp = token >= 0 ? a.dlogp[row] : 0.0f;
    RowGrad r;
    r.lse = a.lse[row];
    r.w = weights_of(r.lse, a.scale);
    const bool empty = r.lse == kNegInf;  // nothing depends on the logits of an empty row
    r.g = -a.scale * dlogp;
    r.dent = ENTROPY && !empty ? a.scale * a.dentropy[row] : 0.0f;
    r.entropy = ENTROPY && !empty ? a.entropy[row] : 0.0f;
    if (empty) r.lse = 0.0f;
    const bool here = token >= 0 && sh.holds(static_cast<int>(token));
    const float x = here ? sh.at(static_cast<int>(token)) : 0.0f;  // read before it may be overwritten
    if (here) __syncthreads();                                     // uniform: all threads have the same token
    write_grad<DT, ENTROPY>(sh, out, r, ax, a.scale);
    if (!here) return;
    __syncthreads();
    if (threadIdx.x == 0)
        store_one<DT>(out, static_cast<int>(token), empty ? 0.0f : grad_of<ENTROPY>(r, x, ax, a.scale) + a.scale * dlogp);
}

// ---------------------------------------------------------------- distillation
//
// q = softmax of the teacher's values at its ids, p = softmax of the student's
// row, both of values times `scale`:
//     loss = sum q_i (log q_i - log p(id_i)),   dlogits = dloss scale (p - q).
// Entries with an id outside the row or a value of -inf do not count; a row
// without any has loss 0 and gradient 0.  The row is read for the sums and
// again for the gradient, the second time mostly from L2.

struct Teacher {
    int id[kMostTeacher];
    float q[kMostTeacher];
    float x[kMostTeacher];  // the student's logit there
};

template <int DT, bool SUMS, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a, int blocks) {
    enter_grid();
    __shared__ Sums part[kWarps];
    __shared__ Sums mine;
    __shared__ float fpart[2][32];
    __shared__ Teacher th;
    const int block = static_cast<int>(blockIdx.x % blocks);
    const int64_t row = blockIdx.x / blocks;
    const void *logits = row_of<DT>(a.logits, row, a.stride);
    const Share<DT> sh(logits, a.cols, block, blocks);
    const float ax = a.scale * kLog2e;

    // the teacher's entries and its softmax; every block has them all
    float largest = kNegInf;
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        const int64_t id = token_at(a.ids, a.i64, row * a.ids_stride + i);
        const int64_t at = row * a.teacher_stride + i;
        float v;
        if (DT == DT_F32 || a.teacher_f32) v = static_cast<const float *>(a.teacher)[at];
        else v = elem_to_f32<DT>(static_cast<const typename ElemOf<DT>::type *>(a.teacher)[at]);
        const bool given = id >= 0 && id < a.cols && v != kNegInf;
        th.id[i] = given ? static_cast<int>(id) : -1;
        th.q[i] = v * a.scale;
        // the loss needs them all, the gradient those that this block writes
        const bool read = given && ((SUMS && block == 0) || sh.holds(static_cast<int>(id)));
        th.x[i] = read ? sh.at(static_cast<int>(id)) : 0.0f;
        if (given) largest = max_nan(largest, th.q[i]);
    }
    __syncthreads();
    largest = block_max_nan(largest, kWarps, fpart[0], kNegInf);
    const bool any = largest != kNegInf;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        th.q[i] = th.id[i] >= 0 ? th.q[i] - largest : kNegInf;
        sum += th.id[i] >= 0 ? expf(th.q[i]) : 0.0f;
    }
    sum = block_sum(sum, kWarps, fpart[1]);
    const float log_sum = logf(sum);

    Sums v = no_sums();
    RowSum r;
    Weights w;
    if constexpr (SUMS) {
        v = pass_over<DT, false>(sh, ax, nullptr, 0, part);
        if (blocks > 1) {
            if (threadIdx.x == 0) mine = v;
            cluster_sync();
            Sums all = *in_block(&mine, 0);
            for (int b = 1; b < blocks; ++b) all = merged(all, *in_block(&mine, b));
            v = all;
            cluster_sync();
        }
        r = finish_row<DT>(v, logits, a.cols, ax, fpart[0]);
        const bool empty = r.careful && r.top == kNegInf;
        w = {r.c, r.inv_s, r.top, r.careful};
        if (block == 0) {
            // in order of the entries, added by the block's fixed tree
            float loss = 0.0f;
            for (int i = threadIdx.x; i < a.k; i += kThreads) {
                const float logq = th.q[i] - log_sum, q = th.id[i] >= 0 ? expf(logq) : 0.0f;
                const float logp = empty ? kNegInf : logp_of(r, th.x[i], ax, a.scale);
                if (q != 0.0f) loss += q * (logq - logp);
            }
            __syncthreads();
            loss = block_sum(loss, kWarps, fpart[1]);
            if (threadIdx.x == 0) {
                if (a.loss) a.loss[row] = any ? loss : 0.0f;
                if (a.lse) a.lse[row] = empty ? kNegInf : lse_of(r, a.scale);
            }
        }
    } else {
        w = weights_of(a.lse[row], a.scale);
    }
    if constexpr (GRAD) {
        const float g = any ? a.dloss[row] * a.scale : 0.0f;
        void *out = row_of<DT>(a.dlogits, row, a.dstride);
        RowGrad rg = {w, g, 0.0f, 0.0f, 0.0f};
        if (!any) rg.w = no_weights();
        // careful rows may be read again by another block: all have to be done before any writes in place
        if (SUMS && w.careful) {
            if (blocks > 1) cluster_sync();
            else __syncthreads();
        }
        write_grad<DT, false>(sh, out, rg, ax, a.scale);
        if (!any) return;
        __syncthreads();
        // entries of one id add up; the first of them writes
        for (int i = threadIdx.x; i < a.k; i += kThreads) {
            const int id = th.id[i];
            if (id < 0 || !sh.holds(id)) continue;
            bool first = true;
            float q = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                if (th.id[j] != id) continue;
                if (j < i) { first = false; break; }
                q += expf(th.q[j] - log_sum);
            }
            if (first) store_one<DT>(out, id, g * (p_of(w, th.x[i], ax) - q));
        }
    }
}

// ---------------------------------------------------------------- launches

// Blocks a row: one where the rows alone fill the device twice, up to a
// cluster of 8 where they are few, each with at least 4096 elements.
inline int blocks_per_row(int64_t rows, int cols, int sms) {
    int blocks = 1;
    while (blocks < 8 && rows * blocks < 2 * static_cast<int64_t>(sms) && cols / (2 * blocks) >= 4096) blocks *= 2;
    return blocks;
}
inline void describe(LaunchInfo *info, int64_t grid) {
    info->grid = static_cast<int>(grid);
    info->block = kThreads;
    info->vec_bytes = 16;
}

template <int DT> cudaError_t logprob_launch(const LogprobArgs &a, int sms, cudaStream_t s, LaunchInfo *info) {
    const int blocks = blocks_per_row(a.rows, a.cols, sms);
    const int64_t grid = a.rows * blocks;
    describe(info, grid);
    return a.top > 0 ? launch_rows(logprob_kernel<DT, true>, dim3(grid), dim3(kThreads), 0, blocks, s, a, blocks)
                     : launch_rows(logprob_kernel<DT, false>, dim3(grid), dim3(kThreads), 0, blocks, s, a, blocks);
}
template <int DT> cudaError_t logprob_grad_launch(const LogprobGradArgs &a, cudaStream_t s, LaunchInfo *info) {
    // no sums: blocks of about 16384 elements, no cluster
    const int blocks = std::max<int>(1, std::min<int64_t>(a.cols / 16384, INT32_MAX / a.rows));
    const int64_t grid = a.rows * blocks;
    describe(info, grid);
    return a.dentropy ? launch_rows(logprob_grad_kernel<DT, true>, dim3(grid), dim3(kThreads), 0, 1, s, a, blocks)
                      : launch_rows(logprob_grad_kernel<DT, false>, dim3(grid), dim3(kThreads), 0, 1, s, a, blocks);
}
template <int DT>
cudaError_t distill_launch(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    const int blocks = blocks_per_row(a.rows, a.cols, sms);
    const int64_t grid = a.rows * blocks;
    describe(info, grid);
    const dim3 g(grid), b(kThreads);
    if (!sums) return launch_rows(distill_kernel<DT, false, true>, g, b, 0, blocks, s, a, blocks);
    return grad ? launch_rows(distill_kernel<DT, true, true>, g, b, 0, blocks, s, a, blocks)
                : launch_rows(distill_kernel<DT, true, false>, g, b, 0, blocks, s, a, blocks);
}

}  // namespace
}  // namespace ew
