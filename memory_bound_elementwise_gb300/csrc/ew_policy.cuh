// ew_policy.cuh -- the clipped policy loss with a divergence term, on rows of
// logits, and its gradient.  Compiled once per element type.
//
// For a row with a token, logp its log probability under softmax(scale * logits):
//     ratio = exp(logp - old_logp)        (1 without an old policy)
//     gain  = min(ratio A, clip(ratio, 1 - low, 1 + high) A)
//     apart = ref_logp - logp,  kl = exp(apart) - apart - 1
//     loss  = -gain + beta kl
//     d loss / d logp = -(ratio A where it is not clipped) + beta (1 - exp(apart))
//     dlogits = dloss (d loss / d logp) scale (1_token - p)
// Rows without a token have loss 0 and gradient 0, and their logits are not read.
//
// The gradient needs the row's sums, so a row is worked over twice.  At the floor
// it crosses DRAM once: policy_stream_kernel keeps it in shared memory in between.
// policy_kernel reads it again, mostly from L2: for rows too short to be worth a
// ring, rows too long, the gradient from a given lse, and where there is no more than
// a row an SM, for which the lists below come late (loss and gradient of 7 rows of
// 79525 bf16 5.9 us, with a ring 7.4; of 100 of 123400 binary32 24 and 32 us).
#pragma once

#include "ew_logits.cuh"

namespace ew {
namespace {

// A token's numbers, and what follows from them and its log probability.
struct PolicyToken {
    float advantage, old_logp, ref_logp, dloss;
};
struct PolicyTerms {
    float loss, slope;  // slope: d loss / d logp
};
// exp(x) - 1 - x.  Near 0, where the difference loses its digits, by the series
// x^2 (1/2! + x/3! + x^2/4! + ..): at 1/2 the first term left out is 4e-8 of the sum.
__device__ __forceinline__ float exp_less_tangent(float x) {
    if (fabsf(x) < 0.5f) {
        float s = 1.0f / 40320.0f;
        s = fmaf(s, x, 1.0f / 5040.0f);
        s = fmaf(s, x, 1.0f / 720.0f);
        s = fmaf(s, x, 1.0f / 120.0f);
        s = fmaf(s, x, 1.0f / 24.0f);
        s = fmaf(s, x, 1.0f / 6.0f);
        s = fmaf(s, x, 0.5f);
        return s * x * x;
    }
    const float e = expm1f(x);
    return e < -kNegInf ? e - x : e;  // infinity or NaN: x adds nothing
}
__device__ __forceinline__ PolicyTerms policy_terms(const PolicyArgs &a, const PolicyToken &t, float logp) {
    // NaN stays: every comparison below is false for it
    const float ratio = a.old_logp ? expf(logp - t.old_logp) : logp == logp ? 1.0f : logp;
    float within = ratio > a.most ? a.most : ratio;
    within = within < a.least ? a.least : within;
    // a ratio past binary32 is still finite: times 0 it is 0
    const bool nothing = t.advantage == 0.0f && ratio == ratio;
    const float gain = nothing ? 0.0f : ratio * t.advantage, bound = nothing ? 0.0f : within * t.advantage;
    const bool clipped = gain > bound;
    PolicyTerms r = {clipped ? -bound : -gain, clipped ? 0.0f : -gain};
    if (a.ref_logp) {
        const float apart = t.ref_logp - logp;
        r.loss = fmaf(a.kl, exp_less_tangent(apart), r.loss);
        r.slope = fmaf(-a.kl, expm1f(apart), r.slope);
    }
    return r;
}
__device__ __forceinline__ PolicyToken policy_token(const PolicyArgs &a, int64_t row, bool grad) {
    return {a.advantage[row], a.old_logp ? a.old_logp[row] : 0.0f, a.ref_logp ? a.ref_logp[row] : 0.0f,
            grad ? a.dloss[row] : 0.0f};
}
// What multiplies 1_token - p.
__device__ __forceinline__ float policy_factor(const PolicyArgs &a, const PolicyToken &t, const PolicyTerms &r) {
    return t.dloss == 0.0f ? 0.0f : t.dloss * r.slope * a.scale;
}
__device__ __forceinline__ bool is_empty(const RowSum &r) { return r.careful && r.top == kNegInf; }
__device__ __forceinline__ void write_results(const PolicyArgs &a, int64_t row, float loss, float logp, float lse) {
    a.loss[row] = loss;
    if (a.logp_out) a.logp_out[row] = logp;
    if (a.lse_out) a.lse_out[row] = lse;
}

// ---------------------------------------------------------------- rows read twice

template <int DT, bool SUMS, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, kResident * kThreads / THREADS) policy_kernel(const __grid_constant__ PolicyArgs a, Split split) {
    enter_grid();
    __shared__ Sums part[THREADS / 32];
    __shared__ Sums mine;
    __shared__ float fpart[32];
    const int blocks = split.blocks(), block = blockIdx.x & (blocks - 1);
    const int64_t row = blockIdx.x >> split.shift;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t token = token_at(a.tokens, a.i64, row);
    if (token < 0 || token >= a.cols) {  // all blocks of the row alike: no barrier is waited for
        if (SUMS && block == 0 && threadIdx.x == 0) write_results(a, row, 0.0f, 0.0f, 0.0f);
        if (GRAD) write_zeros<DT>(row_of<DT>(a.dlogits, row, a.dstride), a.cols, block, split, THREADS);
        return;
    }
    const int col = static_cast<int>(token);
    const void *logits = row_of<DT>(a.logits, row, a.stride);
    const Share<DT> sh(logits, a.cols, block, split);
    const float ax = a.scale * kLog2e;
    const PolicyToken t = policy_token(a, row, GRAD);
    const float x = sh.at(col);  // by every block, before any writes in place
    Weights w;
    bool empty = false;
    float logp;
    if constexpr (SUMS) {
        Chunk<DT> r_chunks[kFlight];
        load_turn<DT, THREADS>(sh, sh.first + static_cast<int>(threadIdx.x), r_chunks);
        float largest, bound;
        Sums v = warp_sums<32, false>(pass_over<DT, false, false, THREADS>(sh, ax, nullptr, 0, r_chunks, largest, bound));
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = sums_of_warps<THREADS / 32, false>(part);
        if (blocks > 1) {
            if (threadIdx.x == 0) mine = v;
            cluster_sync();
            v = cluster_sums<false>(&mine, blocks);
            cluster_arrive();  // the wait is further down: mine has been read
        }
        const RowSum r = finish_row<DT, false>(v, logits, a.cols, ax, fpart);
        w = {r.c, r.inv_s, r.top, r.careful};
        empty = is_empty(r);
        logp = empty ? kNegInf : logp_of(r, x, ax, a.scale);
        if (block == 0 && threadIdx.x == 0)
            write_results(a, row, policy_terms(a, t, logp).loss, logp, empty ? kNegInf : lse_of(r, a.scale));
        if (GRAD && r.careful) {
            // a careful row has been read whole by every block: all are done with it before any writes in place
            if (blocks > 1) {
                cluster_wait();
                cluster_sync();
                cluster_arrive();
            } else {
                __syncthreads();
            }
        }
    } else {
        // every block of the row decides alike
        const float lse = a.lse[row];
        logp = a.logp[row];
        if (lse_holds(lse)) {
            w = weights_of(lse);
        } else {
            const RowSum again = careful_row<DT>(logits, a.cols, ax, fpart);
            if (blocks > 1) cluster_sync();  // all have read the row before any writes in place
            else __syncthreads();
            w = {0.0f, again.inv_s, again.top, true};
            empty = is_empty(again);
        }
    }
    if constexpr (GRAD) {
        void *out = row_of<DT>(a.dlogits, row, a.dstride);
        if (empty) {
            write_zeros<DT>(out, a.cols, block, split, THREADS);
        } else {
            const float factor = policy_factor(a, t, policy_terms(a, t, logp));
            const RowGrad rg = row_grad(w, -factor, 0.0f, 0.0f, 0.0f);
            if (!SUMS) __syncthreads();  // all threads have read the token's logit
            write_grad<DT, false, THREADS>(sh, out, rg, ax, a.scale);
            if (sh.holds(col)) {
                __syncthreads();
                if (threadIdx.x == 0) store_one<DT>(out, col, grad_of<false>(rg, x, ax, a.scale) + factor);
            }
        }
    }
    if (SUMS && blocks > 1) cluster_wait();
}

// ---------------------------------------------------------------- rows held in shared memory
//
// A block walks over rows; one of 512 threads an SM (or a cluster of up to 8 for a
// row), two of 256 for rows up to 96 KiB, which their rings hold (4096 rows of 40000
// bf16 104 us, by one block an SM 115; of 65536, which they do not hold, 190 and 176),
// four of 128 up to 32 KiB.  The block's
// share of a row, from the line in which it begins on, so that a warp's 512 bytes are
// whole lines wherever the row starts (8192 rows of 50257 bf16 336 us, 353 from the
// first chunk on), is `groups` groups of 4 chunks a thread; a ring of kRing groups is
// filled by asynchronous copies in the order of the stream of groups, row after
// row, and a group's place is filled again as soon as the gradient (or, for the
// loss alone, the sum) has used it.  Of a share of more than kRing groups the first
// ones give way while the row is summed; they are copied again, from L2, behind
// the row's last, and their gradient comes last.  That is cheaper than more blocks
// for a row, whose sums take another barrier and a read across the cluster: 2048
// rows of 131072 bf16 took 208 us by clusters of two.  Each thread copies and
// reads its own chunks only: it waits for its own copies and needs no barrier for
// them.  A row has one barrier, between its sums and its gradient; its loss and
// slope are worked out by every thread for itself.
//
// Rows without a token cost a write and no read, so rows are not dealt out by their
// numbers: the rows with a token, in their order, go round the blocks (or
// clusters), and so do those without, from the last block on.  Each block works its
// list out for itself, from all tokens: 8 bytes a row, where a row has thousands.
// 2048 rows of 131072 bf16, a quarter of them without a token, took 188 us by
// numbers and 182 us by lists, both by clusters of two; a block a row takes 157 us.
//
// Tokens, their numbers and logits are read for 32 of the block's rows at once, one
// to a lane: what a row needs comes from a register.

constexpr int kGroup = 4;
constexpr int kRing = 6;
constexpr int kMostGroups = 8;
template <int T> struct Stream {  // T threads
    static constexpr int kGroupChunks = kGroup * T;
    static constexpr int kBlocks = 512 / T;  // an SM's
    static constexpr int kSmem = kRing * kGroupChunks * 16;
    static constexpr int kLooks = 8;         // tokens that a thread looks at together
    static constexpr int kSlab = kLooks * T;
    static constexpr int kList = 4 * T;      // rows of a block's list, and rounds of the blocks in a window of rows
};

// AGAIN: groups of a row that are copied twice; of 1 or more, a row has kRing + AGAIN.
template <int DT, bool GRAD, int THREADS, int AGAIN>
__global__ void __launch_bounds__(THREADS, Stream<THREADS>::kBlocks)
    policy_stream_kernel(const __grid_constant__ PolicyArgs a, Split split, int groups) {
    using T = typename ElemOf<DT>::type;
    using S = Stream<THREADS>;
    constexpr int kGroupChunks = S::kGroupChunks, kWarps = THREADS / 32, kCounts = S::kLooks * kWarps;
    static_assert(kCounts % 32 == 0, "counts go round the lanes");
    enter_grid();
    extern __shared__ uint4 dynamic[];
    __shared__ Sums part[2][kWarps];
    __shared__ Sums mine[2];
    __shared__ float fpart[32];
    __shared__ int list[S::kList + 2];  // with a token from the front, without from the back
    __shared__ int counts[kCounts];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    uint4 *ring = dynamic + tid;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const int blocks = split.blocks(), block = blockIdx.x & (blocks - 1);
    const unsigned step = gridDim.x >> split.shift, me = blockIdx.x >> split.shift;
    if (AGAIN > 0) groups = kRing + AGAIN;
    const float ax = a.scale * kLog2e;
    auto share_of = [&](int64_t row) {
        return Share<DT>(row_of<DT>(a.logits, row, a.stride), a.cols, block, split);
    };
    // the chunk, at or before the share's first, from which a warp's chunks are whole lines
    auto begin_of = [&](const Share<DT> &sh) {
        return sh.first - static_cast<int>(reinterpret_cast<uintptr_t>(sh.row + sh.column(sh.first, 0)) / 16 % 8);
    };
    // -1: none
    auto token_of = [&](int64_t row) {
        const int64_t token = token_at(a.tokens, a.i64, row);
        return token >= 0 && token < a.cols ? static_cast<int>(token) : -1;
    };
    const float per_step = 1.0f / static_cast<float>(step);
    int turn = 0;
#pragma unroll 1
    for (int64_t base = 0; base < a.rows; base += static_cast<int64_t>(step) * S::kList) {
        // The block's rows of this window: ranks among those with a token, and without.
        const int window = static_cast<int>(min(a.rows - base, static_cast<int64_t>(step) * S::kList));
        unsigned with = 0;
#pragma unroll 1
        for (int slab = 0; slab < window; slab += S::kSlab) {
            unsigned given[S::kLooks];
            int64_t token[S::kLooks];  // read together: past the window its last one again
            if (a.i64) {
                const int64_t *from = static_cast<const int64_t *>(a.tokens) + base;
#pragma unroll
                for (int j = 0; j < S::kLooks; ++j) token[j] = from[min(slab + j * THREADS + tid, window - 1)];
            } else {
                const int32_t *from = static_cast<const int32_t *>(a.tokens) + base;
#pragma unroll
                for (int j = 0; j < S::kLooks; ++j) token[j] = from[min(slab + j * THREADS + tid, window - 1)];
            }
#pragma unroll
            for (int j = 0; j < S::kLooks; ++j)
                given[j] = __ballot_sync(kAllLanes, slab + j * THREADS + tid < window && token[j] >= 0 && token[j] < a.cols);
            __syncthreads();  // the counts before, and the list of the window before, have been read
#pragma unroll
            for (int j = 0; j < S::kLooks; ++j)
                if (lane == 0) counts[j * kWarps + warp] = __popc(given[j]);
            __syncthreads();
            // a lane has kOwn counts in a row, and those before them in `upto`
            constexpr int kOwn = kCounts / 32;
            int upto[kOwn + 1] = {};
#pragma unroll
            for (int i = 0; i < kOwn; ++i) upto[i + 1] = upto[i] + counts[lane * kOwn + i];
            int scan = upto[kOwn];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int below = __shfl_up_sync(kAllLanes, scan, d);
                if (lane >= d) scan += below;
            }
            const int before_lane = scan - upto[kOwn];
#pragma unroll
            for (int j = 0; j < S::kLooks; ++j) {
                const int own = j * kWarps + warp, at = slab + j * THREADS + tid;
                if (slab + j * THREADS >= window) break;
                int earlier = before_lane;
#pragma unroll
                for (int i = 1; i < kOwn; ++i) earlier = own % kOwn == i ? before_lane + upto[i] : earlier;
                earlier = __shfl_sync(kAllLanes, earlier, own / kOwn);
                const bool one = given[j] >> lane & 1;
                // its rank among those with a token, or without: a number below 2^24, so that its
                // quotient by the blocks is off by one at most
                const unsigned before = with + earlier + __popc(given[j] & ((1u << lane) - 1u)), rank = one ? before : at - before;
                unsigned round = static_cast<unsigned>(static_cast<float>(rank) * per_step);
                if (round * step > rank) --round;
                if ((round + 1) * step <= rank) ++round;
                const unsigned whose = rank - round * step;
                if (at < window && whose == (one ? me : step - 1 - me)) list[one ? round : S::kList + 1 - round] = at;
            }
            with += __shfl_sync(kAllLanes, scan, 31);
        }
        const int rows = static_cast<int>((with + step - 1 - me) / step), empty_rows = static_cast<int>((window - with + me) / step);
        __syncthreads();

        // Copies: the next group of the stream into the ring; past the last row an empty
        // one, so that the count holds.
        int copy_number = 0, copy_group = 0, copy_place = 0, copy_count = 0;  // chunks of this thread's row from its next one on
        bool copy_before = false;                                             // its next one is before the share's first
        const T *copy_from = nullptr;
        auto start_copies = [&] {
            copy_count = 0;
            if (copy_number < rows) {
                const Share<DT> sh = share_of(base + list[copy_number]);
                const int c = begin_of(sh) + tid;
                copy_from = sh.row + sh.column(c, 0);
                copy_count = sh.end - c;
                copy_before = c < sh.first;
            }
        };
        auto copy_next = [&] {
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                if (u * THREADS < copy_count && !(u == 0 && copy_before))
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(ring_at + (copy_place * kGroup + u) * THREADS * 16),
                                    "l"(copy_from + u * THREADS * Chunk<DT>::kElems) : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
            copy_from += kGroupChunks * Chunk<DT>::kElems;
            copy_count -= kGroupChunks;
            copy_before = false;
            ++copy_group;
            if (AGAIN > 0 && copy_group == groups) start_copies();
            if (copy_group == groups + AGAIN) {
                copy_group = 0;
                ++copy_number;
                start_copies();
            }
            if (++copy_place == kRing) copy_place = 0;
        };
        auto held = [&](int place, int u) {
            const uint4 w = ring[(place * kGroup + u) * THREADS];
            return Chunk<DT>{{w.x, w.y, w.z, w.w}};
        };
        start_copies();
#pragma unroll 1
        for (int q = 0; q < kRing; ++q) copy_next();

#pragma unroll 1
        for (int i = 0; i < empty_rows; ++i) {
            const int64_t row = base + list[S::kList + 1 - i];
            if (block == 0 && tid == 0) write_results(a, row, 0.0f, 0.0f, 0.0f);
            if (GRAD) write_zeros<DT>(row_of<DT>(a.dlogits, row, a.dstride), a.cols, block, split, THREADS);
        }

        int next_place = 0;  // the ring's place of the stream's next group
        auto take_place = [&] {
            const int place = next_place;
            if (++next_place == kRing) next_place = 0;
            return place;
        };
        int my_token = -1;  // of 32 rows, this lane's
        float my_x = 0.0f;
        PolicyToken my = {};
#pragma unroll 1
        for (int number = 0; number < rows; ++number) {
            const int from = number & 31;
            const int64_t row = base + list[number];
            if (from == 0 && number + lane < rows) {
                const int64_t own = base + list[number + lane];
                my_token = token_of(own);
                my = policy_token(a, own, GRAD);
                my_x = share_of(own).at(my_token);
            }
            const int col = __shfl_sync(kAllLanes, my_token, from);
            const Share<DT> sh = share_of(row);
            const int begin = begin_of(sh);
            const bool single = tid < sh.singles;
            const float one = single ? sh.at(sh.single(tid)) : kNegInf;

            PairSums pairs = {kLeastExponent, both(0.0f), both(0.0f)};
            int held_from = next_place + AGAIN;  // the place of the first group that stays
            if (held_from >= kRing) held_from -= kRing;
            auto add_group = [&](int g) {
                const int place = take_place();
                Chunk<DT> r[kGroup];
                const int c0 = begin + g * kGroupChunks;
                if (c0 >= sh.first && c0 + kGroupChunks <= sh.end) {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) r[u] = held(place, u);
                } else {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) {
                        const int c = c0 + u * THREADS + tid;
                        r[u] = c >= sh.first && c < sh.end ? held(place, u) : masked_chunk<DT>();
                    }
                }
                add_chunks<DT, false>(pairs, r, ax);
                if (!GRAD || g < AGAIN) copy_next();
            };
            // A group is complete when only the groups asked for after it are left: kRing - 1
            // while each group used is one more asked for, one less for each that stays.
            static_assert(kRing == 6 && kMostGroups == 8, "one wait for each group below");
            auto left = [](int g) constexpr { return !GRAD || g <= AGAIN ? 5 : g < 5 + AGAIN ? 5 + AGAIN - g : 0; };
            copies_left<5>();
            add_group(0);
            if (groups > 1) { copies_left<left(1)>(); add_group(1); }
            if (groups > 2) { copies_left<left(2)>(); add_group(2); }
            if (groups > 3) { copies_left<left(3)>(); add_group(3); }
            if (groups > 4) { copies_left<left(4)>(); add_group(4); }
            if (groups > 5) { copies_left<left(5)>(); add_group(5); }
            if (groups > 6) { copies_left<left(6)>(); add_group(6); }
            if (groups > 7) { copies_left<left(7)>(); add_group(7); }

            Sums v = warp_sums<32, false>(finished<DT, false>(pairs, single, one, ax));
            if (lane == 0) part[turn][warp] = v;
            __syncthreads();
            v = sums_of_warps<kWarps, false>(part[turn]);
            if (blocks > 1) {
                if (tid == 0) mine[turn] = v;
                cluster_sync();  // the next row's keeps mine[turn] from being written before all have read it
                v = cluster_sums<false>(&mine[turn], blocks);
            }
            turn ^= 1;
            RowSum r;
            if (v.s > 0.0f && v.s < 1e37f) {
                r = {v.c, logf(v.s), 1.0f / v.s, 0.0f, 0.0f, false};
            } else {
                // a careful row is read whole by every thread of every block: all are done with it before any writes in place
                r = careful_row<DT>(sh.row, a.cols, ax, fpart);
                if (blocks > 1) cluster_sync();
            }
            const float x = __shfl_sync(kAllLanes, my_x, from);
            const PolicyToken t = {__shfl_sync(kAllLanes, my.advantage, from), __shfl_sync(kAllLanes, my.old_logp, from),
                                   __shfl_sync(kAllLanes, my.ref_logp, from), __shfl_sync(kAllLanes, my.dloss, from)};
            const bool empty = is_empty(r);
            const float logp = empty ? kNegInf : logp_of(r, x, ax, a.scale);
            const PolicyTerms terms = policy_terms(a, t, logp);
            if (block == 0 && tid == 0) write_results(a, row, terms.loss, logp, empty ? kNegInf : lse_of(r, a.scale));
            if constexpr (GRAD) {
                T *out = static_cast<T *>(row_of<DT>(a.dlogits, row, a.dstride));
                const float factor = policy_factor(a, t, terms);
                const RowGrad rg = row_grad({r.c, r.inv_s, r.top, r.careful}, -factor, 0.0f, 0.0f, 0.0f);
                const int apart = bytes_apart(out, sh);
                const ChunkGrad<DT, false> grad(rg, ax);
                const float at_token = grad_of<false>(rg, x, ax, a.scale) + factor;
                // first the groups that stayed, then those that were copied again
#pragma unroll 1
                for (int i = 0; i < groups; ++i) {
                    const bool stayed = AGAIN == 0 || i < kRing;
                    const int g = stayed ? AGAIN + i : i - kRing;
                    int place = held_from + i;
                    if (place >= kRing) place -= kRing;
                    if (!stayed) {
                        copies_left<kRing - 1>();
                        place = take_place();
                    }
                    if (!r.careful) {
                        const int c0 = begin + g * kGroupChunks + tid;
                        T *to = out + sh.column(c0, 0);
                        if (c0 - tid >= sh.first && c0 - tid + kGroupChunks <= sh.end) {
#pragma unroll
                            for (int u = 0; u < kGroup; ++u)
                                store_chunk<DT>(to + u * THREADS * Chunk<DT>::kElems, grad(held(place, u)), apart, true);
                        } else {
#pragma unroll
                            for (int u = 0; u < kGroup; ++u) {
                                const int c = c0 + u * THREADS;
                                if (c >= sh.first && c < sh.end)
                                    store_chunk<DT>(to + u * THREADS * Chunk<DT>::kElems, grad(held(place, u)), apart,
                                                    c - lane >= sh.first && c - lane + 31 < sh.end);
                            }
                        }
                    }
                    copy_next();  // into this group's place
                }
                if (!r.careful) {
                    if (single) store_one<DT>(out, sh.single(tid), grad_of<false>(rg, one, ax, a.scale));
                    // The token's column, over what the warp that has its chunk has stored (the
                    // whole chunk, where rows lie apart by the lanes before or after, too), or
                    // the thread that has the single element.
                    if (sh.holds(col)) {
                        const bool in_chunk = col >= sh.head && col < sh.tail0;
                        const int owner = in_chunk ? ((col - sh.head) / Chunk<DT>::kElems - begin) % THREADS
                                                   : col < sh.head ? col : sh.n_head + col - sh.tail0;
                        __syncwarp();
                        if (tid == owner) store_one<DT>(out, col, at_token);
                    }
                } else if (empty) {
                    write_zeros<DT>(out, a.cols, block, split, THREADS);
                } else {
                    write_grad_slowly<DT, false>(sh, out, rg, ax, a.scale, THREADS);
                    __syncthreads();
                    if (tid == 0 && sh.holds(col)) store_one<DT>(out, col, at_token);
                }
            }
        }
        copies_left<0>();
    }
    if (blocks > 1) cluster_sync();  // no block leaves while its sums are read
}

// ---------------------------------------------------------------- launches

template <int DT, int THREADS>
cudaError_t policy_twice(const PolicyArgs &a, bool sums, bool grad, int shift, cudaStream_t s, LaunchInfo *info) {
    const Split split = split_of<DT>(a.cols, shift);
    const int64_t grid = a.rows << shift;
    info->grid = static_cast<int>(grid);
    info->block = THREADS;
    info->vec_bytes = 16;
    auto kernel = policy_kernel<DT, false, true, THREADS>;
    if (sums) kernel = grad ? policy_kernel<DT, true, true, THREADS> : policy_kernel<DT, true, false, THREADS>;
    return launch_rows(kernel, dim3(grid), dim3(THREADS), 0, split.blocks(), s, a, split);
}

// Rows that are worked on at once: an SM's blocks, or as many clusters of a row's
// blocks as fit the device (a cluster lies within one of its partitions); asked
// once for each size of block and of cluster on a device (past 15, every time).
template <int THREADS, typename Kernel> cudaError_t rows_at_once(Kernel kernel, int shift, int sms, int *rows) {
    *rows = sms * Stream<THREADS>::kBlocks;
    if (shift == 0) return cudaSuccess;
    constexpr int kKnown = 16;
    static std::atomic<int> known[kKnown][4];  // the loss, and the loss with its gradient, have the same block and memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kKnown && (*rows = known[dev][shift].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms >> shift << shift);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Stream<THREADS>::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << shift;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(rows, kernel, &cfg);
    *rows = std::max(1, *rows);
    if (e == cudaSuccess && dev < kKnown) known[dev][shift].store(*rows, std::memory_order_relaxed);
    return e;
}
// Groups that a row's share takes when 2^shift blocks of THREADS split it, up to 7
// chunks more where a share may begin within a line.
template <int DT, int THREADS> int groups_of(const PolicyArgs &a, int shift) {
    const int64_t each = split_of<DT>(a.cols, shift).each;
    const bool lines = reinterpret_cast<uintptr_t>(a.logits) % 128 == 0 && a.stride * ElemOf<DT>::kBytes % 128 == 0 &&
                       (shift == 0 || each % 8 == 0);
    constexpr int kChunks = Stream<THREADS>::kGroupChunks;
    return static_cast<int>(std::max<int64_t>(1, (each + (lines ? 0 : 7) + kChunks - 1) / kChunks));
}
template <int DT, int THREADS>
cudaError_t policy_stream(const PolicyArgs &a, bool grad, int shift, int sms, cudaStream_t s, LaunchInfo *info) {
    const Split split = split_of<DT>(a.cols, shift);
    const int groups = groups_of<DT, THREADS>(a, shift), again = grad ? std::max(0, groups - kRing) : 0;
    auto kernel = grad ? policy_stream_kernel<DT, true, THREADS, 0> : policy_stream_kernel<DT, false, THREADS, 0>;
    if constexpr (THREADS == 512) {
        if (again == 1) kernel = policy_stream_kernel<DT, true, THREADS, 1>;
        if (again == 2) kernel = policy_stream_kernel<DT, true, THREADS, 2>;
    }
    static std::atomic<uint64_t> allowed[4];
    int at_once = 0;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), Stream<THREADS>::kSmem, &allowed[grad ? 1 + again : 0]);
    if (e == cudaSuccess) e = rows_at_once<THREADS>(kernel, shift, sms, &at_once);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>(a.rows, at_once) << shift;
    info->grid = static_cast<int>(grid);
    info->block = THREADS;
    info->vec_bytes = 16;
    info->smem = Stream<THREADS>::kSmem;
    return launch_rows(kernel, dim3(grid), dim3(THREADS), Stream<THREADS>::kSmem, split.blocks(), s, a, split, groups);
}

template <int DT> cudaError_t policy_launch(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    // The loss alone splits and sums its rows as loss and gradient in one call do, so
    // both give the same bits.
    constexpr int64_t kKiB = 1024;
    const int64_t bytes = static_cast<int64_t>(a.cols) * ElemOf<DT>::kBytes;
    const bool few = a.rows <= sms;
    if (sums && !few && bytes > 24 * kKiB) {
        if (bytes <= 32 * kKiB) return policy_stream<DT, 128>(a, grad, 0, sms, s, info);
        if (groups_of<DT, 256>(a, 0) <= kRing) return policy_stream<DT, 256>(a, grad, 0, sms, s, info);
        int shift = 0;
        while (shift < 3 && groups_of<DT, 512>(a, shift) > kMostGroups) ++shift;
        if (groups_of<DT, 512>(a, shift) <= kMostGroups) return policy_stream<DT, 512>(a, grad, shift, sms, s, info);
    }
    if (!few && bytes <= 32 * kKiB) return policy_twice<DT, kNarrow>(a, sums, grad, 0, s, info);
    return policy_twice<DT, kThreads>(a, sums, grad, split_shift(a.rows, a.cols, sms), s, info);
}

}  // namespace
}  // namespace ew
