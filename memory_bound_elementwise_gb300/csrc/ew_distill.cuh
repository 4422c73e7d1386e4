// ew_distill.cuh -- distillation from a teacher's top logits, loss and gradient.
// Compiled once per element type.
//
// q = softmax of the teacher's values at its ids, p = softmax of the student's
// row, both of values times `scale`:
//     loss = sum q_i (log q_i - log p(id_i)),   dlogits = dloss scale (p - q).
// Entries with an id outside the row or a value of -inf do not count; a row
// without any has loss 0 and gradient 0.
//
// The gradient needs the row's sums, so a row is worked over twice.  At the
// floor it crosses DRAM once: distill_stream_kernel keeps it in shared memory
// in between.  distill_kernel reads it again, mostly from L2: for rows too short to
// be worth a ring, rows too long, and the gradient from a given lse.  4096 rows
// of 65536 bf16 take 179 us (6.0 TB/s, floor 159), 2104 rows of 1000 9 us.
#pragma once

#include "ew_logits.cuh"

namespace ew {
namespace {

// What a block has of a row's teacher: for each entry the student's column
// (-1: does not count), the scaled value (-inf) and the student's logit.
struct Teacher {
    int *id;  // at a multiple of 16 bytes, -1 up to a multiple of 4 entries
    float *t, *x;
    __host__ __device__ static int padded(int k) { return (k + 3) & ~3; }
    __host__ __device__ static int bytes(int k) { return padded(k) * 12; }
    __device__ __forceinline__ Teacher(void *at, int k) : id(static_cast<int *>(at)), t(static_cast<float *>(at) + padded(k)),
                                                          x(static_cast<float *>(at) + 2 * padded(k)) {}
};
struct TeacherEntry {
    int id;
    float t;
};
// An entry as it lies in memory; what it says is worked out when it is needed,
// so that reading it ahead does not wait for it.
template <int DT> struct RawEntry {
    int64_t id;
    uint32_t value;
    __device__ __forceinline__ void read(const DistillArgs &a, int64_t row, int i) {
        id = token_at(a.ids, a.i64, row * a.ids_stride + i);
        const int64_t at = row * a.teacher_stride + i;
        if (DT == DT_F32 || a.teacher_f32) value = static_cast<const uint32_t *>(a.teacher)[at];
        else value = static_cast<const typename ElemOf<DT>::type *>(a.teacher)[at];
    }
    __device__ __forceinline__ TeacherEntry entry(const DistillArgs &a) const {
        float v;
        if (DT == DT_F32 || a.teacher_f32) v = __uint_as_float(value);
        else v = elem_to_f32<DT>(static_cast<typename ElemOf<DT>::type>(value));
        const bool given = id >= 0 && id < a.cols && v != kNegInf;
        return {given ? static_cast<int>(id) : -1, given ? v * a.scale : kNegInf};
    }
};

// The softmax of the teacher's k values, by each warp that needs it for itself.
struct TeacherSum {
    float top, log_sum;
    __device__ __forceinline__ float log_q(float t) const { return t - top - log_sum; }
};
constexpr int kAtOnce = 2;  // entries of a lane whose latencies overlap
__device__ __forceinline__ float teacher_top(const float *t, int k) {
    float top = kNegInf;
    for (int i = threadIdx.x & 31; i < k; i += 32 * kAtOnce)
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) top = max_nan(top, i + 32 * e < k ? t[i + 32 * e] : kNegInf);
    return lanes_max_nan(top, 32);
}
__device__ __forceinline__ TeacherSum teacher_sum(const float *t, int k) {
    const float top = teacher_top(t, k);
    float sum = 0.0f;
    for (int i = threadIdx.x & 31; i < k; i += 32 * kAtOnce)
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const float v = i + 32 * e < k ? t[i + 32 * e] : kNegInf;
            sum += v == kNegInf ? 0.0f : expf(v - top);
        }
    return {top, logf(warp_sum(sum))};
}
// Called by one warp: the row's loss, to all its lanes, and the teacher's
// softmax with it.  With e_i = exp(t_i - top) the loss is
//     sum e_i (t_i - top - log p_i) / sum e_i - log sum e_i,
// two sums that do not wait for one another: in the rows held in shared memory
// this is the longest chain between two barriers.  The first is kept in parts of
// kLossPart, so that terms near the end of binary32 do not overflow it together.
constexpr float kLossPart = 1.0f / (2 * kMostTeacher);  // a power of two
__device__ __forceinline__ float loss_of(const Teacher &th, int k, const RowSum &r, float a, float scale, TeacherSum &q) {
    const bool empty = r.careful && r.top == kNegInf;
    const float top = teacher_top(th.t, k);
    float sum = 0.0f, loss = 0.0f;
    for (int i = threadIdx.x & 31; i < k; i += 32 * kAtOnce)
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const bool given = i + 32 * e < k;
            const float t = given ? th.t[i + 32 * e] : kNegInf, x = given ? th.x[i + 32 * e] : 0.0f;
            const float w = t == kNegInf ? 0.0f : expf(t - top);
            const float logp = empty ? kNegInf : logp_of(r, x, a, scale);
            sum += w;
            if (w != 0.0f) loss += w * kLossPart * (t - top - logp);
        }
    sum = warp_sum(sum);
    q = {top, logf(sum)};
    return warp_sum(loss) / sum / kLossPart - q.log_sum;
}
// Whether any two entries have the same id: a table of at least 4k ids, open
// addressing.  Entries of one id add up to one column; a teacher's top values
// have none, and comparing 256 entries with each other takes as long as the
// gradient of 30000 columns.  Up to kCompared entries are compared all the same.
constexpr int kCompared = 32;
struct IdTable {
    int *slot;
    int mask;
    __host__ __device__ static int slots(int k) {
        int n = 0;
        if (k > kCompared)
            for (n = 8 * kCompared; n < 4 * k;) n *= 2;
        return n;
    }
    __device__ __forceinline__ void clear(int me, int workers) const {
        for (int i = me; i <= mask; i += workers) slot[i] = -1;
    }
    // false where the id is there already
    __device__ __forceinline__ bool add(int id) const {
        int at = static_cast<int>(id * 2654435769u >> __clz(mask));  // the product's first bits
        for (int tries = 0; tries <= mask; ++tries, at = (at + 1) & mask) {
            const int was = atomicCAS(slot + at, -1, id);
            if (was == -1) return true;
            if (was == id) return false;
        }
        return false;  // not reached: more slots than entries
    }
};
// The teacher's columns of the block's share, by `workers` threads of which this
// is number `me`.  Where entries may share an id (`shared_ids`) they add up and
// the first of them writes.
template <int DT>
__device__ __forceinline__ void write_teacher_columns(const Share<DT> &sh, void *out, const Teacher &th, int k,
                                                      const TeacherSum &q, const RowGrad &g, float a, bool shared_ids,
                                                      int me, int workers) {
    for (int i = me; i < k; i += workers) {
        const int id = th.id[i];
        if (id < 0 || !sh.holds(id)) continue;
        float qs = expf(q.log_q(th.t[i]));
        if (shared_ids) {
            int alike = 0, earlier = 0;
            const int4 *ids = reinterpret_cast<const int4 *>(th.id);
#pragma unroll 4
            for (int j = 0; j < k; j += 4) {
                const int4 b = ids[j / 4];
                const int same = (b.x == id) + (b.y == id) + (b.z == id) + (b.w == id);
                alike += same;
                if (j < i) earlier += j + 4 <= i ? same : (b.x == id) + (j + 1 < i && b.y == id) + (j + 2 < i && b.z == id);
            }
            if (earlier) continue;
            for (int j = i + 1; alike > 1 && j < k; ++j)
                if (th.id[j] == id) qs += expf(q.log_q(th.t[j]));
        }
        store_one<DT>(out, id, g.g * (p_of(g.w, th.x[i], a) - qs));
    }
}

// ---------------------------------------------------------------- rows read twice

template <int DT, bool SUMS, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, kResident * kThreads / THREADS) distill_kernel(DistillArgs a, Split split) {
    enter_grid();
    extern __shared__ uint4 dynamic[];
    __shared__ Sums part[THREADS / 32];
    __shared__ Sums mine;
    __shared__ float fpart[32];
    __shared__ int shared_ids;
    const Teacher th(dynamic, a.k);
    const IdTable table = {static_cast<int *>(static_cast<void *>(dynamic)) + 3 * Teacher::padded(a.k), IdTable::slots(a.k) - 1};
    const int blocks = split.blocks(), block = blockIdx.x & (blocks - 1);
    const int64_t row = blockIdx.x >> split.shift;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const void *logits = row_of<DT>(a.logits, row, a.stride);
    const Share<DT> sh(logits, a.cols, block, split);
    const float ax = a.scale * kLog2e;

    Chunk<DT> first_turn[kFlight];  // on its way while the teacher's entries are
    if constexpr (SUMS) load_turn<DT, THREADS>(sh, sh.first + static_cast<int>(threadIdx.x), first_turn);
    // Every block has all entries; of the student's logits the loss (block 0)
    // needs all, the gradient those that this block writes.
    bool mine_counts = false;
    RawEntry<DT> raw;
    if (static_cast<int>(threadIdx.x) < a.k) raw.read(a, row, threadIdx.x);
    if constexpr (GRAD) {
        if (threadIdx.x == 0) shared_ids = a.k > 1 && a.k <= kCompared;
        table.clear(threadIdx.x, THREADS);
        __syncthreads();
    }
    for (int i = threadIdx.x; i < a.k; i += THREADS) {
        if (i >= THREADS) raw.read(a, row, i);
        const TeacherEntry e = raw.entry(a);
        const bool read = e.id >= 0 && ((SUMS && block == 0) || sh.holds(e.id));
        th.id[i] = e.id;
        th.t[i] = e.t;
        th.x[i] = read ? sh.at(e.id) : 0.0f;
        mine_counts = mine_counts || e.id >= 0;
        if (GRAD && a.k > kCompared && e.id >= 0 && !table.add(e.id)) shared_ids = 1;
    }
    if (a.k + static_cast<int>(threadIdx.x) < Teacher::padded(a.k)) th.id[a.k + threadIdx.x] = -1;
    Sums v = no_sums();
    float largest, bound;
    if constexpr (SUMS) v = warp_sums<32, false>(pass_over<DT, false, false, THREADS>(sh, ax, nullptr, 0, first_turn, largest, bound));
    if (lane == 0) part[warp] = v;
    const bool any = __syncthreads_or(mine_counts);

    Weights w;
    RowSum r;
    if constexpr (SUMS) {
        v = sums_of_warps<THREADS / 32, false>(part);
        if (blocks > 1) {
            if (threadIdx.x == 0) mine = v;
            cluster_sync();
            v = cluster_sums<false>(&mine, blocks);
            cluster_arrive();  // the wait is further down: mine has been read
        }
        r = finish_row<DT, false>(v, logits, a.cols, ax, fpart);
        w = {r.c, r.inv_s, r.top, r.careful};
        if (block == 0 && warp == 0) {
            TeacherSum q;
            const float loss = loss_of(th, a.k, r, ax, a.scale, q);
            if (lane == 0) {
                a.loss[row] = any ? loss : 0.0f;
                a.lse[row] = r.careful && r.top == kNegInf ? kNegInf : lse_of(r, a.scale);
            }
        }
    } else {
        // every block of the row decides alike
        const float lse = a.lse[row];
        if (!any || lse_holds(lse)) {
            w = weights_of(lse);
        } else {
            const RowSum again = careful_row<DT>(logits, a.cols, ax, fpart);
            if (blocks > 1) cluster_sync();  // all have read the row before any writes in place
            w = {0.0f, again.inv_s, again.top, true};
        }
    }
    if constexpr (GRAD) {
        const RowGrad rg = row_grad(w, any ? a.dloss[row] * a.scale : 0.0f, 0.0f, 0.0f, 0.0f);
        void *out = row_of<DT>(a.dlogits, row, a.dstride);
        // a careful row has been read whole by every block: all are done with it before any writes in place
        if (SUMS && w.careful) {
            if (blocks > 1) {
                cluster_wait();
                cluster_sync();
                cluster_arrive();
            } else {
                __syncthreads();
            }
        }
        if (any) {
            write_grad<DT, false, THREADS>(sh, out, rg, ax, a.scale);
            __syncthreads();
            // by the last threads: the first warp has the loss to do
            const int me = THREADS - 1 - static_cast<int>(threadIdx.x);
            if ((me & ~31) < a.k)
                write_teacher_columns<DT>(sh, out, th, a.k, teacher_sum(th.t, a.k), rg, ax, shared_ids != 0, me, THREADS);
        } else {
            write_zeros<DT>(out, a.cols, block, split, THREADS);
        }
    }
    if (SUMS && blocks > 1) cluster_wait();
}

// ---------------------------------------------------------------- rows held in shared memory
//
// A block walks over rows; one of 512 streaming threads an SM (or a cluster of
// up to 8 for a row), two of 256 for rows up to 64 KiB, four of 128 up to
// 32 KiB: the shorter the row, the more its barrier weighs, and the blocks cover
// one another's.  The block's share of a row is `groups` groups of 4 chunks a
// streaming thread; a ring of kRing groups is filled by asynchronous copies in
// the order of the stream of groups, row after row, and a group's place is
// filled again as soon as the gradient (or, for the loss alone, the sum) has
// used it.  So kRing - groups groups of rows to come are on their way at any
// time, through the reductions too.  Each thread copies and reads its own chunks
// only: it waits for its own copies and needs no barrier for them.
//
// A row has one barrier, between its sums and its gradient.  Between two of
// them a streaming thread writes one row's gradient and sums the next row.
// What is left is done by warps that do not stream, a quarter as many, so that
// no streaming warp is waited for: they read the teachers ahead, take the
// losses, and write the teacher's columns, whose gradient has to come after all
// others' stores, a row later.  With this work given to streaming warps 4096
// rows of 65536 bf16 took 212 us; now 179, at a floor of 159.  Their chain from
// barrier to barrier must stay shorter than a row's stream: the loss, the
// longest part, is 2 us under load, and has a warp to itself.

constexpr int kGroup = 4;
constexpr int kRing = 6;
template <int T> struct Stream {  // T streaming threads
    static constexpr int kWarps = T / 32;
    static constexpr int kHelpers = T / 4;
    static constexpr int kEntries = 2;                       // of a teacher, a helper's
    static constexpr int kMostEntries = kEntries * kHelpers;
    static constexpr int kGroupChunks = kGroup * T;
    static constexpr int kBlocks = 512 / T;                  // an SM's
    static constexpr int kMostSmem = kRing * kGroupChunks * 16 + 3 * kMostEntries * 12 + 2 * 4 * kMostEntries * 4;
};

template <int DT, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS + Stream<THREADS>::kHelpers, Stream<THREADS>::kBlocks)
    distill_stream_kernel(DistillArgs a, Split split, int groups) {
    using T = typename ElemOf<DT>::type;
    using S = Stream<THREADS>;
    constexpr int kEntries = S::kEntries, kHelpers = S::kHelpers, kGroupChunks = S::kGroupChunks;
    enter_grid();
    extern __shared__ uint4 dynamic[];
    __shared__ Sums part[2][S::kWarps];
    __shared__ Sums mine[2];
    __shared__ float fpart[32];
    __shared__ int shared_ids[4];
    __shared__ TeacherSum teacher_sums[3];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const bool streams = tid < THREADS;
    const int helper = THREADS + kHelpers - 1 - tid;  // from the last on: the last numbers' warp has the loss to do
    uint4 *ring = dynamic + tid;  // a streaming thread's
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    char *teachers = reinterpret_cast<char *>(dynamic + kRing * kGroupChunks);
    const int blocks = split.blocks(), block = blockIdx.x & (blocks - 1);
    const int64_t step = gridDim.x >> split.shift, first_row = blockIdx.x >> split.shift;
    const float ax = a.scale * kLog2e;

    auto share_of = [&](int64_t row) {
        return Share<DT>(row_of<DT>(a.logits, row, a.stride), a.cols, block, split);
    };
    // three teachers: the row's, the one before, whose columns are still to be written, and the next
    auto teacher_of = [&](int third) { return Teacher(teachers + third * Teacher::bytes(a.k), a.k); };
    // the row's sums, after the barrier: the same bits in every thread of the cluster
    auto row_sums = [&](int turn) {
        Sums v = sums_of_warps<S::kWarps, false>(part[turn]);
        if (blocks > 1) {
            if (tid == 0) mine[turn] = v;
            cluster_sync();  // the next row's keeps mine[turn] from being written before all have read it
            v = cluster_sums<false>(&mine[turn], blocks);
        }
        return v;
    };
    auto shortcuts_hold = [](const Sums &v) { return v.s > 0.0f && v.s < 1e37f; };
    // a careful row is read whole by every thread of every block: all are done with it before any writes in place
    auto careful_sums = [&](const void *logits) {
        const RowSum r = careful_row<DT>(logits, a.cols, ax, fpart);
        if (blocks > 1) cluster_sync();
        return r;
    };

    if (streams) {
        // the next group of the stream into the ring; past the last row an empty one, so that the count holds
        int64_t copy_row = first_row;
        int copy_group = 0, copy_place = 0, copy_count = 0;  // chunks of this thread's row from its next one on
        const T *copy_from = nullptr;
        auto start_copies = [&] {
            copy_count = 0;
            if (copy_row < a.rows) {
                const Share<DT> sh = share_of(copy_row);
                copy_from = sh.row + sh.column(sh.first + tid, 0);
                copy_count = sh.end - sh.first - tid;
            }
        };
        auto copy_next = [&] {
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                if (u * THREADS < copy_count)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(ring_at + (copy_place * kGroup + u) * THREADS * 16),
                                    "l"(copy_from + u * THREADS * Chunk<DT>::kElems) : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
            copy_from += kGroupChunks * Chunk<DT>::kElems;
            copy_count -= kGroupChunks;
            if (++copy_group == groups) {
                copy_group = 0;
                copy_row += step;
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

        int place0 = 0;  // the ring's place of the row's first group
        int turn = 0;
#pragma unroll 1
        for (int64_t row = first_row; row < a.rows; row += step, turn ^= 1) {
            const Share<DT> sh = share_of(row);
            const bool single = tid < sh.singles;
            const float one = single ? sh.at(sh.single(tid)) : kNegInf;
            const float dloss = GRAD ? a.dloss[row] : 0.0f;

            PairSums pairs = {kLeastExponent, both(0.0f), both(0.0f)};
            auto add_group = [&](int g) {
                int place = place0 + g;
                if (place >= kRing) place -= kRing;
                Chunk<DT> r[kGroup];
                const int c0 = sh.first + g * kGroupChunks;
                if (c0 + kGroupChunks <= sh.end) {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) r[u] = held(place, u);
                } else {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u)
                        r[u] = c0 + u * THREADS + tid < sh.end ? held(place, u) : masked_chunk<DT>();
                }
                add_chunks<DT, false>(pairs, r, ax);
                if (!GRAD) copy_next();
            };
            // Group g of the row is complete when only the groups after it are left:
            // kRing - 1 - g have been asked for since, or, with one more for each
            // group that the loss alone has used, kRing - 1.
            static_assert(kRing == 6, "one wait for each group below");
            copies_left<5>();
            add_group(0);
            if (groups > 1) { copies_left<GRAD ? 4 : 5>(); add_group(1); }
            if (groups > 2) { copies_left<GRAD ? 3 : 5>(); add_group(2); }
            if (groups > 3) { copies_left<GRAD ? 2 : 5>(); add_group(3); }
            if (groups > 4) { copies_left<GRAD ? 1 : 5>(); add_group(4); }
            if (groups > 5) { copies_left<GRAD ? 0 : 5>(); add_group(5); }

            Sums v = warp_sums<32, false>(finished<DT, false>(pairs, single, one, ax));
            if (lane == 0) part[turn][warp] = v;
            const bool any = __syncthreads_or(0);
            v = row_sums(turn);
            Weights w = {v.c, 0.0f, 0.0f, false};
            if (shortcuts_hold(v)) {
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(w.weight) : "f"(v.s));
            } else {
                const RowSum r = careful_sums(sh.row);
                w = {r.c, r.inv_s, r.top, true};
            }
            if constexpr (GRAD) {
                T *out = static_cast<T *>(row_of<DT>(a.dlogits, row, a.dstride));
                const RowGrad rg = row_grad(w, any ? dloss * a.scale : 0.0f, 0.0f, 0.0f, 0.0f);
                const bool fast = any && !w.careful;
                const int apart = bytes_apart(out, sh);
                const ChunkGrad<DT, false> grad(rg, ax);
#pragma unroll 1
                for (int g = 0; g < groups; ++g) {
                    int place = place0 + g;
                    if (place >= kRing) place -= kRing;
                    if (fast) {
                        const int c0 = sh.first + g * kGroupChunks + tid;
                        T *to = out + sh.column(c0, 0);
                        if (sh.first + (g + 1) * kGroupChunks <= sh.end) {
#pragma unroll
                            for (int u = 0; u < kGroup; ++u)
                                store_chunk<DT>(to + u * THREADS * Chunk<DT>::kElems, grad(held(place, u)), apart, true);
                        } else {
#pragma unroll
                            for (int u = 0; u < kGroup; ++u)
                                if (c0 + u * THREADS < sh.end)
                                    store_chunk<DT>(to + u * THREADS * Chunk<DT>::kElems, grad(held(place, u)), apart,
                                                    c0 - lane + 31 + u * THREADS < sh.end);
                        }
                    }
                    copy_next();  // into this group's place
                }
                if (fast) {
                    if (single) store_one<DT>(out, sh.single(tid), grad_of<false>(rg, one, ax, a.scale));
                } else if (any) {
                    write_grad_slowly<DT, false>(sh, out, rg, ax, a.scale, THREADS);
                } else {
                    write_zeros<DT>(out, a.cols, block, split, THREADS);
                }
            }
            place0 += groups;
            if (place0 >= kRing) place0 -= kRing;
        }
        copies_left<0>();
        __syncthreads();  // the last row's stores precede its teacher's columns
    } else {
        // Entries of the row and of the next one: read a row ahead, and the
        // student's logits there asked for while the row before is summed.
        // Neither is looked at before it is needed: under load a read takes
        // 3 us.  Every block has all entries; of the logits the loss (block 0)
        // needs all, the gradient those that this block writes.
        RawEntry<DT> raw[kEntries] = {};
        TeacherEntry entry[kEntries];
        T x[kEntries] = {};
        auto read_entries = [&](int64_t row) {
#pragma unroll
            for (int e = 0; e < kEntries; ++e)
                if (helper + e * kHelpers < a.k && row < a.rows) raw[e].read(a, row, helper + e * kHelpers);
        };
        auto read_logits = [&](int64_t row) {
            if (row >= a.rows) return;
            const Share<DT> sh = share_of(row);
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                entry[e] = helper + e * kHelpers < a.k ? raw[e].entry(a) : TeacherEntry{-1, kNegInf};
                if (entry[e].id >= 0 && (block == 0 || (GRAD && sh.holds(entry[e].id)))) x[e] = sh.row[entry[e].id];
            }
        };
        read_entries(first_row);
        read_logits(first_row);
        read_entries(first_row + step);
        // two tables of ids: a row's is cleared after its barrier and used again after the next one
        int *slots = reinterpret_cast<int *>(teachers + 3 * Teacher::bytes(a.k));
        auto table_of = [&](int turn) { return IdTable{slots + turn * IdTable::slots(a.k), IdTable::slots(a.k) - 1}; };
        if (GRAD && a.k > kCompared) {
            for (int t = 0; t < 2; ++t) table_of(t).clear(helper, kHelpers);
            if (helper < 4) shared_ids[helper] = 0;
            asm volatile("barrier.sync 1, %0;" :: "n"(kHelpers) : "memory");  // the helpers alone
        }
        int turn = 0, third = 0, quarter = 0;  // the row's number modulo 2, 3 and 4
        bool left = false;        // the row before has columns to be written
        RowGrad left_grad = {};
        auto finish_left = [&](int64_t row, int third, int quarter) {
            const bool shared = a.k <= kCompared ? a.k > 1 : shared_ids[quarter] != 0;
            if (GRAD && left)
                write_teacher_columns<DT>(share_of(row), row_of<DT>(a.dlogits, row, a.dstride), teacher_of(third), a.k,
                                          teacher_sums[third], left_grad, ax, shared, helper, kHelpers);
        };
        int64_t row = first_row;
#pragma unroll 1
        for (; row < a.rows; row += step) {
            const Teacher th = teacher_of(third);
            bool mine_counts = false;
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                const int i = helper + e * kHelpers;
                if (i < a.k) {
                    th.id[i] = entry[e].id;
                    th.t[i] = entry[e].t;
                    th.x[i] = elem_to_f32<DT>(x[e]);
                    mine_counts = mine_counts || entry[e].id >= 0;
                    if (GRAD && a.k > kCompared && entry[e].id >= 0 && !table_of(turn).add(entry[e].id))
                        shared_ids[quarter] = 1;
                } else if (i < Teacher::padded(a.k)) {
                    th.id[i] = -1;
                }
            }
            read_logits(row + step);
            read_entries(row + 2 * step);
            const float dloss = GRAD ? a.dloss[row] : 0.0f;
            const bool any = __syncthreads_or(mine_counts);
            const Sums v = row_sums(turn);
            RowSum r;
            if (shortcuts_hold(v)) {
                r = {v.c, logf(v.s), 0.0f, 0.0f, 0.0f, false};
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv_s) : "f"(v.s));
            } else {
                r = careful_sums(row_of<DT>(a.logits, row, a.stride));
            }
            finish_left(row - step, third == 0 ? 2 : third - 1, quarter + 3 & 3);
            if (GRAD && a.k > kCompared) {  // for the next row but one, whose flag was last read before the barrier
                table_of(turn).clear(helper, kHelpers);
                if (helper == 0) shared_ids[quarter + 2 & 3] = 0;
            }
            if (helper >= kHelpers - 32) {
                TeacherSum q;
                const float loss = loss_of(th, a.k, r, ax, a.scale, q);
                if (lane == 0) teacher_sums[third] = q;  // for its columns, after the next barrier
                if (block == 0 && lane == 0) {
                    a.loss[row] = any ? loss : 0.0f;
                    a.lse[row] = r.careful && r.top == kNegInf ? kNegInf : lse_of(r, a.scale);
                }
            }
            left = any;
            left_grad = row_grad({r.c, r.inv_s, r.top, r.careful}, dloss * a.scale, 0.0f, 0.0f, 0.0f);
            turn ^= 1;
            third = third == 2 ? 0 : third + 1;
            quarter = quarter + 1 & 3;
        }
        __syncthreads();
        finish_left(row - step, third == 0 ? 2 : third - 1, quarter + 3 & 3);
    }
    if (blocks > 1) cluster_sync();  // no block leaves while its sums are read
}

// ---------------------------------------------------------------- launches

// Rows that are worked on at once: an SM's blocks, or as many clusters of a
// row's blocks as fit the device (a cluster lies within one of its
// partitions); asked once for each kernel and size of cluster, on the first
// device that calls.
template <int THREADS, typename Kernel> cudaError_t rows_at_once(Kernel kernel, int shift, int sms, int *rows) {
    *rows = sms * Stream<THREADS>::kBlocks;
    if (shift == 0) return cudaSuccess;
    static std::atomic<int> known[4];  // the loss, and the loss with its gradient, have the same block and memory
    if ((*rows = known[shift].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms >> shift << shift);
    cfg.blockDim = dim3(THREADS + Stream<THREADS>::kHelpers);
    cfg.dynamicSmemBytes = Stream<THREADS>::kMostSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << shift;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(rows, kernel, &cfg);
    if (e == cudaSuccess) known[shift].store(*rows = std::max(1, *rows), std::memory_order_relaxed);
    return e;
}

// Groups that a row's share takes when 2^shift blocks of THREADS split it.
template <int DT, int THREADS> int groups_of(int cols, int shift) {
    return std::max(1, (split_of<DT>(cols, shift).each + Stream<THREADS>::kGroupChunks - 1) / Stream<THREADS>::kGroupChunks);
}
template <int DT, int THREADS>
cudaError_t stream_launch(const DistillArgs &a, bool grad, int shift, int sms, cudaStream_t s, LaunchInfo *info) {
    using S = Stream<THREADS>;
    const Split split = split_of<DT>(a.cols, shift);
    auto kernel = grad ? distill_stream_kernel<DT, true, THREADS> : distill_stream_kernel<DT, false, THREADS>;
    static std::atomic<uint64_t> allowed[2];
    int at_once = 0;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), S::kMostSmem, &allowed[grad]);
    if (e == cudaSuccess) e = rows_at_once<THREADS>(kernel, shift, sms, &at_once);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>(a.rows, at_once) << shift;
    const int smem = kRing * S::kGroupChunks * 16 + 3 * Teacher::bytes(a.k) + 2 * 4 * IdTable::slots(a.k);
    info->grid = static_cast<int>(grid);
    info->block = THREADS + S::kHelpers;
    info->vec_bytes = 16;
    info->smem = smem;
    return launch_rows(kernel, dim3(grid), dim3(THREADS + S::kHelpers), smem, split.blocks(), s, a, split,
                       groups_of<DT, THREADS>(a.cols, shift));
}

template <int DT, int THREADS>
cudaError_t twice_launch(const DistillArgs &a, bool sums, bool grad, int shift, cudaStream_t s, LaunchInfo *info) {
    const Split split = split_of<DT>(a.cols, shift);
    const int64_t grid = a.rows << shift;
    const int smem = Teacher::bytes(a.k) + 4 * IdTable::slots(a.k);
    info->grid = static_cast<int>(grid);
    info->block = THREADS;
    info->vec_bytes = 16;
    info->smem = smem;
    auto kernel = distill_kernel<DT, false, true, THREADS>;
    if (sums) kernel = grad ? distill_kernel<DT, true, true, THREADS> : distill_kernel<DT, true, false, THREADS>;
    return launch_rows(kernel, dim3(grid), dim3(THREADS), smem, split.blocks(), s, a, split);
}

// Which kernel, by the bytes of a row and the teacher's entries.  Measured for
// 8000 bf16 rows, times in us, against the kernel that reads rows twice with 64
// threads a row (up to 32 KiB) or 256:
//     row of    entries   in shared memory   read twice
//     16 KiB       8             63              56
//     24 KiB    8, 64          78, 84          88, 91
//     48 KiB    8, 128        136, 153        156, 176
//    128 KiB    8, 256        335, 410        466, 466
// With more entries than a block's helpers hold (64, 128 or 256) reading twice
// is as fast or faster.  Read twice, 8000 rows of 2 KiB take 24 us with 64
// threads and 69 us with 256.  Where there is an SM for each row, blocks of 256
// streaming threads do from 16 KiB on (100 rows: 5.4 us against 6.9), and longer
// rows are split.
template <int DT>
cudaError_t distill_launch(const DistillArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    // The loss alone splits and sums its rows as loss and gradient in one call
    // do, so both give the same bits.
    constexpr int64_t kKiB = 1024;
    const int64_t bytes = static_cast<int64_t>(a.cols) * ElemOf<DT>::kBytes;
    const bool few = a.rows <= sms;
    if (sums && !few && bytes > 24 * kKiB && bytes <= 32 * kKiB && a.k <= Stream<128>::kMostEntries)
        return stream_launch<DT, 128>(a, grad, 0, sms, s, info);
    if (sums && bytes > (few ? 16 : 32) * kKiB && bytes <= (few ? 32 : 64) * kKiB && a.k <= Stream<256>::kMostEntries)
        return stream_launch<DT, 256>(a, grad, 0, sms, s, info);
    if (sums && bytes > (few ? 32 : 64) * kKiB && a.k <= Stream<512>::kMostEntries) {
        // at most 4 groups a row, so that 2 are on their way
        int shift = 0;
        while (shift < 3 && groups_of<DT, 512>(a.cols, shift) > 4) ++shift;
        while (shift < 3 && a.rows << (shift + 1) <= sms && a.cols >> (shift + 1) >= 4096) ++shift;
        if (groups_of<DT, 512>(a.cols, shift) <= kRing) return stream_launch<DT, 512>(a, grad, shift, sms, s, info);
    }
    if (!few && bytes <= 32 * kKiB) return twice_launch<DT, 64>(a, sums, grad, 0, s, info);
    return twice_launch<DT, kThreads>(a, sums, grad, split_shift(a.rows, a.cols, sms), s, info);
}

}  // namespace
}  // namespace ew
