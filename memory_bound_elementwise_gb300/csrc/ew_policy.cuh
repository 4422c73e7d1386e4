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
// ring, rows too long, and the gradient from a given lse.
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

template <int DT> cudaError_t policy_launch(const PolicyArgs &a, bool sums, bool grad, int sms, cudaStream_t s, LaunchInfo *info) {
    const int64_t bytes = static_cast<int64_t>(a.cols) * ElemOf<DT>::kBytes;
    const bool few = a.rows <= sms;
    if (!few && bytes <= 32 * 1024) return policy_twice<DT, kNarrow>(a, sums, grad, 0, s, info);
    return policy_twice<DT, kThreads>(a, sums, grad, split_shift(a.rows, a.cols, sms), s, info);
}

}  // namespace
}  // namespace ew
