// ew_rows_api.cu -- the row operators' part of the C ABI declared in
// include/ew.h: argument validation and dispatch.  As for the elementwise
// calls, every argument error is found on the host before any CUDA call.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ew_rows.h"

using namespace ew;

namespace {

constexpr int64_t kMaxSize = (int64_t(1) << 31) - (int64_t(1) << 16);  // rows, columns, table rows

bool float_type(int dt) { return dt == EW_F32 || dt == EW_F16 || dt == EW_BF16; }
int bytes_of(ew_dtype dt) { return dt == EW_F32 ? 4 : 2; }
bool size_ok(int64_t v, int64_t least) { return v >= least && v <= kMaxSize; }

// A matrix operand: rows x cols elements of `e` bytes, `stride` elements apart.
struct Operand {
    const void *p;
    int64_t rows, cols, stride;
    int e;
    bool wanted = true;  // an optional operand may be null
};
Operand vec(const void *p, int64_t n, int e, bool wanted = true) { return {p, 1, n, n, e, wanted}; }

ew_status check_operand(const Operand &m) {
    if (m.p == nullptr) return m.wanted && m.rows > 0 && m.cols > 0 ? EW_ERR_NULL_POINTER : EW_OK;
    if (reinterpret_cast<uintptr_t>(m.p) % m.e != 0) return EW_ERR_INVALID_VALUE;
    if (m.stride < m.cols || m.stride > INT64_MAX / 8 / std::max<int64_t>(m.rows, 1)) return EW_ERR_INVALID_VALUE;
    return EW_OK;
}

// Whether two matrices share a byte.  Matrices with one stride may interleave:
// then their rows are compared modulo the stride.
bool share_bytes(const Operand &a, const Operand &b) {
    if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uint64_t ra = static_cast<uint64_t>(a.cols) * a.e, rb = static_cast<uint64_t>(b.cols) * b.e;
    const uint64_t sa = static_cast<uint64_t>(a.stride) * a.e, sb = static_cast<uint64_t>(b.stride) * b.e;
    const uint64_t la = (a.rows - 1) * sa + ra, lb = (b.rows - 1) * sb + rb;
    if (pa >= pb + lb || pb >= pa + la) return false;
    if (sa != sb || (a.rows == 1 && b.rows == 1)) return true;
    const uint64_t d = pa <= pb ? (pb - pa) % sa : sa - (pa - pb) % sa;  // b's rows start d bytes into a's
    return d % sa == 0 || d < ra || d + rb > sa;
}
bool same_place(const Operand &a, const Operand &b) {
    return a.p == b.p && a.e == b.e && a.cols == b.cols && (a.rows <= 1 || a.stride == b.stride);
}

// Overlap rules: an output shares bytes with no other operand, but that output
// `in_place[k]` may be input k itself.
ew_status check_overlap(const Operand *in, int ni, const Operand *out, int no, const bool (*in_place)[2] = nullptr) {
    for (int o = 0; o < no; ++o) {
        for (int i = 0; i < ni; ++i) {
            const bool allowed = in_place != nullptr && i < 2 && in_place[o][i] && same_place(in[i], out[o]);
            if (!allowed && share_bytes(in[i], out[o])) return EW_ERR_OVERLAP;
        }
        for (int q = o + 1; q < no; ++q)
            if (share_bytes(out[o], out[q])) return EW_ERR_OVERLAP;
    }
    return EW_OK;
}

ew_status check_all(const Operand *in, int ni, const Operand *out, int no, const bool (*in_place)[2] = nullptr) {
    const void *p[16];
    int np = 0;
    for (int i = 0; i < ni; ++i) {
        const ew_status st = check_operand(in[i]);
        if (st != EW_OK) return st;
        p[np++] = in[i].rows > 0 ? in[i].p : nullptr;
    }
    for (int o = 0; o < no; ++o) {
        const ew_status st = check_operand(out[o]);
        if (st != EW_OK) return st;
        p[np++] = out[o].rows > 0 ? out[o].p : nullptr;
    }
    const ew_status st = check_overlap(in, ni, out, no, in_place);
    return st != EW_OK ? st : check_pointers(p, np);
}

void record(const LaunchInfo &info, int launches) {
    ew_launch_record &r = launch_record();
    r.launches = launches;
    r.path = info.vec_bytes >= 32 ? EW_PATH_V256 : info.vec_bytes == 16 ? EW_PATH_V128 : EW_PATH_SCALAR;
    r.vec_bytes = info.vec_bytes;
    r.grid = info.grid;
    r.block = info.block;
    r.smem = info.smem;
    r.schedule = EW_SCHED_ONESHOT;
}

ew_status norm_call(ew_dtype dt, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                    ew_dtype wtype, const void *weight, float eps, bool quant, ew_qtype qtype, int64_t group,
                    void *out, int64_t out_stride, float *scales, int64_t scales_stride, void *h_out,
                    int64_t h_stride, float *rstd_out, int64_t rows, int64_t cols, cudaStream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || (weight != nullptr && wtype != dt && wtype != EW_F32)) return EW_ERR_UNSUPPORTED_DTYPE;
    if (!size_ok(rows, 0) || !size_ok(cols, 1) || !(eps >= 0.0f) || std::isinf(eps)) return EW_ERR_INVALID_VALUE;
    if (quant) {
        if (qtype != EW_Q_E4M3 && qtype != EW_Q_I8) return EW_ERR_UNSUPPORTED_DTYPE;
        if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256) return EW_ERR_INVALID_VALUE;
    }
    if (rows == 0) return EW_OK;
    const int e = bytes_of(dt);
    const int64_t groups = !quant ? 0 : group == 0 ? 1 : (cols + group - 1) / group;
    const Operand in[3] = {{x, rows, cols, x_stride, e},
                           {residual, rows, cols, residual_stride, e, false},
                           vec(weight, cols, wtype == EW_F32 ? 4 : e, false)};
    const Operand outs[4] = {{out, rows, cols, out_stride, quant ? 1 : e},
                             {h_out, rows, cols, h_stride, e, false},
                             vec(rstd_out, rows, 4, false),
                             {scales, rows, groups, scales_stride, 4, quant}};
    const bool in_place[4][2] = {{!quant, !quant}, {true, true}, {false, false}, {false, false}};
    const ew_status st = check_all(in, 3, outs, quant ? 4 : 3, in_place);
    if (st != EW_OK) return st;
    int sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    const NormArgs a{x, residual, weight, out, h_out, rstd_out, scales, x_stride, residual_stride, out_stride,
                     h_stride, scales_stride, rows, static_cast<int32_t>(cols), group == 0 ? 0 : __builtin_ctzll(group), eps,
                     1.0f / static_cast<float>(cols),
                     weight != nullptr && wtype == EW_F32, quant && qtype == EW_Q_I8};
    LaunchInfo info;
    ce = (dt == EW_F32 ? norm_f32 : dt == EW_F16 ? norm_f16 : norm_bf16)(quant, a, sms, s, &info);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, 1);
    return EW_OK;
}

// Elements whose rows the embedding's gradient sorts and adds: blocks of 32 positions
// by 256 columns, eight of them to a block, stay below 2^31.
constexpr int64_t kMostSummed = int64_t(1) << 46;

// Workspace of the embedding's gradient, each part at a multiple of 256 bytes.
struct EmbedWork {
    int64_t items0, items1, keys, order, present, partial, bytes;
};
EmbedWork embed_work(int64_t table_rows, int64_t rows, int64_t cols) {
    int64_t at = 0;
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    EmbedWork w;
    w.items0 = take(rows * 8);
    w.items1 = take(rows * 8);
    w.keys = take(rows * 4);
    w.order = take(rows * 4);
    w.present = take((table_rows + 31) / 32 * 4);
    w.partial = take(embed_partial_bytes(rows, cols));
    w.bytes = at;
    return w;
}

bool index_type(int t) { return t == EW_INDEX_I32 || t == EW_INDEX_I64; }
int index_bytes(ew_index t) { return t == EW_INDEX_I64 ? 8 : 4; }
// What multiplies logits: positive, and far from where binary32 ends.
bool scale_ok(float scale) { return scale >= 1.0f / 1048576.0f && scale <= 1048576.0f; }

// The three distillation calls: sums (loss and lse) and grad (dlogits).
ew_status distill_call(bool sums, bool grad, ew_dtype dt, ew_index itype, const void *logits, int64_t stride,
                       const void *ids, int64_t ids_stride, ew_dtype ttype, const void *teacher,
                       int64_t teacher_stride, int64_t k, float scale, const float *dloss, float *loss, float *lse,
                       void *dlogits, int64_t dstride, int64_t rows, int64_t cols, cudaStream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || (ttype != dt && ttype != EW_F32) || !index_type(itype)) return EW_ERR_UNSUPPORTED_DTYPE;
    if (!size_ok(rows, 0) || !size_ok(cols, 1) || k < 1 || k > kMostTeacher || !scale_ok(scale))
        return EW_ERR_INVALID_VALUE;
    if (rows == 0) return EW_OK;
    const int e = bytes_of(dt);
    const Operand in[5] = {{logits, rows, cols, stride, e},
                           {ids, rows, k, ids_stride, index_bytes(itype)},
                           {teacher, rows, k, teacher_stride, bytes_of(ttype)},
                           vec(dloss, grad ? rows : 0, 4),
                           vec(sums ? nullptr : lse, rows, 4, !sums)};
    const Operand out[3] = {{dlogits, grad ? rows : 0, cols, grad ? dstride : cols, e},
                            vec(sums ? loss : nullptr, rows, 4, sums),
                            vec(sums ? lse : nullptr, rows, 4, sums)};
    const bool in_place[3][2] = {{true, false}, {false, false}, {false, false}};
    const ew_status st = check_all(in, 5, out, 3, in_place);
    if (st != EW_OK) return st;
    int sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    const DistillArgs a{logits, ids, teacher, dloss, loss, lse, dlogits, stride, ids_stride, teacher_stride, dstride,
                        rows, static_cast<int32_t>(cols), itype == EW_INDEX_I64, ttype == EW_F32,
                        static_cast<int32_t>(k), scale};
    LaunchInfo info;
    ce = (dt == EW_F32 ? distill_f32 : dt == EW_F16 ? distill_f16 : distill_bf16)(a, sums, grad, sms, s, &info);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, 1);
    return EW_OK;
}

// Rows of partial sums that the norm's backward may use: one for each row up to
// 1280, which is more than its blocks.
constexpr int64_t kNormPartials = 1280;

}  // namespace

extern "C" {

ew_status ew_embed(ew_dtype dt, ew_index itype, const void *table, int64_t table_rows, int64_t table_stride,
                   const void *tokens, float scale, void *out, int64_t out_stride, int64_t rows, int64_t cols,
                   ew_stream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || !index_type(itype)) return EW_ERR_UNSUPPORTED_DTYPE;
    if (!size_ok(rows, 0) || !size_ok(cols, 1) || !size_ok(table_rows, 0)) return EW_ERR_INVALID_VALUE;
    if (rows == 0) return EW_OK;
    const int e = bytes_of(dt);
    const Operand in[2] = {{table, table_rows, cols, table_stride, e}, vec(tokens, rows, index_bytes(itype))};
    const Operand outs[1] = {{out, rows, cols, out_stride, e}};
    const ew_status st = check_all(in, 2, outs, 1);
    if (st != EW_OK) return st;
    int sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    const EmbedArgs a{table, tokens, out, table_rows, table_stride, out_stride, rows, static_cast<int32_t>(cols),
                      itype == EW_INDEX_I64, scale};
    LaunchInfo info;
    ce = launch_embed(dt, a, sms, reinterpret_cast<cudaStream_t>(s), &info);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, 1);
    return EW_OK;
}

int64_t ew_embed_grad_workspace(int64_t table_rows, int64_t rows, int64_t cols) {
    if (!size_ok(table_rows, 0) || !size_ok(rows, 0) || !size_ok(cols, 1)) return -1;
    if (rows > 0 && cols > kMostSummed / rows) return -1;
    return embed_work(table_rows, rows, cols).bytes;
}

ew_status ew_embed_grad(ew_dtype dt, ew_index itype, const void *dout, int64_t dout_stride, const void *tokens,
                        float scale, ew_dtype gtype, void *dtable, int64_t table_rows, int64_t table_stride,
                        int64_t rows, int64_t cols, int accumulate, void *workspace, int64_t workspace_bytes,
                        ew_stream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || (gtype != dt && gtype != EW_F32) || !index_type(itype))
        return EW_ERR_UNSUPPORTED_DTYPE;
    const int64_t need = ew_embed_grad_workspace(table_rows, rows, cols);
    if (need < 0 || workspace_bytes < need || (accumulate != 0 && accumulate != 1) ||
        reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return EW_ERR_INVALID_VALUE;
    if (table_rows == 0 || (rows == 0 && accumulate)) return EW_OK;
    const Operand in[2] = {{dout, rows, cols, dout_stride, bytes_of(dt)},
                           vec(tokens, rows, index_bytes(itype))};
    const Operand out[2] = {{dtable, table_rows, cols, table_stride, bytes_of(gtype)}, vec(workspace, need, 1)};
    const ew_status st = check_all(in, 2, out, 2);
    if (st != EW_OK) return st;
    const EmbedWork w = embed_work(table_rows, rows, cols);
    char *base = static_cast<char *>(workspace);
    const EmbedGradArgs a{dout, tokens, dtable, dout_stride, table_rows, table_stride, rows, static_cast<int32_t>(cols),
                          itype == EW_INDEX_I64, accumulate, scale, reinterpret_cast<uint2 *>(base + w.items0),
                          reinterpret_cast<uint2 *>(base + w.items1), reinterpret_cast<uint32_t *>(base + w.keys),
                          reinterpret_cast<uint32_t *>(base + w.order),
                          accumulate ? nullptr : reinterpret_cast<uint32_t *>(base + w.present),
                          reinterpret_cast<float *>(base + w.partial), 0, 0};
    LaunchInfo info;
    int launches = 0, sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    ce = launch_embed_grad(dt, gtype, a, sms, reinterpret_cast<cudaStream_t>(s), &info, &launches);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, launches);
    return EW_OK;
}

ew_status ew_rmsnorm(ew_dtype dt, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                     ew_dtype wtype, const void *weight, float eps, void *y, int64_t y_stride, void *h_out,
                     int64_t h_stride, float *rstd_out, int64_t rows, int64_t cols, ew_stream_t s) {
    return norm_call(dt, x, x_stride, residual, residual_stride, wtype, weight, eps, false, EW_Q_E4M3, 0, y, y_stride,
                     nullptr, 0, h_out, h_stride, rstd_out, rows, cols, reinterpret_cast<cudaStream_t>(s));
}

ew_status ew_rmsnorm_quant(ew_dtype dt, const void *x, int64_t x_stride, const void *residual,
                           int64_t residual_stride, ew_dtype wtype, const void *weight, float eps, ew_qtype qtype,
                           int64_t group, void *q, int64_t q_stride, float *scales, int64_t scales_stride,
                           void *h_out, int64_t h_stride, float *rstd_out, int64_t rows, int64_t cols,
                           ew_stream_t s) {
    return norm_call(dt, x, x_stride, residual, residual_stride, wtype, weight, eps, true, qtype, group, q, q_stride,
                     scales, scales_stride, h_out, h_stride, rstd_out, rows, cols, reinterpret_cast<cudaStream_t>(s));
}

int64_t ew_rmsnorm_grad_workspace(int64_t rows, int64_t cols) {
    if (!size_ok(rows, 0) || !size_ok(cols, 1)) return -1;
    return std::min(rows, kNormPartials) * cols * 4;
}

ew_status ew_rmsnorm_grad(ew_dtype dt, const void *dy, int64_t dy_stride, const void *h, int64_t h_stride,
                          ew_dtype wtype, const void *weight, const float *rstd, const void *dh, int64_t dh_stride,
                          void *dx, int64_t dx_stride, float *dweight, int64_t rows, int64_t cols, void *workspace,
                          int64_t workspace_bytes, ew_stream_t stream) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || (weight != nullptr && wtype != dt && wtype != EW_F32)) return EW_ERR_UNSUPPORTED_DTYPE;
    const int64_t need = ew_rmsnorm_grad_workspace(rows, cols);
    if (need < 0 || (dweight != nullptr && workspace_bytes < need)) return EW_ERR_INVALID_VALUE;
    if (rows == 0 && dweight == nullptr) return EW_OK;
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return EW_ERR_INVALID_VALUE;
    const int e = bytes_of(dt);
    const Operand in[5] = {{dy, rows, cols, dy_stride, e},
                           {dh, rows, cols, dh_stride, e, false},
                           {h, rows, cols, h_stride, e},
                           vec(weight, cols, wtype == EW_F32 ? 4 : e, false),
                           vec(rstd, rows, 4)};
    const Operand out[3] = {{dx, rows, cols, dx_stride, e},
                            vec(dweight, cols, 4, false),
                            vec(workspace, need / 4, 4, dweight != nullptr && need > 0)};
    const bool in_place[3][2] = {{true, true}, {false, false}, {false, false}};
    const ew_status st = check_all(in, 5, out, dweight != nullptr ? 3 : 2, in_place);
    if (st != EW_OK) return st;
    int sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    const NormGradArgs a{dy, h, weight, dh, rstd, dx, dweight, static_cast<float *>(workspace), dy_stride, h_stride,
                         dh_stride, dx_stride, rows, static_cast<int32_t>(cols),
                         weight != nullptr && wtype == EW_F32};
    LaunchInfo info;
    int launches = 0;
    ce = (dt == EW_F32 ? norm_grad_f32 : dt == EW_F16 ? norm_grad_f16 : norm_grad_bf16)(
        a, std::min(rows, kNormPartials), sms, reinterpret_cast<cudaStream_t>(stream), &info, &launches);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, launches);
    return EW_OK;
}

ew_status ew_logprob(ew_dtype dt, ew_index itype, const void *logits, int64_t stride, const void *tokens, float scale,
                     int64_t top, float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_ids,
                     int64_t rows, int64_t cols, ew_stream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || !index_type(itype)) return EW_ERR_UNSUPPORTED_DTYPE;
    if (!size_ok(rows, 0) || !size_ok(cols, 1) || top < 0 || top > kMostTop || !scale_ok(scale))
        return EW_ERR_INVALID_VALUE;
    if (rows == 0) return EW_OK;
    const Operand in[2] = {{logits, rows, cols, stride, bytes_of(dt)},
                           vec(tokens, rows, index_bytes(itype), logp != nullptr)};
    const Operand out[5] = {vec(logp, rows, 4, false), vec(entropy, rows, 4, false), vec(lse, rows, 4, false),
                            vec(top_logp, rows * top, 4), vec(top_ids, rows * top, 4)};
    const ew_status st = check_all(in, 2, out, top > 0 ? 5 : 3);
    if (st != EW_OK) return st;
    int sms = 0;
    cudaError_t ce = current_sms(&sms);
    if (ce != cudaSuccess) return report_cuda(ce);
    const LogprobArgs a{logits, tokens, logp, entropy, lse, top_logp, top_ids, stride, rows,
                        static_cast<int32_t>(cols), itype == EW_INDEX_I64, static_cast<int32_t>(top), scale};
    LaunchInfo info;
    ce = (dt == EW_F32 ? logprob_f32 : dt == EW_F16 ? logprob_f16 : logprob_bf16)(
        a, sms, reinterpret_cast<cudaStream_t>(s), &info);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, 1);
    return EW_OK;
}

ew_status ew_logprob_grad(ew_dtype dt, ew_index itype, const void *logits, int64_t stride, const void *tokens,
                          const float *lse, const float *entropy, const float *dlogp, const float *dentropy,
                          float scale, void *dlogits, int64_t dstride, int64_t rows, int64_t cols, ew_stream_t s) {
    launch_record() = ew_launch_record{};
    if (!float_type(dt) || !index_type(itype)) return EW_ERR_UNSUPPORTED_DTYPE;
    if (!size_ok(rows, 0) || !size_ok(cols, 1) || !scale_ok(scale)) return EW_ERR_INVALID_VALUE;
    if (rows == 0) return EW_OK;
    const int e = bytes_of(dt);
    const Operand in[6] = {{logits, rows, cols, stride, e},
                           vec(tokens, rows, index_bytes(itype), dlogp != nullptr),
                           vec(lse, rows, 4),
                           vec(entropy, rows, 4, dentropy != nullptr),
                           vec(dlogp, rows, 4, false),
                           vec(dentropy, rows, 4, false)};
    const Operand out[1] = {{dlogits, rows, cols, dstride, e}};
    const bool in_place[1][2] = {{true, false}};
    const ew_status st = check_all(in, 6, out, 1, in_place);
    if (st != EW_OK) return st;
    const LogprobGradArgs a{logits, tokens, lse, entropy, dlogp, dentropy, dlogits, stride, dstride, rows,
                            static_cast<int32_t>(cols), itype == EW_INDEX_I64, scale};
    LaunchInfo info;
    const cudaError_t ce = (dt == EW_F32 ? logprob_grad_f32 : dt == EW_F16 ? logprob_grad_f16 : logprob_grad_bf16)(
        a, reinterpret_cast<cudaStream_t>(s), &info);
    if (ce != cudaSuccess) return report_cuda(ce);
    record(info, 1);
    return EW_OK;
}

ew_status ew_distill(ew_dtype dt, ew_index itype, const void *logits, int64_t stride, const void *ids,
                     int64_t ids_stride, ew_dtype ttype, const void *teacher, int64_t teacher_stride, int64_t k,
                     float scale, float *loss, float *lse, int64_t rows, int64_t cols, ew_stream_t s) {
    return distill_call(true, false, dt, itype, logits, stride, ids, ids_stride, ttype, teacher, teacher_stride, k,
                        scale, nullptr, loss, lse, nullptr, 0, rows, cols, reinterpret_cast<cudaStream_t>(s));
}

ew_status ew_distill_grad(ew_dtype dt, ew_index itype, const void *logits, int64_t stride, const void *ids,
                          int64_t ids_stride, ew_dtype ttype, const void *teacher, int64_t teacher_stride, int64_t k,
                          float scale, const float *lse, const float *dloss, void *dlogits, int64_t dstride,
                          int64_t rows, int64_t cols, ew_stream_t s) {
    return distill_call(false, true, dt, itype, logits, stride, ids, ids_stride, ttype, teacher, teacher_stride, k,
                        scale, dloss, nullptr, const_cast<float *>(lse), dlogits, dstride, rows, cols,
                        reinterpret_cast<cudaStream_t>(s));
}

ew_status ew_distill_step(ew_dtype dt, ew_index itype, const void *logits, int64_t stride, const void *ids,
                          int64_t ids_stride, ew_dtype ttype, const void *teacher, int64_t teacher_stride, int64_t k,
                          float scale, const float *dloss, float *loss, float *lse, void *dlogits, int64_t dstride,
                          int64_t rows, int64_t cols, ew_stream_t s) {
    return distill_call(true, true, dt, itype, logits, stride, ids, ids_stride, ttype, teacher, teacher_stride, k,
                        scale, dloss, loss, lse, dlogits, dstride, rows, cols, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"
