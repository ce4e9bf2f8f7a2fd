// fo_loss_api.cu -- the loss operators' entry points declared in include/fo.h:
// argument validation and kernel launches. Nothing here allocates memory,
// synchronizes or throws.
#include <cmath>

#include "fo.h"
#include "fo_internal.h"
#include "fo_loss.h"

namespace {

constexpr double kLog2E = 1.4426950408889634;
constexpr int64_t kMaxStride = (int64_t)1 << 44;

int64_t element_size(int32_t dtype) { return dtype == FO_LOGITS_F32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == FO_LOGITS_BF16 || dtype == FO_LOGITS_F32 || dtype == FO_LOGITS_F16; }
bool temperature_ok(double t) { return std::isfinite(t) && t >= 0x1p-20 && t <= 0x1p20; }
bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// One array of a call: bytes [lo, hi), empty where the pointer is null.
struct Range {
    uintptr_t lo = 0, hi = 0;
    bool written = false;
    Range() = default;
    Range(const void *p, int64_t bytes, bool w) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo), written(w)
    {
        if (p)
            hi = lo + (uintptr_t)bytes;
    }
};

// A written array may share no byte with any other array of the call.
bool aliases(const Range *r, int n)
{
    for (int a = 0; a < n; ++a)
        for (int b = a + 1; b < n; ++b)
            if ((r[a].written || r[b].written) && r[a].lo < r[b].hi && r[b].lo < r[a].hi)
                return true;
    return false;
}

int64_t outer_rows(const fo_logits_t &x) { return x.rows / x.inner_rows; }

// Elements from the first row's start to the last row's end.
int64_t span(const fo_logits_t &x, int64_t row_stride, int64_t outer_stride)
{
    return (outer_rows(x) - 1) * outer_stride + (x.inner_rows - 1) * row_stride + x.vocab;
}

fo_status_t check_logits(const fo_logits_t *x)
{
    if (!x)
        return FO_ERR_NULL;
    if (x->rows < 0 || x->rows > FO_MAX_LOGIT_ROWS)
        return FO_ERR_SIZE;
    if (!dtype_ok(x->dtype) || !temperature_ok(x->temperature) || x->reserved != 0)
        return FO_ERR_BAD_ARG;
    if (x->rows == 0)
        return FO_OK;
    if (x->vocab < 1 || x->vocab > FO_MAX_ROW_BYTES / element_size(x->dtype))
        return FO_ERR_SIZE;
    if (x->inner_rows < 1 || x->rows % x->inner_rows != 0 || x->row_stride < 0 || x->row_stride > kMaxStride ||
        x->outer_stride < 0 || x->outer_stride > kMaxStride)
        return FO_ERR_BAD_ARG;
    // the last element's offset stays far inside 63 bits
    if ((double)outer_rows(*x) * (double)x->outer_stride + (double)x->inner_rows * (double)x->row_stride > 0x1p60)
        return FO_ERR_SIZE;
    if (!x->data)
        return FO_ERR_NULL;
    if (misaligned(x->data, element_size(x->dtype)))
        return FO_ERR_MISALIGNED;
    return FO_OK;
}

// The gradient's rows must not overlap: either nesting of the two strides.
fo_status_t check_grad(const fo_logits_t &x, const fo_logits_grad_t *g)
{
    if (!g || !g->data)
        return FO_ERR_NULL;
    if (misaligned(g->data, element_size(x.dtype)))
        return FO_ERR_MISALIGNED;
    const int64_t in = x.inner_rows, out = outer_rows(x), v = x.vocab;
    if (g->row_stride < 0 || g->row_stride > kMaxStride || g->outer_stride < 0 || g->outer_stride > kMaxStride ||
        (double)out * (double)g->outer_stride + (double)in * (double)g->row_stride > 0x1p60)
        return FO_ERR_BAD_ARG;
    const bool rows_inside = (in == 1 || g->row_stride >= v) && (out == 1 || g->outer_stride >= (in - 1) * g->row_stride + v);
    const bool outer_inside = (out == 1 || g->outer_stride >= v) && (in == 1 || g->row_stride >= (out - 1) * g->outer_stride + v);
    return rows_inside || outer_inside ? FO_OK : FO_ERR_BAD_ARG;
}

// Whether the gradient takes exactly the logits' place.
bool in_place(const fo_logits_t &x, const fo_logits_grad_t &g)
{
    return x.data == g.data && (x.inner_rows == 1 || x.row_stride == g.row_stride) &&
           (outer_rows(x) == 1 || x.outer_stride == g.outer_stride);
}

fo_status_t check_teacher(const fo_teacher_t *t)
{
    if (!t)
        return FO_ERR_NULL;
    if (t->k < 1 || t->k > FO_MAX_TOP_K)
        return FO_ERR_SIZE;
    if (!dtype_ok(t->dtype) || !temperature_ok(t->temperature) || (t->tail != 0 && t->tail != 1) || t->reserved != 0)
        return FO_ERR_BAD_ARG;
    return FO_OK;
}

fo_status_t check_teacher_arrays(const fo_teacher_t &t)
{
    if (!t.ids || !t.logits)
        return FO_ERR_NULL;
    if (misaligned(t.ids, 4) || misaligned(t.logits, element_size(t.dtype)) || misaligned(t.lse, 4))
        return FO_ERR_MISALIGNED;
    return FO_OK;
}

fo::LogitRows rows_of(const fo_logits_t &x)
{
    fo::LogitRows r;
    r.data = x.data;
    r.rows = x.rows;
    r.vocab = x.vocab;
    r.row_stride = x.row_stride;
    r.inner_rows = x.inner_rows;
    r.outer_stride = x.outer_stride;
    r.inv_t = (float)(1.0 / x.temperature);
    r.c = (float)(kLog2E / x.temperature);
    r.c_lo = (float)(kLog2E / x.temperature - (double)r.c);
    r.d_min = (float)(-160.0 * x.temperature / kLog2E);
    return r;
}

fo::GradRows grad_of(const fo_logits_grad_t *g)
{
    fo::GradRows r = {nullptr, 0, 0};
    if (g) {
        r.data = g->data;
        r.row_stride = g->row_stride;
        r.outer_stride = g->outer_stride;
    }
    return r;
}

fo::Teacher teacher_of(const fo_teacher_t &t)
{
    const float inv_t = (float)(1.0 / t.temperature);
    return fo::Teacher{t.ids, t.logits, t.tail ? t.lse : nullptr, inv_t, (float)(1.0 / t.temperature - (double)inv_t), t.k, t.dtype, t.tail};
}

Range logits_range(const fo_logits_t &x) { return Range(x.data, span(x, x.row_stride, x.outer_stride) * element_size(x.dtype), false); }

Range grad_range(const fo_logits_t &x, const fo_logits_grad_t *g)
{
    return g ? Range(g->data, span(x, g->row_stride, g->outer_stride) * element_size(x.dtype), true) : Range();
}

}  // namespace

extern "C" {

fo_status_t fo_token_logprobs(const fo_logits_t *logits, const int64_t *tokens, int32_t top_k, float *logp,
                              float *entropy, int32_t *top_ids, float *top_logp, float *stats, fo_stream_t stream)
{
    fo_status_t st = check_logits(logits);
    if (st != FO_OK)
        return st;
    if (top_k < 0 || top_k > FO_MAX_TOP_K)
        return FO_ERR_SIZE;
    if (logits->rows == 0)
        return FO_OK;
    const int64_t n = logits->rows;
    if (top_k > logits->vocab)
        return FO_ERR_SIZE;
    if ((logp && !tokens) || (top_k > 0 && (!top_ids || !top_logp)))
        return FO_ERR_NULL;
    if (misaligned(tokens, 8) || misaligned(logp, 4) || misaligned(entropy, 4) || misaligned(stats, 16) ||
        (top_k > 0 && (misaligned(top_ids, 4) || misaligned(top_logp, 4))))
        return FO_ERR_MISALIGNED;
    const Range r[7] = {logits_range(*logits), Range(tokens, 8 * n, false), Range(logp, 4 * n, true),
                        Range(entropy, 4 * n, true), Range(top_k ? top_ids : nullptr, 4 * n * top_k, true),
                        Range(top_k ? top_logp : nullptr, 4 * n * top_k, true), Range(stats, 16 * n, true)};
    if (aliases(r, 7))
        return FO_ERR_ALIAS;
    if (!logp && !entropy && !stats && top_k == 0)
        return FO_OK;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::LogprobArgs a;
    a.in = rows_of(*logits);
    a.tokens = logp ? tokens : nullptr;
    a.k = top_k;
    a.logp = logp;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.stats = reinterpret_cast<float4 *>(stats);
    return fo::cuda_status(fo::launch_token_logprobs(logits->dtype, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_token_logprobs_grad(const fo_logits_t *logits, const int64_t *tokens, int32_t top_k,
                                   const int32_t *top_ids, const float *stats, const float *g_logp,
                                   const float *g_entropy, const float *g_top, const fo_logits_grad_t *grad,
                                   fo_stream_t stream)
{
    fo_status_t st = check_logits(logits);
    if (st != FO_OK)
        return st;
    if (top_k < 0 || top_k > FO_MAX_TOP_K)
        return FO_ERR_SIZE;
    if (logits->rows == 0)
        return FO_OK;
    const int64_t n = logits->rows;
    if (!stats || (g_logp && !tokens) || (g_top && top_k > 0 && !top_ids))
        return FO_ERR_NULL;
    if ((st = check_grad(*logits, grad)) != FO_OK)
        return st;
    if (misaligned(tokens, 8) || misaligned(top_ids, 4) || misaligned(stats, 16) || misaligned(g_logp, 4) ||
        misaligned(g_entropy, 4) || misaligned(g_top, 4))
        return FO_ERR_MISALIGNED;
    const Range r[8] = {grad_range(*logits, grad), in_place(*logits, *grad) ? Range() : logits_range(*logits),
                        Range(tokens, 8 * n, false), Range(top_ids, 4 * n * top_k, false), Range(stats, 16 * n, false),
                        Range(g_logp, 4 * n, false), Range(g_entropy, 4 * n, false), Range(g_top, 4 * n * top_k, false)};
    if (aliases(r, 8))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::LogprobGradArgs a;
    a.in = rows_of(*logits);
    a.out = grad_of(grad);
    a.tokens = g_logp ? tokens : nullptr;
    a.k = g_top ? top_k : 0;
    a.top_ids = top_ids;
    a.stats = reinterpret_cast<const float4 *>(stats);
    a.g_logp = g_logp;
    a.g_entropy = g_entropy;
    a.g_top = g_top;
    return fo::cuda_status(fo::launch_token_logprobs_grad(logits->dtype, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_distill(const fo_logits_t *logits, const fo_teacher_t *teacher, const float *row_weight, float *loss,
                       float *stats, const fo_logits_grad_t *grad, fo_stream_t stream)
{
    fo_status_t st = check_logits(logits);
    if (st != FO_OK)
        return st;
    if ((st = check_teacher(teacher)) != FO_OK)
        return st;
    if (logits->rows == 0)
        return FO_OK;
    const int64_t n = logits->rows, k = teacher->k;
    if ((st = check_teacher_arrays(*teacher)) != FO_OK)
        return st;
    if (grad && (st = check_grad(*logits, grad)) != FO_OK)
        return st;
    if (misaligned(row_weight, 4) || misaligned(loss, 4) || misaligned(stats, 16))
        return FO_ERR_MISALIGNED;
    const Range r[8] = {grad_range(*logits, grad), grad && in_place(*logits, *grad) ? Range() : logits_range(*logits),
                        Range(teacher->ids, 4 * n * k, false),
                        Range(teacher->logits, element_size(teacher->dtype) * n * k, false),
                        Range(teacher->tail ? teacher->lse : nullptr, 4 * n, false), Range(row_weight, 4 * n, false),
                        Range(loss, 4 * n, true), Range(stats, 16 * n, true)};
    if (aliases(r, 8))
        return FO_ERR_ALIAS;
    if (!loss && !stats && !grad)
        return FO_OK;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::DistillArgs a;
    a.in = rows_of(*logits);
    a.teacher = teacher_of(*teacher);
    a.weight = row_weight;
    a.loss = loss;
    a.stats = reinterpret_cast<float4 *>(stats);
    a.grad = grad_of(grad);
    return fo::cuda_status(fo::launch_distill(logits->dtype, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_distill_grad(const fo_logits_t *logits, const fo_teacher_t *teacher, const float *stats,
                            const float *g_loss, const fo_logits_grad_t *grad, fo_stream_t stream)
{
    fo_status_t st = check_logits(logits);
    if (st != FO_OK)
        return st;
    if ((st = check_teacher(teacher)) != FO_OK)
        return st;
    if (logits->rows == 0)
        return FO_OK;
    const int64_t n = logits->rows, k = teacher->k;
    if (!stats || !g_loss)
        return FO_ERR_NULL;
    if ((st = check_teacher_arrays(*teacher)) != FO_OK || (st = check_grad(*logits, grad)) != FO_OK)
        return st;
    if (misaligned(stats, 16) || misaligned(g_loss, 4))
        return FO_ERR_MISALIGNED;
    const Range r[7] = {grad_range(*logits, grad), in_place(*logits, *grad) ? Range() : logits_range(*logits),
                        Range(teacher->ids, 4 * n * k, false),
                        Range(teacher->logits, element_size(teacher->dtype) * n * k, false),
                        Range(teacher->tail ? teacher->lse : nullptr, 4 * n, false), Range(stats, 16 * n, false),
                        Range(g_loss, 4 * n, false)};
    if (aliases(r, 7))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::DistillGradArgs a;
    a.in = rows_of(*logits);
    a.out = grad_of(grad);
    a.teacher = teacher_of(*teacher);
    a.stats = reinterpret_cast<const float4 *>(stats);
    a.g_loss = g_loss;
    return fo::cuda_status(fo::launch_distill_grad(logits->dtype, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
