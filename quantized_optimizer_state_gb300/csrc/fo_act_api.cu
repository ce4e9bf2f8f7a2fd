// fo_act_api.cu -- entry points of the operators on activations, declared in
// include/fo.h: argument validation and kernel launches. Nothing here allocates
// memory, synchronizes or throws.
#include <algorithm>
#include <cmath>

#include "fo.h"
#include "fo_act.h"
#include "fo_check.h"
#include "fo_internal.h"

namespace {

using namespace fo::check;

constexpr int64_t kMaxStride = (int64_t)1 << 40;

int64_t groups_of(int64_t width) { return (width + FO_GROUP - 1) / FO_GROUP; }

// A matrix by itself; `like`, where given, has the sizes and the type it must have.
fo_status_t check_rows(const fo_rows_t *x, bool written, const fo_rows_t *like = nullptr)
{
    if (!x)
        return FO_ERR_NULL;
    if (x->rows < 0 || x->width < 1 || x->width > FO_MAX_ACT_WIDTH || x->rows > FO_MAX_ACT_GROUPS / groups_of(x->width))
        return FO_ERR_SIZE;
    if (!dtype_ok(x->dtype) || x->reserved != 0 || x->row_stride < 0 || x->row_stride > kMaxStride)
        return FO_ERR_BAD_ARG;
    if (like && (x->rows != like->rows || x->width != like->width || x->dtype != like->dtype))
        return FO_ERR_BAD_ARG;
    if (x->rows == 0)
        return FO_OK;
    if ((double)x->rows * (double)x->row_stride > 0x1p58)   // offsets in bytes stay far inside 63 bits
        return FO_ERR_SIZE;
    if (written && x->rows > 1 && x->row_stride < x->width)
        return FO_ERR_BAD_ARG;
    if (!x->data)
        return FO_ERR_NULL;
    if (misaligned(x->data, element_size(x->dtype)))
        return FO_ERR_MISALIGNED;
    return FO_OK;
}

fo_status_t check_kept(const void *codes, const void *steps)
{
    if (!codes || !steps)
        return FO_ERR_NULL;
    return misaligned(codes, 16) || misaligned(steps, 2) ? FO_ERR_MISALIGNED : FO_OK;
}

Range rows_range(const fo_rows_t *x, bool written)
{
    return x ? Range(x->data, ((x->rows - 1) * x->row_stride + x->width) * element_size(x->dtype), written) : Range();
}
Range codes_range(const fo_rows_t &x, const void *codes, bool written)
{
    return Range(codes, x.rows * groups_of(x.width) * FO_GROUP, written);
}
Range steps_range(const fo_rows_t &x, const void *steps, bool written)
{
    return Range(steps, x.rows * groups_of(x.width) * 2, written);
}

// Whether two matrices of one size and stride lie side by side in the rows of one
// buffer: their address ranges overlap, their elements do not.
bool side_by_side(const fo_rows_t &a, const fo_rows_t &b)
{
    const int64_t size = element_size(a.dtype), pitch = a.row_stride * size;
    if (a.row_stride != b.row_stride || pitch == 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.data), y = reinterpret_cast<uintptr_t>(b.data);
    const int64_t apart = (int64_t)((x > y ? x - y : y - x) % (uintptr_t)pitch);
    return apart >= a.width * size && pitch - apart >= a.width * size;
}

// The two matrices a call writes: their ranges may interleave.
bool aliases_beside(const fo_rows_t *first, const fo_rows_t *second, Range *r, int n)
{
    r[n] = rows_range(first, true);
    if (aliases(r, n + 1))
        return true;
    if (!second)
        return false;
    const Range other = rows_range(second, true);
    if (r[n].lo < other.hi && other.lo < r[n].hi && !side_by_side(*first, *second))
        return true;
    r[n] = other;
    return aliases(r, n + 1);
}

fo::RowsIn in_of(const fo_rows_t *x) { return x ? fo::RowsIn{x->data, x->row_stride} : fo::RowsIn{nullptr, 0}; }
fo::RowsOut out_of(const fo_rows_t *x) { return x ? fo::RowsOut{x->data, x->row_stride} : fo::RowsOut{nullptr, 0}; }

bool kind_ok(int kind) { return kind == FO_ACT_SILU || kind == FO_ACT_GELU; }

}  // namespace

extern "C" {

fo_status_t fo_compress(const fo_rows_t *in, int8_t *codes, uint16_t *steps, fo_stream_t stream)
{
    fo_status_t st = check_rows(in, false);
    if (st != FO_OK || in->rows == 0)
        return st;
    if ((st = check_kept(codes, steps)) != FO_OK)
        return st;
    const Range r[3] = {rows_range(in, false), codes_range(*in, codes, true), steps_range(*in, steps, true)};
    if (aliases(r, 3))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    const fo::CompressArgs a = {in->rows, in->width, groups_of(in->width), in_of(in), {codes, steps}};
    return fo::cuda_status(fo::launch_compress(in->dtype, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_expand(const int8_t *codes, const uint16_t *steps, const fo_rows_t *x, fo_stream_t stream)
{
    fo_status_t st = check_rows(x, true);
    if (st != FO_OK || x->rows == 0)
        return st;
    if ((st = check_kept(codes, steps)) != FO_OK)
        return st;
    const Range r[3] = {rows_range(x, true), codes_range(*x, codes, false), steps_range(*x, steps, false)};
    if (aliases(r, 3))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    const fo::ExpandArgs a = {x->rows, x->width, groups_of(x->width), {codes, steps}, out_of(x)};
    return fo::cuda_status(fo::launch_expand(x->dtype, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_activation(fo_act_t kind, const fo_rows_t *in, const fo_rows_t *up, const fo_rows_t *y, int8_t *codes,
                          uint16_t *steps, int8_t *up_codes, uint16_t *up_steps, fo_stream_t stream)
{
    if (!kind_ok((int)kind))
        return FO_ERR_BAD_ARG;
    fo_status_t st = check_rows(in, false);
    if (st != FO_OK || (st = check_rows(y, true, in)) != FO_OK || (up && (st = check_rows(up, false, in)) != FO_OK) || in->rows == 0)
        return st;
    if (codes && ((st = check_kept(codes, steps)) != FO_OK || (up && (st = check_kept(up_codes, up_steps)) != FO_OK)))
        return st;
    Range r[7] = {rows_range(in, false), rows_range(up, false), rows_range(y, true)};
    int n = 3;
    if (codes) {
        r[n++] = codes_range(*in, codes, true);
        r[n++] = steps_range(*in, steps, true);
        if (up) {
            r[n++] = codes_range(*in, up_codes, true);
            r[n++] = steps_range(*in, up_steps, true);
        }
    }
    if (aliases(r, n))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::ActivationArgs a = {in->rows, in->width, groups_of(in->width), in_of(in), in_of(up), out_of(y), {nullptr, nullptr}, {nullptr, nullptr}};
    if (codes) {
        a.kept = {codes, steps};
        if (up)
            a.kept_up = {up_codes, up_steps};
    }
    return fo::cuda_status(fo::launch_activation(in->dtype, (int)kind, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_activation_grad(fo_act_t kind, const int8_t *codes, const uint16_t *steps, const int8_t *up_codes,
                               const uint16_t *up_steps, const fo_rows_t *grad_y, const fo_rows_t *grad_x,
                               const fo_rows_t *grad_up, fo_stream_t stream)
{
    if (!kind_ok((int)kind))
        return FO_ERR_BAD_ARG;
    fo_status_t st = check_rows(grad_y, false);
    if (st != FO_OK || (st = check_rows(grad_x, true, grad_y)) != FO_OK || (grad_up && (st = check_rows(grad_up, true, grad_y)) != FO_OK) ||
        grad_y->rows == 0)
        return st;
    if ((st = check_kept(codes, steps)) != FO_OK || (grad_up && (st = check_kept(up_codes, up_steps)) != FO_OK))
        return st;
    Range r[6] = {rows_range(grad_y, false), codes_range(*grad_y, codes, false), steps_range(*grad_y, steps, false)};
    int n = 3;
    if (grad_up) {
        r[n++] = codes_range(*grad_y, up_codes, false);
        r[n++] = steps_range(*grad_y, up_steps, false);
    }
    if (aliases_beside(grad_x, grad_up, r, n))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    const fo::ActivationGradArgs a = {grad_y->rows, grad_y->width, groups_of(grad_y->width), {codes, steps}, {up_codes, up_steps},
                                      in_of(grad_y), out_of(grad_x), out_of(grad_up)};
    return fo::cuda_status(fo::launch_activation_grad(grad_y->dtype, (int)kind, a, static_cast<cudaStream_t>(stream)));
}

fo_status_t fo_rms_norm(const fo_rows_t *in, const void *weight, int32_t weight_dtype, double eps, const fo_rows_t *y,
                        float *inv_rms, int8_t *codes, uint16_t *steps, fo_stream_t stream)
{
    fo_status_t st = check_rows(in, false);
    if (st != FO_OK || (st = check_rows(y, true, in)) != FO_OK)
        return st;
    if (!(eps >= 0x1p-80 && eps <= 0x1p20) || (weight && !dtype_ok(weight_dtype)))
        return FO_ERR_BAD_ARG;
    if (in->rows == 0)
        return FO_OK;
    if (codes && (!inv_rms || (st = check_kept(codes, steps)) != FO_OK))
        return inv_rms ? st : FO_ERR_NULL;
    if ((weight && misaligned(weight, element_size(weight_dtype))) || (codes && misaligned(inv_rms, 4)))
        return FO_ERR_MISALIGNED;
    const Range r[6] = {rows_range(in, false), rows_range(y, true), Range(weight, in->width * element_size(weight_dtype), false),
                        Range(codes ? inv_rms : nullptr, 4 * in->rows, true), codes_range(*in, codes, true),
                        steps_range(*in, codes ? steps : nullptr, true)};
    if (aliases(r, 6))
        return FO_ERR_ALIAS;
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    fo::NormArgs a = {in->rows, in->width, groups_of(in->width), in_of(in), weight, weight_dtype, (float)eps, out_of(y),
                      codes ? inv_rms : nullptr, {nullptr, nullptr}, 0.0f, false};
    if (codes)
        a.kept = {codes, steps};
    return fo::cuda_status(fo::launch_norm(in->dtype, a, static_cast<cudaStream_t>(stream)));
}

int64_t fo_rms_norm_workspace(int64_t rows, int64_t width)
{
    return rows <= 0 || width <= 0 ? 0 : fo::norm_parts(rows, groups_of(width)) * groups_of(width) * FO_GROUP;
}

fo_status_t fo_rms_norm_grad(const int8_t *codes, const uint16_t *steps, const float *inv_rms, const void *weight,
                             int32_t weight_dtype, const fo_rows_t *grad_y, const fo_rows_t *grad_x, void *grad_weight,
                             float *workspace, fo_stream_t stream)
{
    fo_status_t st = check_rows(grad_y, false);
    if (st != FO_OK || (grad_x && (st = check_rows(grad_x, true, grad_y)) != FO_OK))
        return st;
    if ((weight || grad_weight) && !dtype_ok(weight_dtype))
        return FO_ERR_BAD_ARG;
    if ((weight && misaligned(weight, element_size(weight_dtype))) || (grad_weight && misaligned(grad_weight, element_size(weight_dtype))))
        return FO_ERR_MISALIGNED;
    const int64_t rows = grad_y->rows, width = grad_y->width;
    if (!(grad_x || grad_weight) || (rows == 0 && !grad_weight))
        return FO_OK;
    if (rows > 0) {
        if ((st = check_kept(codes, steps)) != FO_OK)
            return st;
        if (!inv_rms || (grad_weight && !workspace))
            return FO_ERR_NULL;
        if (misaligned(inv_rms, 4) || (grad_weight && misaligned(workspace, 16)))
            return FO_ERR_MISALIGNED;
        const Range r[8] = {rows_range(grad_y, false), codes_range(*grad_y, codes, false), steps_range(*grad_y, steps, false),
                            Range(inv_rms, 4 * rows, false), Range(weight, width * element_size(weight_dtype), false),
                            rows_range(grad_x, true), Range(grad_weight, width * element_size(weight_dtype), true),
                            Range(grad_weight ? workspace : nullptr, 4 * fo_rms_norm_workspace(rows, width), true)};
        if (aliases(r, 8))
            return FO_ERR_ALIAS;
    }
    if ((st = fo::pending_error()) != FO_OK)
        return st;
    const fo::NormGradArgs a = {rows, width, groups_of(width), {codes, steps}, inv_rms, weight, weight_dtype, in_of(grad_y),
                                rows ? out_of(grad_x) : fo::RowsOut{nullptr, 0}, grad_weight, workspace, 0.0f, false};
    return fo::cuda_status(fo::launch_norm_grad(grad_y->dtype, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
