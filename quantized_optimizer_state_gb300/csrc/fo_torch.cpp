// fo_torch.cpp -- the operators on activations and the policy loss as PyTorch
// calls: checks of tensors, their results' memory, and automatic differentiation,
// around the C calls of include/fo.h. The Python modules activations.py and
// losses.py have the documentation.
//
// Host code only. It stands in C++ because a call on small tensors is host time:
// the same steps through ctypes took 13 to 24 us a call, these 6 to 9; forward and
// backward pass by automatic differentiation 200 to 225 us, these 110 to 130, of
// which 75 are the engine's own.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <tuple>
#include <vector>

#include "fo.h"

namespace py = pybind11;

namespace {

using at::ScalarType;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
typedef std::optional<Tensor> Maybe;
typedef std::vector<int64_t> Sizes;

// The binding's exception for a status that is not FO_OK.
void check(const char *fn, fo_status_t status)
{
    if (status == FO_OK)
        return;
    py::gil_scoped_acquire gil;
    py::module_::import("quantized_optimizer_state_gb300.fo").attr("_check")(fn, (int)status);
}

fo_stream_t stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
bool defined(const Maybe &t) { return t.has_value() && t->defined(); }
int64_t groups(int64_t width) { return (width + FO_GROUP - 1) / FO_GROUP; }

// As PyTorch writes it.
const char *type_name(ScalarType t)
{
    switch (t) {
    case ScalarType::BFloat16: return "bfloat16";
    case ScalarType::Half: return "float16";
    case ScalarType::Float: return "float32";
    case ScalarType::Double: return "float64";
    case ScalarType::Char: return "int8";
    case ScalarType::Byte: return "uint8";
    case ScalarType::Short: return "int16";
    case ScalarType::Int: return "int32";
    case ScalarType::Long: return "int64";
    case ScalarType::Bool: return "bool";
    default: return c10::toString(t);
    }
}
const char *type_name(const Tensor &x) { return type_name(x.scalar_type()); }

int32_t dtype_of(const Tensor &x, const char *name)
{
    switch (x.scalar_type()) {
    case ScalarType::BFloat16: return FO_LOGITS_BF16;
    case ScalarType::Float: return FO_LOGITS_F32;
    case ScalarType::Half: return FO_LOGITS_F16;
    default: TORCH_CHECK_TYPE(false, name, " must be bfloat16, float16 or float32, not ", type_name(x)); return -1;
    }
}

// Every call launches on the current device.
void check_device(const Tensor &x, const char *name)
{
    TORCH_CHECK_VALUE(x.is_cuda(), name, ": the library reads and writes device memory: pass CUDA tensors");
    const int current = (int)c10::cuda::current_device();
    TORCH_CHECK_VALUE(x.get_device() == current, name, " is on cuda:", (int)x.get_device(), " but the current device is cuda:", current,
                      "; the library launches on the current device (use torch.cuda.device)");
}

// A contiguous array of n elements of one type at least.
void *array(const Tensor &x, const char *name, ScalarType type, int64_t n)
{
    TORCH_CHECK_VALUE(x.is_cuda(), name, ": the library reads and writes device memory: pass CUDA tensors");
    TORCH_CHECK_VALUE(x.is_contiguous(), name, ": tensors passed to the library must be contiguous");
    TORCH_CHECK_TYPE(x.scalar_type() == type, name, " must be ", type_name(type), ", not ", type_name(x));
    TORCH_CHECK_VALUE(x.numel() >= n, name, " holds ", x.numel(), " elements; the call needs ", n);
    check_device(x, name);
    return x.data_ptr();
}

Tensor empty_like_type(at::IntArrayRef sizes, const Tensor &like) { return at::empty(sizes, like.options()); }
Tensor empty_of(at::IntArrayRef sizes, ScalarType type, const Tensor &like) { return at::empty(sizes, like.options().dtype(type)); }

// --- rows one stride apart -----------------------------------------------------------

// (rows, stride) of the leading dimensions; false where one stride does not cover
// them or the last dimension is not contiguous.
bool rows_of(const Tensor &x, int64_t &rows, int64_t &stride)
{
    const auto shape = x.sizes(), strides = x.strides();
    const int64_t dims = x.dim();
    if (dims < 1 || (strides[dims - 1] != 1 && shape[dims - 1] > 1))
        return false;
    rows = 1;
    stride = shape[dims - 1];
    if (dims == 2) {
        rows = shape[0];
        stride = strides[0];
        return true;
    }
    bool covered = true;
    for (int64_t i = dims - 2; i >= 0; --i) {
        const int64_t n = shape[i];
        if (n == 0) {
            rows = 0;
            return true;
        }
        if (n == 1)
            continue;
        if (rows == 1)
            stride = strides[i];
        else if (strides[i] != stride * rows)
            covered = false;
        rows *= n;
    }
    return covered;
}

fo_rows_t matrix(const Tensor &x, const char *name, const fo_rows_t *like = nullptr)
{
    const int32_t dt = dtype_of(x, name);
    check_device(x, name);
    fo_rows_t m = {x.data_ptr(), 0, x.dim() ? x.size(-1) : 0, 0, dt, 0};
    TORCH_CHECK_VALUE(rows_of(x, m.rows, m.row_stride), name,
                      ": the last dimension must be contiguous and one stride must cover the others (make it contiguous)");
    TORCH_CHECK_VALUE(!like || (m.rows == like->rows && m.width == like->width && dt == like->dtype), name,
                      " must have the other matrices' rows, columns and type");
    return m;
}
fo_rows_t dense(const Tensor &x, int64_t rows, int64_t width, int32_t dt) { return fo_rows_t{x.data_ptr(), rows, width, width, dt, 0}; }

void check_width(const Tensor &x)
{
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1, "a tensor [..., width] of at least one column is needed, not ", x.sizes());
}

// An incoming gradient of the result's shape and type, in a layout that the
// kernels read (an expanded one, for example, is copied).
Tensor readable(const Tensor &grad, at::IntArrayRef shape, ScalarType type)
{
    TORCH_CHECK_VALUE(grad.sizes() == shape && grad.scalar_type() == type, "grad_y must be ", type_name(type), " of shape ", shape,
                      ", not ", type_name(grad), " of shape ", grad.sizes());
    int64_t rows, stride;
    return rows_of(grad, rows, stride) ? grad : grad.contiguous();
}

std::tuple<Tensor, Tensor> compress(const Tensor &x)
{
    check_width(x);
    const fo_rows_t m = matrix(x, "x");
    Sizes shape = x.sizes().vec();
    const int64_t g = groups(m.width);
    shape.back() = g * FO_GROUP;
    Tensor codes = empty_of(shape, ScalarType::Char, x);
    shape.back() = g;
    Tensor steps = empty_of(shape, ScalarType::BFloat16, x);
    check("fo_compress", fo_compress(&m, codes.data_ptr<int8_t>(), static_cast<uint16_t *>(steps.data_ptr()), stream()));
    return {codes, steps};
}

Tensor expand(const Tensor &codes, const Tensor &steps, int64_t width, ScalarType type, const Maybe &out)
{
    const int64_t g = groups(width);
    Sizes shape = codes.sizes().vec(), lead = steps.sizes().vec();
    TORCH_CHECK_VALUE(width >= 1 && !shape.empty() && shape.back() == g * FO_GROUP && lead.size() == shape.size() && lead.back() == g &&
                          std::equal(shape.begin(), shape.end() - 1, lead.begin()),
                      "codes ", codes.sizes(), " and steps ", steps.sizes(), " are not those of ", width, " columns");
    shape.back() = width;
    Tensor x;
    if (defined(out)) {
        x = *out;
        TORCH_CHECK_VALUE(x.sizes() == at::IntArrayRef(shape), "out must be of shape ", shape, ", not ", x.sizes());
    } else {
        check_device(codes, "codes");
        x = empty_of(shape, type, codes);
    }
    const fo_rows_t m = matrix(x, "x");
    const int64_t n = m.rows * g;
    const void *c = array(codes, "codes", ScalarType::Char, n * FO_GROUP), *s = array(steps, "steps", ScalarType::BFloat16, n);
    check("fo_expand", fo_expand(static_cast<const int8_t *>(c), static_cast<const uint16_t *>(s), &m, stream()));
    if (defined(out) && !x.is_inference())
        torch::autograd::impl::bump_version(x);   // a graph that saved it says so
    return x;
}

// --- activation functions ------------------------------------------------------------------

// What the gradient needs beside the kept bytes: codes of x (of a gated kind the
// gate's, then the other half's), then steps.
struct Act {
    int64_t act;
    bool gated, halves;     // halves: gate and other half are those of one tensor
    ScalarType type;
    Sizes shape;            // of the result

    Sizes pack() const
    {
        Sizes v = {act, gated, halves, (int64_t)type};
        v.insert(v.end(), shape.begin(), shape.end());
        return v;
    }
    static Act unpack(const Sizes &v) { return Act{v[0], v[1] != 0, v[2] != 0, (ScalarType)v[3], Sizes(v.begin() + 4, v.end())}; }
    int64_t rows() const
    {
        int64_t n = 1;
        for (size_t i = 0; i + 1 < shape.size(); ++i)
            n *= shape[i];
        return n;
    }
    int64_t kept_groups() const { return rows() * groups(shape.back()); }
    int64_t kept_bytes() const { return kept_groups() * (gated ? 2 : 1) * (FO_GROUP + 2); }
};

struct ActBytes {
    int8_t *codes, *up_codes;
    uint16_t *steps, *up_steps;
    ActBytes(const Tensor &kept, const Act &a)
    {
        const int64_t n = a.kept_groups();
        codes = static_cast<int8_t *>(kept.data_ptr());
        up_codes = a.gated ? codes + n * FO_GROUP : nullptr;
        steps = reinterpret_cast<uint16_t *>(codes + n * FO_GROUP * (a.gated ? 2 : 1));
        up_steps = a.gated ? steps + n : nullptr;
    }
};

std::tuple<Tensor, Tensor, Act> act_forward(const Tensor &x, const Maybe &up, int64_t act, bool gated, bool keep)
{
    check_width(x);
    fo_rows_t m = matrix(x, "x"), u = {};
    Act how = {act, gated, gated && !defined(up), x.scalar_type(), x.sizes().vec()};
    if (how.halves) {
        TORCH_CHECK_VALUE(m.width % 2 == 0, "a gated kind halves the last dimension, which must be even, not ", m.width);
        m.width /= 2;
        how.shape.back() = m.width;
        u = m;
        u.data = static_cast<char *>(m.data) + m.width * x.element_size();
    } else if (gated) {
        TORCH_CHECK_VALUE(up->sizes() == x.sizes(), "up must have the gate's shape ", x.sizes(), ", not ", up->sizes());
        u = matrix(*up, "up", &m);
    }
    Tensor y = empty_like_type(how.shape, x), kept;
    const fo_rows_t to = dense(y, m.rows, m.width, m.dtype);
    if (keep) {
        kept = empty_of({how.kept_bytes()}, ScalarType::Char, x);
        const ActBytes b(kept, how);
        check("fo_activation", fo_activation((fo_act_t)act, &m, gated ? &u : nullptr, &to, b.codes, b.steps, b.up_codes, b.up_steps, stream()));
    } else
        check("fo_activation", fo_activation((fo_act_t)act, &m, gated ? &u : nullptr, &to, nullptr, nullptr, nullptr, nullptr, stream()));
    return {y, kept, how};
}

std::tuple<Tensor, Tensor> act_backward(const Tensor &kept, const Act &how, const Tensor &grad)
{
    const Tensor dy = readable(grad, how.shape, how.type);
    const fo_rows_t m = matrix(dy, "grad_y");
    const ActBytes b(kept, how);
    Sizes shape = how.shape;
    if (how.halves)
        shape.back() *= 2;
    Tensor gx = empty_like_type(shape, dy), gu;
    fo_rows_t to = dense(gx, m.rows, m.width, m.dtype), to_up = to;
    if (how.halves) {
        to.row_stride = to_up.row_stride = 2 * m.width;
        to_up.data = static_cast<char *>(to.data) + m.width * dy.element_size();
    } else if (how.gated) {
        gu = empty_like_type(shape, dy);
        to_up.data = gu.data_ptr();
    }
    check("fo_activation_grad", fo_activation_grad((fo_act_t)how.act, b.codes, b.steps, b.up_codes, b.up_steps, &m, &to,
                                                   how.gated ? &to_up : nullptr, stream()));
    return {gx, gu};
}

// Derivatives are of the first order: a backward pass that is to be
// differentiated gives gradients that refuse it, whether or not what reached it
// asks for a gradient (its result depends on the operator's input too). They
// are made to require one first: the refusing node passes by tensors that do not.
variable_list first_order(variable_list grads)
{
    if (!at::GradMode::is_enabled())
        return grads;
    variable_list made;
    for (const auto &g : grads)
        if (g.defined())
            made.push_back(g.detach().set_requires_grad(true));
    auto refuse = std::make_shared<torch::autograd::DelayedError>("the operators of this library have first derivatives only",
                                                                  (int64_t)made.size());
    made = (*refuse)(std::move(made));
    size_t at = 0;
    for (auto &g : grads)
        if (g.defined())
            g = made[at++];
    return grads;
}

// The same for a backward pass in Python; None for what has no gradient.
std::vector<Maybe> first_order_of(const std::vector<Maybe> &grads)
{
    variable_list list;
    for (const auto &g : grads)
        list.push_back(defined(g) ? *g : Tensor());
    list = first_order(std::move(list));
    std::vector<Maybe> result;
    for (const auto &g : list)
        result.push_back(g.defined() ? Maybe(g) : Maybe());
    return result;
}

struct ActFunction : torch::autograd::Function<ActFunction> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Maybe &up, int64_t act, bool gated)
    {
        auto [y, kept, how] = act_forward(x, up, act, gated, true);
        ctx->save_for_backward({kept});
        ctx->saved_data["how"] = how.pack();
        return y;
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Act how = Act::unpack(ctx->saved_data["how"].toIntVector());
        const c10::cuda::CUDAGuard guard(saved[0].device());
        auto [gx, gu] = act_backward(saved[0], how, grads[0]);
        return first_order({gx, gu, Tensor(), Tensor()});
    }
};

bool differentiable(const Tensor &x, const Maybe &other)
{
    return at::GradMode::is_enabled() && (x.requires_grad() || (defined(other) && other->requires_grad()));
}

Tensor activation(const Tensor &x, const Maybe &up, int64_t act, bool gated)
{
    return differentiable(x, up) ? ActFunction::apply(x, up, act, gated) : std::get<0>(act_forward(x, up, act, gated, false));
}

std::tuple<Tensor, Tensor> activation_forward(const Tensor &x, const Maybe &up, int64_t act, bool gated)
{
    at::NoGradGuard no_grad;
    auto [y, kept, how] = act_forward(x, up, act, gated, true);
    return {y, kept};
}

std::tuple<Tensor, Tensor> activation_backward(const Tensor &kept, int64_t act, bool gated, bool halves, const Sizes &shape, ScalarType type,
                                               const Tensor &grad)
{
    const Act how = {act, gated, halves, type, shape};
    array(kept, "kept", ScalarType::Char, how.kept_bytes());
    return act_backward(kept, how, grad);
}

// --- norm --------------------------------------------------------------------------------------

// Kept bytes of a norm: codes, 1 / rms of each row, steps.
struct NormBytes {
    int8_t *codes;
    float *inv;
    uint16_t *steps;
    NormBytes(const Tensor &kept, int64_t rows, int64_t width)
    {
        codes = static_cast<int8_t *>(kept.data_ptr());
        inv = reinterpret_cast<float *>(codes + rows * groups(width) * FO_GROUP);
        steps = reinterpret_cast<uint16_t *>(inv + rows);
    }
    static int64_t size(int64_t rows, int64_t width) { return rows * (groups(width) * (FO_GROUP + 2) + 4); }
};

const void *weight_of(const Maybe &weight, int64_t width, int32_t &dt)
{
    dt = 0;
    if (!defined(weight))
        return nullptr;
    TORCH_CHECK_VALUE(weight->dim() == 1 && weight->size(0) == width, "weight must be of shape (", width, ",), not ", weight->sizes());
    dt = dtype_of(*weight, "weight");
    return array(*weight, "weight", weight->scalar_type(), width);
}

std::tuple<Tensor, Tensor> norm_forward(const Tensor &x, const Maybe &weight, double eps, bool keep)
{
    check_width(x);
    const fo_rows_t m = matrix(x, "x");
    int32_t wt;
    const void *w = weight_of(weight, m.width, wt);
    Tensor y = empty_like_type(x.sizes(), x), kept;
    const fo_rows_t to = dense(y, m.rows, m.width, m.dtype);
    if (keep) {
        kept = empty_of({NormBytes::size(m.rows, m.width)}, ScalarType::Char, x);
        const NormBytes b(kept, m.rows, m.width);
        check("fo_rms_norm", fo_rms_norm(&m, w, wt, eps, &to, b.inv, b.codes, b.steps, stream()));
    } else
        check("fo_rms_norm", fo_rms_norm(&m, w, wt, eps, &to, nullptr, nullptr, nullptr, stream()));
    return {y, kept};
}

std::tuple<Tensor, Tensor> norm_backward(const Tensor &kept, at::IntArrayRef shape, ScalarType type, const Maybe &weight, const Tensor &grad,
                                         bool need_x, bool need_weight)
{
    const Tensor dy = readable(grad, shape, type);
    const fo_rows_t m = matrix(dy, "grad_y");
    int32_t wt;
    const void *w = weight_of(weight, m.width, wt);
    const NormBytes b(kept, m.rows, m.width);
    Tensor gx, gw, parts;
    fo_rows_t to = {};
    if (need_x) {
        gx = empty_like_type(shape, dy);
        to = dense(gx, m.rows, m.width, m.dtype);
    }
    if (need_weight && w) {
        gw = empty_like_type({m.width}, *weight);
        parts = empty_of({fo_rms_norm_workspace(m.rows, m.width)}, ScalarType::Float, dy);
    }
    check("fo_rms_norm_grad", fo_rms_norm_grad(b.codes, b.steps, b.inv, w, wt, &m, need_x ? &to : nullptr, gw.defined() ? gw.data_ptr() : nullptr,
                                               parts.defined() ? parts.data_ptr<float>() : nullptr, stream()));
    return {gx, gw};
}

struct NormFunction : torch::autograd::Function<NormFunction> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Maybe &weight, double eps)
    {
        auto [y, kept] = norm_forward(x, weight, eps, true);
        ctx->save_for_backward({kept, defined(weight) ? *weight : Tensor()});
        Sizes how = {(int64_t)x.scalar_type()};
        how.insert(how.end(), x.sizes().begin(), x.sizes().end());
        ctx->saved_data["how"] = how;
        return y;
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Sizes how = ctx->saved_data["how"].toIntVector();
        const c10::cuda::CUDAGuard guard(saved[0].device());
        const bool has_weight = saved[1].defined();
        auto [gx, gw] = norm_backward(saved[0], at::IntArrayRef(how).slice(1), (ScalarType)how[0], has_weight ? Maybe(saved[1]) : Maybe(),
                                      grads[0], ctx->needs_input_grad(0), has_weight && ctx->needs_input_grad(1));
        return first_order({gx, gw, Tensor()});
    }
};

Tensor rms_norm(const Tensor &x, const Maybe &weight, double eps)
{
    return differentiable(x, weight) ? NormFunction::apply(x, weight, eps) : std::get<0>(norm_forward(x, weight, eps, false));
}

std::tuple<Tensor, Tensor> rms_norm_forward(const Tensor &x, const Maybe &weight, double eps)
{
    at::NoGradGuard no_grad;
    return norm_forward(x, weight, eps, true);
}

std::tuple<Tensor, Maybe> rms_norm_backward(const Tensor &kept, const Sizes &shape, ScalarType type, const Maybe &weight, const Tensor &grad)
{
    int64_t rows = 1;
    for (size_t i = 0; i + 1 < shape.size(); ++i)
        rows *= shape[i];
    array(kept, "kept", ScalarType::Char, NormBytes::size(rows, shape.back()));
    auto [gx, gw] = norm_backward(kept, shape, type, weight, grad, true, true);
    return {gx, gw.defined() ? Maybe(gw) : Maybe()};
}

// --- policy loss -----------------------------------------------------------------------------------

struct RowStrides {
    int64_t rows, inner, row, outer;
};

// The leading dimensions of logits: one stride, or two of which the first counts
// rows of the second (logits[:, :-1]).
RowStrides row_strides(const Tensor &x, const char *name)
{
    const int64_t dims = x.dim();
    TORCH_CHECK_VALUE(dims >= 1, name, " needs a last dimension (the vocabulary)");
    const auto shape = x.sizes(), strides = x.strides();
    TORCH_CHECK_VALUE(strides[dims - 1] == 1 || shape[dims - 1] <= 1, name, ": the last dimension (the vocabulary) must be contiguous");
    if (dims == 2)
        return {shape[0], std::max<int64_t>(1, shape[0]), strides[0], 0};
    std::vector<std::pair<int64_t, int64_t>> merged;   // (size, stride), where one stride covers two dimensions
    for (int64_t i = 0; i + 1 < dims; ++i) {
        const int64_t n = shape[i], s = strides[i];
        if (n == 1)
            continue;
        if (!merged.empty() && merged.back().second == s * n)
            merged.back() = {merged.back().first * n, s};
        else
            merged.push_back({n, s});
    }
    TORCH_CHECK_VALUE(merged.size() <= 2, name, ": the leading dimensions must be covered by two strides (make it contiguous)");
    if (merged.empty())
        return {1, 1, shape[dims - 1], 0};
    if (merged.size() == 1)
        return {merged[0].first, std::max<int64_t>(1, merged[0].first), merged[0].second, 0};
    return {merged[0].first * merged[1].first, std::max<int64_t>(1, merged[1].first), merged[1].second, merged[0].second};
}

fo_logits_t logits_of(const Tensor &x, double temperature)
{
    const int32_t dt = dtype_of(x, "logits");
    check_device(x, "logits");
    const RowStrides s = row_strides(x, "logits");
    return fo_logits_t{x.data_ptr(), s.rows, x.size(-1), s.row, s.inner, s.outer, temperature, dt, 0};
}

// The layout of a gradient that the caller brings, with that of the logits.
fo_logits_grad_t grad_of(fo_logits_t &x, const Tensor &logits, const Tensor &grad)
{
    TORCH_CHECK_TYPE(grad.scalar_type() == logits.scalar_type(), "grad must be ", type_name(logits), ", as the logits are, not ", type_name(grad));
    TORCH_CHECK_VALUE(grad.sizes() == logits.sizes(), "grad must have the logits' shape ", logits.sizes(), ", not ", grad.sizes());
    check_device(grad, "grad");
    RowStrides s = row_strides(grad, "grad");
    if (s.inner != x.inner_rows) {   // one of the two needs a single stride where the other has two
        if (s.inner == s.rows)
            s.outer = s.row * x.inner_rows;
        else {
            TORCH_CHECK_VALUE(x.inner_rows == x.rows, "grad: its leading dimensions are laid out unlike the logits'");
            x.inner_rows = s.inner;
            x.outer_stride = x.row_stride * s.inner;
        }
    }
    return fo_logits_grad_t{grad.data_ptr(), s.row, s.outer};
}

// A new gradient, whose rows start at the logits' rows' alignment modulo 16 bytes
// where these are contiguous or the rows of a padded matrix (at most 7 elements
// are added to a row).
Tensor new_grad(const Tensor &logits, const fo_logits_t &x, fo_logits_grad_t &to)
{
    if (x.inner_rows == x.rows && x.rows > 1 && x.row_stride > x.vocab && logits.dim() == 2) {
        const int64_t pitch = x.vocab + (x.row_stride - x.vocab) % (16 / logits.element_size());
        const Tensor grad = empty_like_type({x.rows, pitch}, logits).narrow(1, 0, x.vocab);
        to = {grad.data_ptr(), pitch, 0};
        return grad;
    }
    const Tensor grad = empty_like_type(logits.sizes(), logits);
    to = {grad.data_ptr(), x.vocab, x.inner_rows * x.vocab};
    return grad;
}

struct Samples {
    Tensor tokens, old_logp, advantages;
    Maybe ref_logp;
    double clip_low, clip_high, kl_weight;
};

// loss, logp, the gradient and the statistics that are asked for.
std::tuple<Tensor, Tensor, Tensor, Tensor> policy(const Tensor &logits, const Samples &s, const Maybe &weight, double temperature,
                                                  bool with_grad, const Maybe &out, bool with_stats)
{
    TORCH_CHECK_VALUE(logits.dim() >= 1, "logits need a last dimension (the vocabulary)");
    const auto lead = logits.sizes().slice(0, logits.dim() - 1);
    const auto rows = [&](const Tensor &t, const char *name) {
        TORCH_CHECK_VALUE(t.sizes() == lead, name, " must have the logits' leading shape ", lead, ", not ", t.sizes());
        return t.is_contiguous() ? t : t.contiguous();
    };
    const Tensor tokens = rows(s.tokens, "tokens"), old = rows(s.old_logp, "old_logp"), adv = rows(s.advantages, "advantages");
    Tensor ref, w;
    if (defined(s.ref_logp))
        ref = rows(*s.ref_logp, "ref_logp");
    if (defined(weight))
        w = rows(*weight, "row_weight");
    fo_logits_t x = logits_of(logits, temperature);
    fo_policy_t p = {};
    p.tokens = static_cast<const int64_t *>(array(tokens, "tokens", ScalarType::Long, x.rows));
    p.old_logp = static_cast<const float *>(array(old, "old_logp", ScalarType::Float, x.rows));
    p.advantages = static_cast<const float *>(array(adv, "advantages", ScalarType::Float, x.rows));
    p.ref_logp = ref.defined() ? static_cast<const float *>(array(ref, "ref_logp", ScalarType::Float, x.rows)) : nullptr;
    p.clip_low = s.clip_low;
    p.clip_high = s.clip_high;
    p.kl_weight = s.kl_weight;
    const float *pw = w.defined() ? static_cast<const float *>(array(w, "row_weight", ScalarType::Float, x.rows)) : nullptr;
    Tensor loss = empty_of(lead, ScalarType::Float, logits), logp = empty_of(lead, ScalarType::Float, logits), grad, stats;
    fo_logits_grad_t to = {};
    if (defined(out)) {
        grad = *out;
        to = grad_of(x, logits, grad);
    } else if (with_grad)
        grad = new_grad(logits, x, to);
    if (with_stats)
        stats = empty_of({x.rows, FO_LOSS_STATS}, ScalarType::Float, logits);
    check("fo_policy_loss", fo_policy_loss(&x, &p, pw, loss.data_ptr<float>(), logp.data_ptr<float>(),
                                           with_stats ? stats.data_ptr<float>() : nullptr, grad.defined() ? &to : nullptr, stream()));
    if (defined(out) && !grad.is_inference())
        torch::autograd::impl::bump_version(grad);
    return {loss, logp, grad, stats};
}

struct PolicyFunction : torch::autograd::Function<PolicyFunction> {
    static variable_list forward(AutogradContext *ctx, const Tensor &logits, const Tensor &tokens, const Tensor &old_logp,
                                 const Tensor &advantages, const Maybe &ref_logp, double clip_low, double clip_high, double kl_weight,
                                 double temperature)
    {
        auto [loss, logp, grad, stats] =
            policy(logits, Samples{tokens, old_logp, advantages, ref_logp, clip_low, clip_high, kl_weight}, {}, temperature, false, {}, true);
        ctx->save_for_backward({logits, tokens, stats});
        ctx->saved_data["temperature"] = temperature;
        ctx->mark_non_differentiable({logp});
        ctx->set_materialize_grads(false);
        return {loss, logp};
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        variable_list result(9);
        if (!grads[0].defined())
            return result;
        const auto saved = ctx->get_saved_variables();
        const Tensor &logits = saved[0], tokens = saved[1].contiguous();
        const c10::cuda::CUDAGuard guard(logits.device());
        const fo_logits_t x = logits_of(logits, ctx->saved_data["temperature"].toDouble());
        fo_logits_grad_t to = {};
        const Tensor g = grads[0].contiguous(), grad = new_grad(logits, x, to);
        check("fo_policy_loss_grad",
              fo_policy_loss_grad(&x, static_cast<const int64_t *>(array(tokens, "tokens", ScalarType::Long, x.rows)),
                                  saved[2].data_ptr<float>(), static_cast<const float *>(array(g, "g_loss", ScalarType::Float, x.rows)), &to,
                                  stream()));
        result[0] = grad;
        return first_order(std::move(result));
    }
};

std::tuple<Tensor, Tensor> policy_loss(const Tensor &logits, const Tensor &tokens, const Tensor &old_logp, const Tensor &advantages,
                                       const Maybe &ref_logp, double clip_low, double clip_high, double kl_weight, double temperature)
{
    if (at::GradMode::is_enabled() && logits.requires_grad()) {
        const auto o = PolicyFunction::apply(logits, tokens, old_logp.detach(), advantages.detach(),
                                             defined(ref_logp) ? Maybe(ref_logp->detach()) : Maybe(), clip_low, clip_high, kl_weight, temperature);
        return {o[0], o[1]};
    }
    auto [loss, logp, grad, stats] =
        policy(logits, Samples{tokens, old_logp, advantages, ref_logp, clip_low, clip_high, kl_weight}, {}, temperature, false, {}, false);
    return {loss, logp};
}

std::tuple<Tensor, Tensor, Tensor> policy_loss_grad(const Tensor &logits, const Tensor &tokens, const Tensor &old_logp,
                                                    const Tensor &advantages, const Maybe &ref_logp, double clip_low, double clip_high,
                                                    double kl_weight, double temperature, const Maybe &row_weight, const Maybe &out)
{
    at::NoGradGuard no_grad;
    auto [loss, logp, grad, stats] = policy(logits, Samples{tokens, old_logp, advantages, ref_logp, clip_low, clip_high, kl_weight}, row_weight,
                                            temperature, true, out, false);
    return {loss, logp, grad};
}

}  // namespace

// Without the interpreter's lock: a launch waits where its stream's queue is full, and an
// allocation may wait for the device, neither of which other Python threads should.
// Arguments are C++ values by then; what calls Python takes the lock (check).
PYBIND11_MODULE(_fo_torch, m)
{
    const py::call_guard<py::gil_scoped_release> unlocked;
    m.def("compress", &compress, unlocked);
    m.def("expand", &expand, unlocked);
    m.def("activation", &activation, unlocked);
    m.def("activation_forward", &activation_forward, unlocked);
    m.def("activation_backward", &activation_backward, unlocked);
    m.def("rms_norm", &rms_norm, unlocked);
    m.def("rms_norm_forward", &rms_norm_forward, unlocked);
    m.def("rms_norm_backward", &rms_norm_backward, unlocked);
    m.def("policy_loss", &policy_loss, unlocked);
    m.def("policy_loss_grad", &policy_loss_grad, unlocked);
    m.def("first_order", &first_order_of, unlocked);
}
