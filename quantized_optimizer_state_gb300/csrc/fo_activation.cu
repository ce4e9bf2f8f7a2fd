// fo_activation.cu -- activation functions, plain and gated, whose input is kept
// as 8-bit codes for the backward pass.
#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256;

template <class T, int kKind, bool kGated, bool kWide, int kUnits>
__global__ void __launch_bounds__(kThreads) activation_kernel(ActivationArgs a, UnitGrid g)
{
    const uint32_t first = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    Words<T> v[kUnits], up[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Place p = place(first + i * kThreads, g.units, g.per_row, (int)a.width);
        v[i] = load_unit<T, kWide>(a.x, p);
        if (kGated)
            up[i] = load_unit<T, kWide>(a.up, p);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t unit = first + i * kThreads;
        f2 x[kUnit / 2], u[kUnit / 2], y[kUnit / 2];
        widen_unit<T>(v[i], x);
        if (kGated)
            widen_unit<T>(up[i], u);
#pragma unroll
        for (int k = 0; k < kUnit / 2; ++k) {
            y[k] = curve<kKind, kExactType<T>>(x[k]).value;
            if (kGated)
                y[k] = mul2(y[k], u[k]);
        }
        store_unit<T, kWide>(a.y, place(unit, g.units, g.per_row, (int)a.width), narrow_unit<T>(y));
        if (a.kept.codes) {
            keep_unit<T>(a.kept, unit, g.units, v[i], x);
            if (kGated)
                keep_unit<T>(a.kept_up, unit, g.units, up[i], u);
        }
    }
}

template <class T, int kKind, bool kGated, bool kWide, int kUnits>
__global__ void __launch_bounds__(kThreads) activation_grad_kernel(ActivationGradArgs a, UnitGrid g)
{
    const uint32_t first = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    Words<T> dy[kUnits];
    Kept v[kUnits], up[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t unit = first + i * kThreads;
        dy[i] = load_unit<T, kWide>(a.grad_y, place(unit, g.units, g.per_row, (int)a.width));
        v[i] = load_kept(a.kept, unit, g.units);
        if (kGated)
            up[i] = load_kept(a.kept_up, unit, g.units);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        f2 x[kUnit / 2], u[kUnit / 2], d[kUnit / 2], du[kUnit / 2];
        widen_unit<T>(dy[i], d);
        kept_unit(v[i], x);
        if (kGated)
            kept_unit(up[i], u);
#pragma unroll
        for (int k = 0; k < kUnit / 2; ++k) {
            const Curve f = curve<kKind, kExactType<T>>(x[k]);
            if (kGated) {
                du[k] = mul2(d[k], f.value);
                d[k] = mul2(d[k], u[k]);
            }
            d[k] = mul2(d[k], f.slope);
        }
        const Place p = place(first + i * kThreads, g.units, g.per_row, (int)a.width);
        store_unit<T, kWide>(a.grad, p, narrow_unit<T>(d));
        if (kGated)
            store_unit<T, kWide>(a.grad_up, p, narrow_unit<T>(du));
    }
}

template <int kUnits>
unsigned ctas(const UnitGrid &g) { return (g.units + kThreads * kUnits - 1) / (kThreads * kUnits); }

template <class T, int kKind, bool kGated>
cudaError_t launch(const ActivationArgs &a, cudaStream_t stream)
{
    constexpr int kUnits = 2;
    const UnitGrid g = unit_grid(a.rows, a.groups);
    if (wide<T>(a.width, a.x.data, a.x.stride) && wide<T>(a.width, a.up.data, a.up.stride) && wide<T>(a.width, a.y.data, a.y.stride))
        activation_kernel<T, kKind, kGated, true, kUnits><<<ctas<kUnits>(g), kThreads, 0, stream>>>(a, g);
    else
        activation_kernel<T, kKind, kGated, false, kUnits><<<ctas<kUnits>(g), kThreads, 0, stream>>>(a, g);
    count_launch();
    return cudaGetLastError();
}
template <class T, int kKind, bool kGated>
cudaError_t launch(const ActivationGradArgs &a, cudaStream_t stream)
{
    constexpr int kUnits = 2;
    const UnitGrid g = unit_grid(a.rows, a.groups);
    if (wide<T>(a.width, a.grad_y.data, a.grad_y.stride) && wide<T>(a.width, a.grad.data, a.grad.stride) && wide<T>(a.width, a.grad_up.data, a.grad_up.stride))
        activation_grad_kernel<T, kKind, kGated, true, kUnits><<<ctas<kUnits>(g), kThreads, 0, stream>>>(a, g);
    else
        activation_grad_kernel<T, kKind, kGated, false, kUnits><<<ctas<kUnits>(g), kThreads, 0, stream>>>(a, g);
    count_launch();
    return cudaGetLastError();
}
template <class T, class A>
cudaError_t by_kind(int kind, bool gated, const A &a, cudaStream_t stream)
{
    if (kind == kSilu)
        return gated ? launch<T, kSilu, true>(a, stream) : launch<T, kSilu, false>(a, stream);
    return gated ? launch<T, kGelu, true>(a, stream) : launch<T, kGelu, false>(a, stream);
}
template <class A>
cudaError_t by_type(int dtype, int kind, bool gated, const A &a, cudaStream_t stream)
{
    return dtype == 0   ? by_kind<Bf16>(kind, gated, a, stream)
           : dtype == 1 ? by_kind<F32>(kind, gated, a, stream)
                        : by_kind<F16>(kind, gated, a, stream);
}

}  // namespace

cudaError_t launch_activation(int dtype, int kind, const ActivationArgs &a, cudaStream_t stream)
{
    return by_type(dtype, kind, a.up.data != nullptr, a, stream);
}
cudaError_t launch_activation_grad(int dtype, int kind, const ActivationGradArgs &a, cudaStream_t stream)
{
    return by_type(dtype, kind, a.grad_up.data != nullptr, a, stream);
}

}  // namespace fo
