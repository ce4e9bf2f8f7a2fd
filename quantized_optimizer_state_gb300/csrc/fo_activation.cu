// fo_activation.cu -- activation functions, plain and gated, whose input is kept
// as 8-bit codes for the backward pass.
//   y = f(x) [u], dx = dy f'(x^) [u^], du = dy f(x^)
//
// One pass each way, codes made of the registers that hold the input. A pair of
// gate and other half in BF16 is 8.125 bytes forward and as many backward, 26 and
// 28 instructions an element (30 and 31 for gelu) of the 44 that the copy rate
// leaves room for: bound by device memory, 8192 x 14336 BF16 swiglu 142 and 148 us
// (0.99 and 0.95 of the measured copy rate), FP32 1.02 of it over both (the last
// codes are still in the L2 cache; with other layers between, backward takes 152, and
// FP32 4096 x 14336 125 instead of 118). In rows of no alignment instructions bound it:
// 3001 x 2731 FP16 geglu 38 an element forward, 19.0 us and 16.9 backward where the
// bytes alone take 9.8.
#include "fo_act.cuh"

namespace fo {
namespace {

// Threads of a CTA. Short CTAs end, and their successors' loads begin, at more
// times: 8191 x 14337 BF16 swiglu forward 192 us by 128 threads, 216 by 256; 8192 x
// 14336 backward 148 and 154. Aligned forward passes are the other way round (151
// and 142).
template <bool kWide, bool kGrad>
constexpr int kThreads = kWide && !kGrad ? 256 : 128;

template <class T, int kKind, bool kGated, bool kWide, int kUnits>
__global__ void __launch_bounds__((kThreads<kWide, false>)) activation_kernel(ActivationArgs a, UnitGrid g)
{
    constexpr int W = kUnitOf<kWide>, kBlock = kThreads<kWide, false>;
    const uint32_t first = blockIdx.x * (kBlock * kUnits) + threadIdx.x;
    Words<T, W> v[kUnits], up[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Place p = place<W>(first + i * kBlock, g.units, g.per_row, (int)a.width);
        v[i] = load_unit<T, kWide>(a.x, p);
        if (kGated)
            up[i] = load_unit<T, kWide>(a.up, p);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t unit = first + i * kBlock;
        f2 x[W / 2], u[W / 2], y[W / 2];
        widen_unit<T, W>(v[i], x);
        if (kGated)
            widen_unit<T, W>(up[i], u);
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            y[k] = curve<kKind, kExactType<T>>(x[k]).value;
            if (kGated)
                y[k] = mul2(y[k], u[k]);
        }
        store_unit<T, kWide>(a.y, place<W>(unit, g.units, g.per_row, (int)a.width), narrow_unit<T, W>(y));
        if (a.kept.codes) {
            keep_unit<T, W>(a.kept, unit, g.units, v[i], x);
            if (kGated)
                keep_unit<T, W>(a.kept_up, unit, g.units, up[i], u);
        }
    }
}

template <class T, int kKind, bool kGated, bool kWide, int kUnits>
__global__ void __launch_bounds__((kThreads<kWide, true>)) activation_grad_kernel(ActivationGradArgs a, UnitGrid g)
{
    constexpr int W = kUnitOf<kWide>, kBlock = kThreads<kWide, true>;
    const uint32_t first = blockIdx.x * (kBlock * kUnits) + threadIdx.x;
    Words<T, W> dy[kUnits];
    Kept<W> v[kUnits], up[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t unit = first + i * kBlock;
        dy[i] = load_unit<T, kWide>(a.grad_y, place<W>(unit, g.units, g.per_row, (int)a.width));
        v[i] = load_kept<W>(a.kept, unit, g.units);
        if (kGated)
            up[i] = load_kept<W>(a.kept_up, unit, g.units);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        f2 x[W / 2], u[W / 2], d[W / 2], du[W / 2];
        widen_unit<T, W>(dy[i], d);
        kept_unit<W>(v[i], x);
        if (kGated)
            kept_unit<W>(up[i], u);
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            const Curve f = curve<kKind, kExactType<T>>(x[k]);
            if (kGated) {
                du[k] = mul2(d[k], f.value);
                d[k] = mul2(d[k], u[k]);
            }
            d[k] = mul2(d[k], f.slope);
        }
        const Place p = place<W>(first + i * kBlock, g.units, g.per_row, (int)a.width);
        store_unit<T, kWide>(a.grad, p, narrow_unit<T, W>(d));
        if (kGated)
            store_unit<T, kWide>(a.grad_up, p, narrow_unit<T, W>(du));
    }
}

// Units of a thread, all loaded before the first is used: 64 bytes of BF16 input
// on their way (silu of 8192 x 14336 BF16, forward and backward, by CTAs of 256: two
// units 206 us, four 190), 32 where a unit has 16 elements and registers are short.
template <bool kGated, bool kWide>
constexpr int kUnits = kWide ? (kGated ? 2 : 4) : 1;

inline unsigned ctas(const UnitGrid &g, uint32_t each) { return (g.units + each - 1) / each; }

template <class T, int kKind, bool kGated, bool kWide>
void run(const ActivationArgs &a, cudaStream_t stream)
{
    constexpr int N = kUnits<kGated, kWide>;
    const UnitGrid g = unit_grid<kUnitOf<kWide>>(a.rows, a.groups);
    constexpr int kBlock = kThreads<kWide, false>;
    activation_kernel<T, kKind, kGated, kWide, N><<<ctas(g, kBlock * N), kBlock, 0, stream>>>(a, g);
}
template <class T, int kKind, bool kGated, bool kWide>
void run(const ActivationGradArgs &a, cudaStream_t stream)
{
    constexpr int N = kUnits<kGated, kWide>;
    const UnitGrid g = unit_grid<kUnitOf<kWide>>(a.rows, a.groups);
    constexpr int kBlock = kThreads<kWide, true>;
    activation_grad_kernel<T, kKind, kGated, kWide, N><<<ctas(g, kBlock * N), kBlock, 0, stream>>>(a, g);
}

template <class T>
bool all_wide(const ActivationArgs &a)
{
    return wide<T>(a.width, a.x.data, a.x.stride) && wide<T>(a.width, a.up.data, a.up.stride) && wide<T>(a.width, a.y.data, a.y.stride);
}
template <class T>
bool all_wide(const ActivationGradArgs &a)
{
    return wide<T>(a.width, a.grad_y.data, a.grad_y.stride) && wide<T>(a.width, a.grad.data, a.grad.stride) &&
           wide<T>(a.width, a.grad_up.data, a.grad_up.stride);
}

template <class T, int kKind, bool kGated, class A>
cudaError_t launch(const A &a, cudaStream_t stream)
{
    if (all_wide<T>(a))
        run<T, kKind, kGated, true>(a, stream);
    else
        run<T, kKind, kGated, false>(a, stream);
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
