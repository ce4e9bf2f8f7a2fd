// fo_compress.cu -- activations to 8-bit codes and back.
#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;   // units of a thread, all loaded before the first is used

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads) compress_kernel(CompressArgs a, UnitGrid g)
{
    const uint32_t first = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    Words<T> v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        v[i] = load_unit<T, kWide>(a.x, place(first + i * kThreads, g.units, g.per_row, (int)a.width));
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        f2 x[kUnit / 2];
        widen_unit<T>(v[i], x);
        keep_unit<T>(a.kept, first + i * kThreads, g.units, v[i], x);
    }
}

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs a, UnitGrid g)
{
    const uint32_t first = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    Kept k[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        k[i] = load_kept(a.kept, first + i * kThreads, g.units);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        f2 x[kUnit / 2];
        kept_unit(k[i], x);
        store_unit<T, kWide>(a.x, place(first + i * kThreads, g.units, g.per_row, (int)a.width), narrow_unit<T>(x));
    }
}

unsigned ctas(const UnitGrid &g) { return (g.units + kThreads * kUnits - 1) / (kThreads * kUnits); }

template <class T>
cudaError_t launch(const CompressArgs &a, cudaStream_t stream)
{
    const UnitGrid g = unit_grid(a.rows, a.groups);
    if (wide<T>(a.width, a.x.data, a.x.stride))
        compress_kernel<T, true><<<ctas(g), kThreads, 0, stream>>>(a, g);
    else
        compress_kernel<T, false><<<ctas(g), kThreads, 0, stream>>>(a, g);
    count_launch();
    return cudaGetLastError();
}
template <class T>
cudaError_t launch(const ExpandArgs &a, cudaStream_t stream)
{
    const UnitGrid g = unit_grid(a.rows, a.groups);
    if (wide<T>(a.width, a.x.data, a.x.stride))
        expand_kernel<T, true><<<ctas(g), kThreads, 0, stream>>>(a, g);
    else
        expand_kernel<T, false><<<ctas(g), kThreads, 0, stream>>>(a, g);
    count_launch();
    return cudaGetLastError();
}
template <class A>
cudaError_t by_type(int dtype, const A &a, cudaStream_t stream)
{
    return dtype == 0 ? launch<Bf16>(a, stream) : dtype == 1 ? launch<F32>(a, stream) : launch<F16>(a, stream);
}

}  // namespace

cudaError_t launch_compress(int dtype, const CompressArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }
cudaError_t launch_expand(int dtype, const ExpandArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }

}  // namespace fo
