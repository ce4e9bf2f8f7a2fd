// fo_compress.cu -- activations to 8-bit codes and back.
//
// One pass: a group's largest magnitude in registers and one or two shuffles, its
// codes at once. 2 + 1 + 1/16 bytes an element of BF16 either way, 8 to 10
// instructions, so device memory bounds it: 32768 x 14336 BF16 204 us to codes and
// 205 back, 1.03 of the measured copy rate (the last codes written are still in
// the L2 cache). In rows of no alignment the shifting adds about as many
// instructions again: 8191 x 14337 BF16 57 and 65 us, 0.87.
#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256;
// Units of a thread, all loaded before the first is used: 64 bytes of BF16, 32 of
// rows of no alignment to codes (8191 x 14337 57 us, with 64 61), 64 back (65, with 32 68).
template <bool kWide, bool kBack>
constexpr int kUnits = kWide ? 4 : (kBack ? 2 : 1);

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads) compress_kernel(CompressArgs a, UnitGrid g)
{
    constexpr int W = kUnitOf<kWide>, N = kUnits<kWide, false>;
    const uint32_t first = blockIdx.x * (kThreads * N) + threadIdx.x;
    Words<T, W> v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = load_unit<T, kWide>(a.x, place<W>(first + i * kThreads, g.units, g.per_row, (int)a.width));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        f2 x[W / 2];
        widen_unit<T, W>(v[i], x);
        keep_unit<T, W>(a.kept, first + i * kThreads, g.units, v[i], x);
    }
}

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs a, UnitGrid g)
{
    constexpr int W = kUnitOf<kWide>, N = kUnits<kWide, true>;
    const uint32_t first = blockIdx.x * (kThreads * N) + threadIdx.x;
    Kept<W> k[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        k[i] = load_kept<W>(a.kept, first + i * kThreads, g.units);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        f2 x[W / 2];
        kept_unit<W>(k[i], x);
        if constexpr (sizeof(typename T::raw) == 2)
            last_number<T, W>(k[i], x);
        store_unit<T, kWide>(a.x, place<W>(first + i * kThreads, g.units, g.per_row, (int)a.width), narrow_unit<T, W>(x));
    }
}

template <class T, bool kWide>
void run(const CompressArgs &a, cudaStream_t stream)
{
    const UnitGrid g = unit_grid<kUnitOf<kWide>>(a.rows, a.groups);
    constexpr uint32_t kEach = kThreads * kUnits<kWide, false>;
    compress_kernel<T, kWide><<<(g.units + kEach - 1) / kEach, kThreads, 0, stream>>>(a, g);
}
template <class T, bool kWide>
void run(const ExpandArgs &a, cudaStream_t stream)
{
    const UnitGrid g = unit_grid<kUnitOf<kWide>>(a.rows, a.groups);
    constexpr uint32_t kEach = kThreads * kUnits<kWide, true>;
    expand_kernel<T, kWide><<<(g.units + kEach - 1) / kEach, kThreads, 0, stream>>>(a, g);
}

template <class T, class A>
cudaError_t launch(const A &a, cudaStream_t stream)
{
    if (wide<T>(a.width, a.x.data, a.x.stride))
        run<T, true>(a, stream);
    else
        run<T, false>(a, stream);
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
