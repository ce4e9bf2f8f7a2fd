// fo_compress.cu -- activations to 8-bit codes and back.
#include <algorithm>

#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A warp a group, an element a lane.
template <class T>
__global__ void __launch_bounds__(kThreads) compress_kernel(CompressArgs a)
{
    const int64_t step = (int64_t)gridDim.x * kWarps, all = a.rows * a.groups;
    for (int64_t g = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; g < all; g += step) {
        const int64_t r = g / a.groups, c = (g - r * a.groups) * kGroup + (threadIdx.x & 31);
        keep_group(a.kept, g, c < a.width ? load_at<T>(a.x, r, c) : 0.0f);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs a)
{
    const int64_t step = (int64_t)gridDim.x * kWarps, all = a.rows * a.groups;
    for (int64_t g = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; g < all; g += step) {
        const int lane = threadIdx.x & 31;
        const int64_t r = g / a.groups, c = (g - r * a.groups) * kGroup + lane;
        if (c < a.width)
            store_at<T>(a.x, r, c, kept_at(a.kept, g, lane));
    }
}

int64_t ctas_for(int64_t groups) { return std::min<int64_t>((groups + kWarps - 1) / kWarps, (int64_t)sm_count() * 8); }

template <class T>
cudaError_t launch(const CompressArgs &a, cudaStream_t stream)
{
    compress_kernel<T><<<(unsigned)ctas_for(a.rows * a.groups), kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}
template <class T>
cudaError_t launch(const ExpandArgs &a, cudaStream_t stream)
{
    expand_kernel<T><<<(unsigned)ctas_for(a.rows * a.groups), kThreads, 0, stream>>>(a);
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
