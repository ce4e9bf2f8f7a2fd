// fo_activation.cu -- activation functions, plain and gated, whose input is kept
// as 8-bit codes for the backward pass.
#include <algorithm>

#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A warp a group, an element a lane.
template <class T, int kKind, bool kGated>
__global__ void __launch_bounds__(kThreads) activation_kernel(ActivationArgs a)
{
    const int64_t step = (int64_t)gridDim.x * kWarps, all = a.rows * a.groups;
    for (int64_t g = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; g < all; g += step) {
        const int64_t r = g / a.groups, c = (g - r * a.groups) * kGroup + (threadIdx.x & 31);
        const float x = c < a.width ? load_at<T>(a.x, r, c) : 0.0f;
        const float up = kGated && c < a.width ? load_at<T>(a.up, r, c) : 0.0f;
        const float f = curve<kKind, kExactType<T>, false>(x).value;
        if (c < a.width)
            store_at<T>(a.y, r, c, kGated ? __fmul_rn(f, up) : f);
        if (a.kept.codes) {
            keep_group(a.kept, g, x);
            if (kGated)
                keep_group(a.kept_up, g, up);
        }
    }
}

template <class T, int kKind, bool kGated>
__global__ void __launch_bounds__(kThreads) activation_grad_kernel(ActivationGradArgs a)
{
    const int64_t step = (int64_t)gridDim.x * kWarps, all = a.rows * a.groups;
    for (int64_t g = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; g < all; g += step) {
        const int lane = threadIdx.x & 31;
        const int64_t r = g / a.groups, c = (g - r * a.groups) * kGroup + lane;
        if (c >= a.width)
            continue;
        const float dy = load_at<T>(a.grad_y, r, c);
        const Curve f = curve<kKind, kExactType<T>, true>(kept_at(a.kept, g, lane));
        if (kGated) {
            store_at<T>(a.grad, r, c, __fmul_rn(__fmul_rn(dy, kept_at(a.kept_up, g, lane)), f.slope));
            store_at<T>(a.grad_up, r, c, __fmul_rn(dy, f.value));
        } else
            store_at<T>(a.grad, r, c, __fmul_rn(dy, f.slope));
    }
}

int64_t ctas_for(int64_t groups) { return std::min<int64_t>((groups + kWarps - 1) / kWarps, (int64_t)sm_count() * 8); }

template <class T, int kKind, bool kGated>
cudaError_t launch(const ActivationArgs &a, cudaStream_t stream)
{
    activation_kernel<T, kKind, kGated><<<(unsigned)ctas_for(a.rows * a.groups), kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}
template <class T, int kKind, bool kGated>
cudaError_t launch(const ActivationGradArgs &a, cudaStream_t stream)
{
    activation_grad_kernel<T, kKind, kGated><<<(unsigned)ctas_for(a.rows * a.groups), kThreads, 0, stream>>>(a);
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
