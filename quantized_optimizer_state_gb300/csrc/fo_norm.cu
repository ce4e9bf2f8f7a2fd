// fo_norm.cu -- root-mean-square norm whose input is kept as 8-bit codes for the
// backward pass.
//   r = 1 / sqrt(mean x^2 + eps), y = x r w
//   h = x^ r: dx = r (dy w - h mean(dy w h)), dw = sum over rows of dy h
#include <algorithm>

#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Element `c` of row `r`.
template <class T>
__device__ __forceinline__ float load_at(const RowsIn &x, int64_t r, int64_t c)
{
    return T::widen(static_cast<const typename T::raw *>(x.data)[r * x.stride + c]);
}
template <class T>
__device__ __forceinline__ void store_at(const RowsOut &x, int64_t r, int64_t c, float v)
{
    static_cast<typename T::raw *>(x.data)[r * x.stride + c] = T::narrow(v);
}

// A group by a warp, an element a lane.
__device__ __forceinline__ void keep_group(const KeptOut &k, int64_t group, float x)
{
    const float step = step_of(__reduce_max_sync(~0u, magnitude(x)));
    const int lane = threadIdx.x & 31;
    k.codes[group * kGroup + lane] = (int8_t)code_word(x, __frcp_rn(step));
    if (lane == 0)
        k.steps[group] = step_bits(step);
}
__device__ __forceinline__ float kept_at(const KeptIn &k, int64_t group, int lane)
{
    return __fmul_rn((float)k.codes[group * kGroup + lane], step_value(k.steps[group]));
}

__device__ __forceinline__ float weight_at(const void *w, int dtype, int64_t i)
{
    if (!w)
        return 1.0f;
    return dtype == FO_LOGITS_F32    ? static_cast<const float *>(w)[i]
           : dtype == FO_LOGITS_BF16 ? Bf16::widen(static_cast<const uint16_t *>(w)[i])
                                     : F16::widen(static_cast<const uint16_t *>(w)[i]);
}
__device__ __forceinline__ void store_weight(void *w, int dtype, int64_t i, float v)
{
    if (dtype == FO_LOGITS_F32)
        static_cast<float *>(w)[i] = v;
    else
        static_cast<uint16_t *>(w)[i] = dtype == FO_LOGITS_BF16 ? Bf16::narrow(v) : F16::narrow(v);
}

// The sum of v over the CTA, in every thread.
__device__ __forceinline__ float block_sum(float v, float *part)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// 1 / sqrt(mean x^2 + eps) from the sum of squares of x / scale.
__device__ __forceinline__ float inverse_rms(float sum, float scale, const NormArgs &a)
{
    const float mean = sum / (float)a.width;
    return 1.0f / scale / sqrtf(mean + a.eps / scale / scale);
}

// A row a CTA.
template <class T>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs a)
{
    __shared__ float part[kWarps];
    const int64_t r = blockIdx.x;
    float sum = 0.0f, most = 0.0f;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float x = load_at<T>(a.x, r, c);
        sum = __fmaf_rn(x, x, sum);
    }
    sum = block_sum(sum, part);
    float scale = 1.0f;
    if (!(sum < 0x1p120f)) {   // rare: x^2 may lie outside FP32, or x is not finite
        for (int64_t c = threadIdx.x; c < a.width; c += kThreads)
            most = max_nan(most, fabsf(load_at<T>(a.x, r, c)));
#pragma unroll
        for (int o = 16; o; o >>= 1)
            most = max_nan(most, __shfl_xor_sync(~0u, most, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x / 32] = most;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i)
            most = max_nan(most, part[i]);
        scale = most < kInf ? 0x1p96f : kNan;
        sum = 0.0f;
        for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
            const float x = load_at<T>(a.x, r, c) / scale;
            sum = __fmaf_rn(x, x, sum);
        }
        sum = block_sum(sum, part);
    }
    const float inv = inverse_rms(sum, scale, a);
    if (threadIdx.x == 0 && a.inv_rms)
        a.inv_rms[r] = inv;
    for (int64_t g = threadIdx.x / 32; g < a.groups; g += kWarps) {
        const int64_t c = g * kGroup + (threadIdx.x & 31);
        const float x = c < a.width ? load_at<T>(a.x, r, c) : 0.0f;
        if (c < a.width)
            store_at<T>(a.y, r, c, __fmul_rn(__fmul_rn(x, inv), weight_at(a.weight, a.weight_dtype, c)));
        if (a.kept.codes)
            keep_group(a.kept, r * a.groups + g, x);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(NormGradArgs a)
{
    __shared__ float part[kWarps];
    const int64_t r = blockIdx.x;
    const float inv = a.inv_rms[r];
    float dot = 0.0f;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float h = __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), inv);
        dot = __fmaf_rn(__fmul_rn(load_at<T>(a.grad_y, r, c), weight_at(a.weight, a.weight_dtype, c)), h, dot);
    }
    const float mean = block_sum(dot, part) / (float)a.width;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float h = __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), inv);
        const float g = __fmul_rn(load_at<T>(a.grad_y, r, c), weight_at(a.weight, a.weight_dtype, c));
        store_at<T>(a.grad, r, c, __fmul_rn(inv, __fmaf_rn(-h, mean, g)));
    }
}

// Columns by a thread each, rows part, part + parts, ... by a CTA.
template <class T>
__global__ void __launch_bounds__(kThreads) norm_weight_parts_kernel(NormGradArgs a)
{
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= a.width)
        return;
    float sum = 0.0f;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float h = __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), a.inv_rms[r]);
        sum = __fmaf_rn(load_at<T>(a.grad_y, r, c), h, sum);
    }
    a.parts[blockIdx.x * a.width + c] = sum;
}

// The parts of 32 columns by a CTA: eight chains a column, joined pairwise.
__global__ void __launch_bounds__(kThreads) norm_weight_kernel(NormGradArgs a, int parts)
{
    __shared__ float part[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f;
    for (int p = warp; c < a.width && p < parts; p += kWarps)
        sum += a.parts[p * a.width + c];
    part[warp][lane] = sum;
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) {
        __syncthreads();
        if (warp < o)
            part[warp][lane] += part[warp + o][lane];
    }
    if (warp == 0 && c < a.width)
        store_weight(a.grad_weight, a.weight_dtype, c, part[0][lane]);
}

template <class T>
cudaError_t launch(const NormArgs &a, cudaStream_t stream)
{
    norm_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}
template <class T>
cudaError_t launch(const NormGradArgs &a, cudaStream_t stream)
{
    if (a.grad.data) {
        norm_grad_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
        count_launch();
    }
    if (a.grad_weight) {
        const int parts = (int)std::min<int64_t>(a.rows, FO_NORM_PARTS);
        const unsigned columns = (unsigned)((a.width + kThreads - 1) / kThreads);
        if (parts) {
            norm_weight_parts_kernel<T><<<dim3((unsigned)parts, columns), kThreads, 0, stream>>>(a);
            count_launch();
        }
        norm_weight_kernel<<<(unsigned)((a.width + 31) / 32), kThreads, 0, stream>>>(a, parts);
        count_launch();
    }
    return cudaGetLastError();
}
template <class A>
cudaError_t by_type(int dtype, const A &a, cudaStream_t stream)
{
    return dtype == 0 ? launch<Bf16>(a, stream) : dtype == 1 ? launch<F32>(a, stream) : launch<F16>(a, stream);
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }
cudaError_t launch_norm_grad(int dtype, const NormGradArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }

}  // namespace fo
