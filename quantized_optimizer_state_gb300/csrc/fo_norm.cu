// fo_norm.cu -- root-mean-square norm whose input is kept as 8-bit codes for the
// backward pass.
//   r = 1 / sqrt(mean x^2 + eps), y = x r w
//   h = x^ r: dx = r (dy w - h mean(dy w h)), dw = sum over rows of dy h
#include <algorithm>

#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// --- 1 / rms -----------------------------------------------------------------------

// Squares of a row whose sum reaches 2^120 may lie outside FP32: such rows, which
// are rare, are summed again at 2^-96 of their size, where a sum that is not
// finite means that the row holds a NaN or an infinity.
constexpr float kLargeSum = 0x1p120f, kDown = 0x1p-96f;

// 1 / sqrt(m) for m in [2^-80, 2^121]: the hardware's approximation and a step of Newton's.
__device__ __forceinline__ float reciprocal_root(float m)
{
    const float y = rsqrt_approx(m), e = __fmaf_rn(-__fmul_rn(m, y), y, 1.0f);
    return __fmaf_rn(__fmul_rn(0.5f, y), e, y);
}
__device__ __forceinline__ float inverse_rms(float sum, const NormArgs &a) { return reciprocal_root(__fmaf_rn(sum, a.inv_width, a.eps)); }
__device__ __forceinline__ float inverse_rms_down(float sum, const NormArgs &a)
{
    return sum < kInf ? __fmul_rn(reciprocal_root(__fmul_rn(sum, a.inv_width)), kDown) : kNan;
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


// The weight of a unit; 1 without one.
__device__ __forceinline__ void weight_unit(const void *w, int dtype, bool aligned, const Place &p, f2 (&x)[kUnit / 2])
{
    if (w && aligned && p.left >= kUnit) {
        if (dtype == FO_LOGITS_F32) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.col));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.col) + 1);
            x[0] = pk(a.x, a.y);
            x[1] = pk(a.z, a.w);
            x[2] = pk(b.x, b.y);
            x[3] = pk(b.z, b.w);
            return;
        }
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + p.col));
        if (dtype == FO_LOGITS_BF16)
            widen_vec<Bf16>(a, x);
        else
            widen_vec<F16>(a, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i)
        x[i] = pk(2 * i < p.left ? weight_at(w, dtype, p.col + 2 * i) : 0.0f, 2 * i + 1 < p.left ? weight_at(w, dtype, p.col + 2 * i + 1) : 0.0f);
}

__device__ __forceinline__ float both(f2 v)
{
    float a, b;
    unpk(v, a, b);
    return __fadd_rn(a, b);
}

// The sum of v over the kLanes threads of a row, in every one of them. More than
// a warp: they are a CTA, and `part` holds its warps' sums (two sets in turn, so
// that one barrier a sum is enough).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float *part)
{
#pragma unroll
    for (int o = (kLanes < 32 ? kLanes : 32) / 2; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    if constexpr (kLanes > 32) {
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x / 32] = v;
        __syncthreads();
        v = part[threadIdx.x % (kLanes / 32)];
#pragma unroll
        for (int o = kLanes / 64; o; o >>= 1)
            v += __shfl_xor_sync(~0u, v, o);
    }
    return v;
}

// The place of unit u of row r; beyond the rows, and beyond the row's units, it is none.
__device__ __forceinline__ Place row_place(int r, int rows, int u, int units, int width)
{
    Place p;
    const bool there = r < rows && u < units;
    p.row = there ? r : -1;
    p.col = u * kUnit;
    p.left = there ? width - p.col : -64;
    return p;
}

template <int kLanes>
constexpr int kBlockOf = kLanes > 32 ? kLanes : kThreads;   // threads of a CTA

// --- rows held in registers --------------------------------------------------------------

// A team of kLanes threads to a row, each thread with kVecs of its units (kLanes
// apart) and their weights. A team takes rows a grid apart, the next one's loads
// on their way while one is worked on.
constexpr int kThreadsPerSm = 1024;   // of norm_kernel
template <int kVecs>
constexpr int kGradThreadsPerSm = kVecs == 1 ? 1024 : 512;   // of norm_grad_kernel
template <class T, bool kWide, int kLanes, int kVecs>
__global__ void __launch_bounds__(kBlockOf<kLanes>, kThreadsPerSm / kBlockOf<kLanes>) norm_kernel(NormArgs a)
{
    __shared__ float part[4][kLanes > 32 ? kLanes / 32 : 1];
    constexpr int kTeams = kBlockOf<kLanes> / kLanes;
    const int lane = threadIdx.x % kLanes, units = (int)a.groups * 4, rows = (int)a.rows, width = (int)a.width;
    const int step = gridDim.x * kTeams;
    int r = blockIdx.x * kTeams + threadIdx.x / kLanes;
    Words<T> next[kVecs];
    f2 w[kVecs][kUnit / 2];
    const auto fetch = [&](int row) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            next[k] = load_unit<T, kWide>(a.x, row_place(row, rows, lane + k * kLanes, units, width));
    };
    fetch(r);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        weight_unit(a.weight, a.weight_dtype, a.weight_aligned, row_place(0, 1, lane + k * kLanes, units, width), w[k]);
    int turn = 0;
    // every thread takes as many turns as the CTA's first team: barriers and shuffles are all threads'
    for (int base = blockIdx.x * kTeams; base < rows; base += step, r += step, turn ^= 2) {
        // what needs no sum comes first, so that less waits for it
        f2 x[kVecs][kUnit / 2];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            widen_unit<T>(next[k], x[k]);
            if (a.kept.codes)
                keep_unit<T>(a.kept, (uint32_t)r * units + lane + k * kLanes, r < rows && lane + k * kLanes < units ? ~0u : 0u, next[k], x[k]);
        }
        fetch(r + step);
        const auto squares = [&](float scale) {
            f2 sum = 0;
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
#pragma unroll
                for (int j = 0; j < kUnit / 2; ++j) {
                    const f2 v = scale != 1.0f ? mul2(x[k][j], splat(scale)) : x[k][j];
                    sum = fma2(v, v, sum);
                }
            return both(sum);
        };
        const float sum = row_sum<kLanes>(squares(1.0f), part[turn]);
        const bool large = !(sum < kLargeSum);
        float inv = inverse_rms(sum, a);
        if (kLanes > 32 ? large : __any_sync(~0u, large)) {   // the same in a CTA; other rows of a warp keep theirs
            const float down = inverse_rms_down(row_sum<kLanes>(squares(kDown), part[turn + 1]), a);
            inv = large ? down : inv;
        }
        if (lane == 0 && a.inv_rms && r < rows)
            a.inv_rms[r] = inv;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
#pragma unroll
            for (int j = 0; j < kUnit / 2; ++j)
                x[k][j] = mul2(mul2(x[k][j], splat(inv)), w[k][j]);
            store_unit<T, kWide, (kLanes < 32 ? kLanes : 32)>(a.y, row_place(r, rows, lane + k * kLanes, units, width), narrow_unit<T>(x[k]));
        }
    }
}

// A unit of dy and of the kept x, as loaded.
template <class T>
struct GradUnit {
    Words<T> dy;
    Kept x;
};

// The same for the gradient; the weight's gradient of a thread's columns is added
// up in registers. A CTA's teams are joined in shared memory and leave one row of
// partial sums.
template <class T, bool kWide, int kLanes, int kVecs>
__global__ void __launch_bounds__(kBlockOf<kLanes>, kGradThreadsPerSm<kVecs> / kBlockOf<kLanes>) norm_grad_kernel(NormGradArgs a)
{
    constexpr int kTeams = kBlockOf<kLanes> / kLanes;
    __shared__ float part[2][kLanes > 32 ? kLanes / 32 : 1];
    __shared__ __align__(16) float joined[kTeams > 1 ? kTeams : 1][kTeams > 1 ? kLanes * kVecs * kUnit : 4];
    const int lane = threadIdx.x % kLanes, team = threadIdx.x / kLanes, units = (int)a.groups * 4, rows = (int)a.rows, width = (int)a.width;
    f2 w[kVecs][kUnit / 2], dw[kVecs][kUnit / 2];
    const int step = gridDim.x * kTeams;
    GradUnit<T> next[kVecs];
    float next_inv;
    const auto fetch = [&](int r) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int u = lane + k * kLanes;
            const Place p = row_place(r, rows, u, units, width);
            next[k].dy = load_unit<T, kWide>(a.grad_y, p);
            next[k].x = load_kept(a.kept, (uint32_t)r * units + u, p.row < 0 ? 0u : ~0u);
        }
        next_inv = r < rows ? __ldg(a.inv_rms + r) : 0.0f;
    };
    int r = blockIdx.x * kTeams + team;
    fetch(r);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        weight_unit(a.weight, a.weight_dtype, a.weight_aligned, row_place(0, 1, lane + k * kLanes, units, width), w[k]);
#pragma unroll
        for (int j = 0; j < kUnit / 2; ++j)
            dw[k][j] = 0;
    }
    int turn = 0;
    for (int base = blockIdx.x * kTeams; base < rows; base += step, r += step, turn ^= 1) {
        f2 t[kVecs][kUnit / 2], h[kVecs][kUnit / 2], dot = 0;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            widen_unit<T>(next[k].dy, t[k]);
            kept_unit(next[k].x, h[k], next_inv);
#pragma unroll
            for (int j = 0; j < kUnit / 2; ++j) {
                dw[k][j] = fma2(t[k][j], h[k][j], dw[k][j]);
                t[k][j] = mul2(t[k][j], w[k][j]);
                dot = fma2(t[k][j], h[k][j], dot);
            }
        }
        const float inv = next_inv;
        fetch(r + step);
        if (a.grad.data) {
            const f2 mean = splat(-__fmul_rn(row_sum<kLanes>(both(dot), part[turn]), a.inv_width));
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
#pragma unroll
                for (int j = 0; j < kUnit / 2; ++j)
                    t[k][j] = mul2(fma2(h[k][j], mean, t[k][j]), splat(inv));
                store_unit<T, kWide, (kLanes < 32 ? kLanes : 32)>(a.grad, row_place(r, rows, lane + k * kLanes, units, width), narrow_unit<T>(t[k]));
            }
        }
    }
    if (!a.grad_weight)
        return;
    float *const to = a.parts + (int64_t)blockIdx.x * a.groups * kGroup;
    if constexpr (kTeams > 1) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
            for (int j = 0; j < kUnit / 2; ++j)
                *reinterpret_cast<f2 *>(&joined[team][(lane + k * kLanes) * kUnit + 2 * j]) = dw[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < units * kUnit; c += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kTeams; ++i)
                sum += joined[i][c];
            to[c] = sum;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int u = lane + k * kLanes;
            if (u < units)
#pragma unroll
                for (int j = 0; j < kUnit / 4; ++j)
                    reinterpret_cast<ulonglong2 *>(to + u * kUnit)[j] = make_ulonglong2(dw[k][2 * j], dw[k][2 * j + 1]);
        }
    }
}

// The parts of 32 columns by a CTA: 32 chains a column, joined pairwise.
constexpr int kJoin = 32;
__global__ void __launch_bounds__(kJoin * 32) norm_weight_kernel(NormGradArgs a, int parts)
{
    __shared__ float part[kJoin][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane, pitch = a.groups * kGroup;
    float sum = 0.0f;
#pragma unroll 8
    for (int p = warp; p < parts; p += kJoin)
        sum += a.parts[p * pitch + c];
    part[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(part[lane][warp]);   // column `warp`, its chains across the lanes
    if (lane == 0 && (int64_t)blockIdx.x * 32 + warp < a.width)
        store_weight(a.grad_weight, a.weight_dtype, (int64_t)blockIdx.x * 32 + warp, sum);
}

// --- longer rows: read again from the L2 cache -----------------------------------------------

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
    const float step = step_of<false>(__reduce_max_sync(~0u, __float_as_uint(x) & 0x7fffffffu));
    const int lane = threadIdx.x & 31;
    k.codes[group * kGroup + lane] = (int8_t)__float_as_uint(__fmaf_rn(x, step_reciprocal(step), kRound));
    if (lane == 0)
        k.steps[group] = step_bits(step);
}
__device__ __forceinline__ float kept_at(const KeptIn &k, int64_t group, int lane)
{
    return __fmul_rn((float)k.codes[group * kGroup + lane], step_value(k.steps[group]));
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

// A row a CTA.
template <class T>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormArgs a)
{
    __shared__ float part[kWarps];
    const int64_t r = blockIdx.x;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float x = load_at<T>(a.x, r, c);
        sum = __fmaf_rn(x, x, sum);
    }
    sum = block_sum(sum, part);
    float inv = inverse_rms(sum, a);
    if (!(sum < kLargeSum)) {   // the same in the whole CTA
        sum = 0.0f;
        for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
            const float x = __fmul_rn(load_at<T>(a.x, r, c), kDown);
            sum = __fmaf_rn(x, x, sum);
        }
        inv = inverse_rms_down(block_sum(sum, part), a);
    }
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
__global__ void __launch_bounds__(kThreads) norm_long_grad_kernel(NormGradArgs a)
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
__global__ void __launch_bounds__(kThreads) norm_long_weight_kernel(NormGradArgs a)
{
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= a.groups * kGroup)
        return;
    float sum = 0.0f;
    for (int64_t r = blockIdx.x; c < a.width && r < a.rows; r += gridDim.x) {
        const float h = __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), a.inv_rms[r]);
        sum = __fmaf_rn(load_at<T>(a.grad_y, r, c), h, sum);
    }
    a.parts[blockIdx.x * a.groups * kGroup + c] = sum;
}


constexpr int64_t kMaxUnits = 2048;   // of a row in registers: 16384 elements

template <class T, bool kWide, int kLanes, int kVecs>
cudaError_t launch(const NormArgs &a, cudaStream_t stream)
{
    constexpr int kBlock = kBlockOf<kLanes>, kTeams = kBlock / kLanes;
    const int64_t ctas = std::min((a.rows + kTeams - 1) / kTeams, (int64_t)sm_count() * (kThreadsPerSm / kBlock));
    norm_kernel<T, kWide, kLanes, kVecs><<<(unsigned)ctas, kBlock, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}
template <class T, bool kWide>
cudaError_t launch(const NormArgs &a, cudaStream_t stream)
{
    // 32 bytes of x a thread. 16384 x 4096: BF16 with one unit a thread 65 us, two
    // 57, four 71 (spills); FP32 99 with one, 108 with two. 131072 x 128 BF16 18.2
    // with one, 17.3 with two.
    constexpr int k = sizeof(typename T::raw) == 2 ? 2 : 1;
    const int64_t units = a.groups * 4;
    if (units <= 4)
        return launch<T, kWide, 4, 1>(a, stream);
    if (units <= 8)
        return launch<T, kWide, 8 / k, k>(a, stream);
    if (units <= 16)
        return launch<T, kWide, 16 / k, k>(a, stream);
    if (units <= 32)
        return launch<T, kWide, 32 / k, k>(a, stream);
    if (units <= 64)
        return launch<T, kWide, 32, 2>(a, stream);
    if (units <= 128)
        return launch<T, kWide, 128 / k, k>(a, stream);
    if (units <= 256)
        return launch<T, kWide, 256 / k, k>(a, stream);
    if (units <= 512)
        return launch<T, kWide, 512 / k, k>(a, stream);
    if (units <= 1024)
        return launch<T, kWide, 1024 / k, k>(a, stream);
    return launch<T, kWide, 1024, 2>(a, stream);
}
template <class T>
cudaError_t launch(NormArgs a, cudaStream_t stream)
{
    a.inv_width = (float)(1.0 / (double)a.width);
    a.weight_aligned = (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
    if (a.groups * 4 <= kMaxUnits)
        return wide<T>(a.width, a.x.data, a.x.stride) && wide<T>(a.width, a.y.data, a.y.stride) ? launch<T, true>(a, stream) : launch<T, false>(a, stream);
    norm_long_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

// The CTAs that are on the device at once, or one for each set of teams; the
// parts they leave are then added up.
template <class T, bool kWide, int kLanes, int kVecs>
int launch_parts(const NormGradArgs &a, cudaStream_t stream)
{
    constexpr int kBlock = kBlockOf<kLanes>, kTeams = kBlock / kLanes;
    const int64_t fit = std::min<int64_t>(FO_NORM_PARTS, (int64_t)sm_count() * std::max(1, kGradThreadsPerSm<kVecs> / kBlock));
    const int ctas = (int)std::min<int64_t>((a.rows + kTeams - 1) / kTeams, fit);
    norm_grad_kernel<T, kWide, kLanes, kVecs><<<ctas, kBlock, 0, stream>>>(a);
    count_launch();
    return ctas;
}
template <class T, bool kWide>
int launch_parts(const NormGradArgs &a, cudaStream_t stream)
{
    const int64_t units = a.groups * 4;
    // A warp with two units a thread where they hold the row, one unit a thread of
    // more warps beyond (65536 x 512 FP32 49 us, by 64 threads 61; 65536 x 768 BF16
    // by 64 threads 59, by 128 56; 16384 x 4096 BF16 64.6 and 63.6); 4096 x 16384
    // BF16 by 512 threads of four units 125, by 1024 of two 96.
    if (units <= 4)
        return launch_parts<T, kWide, 4, 1>(a, stream);
    if (units <= 8)
        return launch_parts<T, kWide, 4, 2>(a, stream);
    if (units <= 16)
        return launch_parts<T, kWide, 8, 2>(a, stream);
    if (units <= 32)
        return launch_parts<T, kWide, 16, 2>(a, stream);
    if (units <= 64)
        return launch_parts<T, kWide, 32, 2>(a, stream);
    if (units <= 128)
        return launch_parts<T, kWide, 128, 1>(a, stream);
    if (units <= 256)
        return launch_parts<T, kWide, 256, 1>(a, stream);
    if (units <= 512)
        return launch_parts<T, kWide, 512, 1>(a, stream);
    if (units <= 1024)
        return launch_parts<T, kWide, 1024, 1>(a, stream);
    return launch_parts<T, kWide, 1024, 2>(a, stream);
}
template <class T>
cudaError_t launch(NormGradArgs a, cudaStream_t stream)
{
    a.inv_width = (float)(1.0 / (double)a.width);
    a.weight_aligned = (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
    int parts = 0;
    if (a.rows > 0 && a.groups * 4 <= kMaxUnits)
        parts = wide<T>(a.width, a.grad_y.data, a.grad_y.stride) && wide<T>(a.width, a.grad.data, a.grad.stride) ? launch_parts<T, true>(a, stream)
                                                                                               : launch_parts<T, false>(a, stream);
    else if (a.rows > 0) {
        if (a.grad.data) {
            norm_long_grad_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
            count_launch();
        }
        if (a.grad_weight) {
            parts = (int)std::min<int64_t>(a.rows, FO_NORM_PARTS);
            norm_long_weight_kernel<T><<<dim3((unsigned)parts, (unsigned)((a.groups * kGroup + kThreads - 1) / kThreads)), kThreads, 0, stream>>>(a);
            count_launch();
        }
    }
    if (a.grad_weight) {
        norm_weight_kernel<<<(unsigned)a.groups, kJoin * 32, 0, stream>>>(a, parts);
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
