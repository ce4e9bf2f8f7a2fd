// fo_norm.cu -- root-mean-square norm whose input is kept as 8-bit codes for the
// backward pass.
//   r = 1 / sqrt(mean x^2 + eps), y = x r w
//   h = x^ r: dx = r (dy w - h mean(dy w h)), dw = sum over rows of dy h
//
// A row stays in registers between its sum and its result, so that every byte
// crosses device memory once: 5.0625 bytes an element of BF16 either way. The
// codes need no sum and come before it is waited for; the weight's gradient is
// summed in registers over the rows that a team takes, and a second, small launch
// adds up what the CTAs left (3 us). 16384 x 4096 BF16: 56 and 56 us, 0.89 of the
// measured copy rate, 15 and 18 instructions an element; FP32 98 and 91, 0.95. The
// backward passes are those right after their forward passes, which find the last
// codes in the L2 cache: with other layers between they take 64 and 97.
// What is missing are the waits of a CTA for a row's sum: rows two ahead instead of
// one changed nothing. Rows of 128 take 16.6 and 15.5 us (18.5 with other layers
// between) for 131072, where the bytes alone take 12.6. Rows of no alignment are bound by instructions and
// occupancy: 8191 x 4099 BF16 50 and 65 us where the bytes take 25 each.
#include <algorithm>

#include "fo_act.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// --- sums ------------------------------------------------------------------------------

// A sum of products that keeps what its roundings lose (W. Kahan, "Further remarks on
// reducing truncation errors", CACM 8(1), 1965): off by 2 roundings, whatever the
// number of terms. One after another like terms are all rounded the same way:
// 20 million equal squares, 78000 a thread, came out 9e-4 off.
struct LongSum {
    float sum = 0.0f, over = 0.0f;   // `over`: what is in the sum too much
    __device__ __forceinline__ void add(float a, float b = 1.0f)
    {
        const float y = __fmaf_rn(a, b, -over), t = __fadd_rn(sum, y);
        over = fabsf(t) < kInf ? __fsub_rn(__fsub_rn(t, sum), y) : 0.0f;   // infinities go on as such
        sum = t;
    }
    // The sum of a warp's sums, in every lane: pairs with the rest of their addition,
    // whichever is larger (D. Knuth, "The Art of Computer Programming", vol. 2, 4.2.2).
    __device__ __forceinline__ float warp() const
    {
        float s = sum, rest = -over;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float b = __shfl_xor_sync(~0u, s, o), t = __fadd_rn(s, b), from_b = __fsub_rn(t, s);
            const float lost = __fadd_rn(__fsub_rn(s, __fsub_rn(t, from_b)), __fsub_rn(b, from_b));
            rest = __fadd_rn(rest, __shfl_xor_sync(~0u, rest, o));
            rest = fabsf(t) < kInf ? __fadd_rn(rest, lost) : 0.0f;
            s = t;
        }
        return __fadd_rn(s, rest);
    }
};

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
template <int W>
__device__ __forceinline__ void weight_unit(const void *w, int dtype, bool aligned, const Place &p, f2 (&x)[W / 2])
{
    if (w && aligned && p.left >= W) {
#pragma unroll
        for (int i = 0; i < W / 8; ++i) {
            f2(&to)[4] = *reinterpret_cast<f2(*)[4]>(&x[4 * i]);
            if (dtype == FO_LOGITS_F32) {
                const float4 *const at = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.col) + 2 * i;
                const float4 a = __ldg(at), b = __ldg(at + 1);
                to[0] = pk(a.x, a.y);
                to[1] = pk(a.z, a.w);
                to[2] = pk(b.x, b.y);
                to[3] = pk(b.z, b.w);
            } else {
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + p.col) + i);
                if (dtype == FO_LOGITS_BF16)
                    widen_vec<Bf16>(a, to);
                else
                    widen_vec<F16>(a, to);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        x[i] = pk(2 * i < p.left ? weight_at(w, dtype, p.col + 2 * i) : 0.0f, 2 * i + 1 < p.left ? weight_at(w, dtype, p.col + 2 * i + 1) : 0.0f);
}

__device__ __forceinline__ float both(f2 v)
{
    float a, b;
    unpk(v, a, b);
    return __fadd_rn(a, b);
}

// A row is worked on by a team: kLanes threads of a warp, or (kLanes = 0) a whole
// CTA, of as many warps as the row fills, kWarps at most. The sum of v over the
// team, in every one of its threads. `part` holds a CTA's warps' sums, and zeros
// for the warps that it does not have; two sets in turn, so that one barrier a sum
// is enough.
template <int kLanes, int kWarps>
__device__ __forceinline__ float row_sum(float v, float *part)
{
#pragma unroll
    for (int o = (kLanes ? kLanes : 32) / 2; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    if constexpr (kLanes == 0) {
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x / 32] = v;
        __syncthreads();
        f2 sum = 0, other = 0;
#pragma unroll
        for (int i = 0; i < (kWarps + 3) / 4; ++i) {
            const ulonglong2 s = reinterpret_cast<const ulonglong2 *>(part)[i];
            sum = add2(sum, s.x);
            other = add2(other, s.y);
        }
        v = both(add2(sum, other));
    }
    return v;
}

// The place of unit u of row r; beyond the rows, and beyond the row's units, it is none.
template <int W>
__device__ __forceinline__ Place row_place(int r, int rows, int u, int units, int width)
{
    Place p;
    const bool there = r < rows && u < units;
    p.row = there ? r : -1;
    p.last = u + 1 >= units;
    p.col = u * W;
    p.left = there ? width - p.col : -64;
    return p;
}

// A unit at an address that moves on with the rows; where rows line up with no
// vector, registers are short, and it is computed from the place.
template <class T, bool kWide>
__device__ __forceinline__ Words<T, kUnitOf<kWide>> load(const RowsIn &x, const typename T::raw *at, const Place &p)
{
    if constexpr (kWide)
        return load_unit<T, kWide>(at, p);
    else
        return load_unit<T, kWide>(x, p);
}
template <class T, bool kWide, int kLanes>
__device__ __forceinline__ void store(const RowsOut &x, typename T::raw *at, const Place &p, const Words<T, kUnitOf<kWide>> &v)
{
    if constexpr (!kWide)
        at = static_cast<typename T::raw *>(x.data) + (int64_t)p.row * x.stride + p.col;
    store_unit<T, kWide, (kLanes ? kLanes : 32)>(at, p, v);
}

// --- rows held in registers --------------------------------------------------------------

// Each thread of a team has kVecs units of the row (a team apart) and their
// weights. A team takes rows a grid apart, the next one's loads on their way while
// one is worked on. kBlock: threads of a CTA at most, kCtas: on an SM at least.
template <class T, bool kWide, int kLanes, int kVecs, int kBlock, int kCtas>
__global__ void __launch_bounds__(kBlock, kCtas) norm_kernel(NormArgs a)
{
    typedef typename T::raw raw;
    constexpr int W = kUnitOf<kWide>, kWarps = kBlock / 32;
    __shared__ __align__(16) float part[4][32];
    for (int i = threadIdx.x; kLanes == 0 && i < 4 * 32; i += blockDim.x)
        part[i / 32][i % 32] = 0.0f;
    __syncthreads();
    const int lanes = kLanes ? kLanes : blockDim.x, teams = kLanes ? kBlock / (kLanes ? kLanes : 1) : 1;
    const int lane = kLanes ? threadIdx.x % lanes : threadIdx.x;
    const int units = (int)a.groups * (32 / W), rows = (int)a.rows, width = (int)a.width;
    const int step = gridDim.x * teams;
    int r = blockIdx.x * teams + (kLanes ? threadIdx.x / lanes : 0);
    Words<T, W> next[kVecs];
    f2 w[kVecs][W / 2];
    const raw *from = static_cast<const raw *>(a.x.data) + (int64_t)r * a.x.stride + lane * W;
    raw *to = static_cast<raw *>(a.y.data) + (int64_t)r * a.y.stride + lane * W;
    const auto fetch = [&](int row) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            next[k] = load<T, kWide>(a.x, from + k * lanes * W, row_place<W>(row, rows, lane + k * lanes, units, width));
        from += step * a.x.stride;
    };
    fetch(r);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        weight_unit<W>(a.weight, a.weight_dtype, a.weight_aligned, row_place<W>(0, 1, lane + k * lanes, units, width), w[k]);
    int turn = 0;
    // every thread takes as many turns as the CTA's first team: barriers and shuffles are all threads'
    for (int base = blockIdx.x * teams; base < rows; base += step, r += step, turn ^= 2) {
        // what needs no sum comes first, so that less waits for it
        f2 x[kVecs][W / 2];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int u = lane + k * lanes;
            widen_unit<T, W>(next[k], x[k]);
            if (a.kept.codes)
                keep_unit<T, W>(a.kept, (uint32_t)r * units + u, r < rows && u < units ? ~0u : 0u, next[k], x[k]);
        }
        fetch(r + step);
        const auto squares = [&](float scale) {
            f2 sum = 0;
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const f2 v = scale != 1.0f ? mul2(x[k][j], splat(scale)) : x[k][j];
                    sum = fma2(v, v, sum);
                }
            return both(sum);
        };
        const float sum = row_sum<kLanes, kWarps>(squares(1.0f), part[turn]);
        const bool large = !(sum < kLargeSum);
        float inv = inverse_rms(sum, a);
        if (kLanes ? __any_sync(~0u, large) : large) {   // the same in a CTA; other rows of a warp keep theirs
            const float down = inverse_rms_down(row_sum<kLanes, kWarps>(squares(kDown), part[turn + 1]), a);
            inv = large ? down : inv;
        }
        if (lane == 0 && a.inv_rms && r < rows)
            a.inv_rms[r] = inv;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
#pragma unroll
            for (int j = 0; j < W / 2; ++j)
                x[k][j] = mul2(mul2(x[k][j], splat(inv)), w[k][j]);
            store<T, kWide, kLanes>(a.y, to + k * lanes * W, row_place<W>(r, rows, lane + k * lanes, units, width), narrow_unit<T, W>(x[k]));
        }
        to += step * a.y.stride;
    }
}

// The same for the gradient; the weight's gradient of a thread's columns is added
// up in registers. A CTA's teams are joined in shared memory and leave one row of
// partial sums.
template <class T, bool kWide, int kLanes, int kVecs, int kBlock, int kCtas>
__global__ void __launch_bounds__(kBlock, kCtas) norm_grad_kernel(NormGradArgs a)
{
    typedef typename T::raw raw;
    constexpr int W = kUnitOf<kWide>, kTeams = kLanes ? kBlock / (kLanes ? kLanes : 1) : 1, kWarps = kBlock / 32;
    // h = x^ r with one rounding in FP32 (16384 x 4096 91 us, with two 103: a register less);
    // in 16-bit types with two, of which neither reaches the results' own (4096 x 16384
    // 115 us, with one 117).
    constexpr bool kOnce = kExactType<T>;
    __shared__ __align__(16) float part[2][32];
    for (int i = threadIdx.x; kLanes == 0 && i < 2 * 32; i += blockDim.x)
        part[i / 32][i % 32] = 0.0f;
    __syncthreads();
    __shared__ __align__(16) float joined[kTeams][kTeams > 1 ? kLanes * kVecs * W : 4];
    const int lanes = kLanes ? kLanes : blockDim.x;
    const int lane = kLanes ? threadIdx.x % lanes : threadIdx.x, team = kLanes ? threadIdx.x / lanes : 0;
    const int units = (int)a.groups * (32 / W), rows = (int)a.rows, width = (int)a.width;
    f2 w[kVecs][W / 2], dw[kVecs][W / 2];
    const int step = gridDim.x * kTeams;
    Words<T, W> next[kVecs];
    Kept<W> next_x[kVecs];
    float next_inv;
    int r = blockIdx.x * kTeams + team;
    const raw *from = static_cast<const raw *>(a.grad_y.data) + (int64_t)r * a.grad_y.stride + lane * W;
    raw *to = static_cast<raw *>(a.grad.data) + (int64_t)r * a.grad.stride + lane * W;
    const auto fetch = [&](int r) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int u = lane + k * lanes;
            const Place p = row_place<W>(r, rows, u, units, width);
            next[k] = load<T, kWide>(a.grad_y, from + k * lanes * W, p);
            next_x[k] = load_kept<W>(a.kept, (uint32_t)r * units + u, p.row < 0 ? 0u : ~0u);
        }
        next_inv = r < rows ? __ldg(a.inv_rms + r) : 0.0f;
        from += step * a.grad_y.stride;
    };
    fetch(r);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        weight_unit<W>(a.weight, a.weight_dtype, a.weight_aligned, row_place<W>(0, 1, lane + k * lanes, units, width), w[k]);
#pragma unroll
        for (int j = 0; j < W / 2; ++j)
            dw[k][j] = 0;
    }
    int turn = 0;
    for (int base = blockIdx.x * kTeams; base < rows; base += step, r += step, turn ^= 1) {
        f2 t[kVecs][W / 2], h[kVecs][W / 2], dot = 0;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            widen_unit<T, W>(next[k], t[k]);
            kept_unit<W, kOnce>(next_x[k], h[k], next_inv);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                dw[k][j] = fma2(t[k][j], h[k][j], dw[k][j]);
                t[k][j] = mul2(t[k][j], w[k][j]);
                dot = fma2(t[k][j], h[k][j], dot);
            }
        }
        const float inv = next_inv;
        fetch(r + step);
        if (a.grad.data) {
            const f2 mean = splat(-__fmul_rn(row_sum<kLanes, kWarps>(both(dot), part[turn]), a.inv_width));
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
#pragma unroll
                for (int j = 0; j < W / 2; ++j)
                    t[k][j] = mul2(fma2(h[k][j], mean, t[k][j]), splat(inv));
                store<T, kWide, kLanes>(a.grad, to + k * lanes * W, row_place<W>(r, rows, lane + k * lanes, units, width), narrow_unit<T, W>(t[k]));
            }
            to += step * a.grad.stride;
        }
    }
    if (!a.grad_weight)
        return;
    float *const sums = a.parts + (int64_t)blockIdx.x * a.groups * kGroup;
    if constexpr (kTeams > 1) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
            for (int j = 0; j < W / 2; ++j)
                *reinterpret_cast<f2 *>(&joined[team][(lane + k * lanes) * W + 2 * j]) = dw[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < units * W; c += kBlock) {
            LongSum sum;
#pragma unroll
            for (int i = 0; i < kTeams; ++i)
                sum.add(joined[i][c]);
            sums[c] = sum.sum;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int u = lane + k * lanes;
            if (u < units)
#pragma unroll
                for (int j = 0; j < W / 4; ++j)
                    reinterpret_cast<ulonglong2 *>(sums + u * W)[j] = make_ulonglong2(dw[k][2 * j], dw[k][2 * j + 1]);
        }
    }
}

// The parts of 32 columns by a CTA: 32 chains a column, joined pairwise, without what
// roundings lose: each part has been rounded in its CTA, one after another by as many
// rows as a thread takes (a 152th of them or fewer), and this adds one rounding to
// that. 304 parts of 4096 columns 3.2 us (by 256 threads a CTA 8.5; plain sums 2.9).
constexpr int kJoin = 32;
__global__ void __launch_bounds__(kJoin * 32) norm_weight_kernel(NormGradArgs a, int parts)
{
    __shared__ float part[2][kJoin][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane, pitch = a.groups * kGroup;
    LongSum sum;
#pragma unroll 8
    for (int p = warp; p < parts; p += kJoin)
        sum.add(a.parts[p * pitch + c]);
    part[0][warp][lane] = sum.sum;
    part[1][warp][lane] = sum.over;
    __syncthreads();
    sum.sum = part[0][lane][warp];   // column `warp`, its chains across the lanes
    sum.over = part[1][lane][warp];
    const float all = sum.warp();
    if (lane == 0 && (int64_t)blockIdx.x * 32 + warp < a.width)
        store_weight(a.grad_weight, a.weight_dtype, (int64_t)blockIdx.x * 32 + warp, all);
}

// --- rows beyond kMaxWidth --------------------------------------------------------------
//
// An element a thread and a row a CTA: the first, simple form. The forward pass reads
// x twice, the backward pass the codes and grad_y three times, the last time in a
// launch of its own by columns; what the L2 cache does not hold comes from device
// memory again. Bound by the loads that a thread waits for one after another: 4096 x
// 16640 BF16 172 us forward and 411 backward where the bytes take 102 together, one row
// of 131072, one CTA, 392 and 414.

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
    LongSum squares;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float x = load_at<T>(a.x, r, c);
        squares.add(x, x);
    }
    const float sum = block_sum(squares.sum, part);
    float inv = inverse_rms(sum, a);
    if (!(sum < kLargeSum)) {   // the same in the whole CTA
        squares = LongSum();
        for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
            const float x = __fmul_rn(load_at<T>(a.x, r, c), kDown);
            squares.add(x, x);
        }
        inv = inverse_rms_down(block_sum(squares.sum, part), a);
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
    LongSum dot;
    for (int64_t c = threadIdx.x; c < a.width; c += kThreads) {
        const float h = __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), inv);
        dot.add(__fmul_rn(load_at<T>(a.grad_y, r, c), weight_at(a.weight, a.weight_dtype, c)), h);
    }
    const float mean = block_sum(dot.sum, part) / (float)a.width;
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
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.groups * kGroup)
        return;
    LongSum sum;
    for (int64_t r = blockIdx.y; c < a.width && r < a.rows; r += gridDim.y)
        sum.add(load_at<T>(a.grad_y, r, c), __fmul_rn(kept_at(a.kept, r * a.groups + c / kGroup, (int)(c % kGroup)), a.inv_rms[r]));
    a.parts[blockIdx.y * a.groups * kGroup + c] = sum.sum;
}


constexpr int64_t kMaxWidth = 16384;   // of a row in registers

// CTAs of `block` threads that an SM holds at once, by the launch bounds.
constexpr int64_t ctas_per_sm(int block, int most, int ctas) { return most * ctas / block; }

// A grid of as many CTAs as the device holds at once, or as the rows need.
template <class T, bool kWide, int kLanes, int kVecs, int kBlock, int kCtas>
int run(const NormArgs &a, int block, cudaStream_t stream)
{
    const int64_t teams = kLanes ? block / (kLanes ? kLanes : 1) : 1;
    const int64_t ctas = std::min((a.rows + teams - 1) / teams, sm_count() * ctas_per_sm(block, kBlock, kCtas));
    norm_kernel<T, kWide, kLanes, kVecs, kBlock, kCtas><<<(unsigned)ctas, block, 0, stream>>>(a);
    count_launch();
    return (int)ctas;
}
template <class T, bool kWide, int kLanes, int kVecs, int kBlock, int kCtas>
int run(const NormGradArgs &a, int block, cudaStream_t stream)
{
    const int64_t teams = kLanes ? block / (kLanes ? kLanes : 1) : 1;
    const int64_t fit = std::min(norm_parts(a.rows, a.groups), sm_count() * ctas_per_sm(block, kBlock, kCtas));
    const int64_t ctas = std::min((a.rows + teams - 1) / teams, fit);
    norm_grad_kernel<T, kWide, kLanes, kVecs, kBlock, kCtas><<<(unsigned)ctas, block, 0, stream>>>(a);
    count_launch();
    return (int)ctas;
}

// Teams of a warp's lanes, kVecs units each.
template <class T, bool kWide, int kVecs, int kCtas, class A>
int by_lanes(const A &a, int64_t units, cudaStream_t stream)
{
    if (units <= 4 * kVecs)
        return run<T, kWide, 4, kVecs, kThreads, kCtas>(a, kThreads, stream);
    if (units <= 8 * kVecs)
        return run<T, kWide, 8, kVecs, kThreads, kCtas>(a, kThreads, stream);
    if (units <= 16 * kVecs)
        return run<T, kWide, 16, kVecs, kThreads, kCtas>(a, kThreads, stream);
    return run<T, kWide, 32, kVecs, kThreads, kCtas>(a, kThreads, stream);
}
inline int block_for(int64_t units, int vecs) { return (int)((units + 32 * vecs - 1) / (32 * vecs)) * 32; }

// Registers of a thread hold 32 bytes of a row and as much of the next one. In us
// (forward), 16384 x 4096: BF16 with one unit of 8 a thread 65, two 57, four 71
// (spills); FP32 99 with one, 108 with two. 131072 x 128 BF16 18.2 with one, 17.3
// with two.
template <class T, bool kWide>
int by_size(const NormArgs &a, cudaStream_t stream)
{
    const int64_t units = a.groups * (32 / kUnitOf<kWide>);
    constexpr int k = kWide && sizeof(typename T::raw) == 2 ? 2 : 1;
    if (units <= 32 * k)
        return by_lanes<T, kWide, k, 4>(a, units, stream);
    const int block = block_for(units, k);
    if (block <= 512)
        return run<T, kWide, 0, k, 512, 2>(a, block, stream);
    if constexpr (kWide)
        if (block > 1024)
            return run<T, kWide, 0, 2, 1024, 1>(a, block_for(units, 2), stream);
    return run<T, kWide, 0, k, 1024, 1>(a, block, stream);
}

// The gradient: a warp with two units a thread where they hold the row, one unit a
// thread of more warps beyond (65536 x 512 FP32 49 us, by 64 threads 61; 65536 x
// 768 BF16 by 64 threads 59, by 128 56; 16384 x 4096 BF16 64.6 and 63.6; 4096 x
// 16384 BF16 by 512 threads of four units 125, by 1024 of two 96). Two CTAs of 544
// or 576 threads fit an SM at 56 registers; up to 512 threads have 64, without which
// 16384 x 4096 takes 65 us instead of 57.
template <class T, bool kWide>
int by_size(const NormGradArgs &a, cudaStream_t stream)
{
    const int64_t units = a.groups * (32 / kUnitOf<kWide>);
    constexpr int k = kWide ? 2 : 1;
    if (units <= 32 * k)
        return by_lanes<T, kWide, k, 2>(a, units, stream);
    const int block = block_for(units, 1);
    if constexpr (!kWide) {
        if (block <= 576)
            return run<T, kWide, 0, 1, 576, 1>(a, block, stream);
    } else if (block <= 512)
        return run<T, kWide, 0, 1, 512, 2>(a, block, stream);
    else if (block <= 576)
        return run<T, kWide, 0, 1, 576, 2>(a, block, stream);
    if constexpr (kWide)
        if (block > 1024)
            return run<T, kWide, 0, 2, 1024, 1>(a, block_for(units, 2), stream);
    return run<T, kWide, 0, 1, 1024, 1>(a, block, stream);
}

template <class T>
cudaError_t launch(NormArgs a, cudaStream_t stream)
{
    a.inv_width = (float)(1.0 / (double)a.width);
    a.weight_aligned = (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
    if (a.width <= kMaxWidth) {
        wide<T>(a.width, a.x.data, a.x.stride) && wide<T>(a.width, a.y.data, a.y.stride) ? by_size<T, true>(a, stream) : by_size<T, false>(a, stream);
        return cudaGetLastError();
    }
    norm_long_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <class T>
cudaError_t launch(NormGradArgs a, cudaStream_t stream)
{
    a.inv_width = (float)(1.0 / (double)a.width);
    a.weight_aligned = (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
    int parts = 0;
    if (a.rows > 0 && a.width <= kMaxWidth)
        parts = wide<T>(a.width, a.grad_y.data, a.grad_y.stride) && wide<T>(a.width, a.grad.data, a.grad.stride) ? by_size<T, true>(a, stream)
                                                                                                                 : by_size<T, false>(a, stream);
    else if (a.rows > 0) {
        if (a.grad.data) {
            norm_long_grad_kernel<T><<<(unsigned)a.rows, kThreads, 0, stream>>>(a);
            count_launch();
        }
        if (a.grad_weight) {
            parts = (int)norm_parts(a.rows, a.groups);
            norm_long_weight_kernel<T><<<dim3((unsigned)((a.groups * kGroup + kThreads - 1) / kThreads), (unsigned)parts), kThreads, 0, stream>>>(a);
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
