// fo_loss.cuh -- device helpers shared by the loss operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fo_loss.h"

namespace fo {

// Element types by fo_logit_dtype_t.
struct Bf16 {
    typedef uint16_t raw;
    static constexpr float kShift = 0x1p24f;   // see grad_exp
    static __device__ __forceinline__ float widen(raw v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ raw narrow(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};
struct F16 {
    typedef uint16_t raw;
    static constexpr float kShift = 0x1p24f;
    static __device__ __forceinline__ float widen(raw v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ raw narrow(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
struct F32 {
    typedef float raw;
    static constexpr float kShift = 1.0f;
    static __device__ __forceinline__ float widen(raw v) { return v; }
    static __device__ __forceinline__ raw narrow(float f) { return f; }
};

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int64_t row_offset(const LogitRows &x, int64_t r, int64_t row_stride, int64_t outer_stride)
{
    if (x.inner_rows >= x.rows)
        return r * row_stride;
    const int64_t o = r / x.inner_rows;
    return o * outer_stride + (r - o * x.inner_rows) * row_stride;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// d = x - m, held where 2^(d c) is 0 but d c and its products are finite.
__device__ __forceinline__ float distance(float x, float m, const LogitRows &in) { return max_nan(__fsub_rn(x, m), in.d_min); }

// T::kShift 2^(d c), for a gradient, with t = d c. A gradient of 16 bits takes
// the exponential 24 powers of two higher, so that probabilities down to
// FP32's smallest subnormal are kept at no cost (the factor that it is
// multiplied with is 2^-24 of itself). One of 32 bits adds the first-order
// effect of what the rounding of t left, 3 roundings of t being 1e-5 of a
// probability of 1e-27.
template <class T>
__device__ __forceinline__ float grad_exp(float d, const LogitRows &in, float &t)
{
    t = __fmul_rn(d, in.c);
    if (sizeof(typename T::raw) == 2)
        return exp2_approx(__fmaf_rn(d, in.c, 24.0f));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    const float r = __fmaf_rn(d, in.c_lo, __fmaf_rn(d, in.c, -t));
    return __fmaf_rn(e, __fmul_rn(r, kLn2), e);
}

// A 32-bit key that orders as the logits do: -0 equals +0, NaN is the largest.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (v != v)
        return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The same with the id below it: larger keys come first, no two are equal.
__device__ __forceinline__ uint64_t entry_key(float v, uint32_t id) { return ((uint64_t)order_key(v) << 32) | (0xffffffffu - id); }
__device__ __forceinline__ uint32_t entry_id(uint64_t key) { return 0xffffffffu - (uint32_t)key; }

// The maximum to subtract: 0 for a row that is all -inf, so that x - m is
// -inf and not NaN.
__device__ __forceinline__ float safe_max(float m) { return m == -kInf ? 0.0f : m; }

// log p of a logit, given m, Z and ln Z; -inf in a row without a distribution.
// In double, for the few entries of a row that need it: beside a logit of the
// type's lowest value the difference may lie outside FP32 although what it is
// weighted with brings it back.
__device__ __forceinline__ double log_prob(float x, float m, float z, float ln_z, float inv_t)
{
    return z == 0.0f ? -(double)kInf : ((double)x - (double)safe_max(m)) * (double)inv_t - (double)ln_z;
}

__device__ __forceinline__ float load_dtype(const void *p, int64_t i, int dtype)
{
    if (dtype == 1)
        return static_cast<const float *>(p)[i];
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    return dtype == 0 ? Bf16::widen(v) : F16::widen(v);
}

}  // namespace fo
