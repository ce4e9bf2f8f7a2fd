// fo_act.cuh -- device helpers of the operators on activations: the 8-bit code
// of a group of 32 elements, and the activation functions.
//
// Code: with a = max |x| of the group,
//   step = the smallest BF16 number that is at least max(a / 127, 2^-126),
//   code = rint(x r), r = RN(1 / step), the product not rounded before;
//   x^ = code * step, exact in FP32 (7 bits by 8).
// A step is never 0, so that no division by it needs a guard, and one rounded
// up never lets a code leave -127..127. NaN or an infinity in a group makes its
// step NaN, and with it all that the group decodes to.
#pragma once

#include <cstdint>

#include "fo_act.h"
#include "fo_loss.cuh"

namespace fo {

// The bits of |x| of a value in FP32, as an unsigned number: it orders as |x|
// does, infinity and NaN above everything finite.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The step of a group whose largest magnitude has these bits. a times RN(1/127)
// is within a rounding and a half of a / 127: cut to BF16 it is at most two
// BF16 numbers short of the smallest s with 127 s >= a, a product that is exact.
__device__ __forceinline__ float step_of(uint32_t magnitude_bits)
{
    if (magnitude_bits >= 0x7f800000u)
        return kNan;
    const float a = __uint_as_float(magnitude_bits);
    uint32_t s = __float_as_uint(fmaxf(__fmul_rn(a, 0x1.020408p-7f), 0x1p-126f)) & 0xffff0000u;
    s += __fmul_rn(127.0f, __uint_as_float(s)) < a ? 0x10000u : 0u;
    s += __fmul_rn(127.0f, __uint_as_float(s)) < a ? 0x10000u : 0u;
    return __uint_as_float(s);
}

__device__ __forceinline__ uint16_t step_bits(float step) { return (uint16_t)(__float_as_uint(step) >> 16); }
__device__ __forceinline__ float step_value(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }

// In the sum of x r and 1.5 2^23 the last place is 1: the one rounding of the
// fused operation is rint(x r), whose lowest byte is the code.
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ uint32_t code_word(float x, float r) { return __float_as_uint(__fmaf_rn(x, r, kRound)); }

// --- activation functions --------------------------------------------------------------

enum : int { kSilu = 0, kGelu = 1 };

// f(x) and, with kSlope, its derivative. kExact: for FP32, whose results keep
// what 16-bit ones lose in their own rounding: the exponential's argument in two
// parts, the reciprocal with a step of Newton's.
struct Curve {
    float value, slope;
};

// e^-(u v), u v >= 0
template <bool kExact>
__device__ __forceinline__ float exp_minus(float u, float v)
{
    constexpr float kHigh = 1.44269504088896341f, kLow = (float)(1.44269504088896341 - (double)1.44269504088896341f);
    const float p = __fmul_rn(u, v), t = __fmul_rn(-p, kHigh);
    if (!kExact)
        return exp2_approx(t);
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    // t, p and kHigh as they were rounded, to first order
    const float rest = __fmaf_rn(-__fmaf_rn(u, v, -p), kHigh, __fmaf_rn(-p, kLow, __fmaf_rn(-p, kHigh, -t)));
    return __fmaf_rn(e, __fmul_rn(rest, kLn2), e);
}

template <bool kExact>
__device__ __forceinline__ float reciprocal(float x)
{
    const float y = rcp_approx(x);
    return kExact ? __fmaf_rn(y, __fmaf_rn(-x, y, 1.0f), y) : y;
}

// silu(x) = x s with s = 1 / (1 + e^-x), silu'(x) = s (1 + x (1 - s)). From
// e = e^-|x|, both s and 1 - s are quotients without cancellation. Below -120
// everything is 0 in FP32, and so is the limit at -inf.
template <bool kExact, bool kSlope>
__device__ __forceinline__ Curve silu(float x)
{
    x = max_nan(x, -120.0f);
    const float e = exp_minus<kExact>(fminf(fabsf(x), 200.0f), 1.0f);
    const float big = reciprocal<kExact>(__fadd_rn(1.0f, e)), small = __fmul_rn(e, big);
    const float s = x >= 0.0f ? big : small, rest = x >= 0.0f ? small : big;
    Curve c;
    c.value = __fmul_rn(x, s);
    c.slope = kSlope ? __fmul_rn(s, __fmaf_rn(x, rest, 1.0f)) : 0.0f;
    return c;
}

// gelu(x) = x Phi(x), gelu'(x) = Phi(x) + x phi(x). The normal distribution's
// tail Phi(-u) is Q(1 / (1 + 0.3 u)) e^(-u^2 / 2), Q the polynomial of degree 8
// with the least relative error on u in [0, 15] (5.8e-8; 3.6e-7 as evaluated in
// FP32), so that far on the negative side the result keeps its relative
// precision, which 1 + erf(x / sqrt 2) loses. Beyond 15 the tail is 0 in FP32.
template <bool kExact, bool kSlope>
__device__ __forceinline__ Curve gelu(float x)
{
    x = max_nan(x, -15.0f);
    const float u = fminf(fabsf(x), 15.0f);
    const float e = exp_minus<kExact>(u, 0.5f * u), t = reciprocal<kExact>(__fmaf_rn(0.3f, u, 1.0f));
    float q = 0x1.3ac79cp-5f;
    q = __fmaf_rn(q, t, -0x1.5aeb4cp-3f);
    q = __fmaf_rn(q, t, 0x1.d54246p-3f);
    q = __fmaf_rn(q, t, -0x1.3b91b6p-4f);
    q = __fmaf_rn(q, t, 0x1.24ab96p-3f);
    q = __fmaf_rn(q, t, 0x1.832e2ap-4f);
    q = __fmaf_rn(q, t, 0x1.f38cbcp-4f);
    q = __fmaf_rn(q, t, 0x1.e96612p-4f);
    q = __fmaf_rn(q, t, 0x1.f6f9aap-18f);
    const float tail = __fmul_rn(q, e), cdf = x >= 0.0f ? __fsub_rn(1.0f, tail) : tail;
    Curve c;
    c.value = __fmul_rn(x, cdf);
    // x phi(x) with |x| held at 15 as in e; NaN stays NaN
    c.slope = kSlope ? __fmaf_rn(__fmul_rn(x > 15.0f ? 15.0f : x, 0.398942280401432678f), e, cdf) : 0.0f;
    return c;
}

template <int kKind, bool kExact, bool kSlope>
__device__ __forceinline__ Curve curve(float x)
{
    return kKind == kSilu ? silu<kExact, kSlope>(x) : gelu<kExact, kSlope>(x);
}

template <class T>
constexpr bool kExactType = sizeof(typename T::raw) == 4;

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

}  // namespace fo
