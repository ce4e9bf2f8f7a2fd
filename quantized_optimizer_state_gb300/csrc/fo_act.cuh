// fo_act.cuh -- device helpers of the operators on activations: the 8-bit code
// of a group of 32 elements, and the activation functions.
//
// Code: with a = max |x| of the group,
//   step = the smallest BF16 number that is at least max(a / 127, 2^-126),
//   code = rint(x r), r = RN(1 / step), the product not rounded before;
//   x^ = code * step, exact in FP32 (7 bits by 8).
// A step is never 0, so that no division by it needs a guard, and one rounded
// up never lets a code leave -127..127. NaN or an infinity in a group makes its
// step NaN, and with it all that the group decodes to. Rounded up, 127 steps may
// be more than a 16-bit type's largest number where the group's largest is near it
// (see last_number). They stay within FP32: that of its largest number is
// (1 + 2^-6) 2^121, which goes into it 126 times, and the next smaller step 127 times.
#pragma once

#include <cstdint>

#include "fo_act.h"
#include "fo_loss.cuh"

namespace fo {

// The step of a group whose largest magnitude a has these bits. kBelow is less
// than 1 / 127 by 3 roundings, so that t = RN(a kBelow) is below a / 127, but
// by less than 2^-21 of it. Cut to BF16, t is then the largest BF16 number below
// a / 127, and the next one is the step: also where a / 127 is a BF16 number
// itself. Only where it lies above one by less than 2^-21, which the 8 or 11 bits
// of a BF16 or FP16 value do not reach, is that one short: 127 s, which is
// exact, says so. An infinity's t becomes NaN by the last addition; that of NaN
// runs over, and is taken back.
template <bool kFewBits>
__device__ __forceinline__ float step_of(uint32_t magnitude_bits)
{
    constexpr float kBelow = 0x1.020402p-7f;
    const float a = __uint_as_float(magnitude_bits);
    const uint32_t t = max(__float_as_uint(__fmul_rn(a, kBelow)), 0x007fffffu);   // at least just below 2^-126
    uint32_t s = min((t & 0xffff0000u) + 0x10000u, 0x7fc00000u);
    if (!kFewBits && __fmul_rn(127.0f, __uint_as_float(s)) < a)
        s += 0x10000u;
    return __uint_as_float(s);
}

__device__ __forceinline__ uint16_t step_bits(float step) { return (uint16_t)(__float_as_uint(step) >> 16); }
__device__ __forceinline__ float step_value(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }

// In the sum of x r and 1.5 2^23 the last place is 1: the one rounding of the
// fused operation is rint(x r), whose lowest byte is the code.
constexpr float kRound = 12582912.0f;

// --- activation functions --------------------------------------------------------------

enum : int { kSilu = 0, kGelu = 1 };

// Both functions are, with u = |x|,
//   f(x) = max(x, 0) - u q(u),   f'(x) = v(u) for x < 0, 1 - v(u) else
//   silu: q = e / (1 + e), e = e^-u;         v = q (1 - u / (1 + e))
//   gelu: q = the normal tail Phi(-u) = Q(1 / (1 + 0.3 u)) e^(-u^2 / 2), Q a
//         polynomial;                        v = q - u phi(u)
// so that far on the negative side results keep their relative precision, which
// 1 - s and 1 + erf lose, as long as they are normal numbers, and the limit at -inf is
// 0. u is held at 120 (15), beyond which u q and v are 0 in FP32. The hardware's
// exponential gives 0 below 2^-126, from u = 87.3 on, where u e^-u is a normal number
// up to 92: 16-bit silu takes it 2^24 larger. gelu's values are below 2^-127 where its
// exponential is, and its slope 0 from 13.2 on instead of 5 2^-126 and less: there it
// stays as it is (shifted, geglu 8192 x 14336 BF16 forward took 163 us instead of 145:
// two registers more). Pairs of values: two operations an
// instruction. Below, q and v are formed with their signs turned, which saves
// negations.
// kExact is for FP32, whose results keep what 16-bit ones lose in their own
// rounding: the exponential's argument in two parts, the reciprocal with a step of
// Newton's, and Q of degree 8 instead of 6. Q has the least relative error for u
// in [0, 15]: 5.8e-8 and 1.9e-6, as evaluated in FP32 3.7e-7 and 2.2e-6.
struct Curve {
    f2 value, slope;
};

constexpr float kLog2E = 1.44269504088896341f;

// e^-(u v), u v >= 0, for FP32
__device__ __forceinline__ f2 exp_minus(f2 u, f2 v)
{
    constexpr float kLow = (float)(1.44269504088896341 - (double)kLog2E);
    const f2 p = mul2(u, v), t = mul2(p, splat(-kLog2E));
    float a, b;
    unpk(t, a, b);
    asm("ex2.approx.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.f32 %0, %0;" : "+f"(b));
    // t, p and kLog2E as they were rounded, to first order
    const f2 e = pk(a, b), minus = splat(-1.0f), np = mul2(p, minus), lost = fma2(u, v, np);
    const f2 rest = fma2(lost, splat(-kLog2E), fma2(np, splat(kLow), fma2(np, splat(kLog2E), mul2(t, minus))));
    return fma2(e, mul2(rest, splat(kLn2)), e);
}

// 2^(p c), p c <= 0, for 16-bit types. exp2_approx gives 0 for what is below 2^-126;
// kBelow: it takes 2^24 times the result, and the product keeps what is below.
template <bool kBelow>
__device__ __forceinline__ f2 exp2_short(f2 p, float c)
{
    float a, b;
    unpk(kBelow ? fma2(p, splat(c), splat(24.0f)) : mul2(p, splat(c)), a, b);
    const f2 e = pk(exp2_approx(a), exp2_approx(b));
    return kBelow ? mul2(e, splat(0x1p-24f)) : e;
}

template <bool kExact>
__device__ __forceinline__ f2 reciprocal(f2 x)
{
    float a, b;
    unpk(x, a, b);
    const f2 y = pk(rcp_approx(a), rcp_approx(b));
    return kExact ? fma2(y, fma2(mul2(x, splat(-1.0f)), y, splat(1.0f)), y) : y;
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <int kKind, bool kExact>
__device__ __forceinline__ Curve curve(f2 x)
{
    constexpr float kFar = kKind == kSilu ? 120.0f : 15.0f;
    float a, b;
    unpk(x, a, b);
    const f2 u = pk(min_nan(fabsf(a), kFar), min_nan(fabsf(b), kFar));
    f2 nq, nv;   // -q and -v
    if (kKind == kSilu) {
        const f2 e = kExact ? exp_minus(u, splat(1.0f)) : exp2_short<true>(u, -kLog2E);
        const f2 n = reciprocal<kExact>(fma2(e, splat(-1.0f), splat(-1.0f)));   // -1 / (1 + e)
        nq = mul2(e, n);
        nv = mul2(nq, fma2(u, n, splat(1.0f)));
    } else {
        const f2 e = kExact ? exp_minus(u, mul2(u, splat(0.5f))) : exp2_short<false>(mul2(u, u), -0.5f * kLog2E), t = reciprocal<kExact>(fma2(u, splat(0.3f), splat(1.0f)));
        f2 q;
        const auto next = [&](float c) { q = fma2(q, t, splat(c)); };
        if (kExact) {
            q = splat(-0x1.3ac79cp-5f);
            next(0x1.5aeb4cp-3f);
            next(-0x1.d54246p-3f);
            next(0x1.3b91b6p-4f);
            next(-0x1.24ab96p-3f);
            next(-0x1.832e2ap-4f);
            next(-0x1.f38cbcp-4f);
            next(-0x1.e96612p-4f);
            next(-0x1.f6f9aap-18f);
        } else {
            q = splat(0x1.5a7e80p-4f);
            next(-0x1.ecb18ep-3f);
            next(0x1.8e7f86p-5f);
            next(-0x1.517030p-3f);
            next(-0x1.b50fb0p-4f);
            next(-0x1.f0bdc4p-4f);
            next(0x1.4eab20p-14f);
        }
        nq = mul2(q, e);
        nv = fma2(mul2(u, splat(0.398942280401432678f)), e, nq);
    }
    Curve c;
    c.value = fma2(u, nq, pk(fmaxf(a, 0.0f), fmaxf(b, 0.0f)));   // NaN by u
    // v where x has a sign, 1 - v where it has none
    const auto slope = [](float v, float x) {
        const uint32_t sign = __float_as_uint(x);
        const float one = __uint_as_float(~(uint32_t)((int32_t)sign >> 31) & 0x3f800000u);
        return __fadd_rn(one, __uint_as_float(__float_as_uint(v) ^ (sign & 0x80000000u)));
    };
    float p, q;
    unpk(nv, p, q);
    c.slope = pk(slope(p, a), slope(q, b));
    return c;
}

template <class T>
constexpr bool kExactType = sizeof(typename T::raw) == 4;

// --- units -----------------------------------------------------------------------------
//
// A thread works on units of W contiguous elements, neighbouring lanes on
// neighbouring units. Where rows line up with vectors of 16 bytes (kWide) W is 8,
// four lanes to a group: 16 bytes of a 16-bit type a lane and load, whole lines a
// warp. Elsewhere it is 16, two lanes to a group: what the shifting of vectors
// and their edges cost is for twice the elements. Units are numbered
// through the rows, 32 / W to a group, so that unit q has the codes from W q on.

template <bool kWide>
constexpr int kUnitOf = kWide ? 8 : 16;

// Division of numbers below 2^31 by a fixed one: n / d = (n m / 2^32 + n) / 2^shift
// (T. Granlund, P. Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994).
struct Divisor {
    uint32_t d, m, shift;
};
inline Divisor divisor(uint32_t d)
{
    Divisor r = {d, 0, 0};
    while (r.shift < 31 && (1u << r.shift) < d)
        ++r.shift;
    r.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << r.shift) - d)) / d + 1);
    return r;
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor &d) { return (__umulhi(n, d.m) + n) >> d.shift; }

// Where a unit lies. `left`: elements of the row from its first one on (0 or
// less beyond the row's end). Beyond the last row: row -1, and `left` far below 0.
struct Place {
    int row, col, left;
    bool last;   // of its row's units
};
template <int W>
__device__ __forceinline__ Place place(uint32_t unit, uint32_t units, const Divisor &per_row, int width)
{
    const uint32_t r = quotient(unit, per_row);
    Place p;
    p.row = unit < units ? (int)r : -1;
    p.last = unit - r * per_row.d + 1 == per_row.d;
    p.col = (int)((unit - r * per_row.d) * W);
    p.left = unit < units ? width - p.col : -64;
    return p;
}

// The 32-bit words of a unit, as they lie in memory.
template <class T, int W>
struct Words {
    static constexpr int kN = W * sizeof(typename T::raw) / 4;
    uint32_t w[kN];
};

// Whether every unit of a matrix lies wholly in its row and in aligned vectors of
// 16 bytes (kWide below; so it is where widths and strides are multiples of 8 and
// the matrix starts at such a boundary), or wholly beyond its width.
template <class T>
inline bool wide(int64_t width, const void *data, int64_t stride)
{
    return width % kUnitOf<true> == 0 && (reinterpret_cast<uintptr_t>(data) & 15) == 0 && stride * (int64_t)sizeof(typename T::raw) % 16 == 0;
}

// The words from element `from` on of a longer run of them; `from` < 8 of 16 bits
// or < 4 of 32. Three (two) steps, by the bits of `from`.
template <class T, int kIn, int kOut>
__device__ __forceinline__ void shifted(uint32_t (&in)[kIn], int from, uint32_t (&out)[kOut])
{
    constexpr bool kHalves = sizeof(typename T::raw) == 2;
    const int words = kHalves ? from >> 1 : from;
#pragma unroll
    for (int i = 0; i + 2 < kIn; ++i)
        in[i] = words & 2 ? in[i + 2] : in[i];
#pragma unroll
    for (int i = 0; i + 1 < kIn; ++i)
        in[i] = words & 1 ? in[i + 1] : in[i];
#pragma unroll
    for (int i = 0; i < kOut; ++i)
        out[i] = kHalves ? __funnelshift_r(in[i], in[i + 1 < kIn ? i + 1 : i], from & 1 ? 16 : 0) : in[i];
}

// n ones, for n below 32; none for n <= 0.
__device__ __forceinline__ uint32_t low_bits(int n) { return n > 0 ? ~(~0u << min(n, 31)) : 0u; }

template <class T>
__device__ __forceinline__ void load_vector(const uint4 *at, uint32_t *w)
{
    const uint4 a = __ldcs(at);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = a.z;
    w[3] = a.w;
}

// A unit; 0 beyond the row's end. No byte outside the row is read. Without kWide
// the row may start anywhere: the aligned vectors that hold the unit are read
// and shifted.
template <class T, bool kWide, int W = kUnitOf<kWide>>
__device__ __forceinline__ Words<T, W> load_unit(const typename T::raw *at, const Place &p)
{
    typedef typename T::raw raw;
    constexpr int kSize = sizeof(raw), kVecs = W * kSize / 16;
    Words<T, W> v;
#pragma unroll
    for (int i = 0; i < Words<T, W>::kN; ++i)
        v.w[i] = 0;
    if (kWide) {
        if (p.left > 0)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                load_vector<T>(reinterpret_cast<const uint4 *>(at) + i, v.w + 4 * i);
        return v;
    }
    const int phase = (int)((reinterpret_cast<uintptr_t>(at) & 15) / kSize);
    if (phase == 0 && p.left >= W) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            load_vector<T>(reinterpret_cast<const uint4 *>(at) + i, v.w + 4 * i);
    } else if (p.col >= phase && p.left + phase >= (kVecs + 1) * 16 / kSize) {
        uint32_t in[4 * (kVecs + 1)];
#pragma unroll
        for (int i = 0; i <= kVecs; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(at - phase) + i);
            in[4 * i] = a.x; in[4 * i + 1] = a.y; in[4 * i + 2] = a.z; in[4 * i + 3] = a.w;
        }
        shifted<T>(in, phase, v.w);
    } else {
        raw *e = reinterpret_cast<raw *>(v.w);
        const uint32_t there = low_bits(p.left);
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (there >> i & 1)
                e[i] = at[i];
    }
    return v;
}

template <class T, bool kWide>
__device__ __forceinline__ Words<T, kUnitOf<kWide>> load_unit(const RowsIn &x, const Place &p)
{
    return load_unit<T, kWide>(static_cast<const typename T::raw *>(x.data) + (int64_t)p.row * x.stride + p.col, p);
}

// Stores a unit. Without kWide by all lanes of a warp, whose units follow one
// another: a lane stores the aligned vectors that begin in the unit before its
// own and end in its own, with what that unit's lane hands over; what has no such
// lane goes element by element. Runs of kRun lanes have units that follow one another.
template <class T, bool kWide, int kRun = 32, int W = kUnitOf<kWide>>
__device__ __forceinline__ void store_unit(typename T::raw *at, const Place &p, const Words<T, W> &v)
{
    typedef typename T::raw raw;
    constexpr int kSize = sizeof(raw), kVecs = W * kSize / 16, kN = Words<T, W>::kN;
    if (kWide) {
        if (p.left > 0)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                __stcs(reinterpret_cast<uint4 *>(at) + i, make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]));
        return;
    }
    const int phase = (int)((reinterpret_cast<uintptr_t>(at) & 15) / kSize), lane = threadIdx.x % kRun;
    constexpr int kOver = kSize == 2 ? 4 : 3;   // words that a unit hands over at most
    uint32_t in[kOver + kN], out[kN];
#pragma unroll
    for (int i = 0; i < kOver; ++i)
        in[i] = __shfl_up_sync(~0u, v.w[kN - kOver + i], 1);
#pragma unroll
    for (int i = 0; i < kN; ++i)
        in[kOver + i] = out[i] = v.w[i];
    const bool before = lane > 0 && p.col > 0, after = lane < kRun - 1 && !p.last;
    int lo = 0, hi = p.left;             // places of `out`, from the vectors' first on, that are the row's
    if (phase) {
        shifted<T>(in, (kSize == 2 ? 8 : 3) - phase, out);
        lo = before ? 0 : phase;
        hi = p.left + phase;
        if (!after) {                    // the unit's last elements
            const raw *e = reinterpret_cast<const raw *>(v.w);
            const uint32_t there = low_bits(p.left) & ~low_bits(W - phase);
#pragma unroll
            for (int i = W - 16 / kSize + 1; i < W; ++i)
                if (there >> i & 1)
                    at[i] = e[i];
        }
    }
    raw *const to = at - phase;
    const raw *e = reinterpret_cast<const raw *>(out);
    constexpr int kPer = 16 / kSize;
    const uint32_t there = low_bits(hi) & ~low_bits(lo), all = (1u << kPer) - 1;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint32_t mine = there >> kPer * i & all;
        if (mine == all)
            __stcs(reinterpret_cast<uint4 *>(to) + i, make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]));
        else if (mine)
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (mine >> k & 1)
                    to[kPer * i + k] = e[kPer * i + k];
    }
}

template <class T, bool kWide, int W>
__device__ __forceinline__ void store_unit(const RowsOut &x, const Place &p, const Words<T, W> &v)
{
    store_unit<T, kWide>(static_cast<typename T::raw *>(x.data) + (int64_t)p.row * x.stride + p.col, p, v);
}

// A unit's values in pairs, and back, rounded once.
template <class T, int W>
__device__ __forceinline__ void widen_unit(const Words<T, W> &v, f2 (&x)[W / 2])
{
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        if constexpr (sizeof(typename T::raw) == 2)
            x[i] = T::widen2(v.w[i]);
        else
            x[i] = pk(__uint_as_float(v.w[2 * i]), __uint_as_float(v.w[2 * i + 1]));
}
template <class T, int W>
__device__ __forceinline__ Words<T, W> narrow_unit(const f2 (&x)[W / 2])
{
    Words<T, W> v;
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        if constexpr (sizeof(typename T::raw) == 2)
            v.w[i] = T::narrow2(x[i]);
        else {
            float a, b;
            unpk(x[i], a, b);
            v.w[2 * i] = __float_as_uint(a);
            v.w[2 * i + 1] = __float_as_uint(b);
        }
    return v;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The step of the group that this lane's unit and those of the 32 / W - 1 lanes
// beside it make up. As unsigned numbers the magnitudes of any of the types order
// as their values do, infinity and NaN on top: two 16-bit ones to a word.
template <class T, int W>
__device__ __forceinline__ float group_step(const Words<T, W> &v)
{
    constexpr bool kHalves = sizeof(typename T::raw) == 2;
    const auto most = [](uint32_t a, uint32_t b) { return kHalves ? max_u16x2(a, b) : max(a, b); };
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < Words<T, W>::kN; ++i)
        m = most(m, v.w[i] & (kHalves ? 0x7fff7fffu : 0x7fffffffu));
#pragma unroll
    for (int o = 1; o < 32 / W; o *= 2)
        m = most(m, __shfl_xor_sync(~0u, m, o));
    if constexpr (kHalves)
        m = __float_as_uint(T::widen((typename T::raw)max(m & 0xffffu, m >> 16)));
    return step_of<kHalves>(m);
}

// RN(1 / step): the hardware's approximation and a step of Newton's, which is
// the correctly rounded reciprocal of every FP32 number in [2^-100, 2^100]
// (enumerated by fo_verify_fast_arithmetic) and, steps and their reciprocals being
// normal numbers, of their multiples by powers of two.
__device__ __forceinline__ float step_reciprocal(float step)
{
    const float y = rcp_approx(step);
    return __fmaf_rn(y, __fmaf_rn(-step, y, 1.0f), y);
}

// The lowest bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of a unit, as one vector.
template <int W>
struct CodeVec {
    typedef uint2 type;
};
template <>
struct CodeVec<16> {
    typedef uint4 type;
};

// The codes and the step of unit `unit` of a matrix of `units` units.
template <class T, int W>
__device__ __forceinline__ void keep_unit(const KeptOut &k, uint32_t unit, uint32_t units, const Words<T, W> &v, const f2 (&x)[W / 2])
{
    const float step = group_step<T, W>(v);
    const f2 r = splat(step_reciprocal(step)), round = splat(kRound);
    uint32_t c[W];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        float a, b;
        unpk(fma2(x[i], r, round), a, b);
        c[2 * i] = __float_as_uint(a);
        c[2 * i + 1] = __float_as_uint(b);
    }
    if (unit < units) {
        typename CodeVec<W>::type codes;
        codes.x = low_bytes(c[0], c[1], c[2], c[3]);
        codes.y = low_bytes(c[4], c[5], c[6], c[7]);
        if constexpr (W == 16) {
            codes.z = low_bytes(c[8], c[9], c[10], c[11]);
            codes.w = low_bytes(c[12], c[13], c[14], c[15]);
        }
        // Without the streaming hint that the results have: a backward pass right after
        // its forward pass finds the last of them in the L2 cache (norm of 16384 x 4096
        // BF16 56 us; 64 with the hint, and with other layers between the two). What they
        // take of the cache from an operator that reads the results next was not measured.
        reinterpret_cast<typename CodeVec<W>::type *>(k.codes)[unit] = codes;
        if (unit % (32 / W) == 0)
            k.steps[unit / (32 / W)] = step_bits(step);
    }
}

// A unit's codes and step as loaded, and the values x^ they stand for. A code
// becomes the low byte of 2^23 + 128 + code, from which FP32 takes the rest away.
// `factor` is multiplied into the step first, or (kOnce) x^ by it, which rounds once
// and takes an instruction a pair more.
template <int W>
struct Kept {
    typename CodeVec<W>::type codes;
    uint16_t step;
};
template <int W>
__device__ __forceinline__ Kept<W> load_kept(const KeptIn &k, uint32_t unit, uint32_t units)
{
    Kept<W> v = {};
    if (unit < units) {
        v.codes = __ldcs(reinterpret_cast<const typename CodeVec<W>::type *>(k.codes) + unit);
        v.step = __ldg(k.steps + unit / (32 / W));
    }
    return v;
}
template <int W, bool kOnce = false>
__device__ __forceinline__ void kept_unit(const Kept<W> &v, f2 (&x)[W / 2], float factor = 1.0f)
{
    const f2 base = splat(-(8388608.0f + 128.0f)), step = splat(kOnce ? step_value(v.step) : __fmul_rn(step_value(v.step), factor));
    uint32_t words[W / 4] = {v.codes.x, v.codes.y};
    if constexpr (W == 16) {
        words[2] = v.codes.z;
        words[3] = v.codes.w;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        const uint32_t w = words[i / 2] ^ 0x80808080u;
        const f2 n = pk(__uint_as_float(__byte_perm(w, 0x4b000000u, i % 2 ? 0x7442 : 0x7440)),
                        __uint_as_float(__byte_perm(w, 0x4b000000u, i % 2 ? 0x7443 : 0x7441)));
        x[i] = mul2(add2(n, base), step);
        if (kOnce)
            x[i] = mul2(x[i], splat(factor));
    }
}

// x^ of a unit as numbers of type T: one beyond T's largest number becomes that
// number where it is less than a step beyond, so that the element itself may be a
// number of T (of codes made from T's numbers every one is); else infinity. A
// comparison a unit asks for it: 8192 x 14336 FP16 to codes and back 98 us with it
// and without.
template <class T, int W>
__device__ __forceinline__ void last_number(const Kept<W> &v, f2 (&x)[W / 2])
{
    const float step = step_value(v.step);
    if (!(__fmul_rn(127.0f, step) > T::kLargest))
        return;
    const auto stop = [&](float a) {
        const float over = __fsub_rn(fabsf(a), T::kLargest);   // exact where it matters: both are multiples of the step's last place
        return over > 0.0f && over <= step ? copysignf(T::kLargest, a) : a;
    };
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        float a, b;
        unpk(x[i], a, b);
        x[i] = pk(stop(a), stop(b));
    }
}

// The grid of a launch over all units, kUnits a thread.
struct UnitGrid {
    uint32_t units;
    Divisor per_row;
};
template <int W>
inline UnitGrid unit_grid(int64_t rows, int64_t groups)
{
    return UnitGrid{(uint32_t)(rows * groups * (32 / W)), divisor((uint32_t)(groups * (32 / W)))};
}

}  // namespace fo
