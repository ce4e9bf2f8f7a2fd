// fo_loss.cuh -- device helpers shared by the loss operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "fo_internal.h"
#include "fo_loss.h"
#include "fo_pair.cuh"

namespace fo {

// Element types by fo_logit_dtype_t. A vector is 16 bytes, kPerVec elements.
struct Bf16 {
    typedef uint16_t raw;
    static constexpr int kPerVec = 8;
    static constexpr float kShift = 0x1p24f;              // see grad_exp
    static constexpr uint32_t kKeyBits = 0xffff0000u;     // the part of an order key that differs between values
    static __device__ __forceinline__ float widen(raw v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ raw narrow(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
    static __device__ __forceinline__ f2 widen2(uint32_t w) { return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
    static __device__ __forceinline__ uint32_t narrow2(f2 v)
    {
        float lo, hi;
        unpk(v, lo, hi);
        uint32_t d;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // whether either element of a is greater than b's
    static __device__ __forceinline__ bool any_gt2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("{\n .reg .pred p, q;\n setp.gt.bf16x2 p|q, %1, %2;\n or.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(d) : "r"(a), "r"(b));
        return d != 0;
    }
    static __device__ __forceinline__ uint32_t twice(float f) { return (uint32_t)narrow(f) * 0x10001u; }
    static constexpr float kLargest = 0x1.fep127f;        // the largest finite value
    static __device__ __forceinline__ bool finite(float f) { return fabsf(f) < 0x1p126f; }
};
struct F16 {
    typedef uint16_t raw;
    static constexpr int kPerVec = 8;
    static constexpr float kShift = 0x1p24f;
    static constexpr uint32_t kKeyBits = 0xffffe000u;
    static __device__ __forceinline__ float widen(raw v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ raw narrow(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ f2 widen2(uint32_t w) { return pk(widen((raw)w), widen((raw)(w >> 16))); }
    static __device__ __forceinline__ uint32_t narrow2(f2 v)
    {
        float lo, hi;
        unpk(v, lo, hi);
        uint32_t d;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ bool any_gt2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("{\n .reg .pred p, q;\n setp.gt.f16x2 p|q, %1, %2;\n or.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(d) : "r"(a), "r"(b));
        return d != 0;
    }
    static __device__ __forceinline__ uint32_t twice(float f) { return (uint32_t)narrow(f) * 0x10001u; }
    static constexpr float kLargest = 65504.0f;
    static __device__ __forceinline__ bool finite(float f) { return fabsf(f) < 65000.0f; }
};
struct F32 {
    typedef float raw;
    static constexpr int kPerVec = 4;
    static constexpr float kShift = 1.0f;
    static constexpr uint32_t kKeyBits = 0xffffffffu;
    static __device__ __forceinline__ float widen(raw v) { return v; }
    static __device__ __forceinline__ raw narrow(float f) { return f; }
    static constexpr float kLargest = 0x1.fffffep127f;
    static __device__ __forceinline__ bool finite(float f) { return fabsf(f) < 0x1p126f; }
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

// The id of an entry's key: order_key above, the complement of the id below it.
__device__ __forceinline__ uint32_t entry_id(uint64_t key) { return 0xffffffffu - (uint32_t)key; }

// The maximum to subtract: 0 for a row that is all -inf, so that x - m is
// -inf and not NaN.
__device__ __forceinline__ float safe_max(float m) { return m == -kInf ? 0.0f : m; }

// (x - m) / 4, finite for any two finite logits: beside one of the type's
// lowest value the difference itself may lie outside FP32, although what it is
// weighted or divided by brings it back.
__device__ __forceinline__ float quarter_distance(float x, float m) { return __fsub_rn(0.25f * x, 0.25f * safe_max(m)); }

// log p of a logit, given m, Z and ln Z; -inf in a row without a distribution.
__device__ __forceinline__ float log_prob(float x, float m, float z, float ln_z, float inv_t)
{
    return z == 0.0f ? -kInf : __fmaf_rn(quarter_distance(x, m), 4.0f * inv_t, -ln_z);
}

// --- a row, in 16-byte vectors -------------------------------------------------

// The pairs of FP32 values of a vector, and back.
template <class T>
__device__ __forceinline__ void widen_vec(const uint4 &v, f2 (&x)[T::kPerVec / 2])
{
    x[0] = T::widen2(v.x);
    x[1] = T::widen2(v.y);
    x[2] = T::widen2(v.z);
    x[3] = T::widen2(v.w);
}
template <>
__device__ __forceinline__ void widen_vec<F32>(const uint4 &v, f2 (&x)[2])
{
    x[0] = pk(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = pk(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <class T>
__device__ __forceinline__ uint4 narrow_vec(const f2 (&x)[T::kPerVec / 2])
{
    return make_uint4(T::narrow2(x[0]), T::narrow2(x[1]), T::narrow2(x[2]), T::narrow2(x[3]));
}
template <>
__device__ __forceinline__ uint4 narrow_vec<F32>(const f2 (&x)[2])
{
    float a, b, c, d;
    unpk(x[0], a, b);
    unpk(x[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// The vector's elements raised to `floor_` where they are below it. NaN stays.
template <class T>
__device__ __forceinline__ uint4 raise(const uint4 &v, uint32_t floor_)
{
    return make_uint4(T::max2(v.x, floor_), T::max2(v.y, floor_), T::max2(v.z, floor_), T::max2(v.w, floor_));
}
template <class T>
__device__ __forceinline__ uint4 raise(const uint4 &v, float floor_)
{
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(v.x), floor_)), __float_as_uint(max_nan(__uint_as_float(v.y), floor_)),
                      __float_as_uint(max_nan(__uint_as_float(v.z), floor_)), __float_as_uint(max_nan(__uint_as_float(v.w), floor_)));
}

// A row lies in vectors counted from the 16-byte boundary at or before its
// first element, which is element `phase` of vector 0. The first and the last
// vector may reach beyond the row.
template <class T>
struct Row {
    typedef typename T::raw raw;
    const raw *x;      // the row
    int phase, vocab;
    int vecs;          // vectors that hold elements of the row
    int full0, full1;  // those wholly inside it: [full0, full1)

    __device__ __forceinline__ Row(const LogitRows &in, int64_t r)
        : x(static_cast<const raw *>(in.data) + row_offset(in, r, in.row_stride, in.outer_stride)), vocab((int)in.vocab)
    {
        phase = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(raw));
        vecs = (phase + vocab + T::kPerVec - 1) / T::kPerVec;
        full0 = phase ? 1 : 0;
        full1 = (phase + vocab) / T::kPerVec;
    }
    // The element that vector i holds at place e, as an id (outside [0, vocab) beyond the row's ends).
    __device__ __forceinline__ int id(int i, int e) const { return i * T::kPerVec + e - phase; }
    __device__ __forceinline__ const uint4 *vec(int i) const { return reinterpret_cast<const uint4 *>(x - phase) + i; }
};

// Vector i of a row; where it reaches beyond the row's ends, the row's elements
// one by one (no byte outside the row is read) and -inf beside them.
template <class T>
__device__ __forceinline__ uint4 load_vec(const Row<T> &row, int i)
{
    if (i >= row.full0 && i < row.full1)
        return __ldcs(row.vec(i));
    uint4 v;
    typename T::raw *e = reinterpret_cast<typename T::raw *>(&v);
#pragma unroll
    for (int k = 0; k < T::kPerVec; ++k) {
        const int id = row.id(i, k);
        e[k] = id >= 0 && id < row.vocab ? row.x[id] : T::narrow(-kInf);
    }
    return v;
}

// The elementwise largest of a vector's packed words (one word for the 16-bit
// types, whose two halves are kept apart; the value itself for FP32). NaN stays.
template <class T>
struct Largest {
    uint32_t w;
    static __device__ __forceinline__ Largest none() { return Largest{T::twice(-kInf)}; }
    static __device__ __forceinline__ Largest of(const uint4 &v) { return Largest{T::max2(T::max2(v.x, v.y), T::max2(v.z, v.w))}; }
    __device__ __forceinline__ Largest with(Largest o) const { return Largest{T::max2(w, o.w)}; }
    __device__ __forceinline__ bool above(uint32_t bound) const { return T::any_gt2(w, bound); }
    __device__ __forceinline__ float lo() const { return T::widen((typename T::raw)w); }
    __device__ __forceinline__ float hi() const { return T::widen((typename T::raw)(w >> 16)); }
    __device__ __forceinline__ float value() const { return fmaxf(lo(), hi()); }         // of what is not NaN
    __device__ __forceinline__ float value_nan() const { return max_nan(lo(), hi()); }   // NaN where there is one
    static __device__ __forceinline__ uint32_t bound(float f) { return T::twice(f); }
};
template <>
struct Largest<F32> {
    float w;
    static __device__ __forceinline__ Largest none() { return Largest{-kInf}; }
    static __device__ __forceinline__ Largest of(const uint4 &v)
    {
        return Largest{max_nan(max3_nan(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)), __uint_as_float(v.w))};
    }
    __device__ __forceinline__ Largest with(Largest o) const { return Largest{max_nan(w, o.w)}; }
    __device__ __forceinline__ bool above(float bound) const { return w > bound; }
    __device__ __forceinline__ float value() const { return w; }
    __device__ __forceinline__ float value_nan() const { return w; }
    static __device__ __forceinline__ float bound(float f) { return f; }
};

// Statistics of a set of logits: m a reference near their maximum (at most
// 2^32 below it in 2^((x-m)c)), z = sum 2^((x-m)c), w = sum 2^t t with
// t = (x-m)c (entropy; else unused). An empty set: {-inf, 0, 0}.
struct Stat {
    float m, z, w;
};

template <bool kEntropy>
__device__ __forceinline__ void rescale(Stat &s, float m, const LogitRows &in)
{
    const float t = __fmul_rn(max_nan(__fsub_rn(s.m, m), in.d_min), in.c);   // s.m = -inf: 2^-160, which is 0
    const float f = exp2_approx(t);
    if (kEntropy)
        s.w = __fmul_rn(__fmaf_rn(t, s.z, s.w), f);
    s.z = __fmul_rn(s.z, f);
    s.m = m;
}

// Over the first `n` lanes of a warp (a power of two), in every lane of them.
template <bool kEntropy>
__device__ __forceinline__ Stat warp_join(Stat s, const LogitRows &in, int n = 32)
{
    float m = s.m;
    for (int o = n / 2; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (m != -kInf)
        rescale<kEntropy>(s, m, in);
    for (int o = n / 2; o; o >>= 1) {
        s.z += __shfl_xor_sync(~0u, s.z, o);
        if (kEntropy)
            s.w += __shfl_xor_sync(~0u, s.w, o);
    }
    return s;
}

// Among the first kN threads of a CTA.
template <int kN>
__device__ __forceinline__ void barrier_among()
{
    asm volatile("bar.sync 1, %0;" ::"n"(kN) : "memory");
}

// Over the first kN threads of a CTA: the result in every one of them. `part`
// is shared memory of kN / 32 entries.
template <bool kEntropy, int kN>
__device__ __forceinline__ Stat block_join(Stat s, Stat *part, const LogitRows &in)
{
    s = warp_join<kEntropy>(s, in);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = s;
    barrier_among<kN>();
    return warp_join<kEntropy>(part[threadIdx.x % (kN / 32)], in, kN / 32);
}

// One thread's statistics while it walks over its vectors. An exponential
// costs one fused multiply-add, 2^(x c - M): M is the reference m times c,
// rounded, and the rounding is undone at the end. m follows the maximum
// loosely: it is moved where a vector reaches 16 powers of two above it, which
// after the first vector is rare, and saves the rescaling of most vectors.
// `careful` marks references beside which x c - M does not do: M of 2^24 and more,
// NaN among them (the rounding of M, up to half of its last place, is undone by
// 2^(M - m c), which must stay near 1: for a mask value of -1e9 at T = 0.1 that
// rounding may be 2^9, and the sums would be infinities and zeros), and, for the
// entropy, those next to the type's lowest value. Vectors are then taken element
// by element through x - m.
template <class T, bool kEntropy>
struct Running {
    float m, ref;                       // the reference and RN(m c)
    f2 z, w;
    Largest<T> top;                     // the largest seen; NaN stays
    decltype(Largest<T>::bound(0.0f)) limit, floor_;
    bool careful;

    __device__ __forceinline__ Running()
        : m(-kInf), ref(0.0f), z(0), w(0), top(Largest<T>::none()), limit(Largest<T>::bound(-kInf)), floor_(limit), careful(kEntropy)
    {
    }

    // Moves the reference up to the largest seen.
    __device__ __forceinline__ void move(const LogitRows &in)
    {
        const float to = top.value(), reach = __fmul_rn(-in.d_min, 1.02f);
        const float low = to - fmaxf(reach, fabsf(to) * 0x1p-6f);   // where 2^t is 0, at the type's precision
        const float r = __fmul_rn(to, in.c);
        const bool c = !(fabsf(r) < 0x1p24f) || (kEntropy && !T::finite(low));
        // From what the sums were taken beside to what they are taken beside
        // from here on: each is m c, rounded to `ref` where it is not careful.
        float t;
        if (careful)
            t = c ? __fmul_rn(to == m ? 0.0f : __fsub_rn(m, to), in.c) : __fmaf_rn(m, in.c, -r);
        else
            t = c ? __fmaf_rn(-to, in.c, ref) : __fsub_rn(ref, r);
        t = max_nan(t, -160.0f);
        const float f = m == -kInf ? 0.0f : exp2_approx(t);
        if (kEntropy)
            w = mul2(fma2(splat(t), z, w), splat(f));
        z = mul2(z, splat(f));
        m = to;
        ref = r;
        careful = c;
        // -d_min c = 160; +inf is above every limit, so that it becomes the reference
        limit = Largest<T>::bound(c ? to : fminf(__fmaf_rn(-in.d_min, 0.1f, to), T::kLargest));
        floor_ = Largest<T>::bound(low);
    }

    // Vectors at a time: one look at the reference for all, and their sum is
    // formed first, so that the chains of additions into z and w stay short.
    template <int N>
    __device__ __forceinline__ void add(const uint4 (&v)[N], const LogitRows &in)
    {
        Largest<T> most = Largest<T>::of(v[0]);
#pragma unroll
        for (int j = 1; j < N; ++j)
            most = most.with(Largest<T>::of(v[j]));
        top = top.with(most);
        if (most.above(limit))
            move(in);
        constexpr int kPairs = T::kPerVec / 2;
        f2 sums[N], weighted = 0;
        const f2 c = splat(in.c), r = splat(-ref);
        const float at = safe_max(m);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            f2 x[kPairs], e[kPairs];
            float a, b;
            if (!careful) {
                if (kEntropy)
                    widen_vec<T>(raise<T>(v[j], floor_), x);
                else
                    widen_vec<T>(v[j], x);
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    x[i] = fma2(x[i], c, r);
            } else {
                widen_vec<T>(v[j], x);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    unpk(x[i], a, b);
                    x[i] = pk(__fmul_rn(distance(a, at, in), in.c), __fmul_rn(distance(b, at, in), in.c));
                }
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                unpk(x[i], a, b);
                e[i] = pk(exp2_approx(a), exp2_approx(b));
                if (kEntropy)
                    weighted = fma2(e[i], x[i], weighted);
            }
#pragma unroll
            for (int n = kPairs / 2; n; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i)
                    e[i] = add2(e[i], e[i + n]);
            sums[j] = e[0];
        }
#pragma unroll
        for (int n = N / 2; n; n >>= 1)
#pragma unroll
            for (int j = 0; j < n; ++j)
                sums[j] = add2(sums[j], sums[j + n]);
        z = add2(z, sums[0]);
        if (kEntropy)
            w = add2(w, weighted);
    }

    __device__ __forceinline__ void add(const uint4 &v, const LogitRows &in)
    {
        const uint4 one[1] = {v};
        add(one, in);
    }

    __device__ __forceinline__ Stat stat(const LogitRows &in) const
    {
        float a, b;
        unpk(z, a, b);
        Stat s = {m, __fadd_rn(a, b), 0.0f};
        unpk(w, a, b);
        if (kEntropy)
            s.w = __fadd_rn(a, b);
        if (!careful && m != -kInf) {   // from 2^ref to 2^(m c)
            const float d = __fmaf_rn(m, in.c, -ref), f = exp2_approx(-d);
            if (kEntropy)
                s.w = __fmul_rn(__fmaf_rn(-d, s.z, s.w), f);
            s.z = __fmul_rn(s.z, f);
        }
        return s;
    }
};

// --- clusters, and a ring of bulk copies --------------------------------------------

__device__ __forceinline__ uint32_t shared_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of `p`, of this CTA's shared memory, in that of another CTA of the cluster.
__device__ __forceinline__ uint32_t map_shared(const void *p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(shared_address(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t a)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// This CTA's vectors of a row: [v0, v0 + n).
struct Part {
    int v0, n;
};
template <class T>
__device__ __forceinline__ Part part_of(const Row<T> &row, uint32_t rank, uint32_t size)
{
    const int per = (row.vecs + (int)size - 1) / (int)size;
    const int v0 = min((int)rank * per, row.vecs);
    return Part{v0, min(per, row.vecs - v0)};
}

// mbarriers. A wait is bounded (each try sleeps in the hardware for a while):
// something that never comes gives false, not a hang.
__device__ __forceinline__ void barrier_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_address(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_address(bar)) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_address(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_wait(uint64_t *bar, uint32_t parity)
{
    for (int i = 0; i < 1 << 20; ++i) {
        uint32_t done;
        asm volatile("{\n .reg .pred p;\n"
                     " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done)
                     : "r"(shared_address(bar)), "r"(parity)
                     : "memory");
        if (done)
            return true;
    }
    return false;
}

// The same by all lanes of a warp, which agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) { return __all_sync(~0u, barrier_wait(bar, parity)); }

// A place in the ring of stages and how often it has been used, modulo 2.
template <int kStages>
struct Cursor {
    int at = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == kStages) {
            at = 0;
            turn ^= 1;
        }
    }
};

// What the L2 cache does with lines that are read: keeps them longest, or lets them go first.
__device__ __forceinline__ uint64_t keep_policy()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t drop_policy()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Starts the copy of vectors [i0, i1) of a row into a stage, by one warp. The
// vectors wholly inside the row come by a bulk copy; those that reach beyond
// its ends element by element (no byte outside the row is read), filled up
// with -inf. `full` counts the copy's bytes and two arrivals.
template <class T>
__device__ __forceinline__ void fill_stage(const Row<T> &row, int i0, int i1, uint4 *stage, uint64_t *full, uint64_t policy)
{
    typedef typename T::raw raw;
    const int lane = threadIdx.x & 31;
    const int lo = max(i0, row.full0), hi = min(i1, row.full1);
    if (lane == 0) {
        const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16u : 0u;
        barrier_expect(full, bytes);
        if (bytes)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                             shared_address(stage + (lo - i0))),
                         "l"(row.vec(lo)), "r"(bytes), "r"(shared_address(full)), "l"(policy)
                         : "memory");
    }
    if (lo > i0 || hi < i1) {
        const int side = lane / T::kPerVec, e = lane % T::kPerVec;
        const int i = side == 0 ? 0 : row.vecs - 1;
        if (side < 2 && (i < row.full0 || i >= row.full1) && i >= i0 && i < i1) {
            const int id = row.id(i, e);
            raw v = T::narrow(-kInf);
            if (id >= 0 && id < row.vocab)
                v = row.x[id];
            reinterpret_cast<raw *>(stage + (i - i0))[e] = v;
        }
        __syncwarp();
    }
    if (lane == 0)
        barrier_arrive(full);
}

// Stores into another CTA's shared memory of the cluster (launched as one), and
// an arrival at a barrier there that the stores before it precede.
__device__ __forceinline__ void st_cluster(uint32_t at, float a, float b)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// --- gradients -----------------------------------------------------------------

// Sets bit `at`; whether it was set before.
__device__ __forceinline__ bool claim(uint32_t *bits, int at) { return atomicOr(bits + at / 32, 1u << at % 32) >> at % 32 & 1; }

// Element e of a stored vector goes to its place in the gradient's row.
template <class T>
__device__ __forceinline__ void store_edge(typename T::raw *g, const Row<T> &row, int i, const uint4 &v)
{
    const typename T::raw *e = reinterpret_cast<const typename T::raw *>(&v);
#pragma unroll
    for (int k = 0; k < T::kPerVec; ++k) {
        const int id = row.id(i, k);
        if (id >= 0 && id < row.vocab)
            g[id] = e[k];
    }
}

__device__ __forceinline__ void store_stream(void *p, const uint4 &v) { __stcs(static_cast<uint4 *>(p), v); }

// Whether vectors of the logits' row are vectors of the gradient's too.
template <class T>
__device__ __forceinline__ bool same_phase(const Row<T> &row, const typename T::raw *g)
{
    return ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(row.x)) & 15) == 0;
}

// grad_exp for a pair, d not held at d_min (e is 0 there; t may be -inf).
template <class T>
__device__ __forceinline__ f2 grad_exp2(f2 d, const LogitRows &in, f2 &t)
{
    const f2 c = splat(in.c);
    float a, b;
    t = mul2(d, c);
    if (sizeof(typename T::raw) == 2) {
        unpk(fma2(d, c, splat(24.0f)), a, b);
        return pk(exp2_approx(a), exp2_approx(b));
    }
    unpk(t, a, b);
    asm("ex2.approx.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.f32 %0, %0;" : "+f"(b));
    const f2 e = pk(a, b), minus_one = splat(-1.0f);
    const f2 r = fma2(d, splat(in.c_lo), fma2(d, c, mul2(t, minus_one)));
    return fma2(e, mul2(r, splat(kLn2)), e);
}

// --- launches ------------------------------------------------------------------

constexpr int kMaxCluster = 8;

// Lets a kernel take the dynamic shared memory that the device has beside its
// static part. The limit belongs to the kernel on its device, and threads that
// launch it share it: so it is set once, to the most there is, and never to what
// one call needs, which would refuse another thread's larger launch. `done` has
// a bit for each device; beyond 64 of them it is set each time, to the same value.
template <class Args>
cudaError_t allow_shared(void (*kernel)(Args), std::atomic<uint64_t> &done)
{
    int dev = 0, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (e == cudaSuccess && (done.load(std::memory_order_acquire) & bit))
        return cudaSuccess;
    cudaFuncAttributes attr;
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess)
        e = cudaFuncGetAttributes(&attr, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)attr.sharedSizeBytes);
    if (e != cudaSuccess)
        (void)cudaGetLastError();
    else
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A row by a cluster of `size` CTAs.
template <auto kKernel, class Args>
cudaError_t launch_cluster(const Args &a, int64_t rows, int size, size_t shared_bytes, int threads, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = cudaSuccess;
    if (shared_bytes > 32 * 1024)   // with the static part, beyond what a kernel gets unasked
        e = allow_shared(kKernel, allowed);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * size));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = size > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kKernel, a);
    count_launch();
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

// Vectors of a row of `row_bytes` bytes at any alignment, and of one CTA's part of it.
inline int64_t row_vecs(int64_t row_bytes) { return (row_bytes + 30) / 16; }
inline int64_t part_vecs(int64_t row_bytes, int size) { return (row_vecs(row_bytes) + size - 1) / size; }

}  // namespace fo
