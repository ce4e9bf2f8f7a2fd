// fo_distill.cu -- distillation from a teacher's top logits: loss, and its
// gradient in the same pass or from saved statistics.
#include "fo_internal.h"
#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kThreads = 512;

struct Row {
    float m, z, rest;   // rest: the part of Z of tokens that are not listed
};

__device__ __forceinline__ Row join(Row a, Row b, float c)
{
    Row r;
    r.m = fmaxf(a.m, b.m);
    const float mm = safe_max(r.m);
    const float ea = a.z == 0.0f ? 0.0f : exp2_approx((a.m - mm) * c), eb = b.z == 0.0f ? 0.0f : exp2_approx((b.m - mm) * c);
    r.z = a.z * ea + b.z * eb;
    r.rest = a.rest * ea + b.rest * eb;
    return r;
}

struct Shared {
    int32_t ids[FO_MAX_TOP_K];
    float q[FO_MAX_TOP_K], logq[FO_MAX_TOP_K];
    float sum_q, q_rest;
    bool bad;
};

__device__ __forceinline__ int listed(const Shared &s, int k, int64_t j)
{
    for (int i = 0; i < k; ++i)
        if (s.ids[i] == j)
            return i;
    return -1;
}

// The teacher's row: ids, q and log q.
__device__ void read_teacher(Shared &s, const Teacher &t, int64_t r, int64_t v)
{
    const int i = threadIdx.x;
    if (i < t.k) {
        s.ids[i] = t.ids[r * t.k + i];
        s.logq[i] = s.ids[i] < 0 ? -kInf : load_dtype(t.logits, r * t.k + i, t.dtype) * t.inv_t;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float m = -kInf;
        s.bad = false;
        for (int e = 0; e < t.k; ++e) {
            m = fmaxf(m, s.logq[e]);
            s.bad = s.bad || s.ids[e] >= v;
        }
        m = safe_max(m);
        float z = 0.0f;
        for (int e = 0; e < t.k; ++e)
            z += expf(s.logq[e] - m);
        const float norm = t.tail ? (t.lse ? t.lse[r] : 0.0f) : z == 0.0f ? 0.0f : m + logf(z);
        float sum = 0.0f;
        for (int e = 0; e < t.k; ++e) {
            s.logq[e] -= norm;
            s.q[e] = expf(s.logq[e]);
            sum += s.q[e];
        }
        s.q_rest = t.tail ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
        s.sum_q = t.tail ? fmaxf(1.0f, sum) : z == 0.0f ? 0.0f : 1.0f;
        if (s.bad)
            s.sum_q = __int_as_float(0x7fffffff);
    }
    __syncthreads();
}

template <class T>
__device__ void write_grad(typename T::raw *g, const typename T::raw *x, const LogitRows &in, const Shared &s, int k,
                           float m, float z, float a, float b, float scale)
{
    const float mm = safe_max(m), inv_z = z == 0.0f ? 0.0f : 1.0f / z;
    const bool zero = scale == 0.0f || z == 0.0f;
    for (int64_t j = threadIdx.x; j < in.vocab; j += kThreads) {
        float d = 0.0f;
        if (!zero) {
            const int first = listed(s, k, j);
            float q = 0.0f;
            for (int i = first; i >= 0 && i < k; ++i)
                if (s.ids[i] == j)
                    q += s.q[i];
            float t;
            const float e = grad_exp<T>(distance(T::widen(x[j]), mm, in), in, t);
            d = (first < 0 ? e * (inv_z / T::kShift * (a - b)) : __fmaf_rn(e, inv_z / T::kShift * a, -q)) * scale;
        }
        g[j] = T::narrow(d);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a)
{
    __shared__ Shared sh;
    __shared__ Row part[kThreads / 32];
    const int64_t r = blockIdx.x, v = a.in.vocab;
    const float weight = a.weight ? a.weight[r] : 1.0f, c = a.in.c;
    const typename T::raw *x = static_cast<const typename T::raw *>(a.in.data) + row_offset(a.in, r, a.in.row_stride, a.in.outer_stride);
    typename T::raw *g = static_cast<typename T::raw *>(a.grad.data);
    if (g)
        g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
    if (weight == 0.0f) {
        if (threadIdx.x == 0 && a.loss)
            a.loss[r] = 0.0f;
        if (g)
            write_grad<T>(g, x, a.in, sh, 0, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    read_teacher(sh, a.teacher, r, v);
    Row s = {-kInf, 0.0f, 0.0f};
    // sums of 16 first: a chain of roundings of equal terms does not average out
    for (int64_t j = threadIdx.x; j < v; j += 16 * kThreads) {
        Row b = {-kInf, 0.0f, 0.0f};
        for (int64_t i = j; i < v && i < j + 16 * kThreads; i += kThreads) {
            const float xv = T::widen(x[i]);
            const float one = xv - xv == 0.0f ? 1.0f : xv - xv;
            if (xv != -kInf)
                b = join(b, Row{xv != xv ? b.m : xv, one, listed(sh, a.teacher.k, i) < 0 ? one : 0.0f}, c);
        }
        s = join(s, b, c);
    }
    for (int o = 16; o; o >>= 1)
        s = join(s, Row{__shfl_xor_sync(~0u, s.m, o), __shfl_xor_sync(~0u, s.z, o), __shfl_xor_sync(~0u, s.rest, o)}, c);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = part[0];
    for (int i = 1; i < kThreads / 32; ++i)
        s = join(s, part[i], c);
    const float b = sh.q_rest == 0.0f || s.rest == 0.0f ? 0.0f : sh.q_rest * s.z / s.rest;
    if (threadIdx.x == 0) {
        const float ln_z = logf(s.z);
        double sum = 0.0;
        for (int i = 0; i < a.teacher.k; ++i) {
            const int32_t id = sh.ids[i];
            if (id >= 0 && id < v && sh.q[i] > 0.0f)
                sum += (double)sh.q[i] * ((double)sh.logq[i] - log_prob(T::widen(x[id]), s.m, s.z, ln_z, a.in.inv_t));
        }
        if (sh.q_rest > 0.0f)
            sum += sh.q_rest * (logf(sh.q_rest) - (s.rest == 0.0f ? -kInf : logf(s.rest) - ln_z));
        float loss = (float)sum;
        if (sh.bad || s.z != s.z)
            loss = __int_as_float(0x7fffffff);
        if (a.loss)
            a.loss[r] = loss * weight;
        if (a.stats)
            a.stats[r] = make_float4(s.m, s.z, sh.sum_q, b);
    }
    __syncthreads();
    if (g)
        write_grad<T>(g, x, a.in, sh, a.teacher.k, s.m, s.z, sh.sum_q, b, weight * a.in.inv_t);
}

template <class T>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(DistillGradArgs a)
{
    __shared__ Shared sh;
    const int64_t r = blockIdx.x;
    const typename T::raw *x = static_cast<const typename T::raw *>(a.in.data) + row_offset(a.in, r, a.in.row_stride, a.in.outer_stride);
    typename T::raw *g = static_cast<typename T::raw *>(a.out.data) + row_offset(a.in, r, a.out.row_stride, a.out.outer_stride);
    read_teacher(sh, a.teacher, r, a.in.vocab);
    const float gl = a.g_loss[r];
    const float4 st = gl == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : a.stats[r];
    write_grad<T>(g, x, a.in, sh, a.teacher.k, st.x, st.y, st.z, st.w, gl * a.in.inv_t);
}

}  // namespace

cudaError_t launch_distill(int dtype, const DistillArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)a.in.rows;
    if (dtype == 0)
        distill_kernel<Bf16><<<grid, kThreads, 0, stream>>>(a);
    else if (dtype == 1)
        distill_kernel<F32><<<grid, kThreads, 0, stream>>>(a);
    else
        distill_kernel<F16><<<grid, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_distill_grad(int dtype, const DistillGradArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)a.in.rows;
    if (dtype == 0)
        distill_grad_kernel<Bf16><<<grid, kThreads, 0, stream>>>(a);
    else if (dtype == 1)
        distill_grad_kernel<F32><<<grid, kThreads, 0, stream>>>(a);
    else
        distill_grad_kernel<F16><<<grid, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fo
