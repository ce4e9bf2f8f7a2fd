// fo_logprobs.cu -- log probabilities of given tokens with entropy and top
// alternatives, and their gradient.
#include "fo_internal.h"
#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kThreads = 512;

// Running statistics: m, Z = sum 2^((x-m)c), W = sum 2^t t with t = (x-m)c.
struct Stat {
    float m, z, w;
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c)
{
    Stat r;
    r.m = fmaxf(a.m, b.m);
    const float mm = safe_max(r.m);
    // the floor keeps W finite where one part's values are the type's lowest
    const float da = a.z == 0.0f ? 0.0f : fmaxf((a.m - mm) * c, -1e30f);
    const float db = b.z == 0.0f ? 0.0f : fmaxf((b.m - mm) * c, -1e30f);
    const float ea = exp2_approx(da), eb = exp2_approx(db);
    r.z = a.z * ea + b.z * eb;
    r.w = (a.w + da * a.z) * ea + (b.w + db * b.z) * eb;
    return r;
}

template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a)
{
    __shared__ Stat part[kThreads / 32];
    __shared__ unsigned long long best[kThreads / 32];
    const int64_t r = blockIdx.x;
    const typename T::raw *x = static_cast<const typename T::raw *>(a.in.data) + row_offset(a.in, r, a.in.row_stride, a.in.outer_stride);
    const int64_t v = a.in.vocab;
    const float c = a.in.c;
    Stat s = {-kInf, 0.0f, 0.0f};
    // sums of 16 first: a chain of roundings of equal terms does not average out
    for (int64_t j = threadIdx.x; j < v; j += 16 * kThreads) {
        Stat b = {-kInf, 0.0f, 0.0f};
        for (int64_t i = j; i < v && i < j + 16 * kThreads; i += kThreads) {
            const float xv = T::widen(x[i]);
            if (xv != -kInf)
                b = join(b, Stat{xv != xv ? b.m : xv, xv - xv == 0.0f ? 1.0f : xv - xv, 0.0f}, c);
        }
        s = join(s, b, c);
    }
    for (int o = 16; o; o >>= 1)
        s = join(s, Stat{__shfl_xor_sync(~0u, s.m, o), __shfl_xor_sync(~0u, s.z, o), __shfl_xor_sync(~0u, s.w, o)}, c);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = part[0];
    for (int i = 1; i < kThreads / 32; ++i)
        s = join(s, part[i], c);
    const float ln_z = logf(s.z);
    if (threadIdx.x == 0) {
        const float h = s.z == 0.0f ? 0.0f : ln_z - kLn2 * (s.w / s.z);
        if (a.logp) {
            const int64_t t = a.tokens[r];
            a.logp[r] = t < 0 ? 0.0f : t >= v ? __int_as_float(0x7fffffff) : (float)log_prob(T::widen(x[t]), s.m, s.z, ln_z, a.in.inv_t);
        }
        if (a.entropy)
            a.entropy[r] = h;
        if (a.stats)
            a.stats[r] = make_float4(s.m, s.z, h, 0.0f);
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.k; ++k) {
        unsigned long long b = 0;
        for (int64_t j = threadIdx.x; j < v; j += kThreads) {
            const unsigned long long key = entry_key(T::widen(x[j]), (uint32_t)j);
            if (key < last && key > b)
                b = key;
        }
        for (int o = 16; o; o >>= 1) {
            const unsigned long long q = __shfl_xor_sync(~0u, b, o);
            b = q > b ? q : b;
        }
        if ((threadIdx.x & 31) == 0)
            best[threadIdx.x >> 5] = b;
        __syncthreads();
        last = best[0];
        for (int i = 1; i < kThreads / 32; ++i)
            last = best[i] > last ? best[i] : last;
        __syncthreads();
        if (threadIdx.x == 0) {
            const uint32_t id = entry_id(last);
            a.top_ids[r * a.k + k] = (int32_t)id;
            a.top_logp[r * a.k + k] = (float)log_prob(T::widen(x[id]), s.m, s.z, ln_z, a.in.inv_t);
        }
    }
}

// dx_j = (1/T) [ sum of the weights of entries at j - p_j (G + h (ln p_j + H)) ],
// G the sum of all entries' weights, the entries being the token and the top ids.
template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(LogprobGradArgs a)
{
    __shared__ int64_t ids[FO_MAX_TOP_K + 1];
    __shared__ float weight[FO_MAX_TOP_K + 1];
    const int64_t r = blockIdx.x;
    const typename T::raw *x = static_cast<const typename T::raw *>(a.in.data) + row_offset(a.in, r, a.in.row_stride, a.in.outer_stride);
    typename T::raw *g = static_cast<typename T::raw *>(a.out.data) + row_offset(a.in, r, a.out.row_stride, a.out.outer_stride);
    const int64_t v = a.in.vocab;
    const float4 st = a.stats[r];
    const float m = safe_max(st.x), inv_z = st.y == 0.0f ? 0.0f : 1.0f / st.y, ln_z = logf(st.y);
    const float h = a.g_entropy ? a.g_entropy[r] : 0.0f;
    if (threadIdx.x <= a.k) {
        const int i = (int)threadIdx.x - 1;
        ids[threadIdx.x] = i < 0 ? (a.g_logp ? a.tokens[r] : -1) : a.top_ids[r * a.k + i];
        weight[threadIdx.x] = i < 0 ? (a.g_logp ? a.g_logp[r] : 0.0f) : a.g_top[r * a.k + i];
    }
    __syncthreads();
    float sum = 0.0f;
    bool any = h != 0.0f;
    for (int i = 0; i <= a.k; ++i) {
        if (ids[i] >= 0) {
            any = any || weight[i] != 0.0f;
            sum += weight[i];
        }
        if (ids[i] >= v && weight[i] != 0.0f)
            sum = __int_as_float(0x7fffffff);
    }
    const bool zero = !any || st.y == 0.0f;
    for (int64_t j = threadIdx.x; j < v; j += kThreads) {
        float d = 0.0f;
        if (!zero) {
            float w = 0.0f;
            for (int i = 0; i <= a.k; ++i)
                if (ids[i] == j)
                    w += weight[i];
            float t;
            const float e = grad_exp<T>(distance(T::widen(x[j]), m, a.in), a.in, t);
            const float b = h == 0.0f ? 0.0f : h * (__fmaf_rn(t, kLn2, -ln_z) + st.z);
            d = (w - e * (inv_z / T::kShift * (sum + b))) * a.in.inv_t;
        }
        g[j] = T::narrow(d);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(int dtype, const LogprobArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)a.in.rows;
    if (dtype == 0)
        logprobs_kernel<Bf16><<<grid, kThreads, 0, stream>>>(a);
    else if (dtype == 1)
        logprobs_kernel<F32><<<grid, kThreads, 0, stream>>>(a);
    else
        logprobs_kernel<F16><<<grid, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_grad(int dtype, const LogprobGradArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)a.in.rows;
    if (dtype == 0)
        logprobs_grad_kernel<Bf16><<<grid, kThreads, 0, stream>>>(a);
    else if (dtype == 1)
        logprobs_grad_kernel<F32><<<grid, kThreads, 0, stream>>>(a);
    else
        logprobs_grad_kernel<F16><<<grid, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fo
