// fo_policy.cu -- the clipped loss of policy training on sampled tokens, with a KL
// term, and its gradient in the same call. (The gradient from saved statistics is
// that of the token's log probability: fo_logprobs.cu.)
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256;

// A row's loss and its derivative by the log probability.
struct RowLoss {
    float loss, slope;
};

// e^k - k - 1. Its terms cancel for small k, whose series is taken instead (to
// k^11 / 11!: 2^-11 to that power is below 2^-25 of k^2 / 2).
__device__ __forceinline__ float exp_rest(float k)
{
    if (k == kInf)
        return kInf;
    if (fabsf(k) >= 0.5f)
        return __fsub_rn(__fsub_rn(expf(k), k), 1.0f);
    float s = 1.0f;
#pragma unroll
    for (int n = 11; n >= 3; --n)
        s = __fmaf_rn(__fmul_rn(k, 1.0f / (float)n), s, 1.0f);
    return __fmul_rn(__fmul_rn(0.5f * k, k), s);
}

__device__ __forceinline__ RowLoss row_loss(const PolicyArgs &a, int64_t r, float logp)
{
    RowLoss o = {0.0f, 0.0f};
    const float adv = a.advantages[r];
    if (adv != 0.0f) {
        const float q = expf(__fsub_rn(logp, a.old_logp[r]));
        const bool inside = adv >= 0.0f ? q <= a.ratio_high : q >= a.ratio_low;
        o.loss = -__fmul_rn(inside ? q : adv >= 0.0f ? a.ratio_high : a.ratio_low, adv);
        o.slope = inside ? o.loss : 0.0f;
        if (adv != adv || q != q)
            o.loss = o.slope = kNan;
    }
    if (a.ref_logp) {
        const float k = __fsub_rn(a.ref_logp[r], logp);
        o.loss = __fmaf_rn(a.kl_weight, exp_rest(k), o.loss);
        o.slope = __fmaf_rn(a.kl_weight, -expm1f(k), o.slope);
    }
    return o;
}

// A row a CTA, two passes.
template <class T>
__global__ void __launch_bounds__(kThreads) policy_kernel(PolicyArgs a)
{
    typedef typename T::raw raw;
    __shared__ Stat part[kThreads / 32];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x, token = a.tokens[r];
    const Row<T> row(a.in, r);
    raw *g = static_cast<raw *>(a.grad.data);
    if (g)
        g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
    const bool aligned = g && same_phase(row, g);
    const auto write = [&](int i, const uint4 &v) {
        if (aligned && i >= row.full0 && i < row.full1)
            store_stream(g + row.id(i, 0), v);
        else
            store_edge<T>(g, row, i, v);
    };
    const float weight = a.weight ? a.weight[r] : 1.0f;
    if (token < 0 || weight == 0.0f) {
        if (tid == 0) {
            if (a.loss)
                a.loss[r] = 0.0f;
            if (a.logp)
                a.logp[r] = 0.0f;
            if (a.stats)
                a.stats[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        for (int i = tid; g && i < row.vecs; i += kThreads)
            write(i, make_uint4(0, 0, 0, 0));
        return;
    }
    const bool there = token < row.vocab;
    const float x = there ? T::widen(row.x[token]) : kNan;
    Running<T, false> run;
    for (int i = tid; i < row.vecs; i += kThreads)
        run.add(load_vec(row, i), a.in);
    const Stat s = block_join<false, kThreads>(run.stat(a.in), part, a.in);   // every thread has read x
    const float z = there ? s.z : kNan;
    const float logp = z == 0.0f ? -kInf : z != z ? kNan : log_prob(x, s.m, z, logf(z), a.in.inv_t);
    const RowLoss o = row_loss(a, r, logp);
    if (tid == 0) {
        if (a.loss)
            a.loss[r] = __fmul_rn(o.loss, weight);
        if (a.logp)
            a.logp[r] = logp;
        if (a.stats)
            a.stats[r] = make_float4(s.m, z, o.slope, 0.0f);
    }
    if (!g)
        return;
    const float scaled = __fmul_rn(o.slope, weight), slope = z == 0.0f ? 0.0f : fabsf(scaled) < kInf ? scaled * a.in.inv_t : kNan;
    const float f = z == 0.0f ? 0.0f : -slope * (1.0f / z) / T::kShift, mm = safe_max(s.m);
    for (int i = tid; i < row.vecs; i += kThreads)
        write(i, grad_vec<T>(load_vec(row, i), splat(-mm), splat(f), a.in));
    __syncthreads();
    if (tid == 0 && there) {
        float t;
        g[token] = T::narrow(z == 0.0f ? 0.0f : __fmaf_rn(grad_exp<T>(distance(x, mm, a.in), a.in, t), f, slope));
    }
}

template <class T>
cudaError_t launch(const PolicyArgs &a, cudaStream_t stream)
{
    policy_kernel<T><<<(unsigned)a.in.rows, kThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_policy(int dtype, const PolicyArgs &a, cudaStream_t stream)
{
    return dtype == 0 ? launch<Bf16>(a, stream) : dtype == 1 ? launch<F32>(a, stream) : launch<F16>(a, stream);
}

}  // namespace fo
