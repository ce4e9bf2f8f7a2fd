// fo_distill.cu -- distillation from a teacher's top logits: loss, and its
// gradient in the same pass or from saved statistics.
#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kPartBytes = 64 * 1024;
constexpr int kEntryWarps = FO_MAX_TOP_K / 32;   // warps that hold an entry a thread

// The teacher's row: ids (-1: none), q and ln q.
struct Entries {
    int32_t ids[FO_MAX_TOP_K];
    float q[FO_MAX_TOP_K], logq[FO_MAX_TOP_K];
    float sum;      // A: sum of q and of the rest; NaN where an id is out of range
    float rest;     // the mass that is not listed (0 without tail)
};

// By one warp.
__device__ __forceinline__ void read_teacher(Entries &s, const Teacher &t, int64_t r, int vocab)
{
    const int lane = threadIdx.x & 31;
    float y[kEntryWarps], m = -kInf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kEntryWarps; ++i) {
        const int e = lane + 32 * i;
        const int32_t id = e < t.k ? t.ids[r * t.k + e] : -1;
        y[i] = id < 0 ? -kInf : load_dtype(t.logits, r * t.k + e, t.dtype) * t.inv_t;
        m = fmaxf(m, y[i]);
        bad = bad || id >= vocab;
        s.ids[e] = id;
    }
    bad = __any_sync(~0u, bad);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    m = safe_max(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kEntryWarps; ++i)
        z += expf(y[i] - m);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        z += __shfl_xor_sync(~0u, z, o);
    const float norm = t.tail ? (t.lse ? t.lse[r] : 0.0f) : z == 0.0f ? 0.0f : m + logf(z);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kEntryWarps; ++i) {
        const float lq = y[i] - norm, q = expf(lq);
        sum += q;
        s.q[lane + 32 * i] = q;
        s.logq[lane + 32 * i] = lq;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) {
        s.rest = t.tail ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
        s.sum = bad ? __int_as_float(0x7fffffff) : t.tail ? fmaxf(1.0f, sum) : z == 0.0f ? 0.0f : 1.0f;
    }
}

// The weight of all entries with the id of entry k, and whether k is the first of them.
__device__ __forceinline__ float merged_q(const Entries &s, int n, int k, bool &first)
{
    const int32_t id = s.ids[k];
    float q = 0.0f;
    first = true;
    for (int i = 0; i < n; ++i)
        if (s.ids[i] == id) {
            q += s.q[i];
            first = first && i >= k;
        }
    return q;
}

// 2^t f for a vector of logits: the gradient of tokens that are not listed.
template <class T>
__device__ __forceinline__ uint4 grad_vec(const uint4 &v, f2 nm, f2 f, const LogitRows &in)
{
    f2 x[T::kPerVec / 2];
    widen_vec<T>(v, x);
#pragma unroll
    for (int k = 0; k < T::kPerVec / 2; ++k) {
        f2 d = add2(x[k], nm), t;
        if (sizeof(typename T::raw) == 4) {
            float a, b;
            unpk(d, a, b);
            d = pk(max_nan(a, in.d_min), max_nan(b, in.d_min));
        }
        x[k] = mul2(grad_exp2<T>(d, in, t), f);
    }
    return narrow_vec<T>(x);
}

template <class T>
__device__ __forceinline__ float grad_listed(float x, float m, float q, float a, float inv_z, float scale, const LogitRows &in)
{
    float t;
    const float e = grad_exp<T>(distance(x, m, in), in, t);
    return __fmaf_rn(e, inv_z / T::kShift * a, -q) * scale;
}

// What a CTA's part of a row adds to the row.
struct PartSums {
    Stat rest;      // m, z of the tokens that are not listed (w unused)
    Stat listed;    // of those that are
    float q;        // sum of q over the entries in the part
    double dot;     // sum of q (x - listed.m) over them
};

struct Shared {
    uint64_t bar;
    Entries t;
    Stat part[kWarps + 1];
    Stat listed[kEntryWarps];
    double dot[kEntryWarps];
    float q[kEntryWarps];
    PartSums mine;   // read by the other CTAs of the cluster
};

__device__ __forceinline__ Stat ld_cluster_stat(uint32_t at)
{
    return Stat{ld_cluster_f32(at), ld_cluster_f32(at + 4), 0.0f};
}

// One row by a cluster of CTAs, each holding a part of it in shared memory:
// logits are read from device memory once, by bulk copies, for the loss and the
// gradient. The listed tokens' logits are taken out of the part (replaced by
// -inf) before the pass, so that what is summed is the rest alone: 1 - sum p
// would lose a small rest. For the same reason the rest keeps a maximum of its
// own: it may lie further below the listed logits than FP32's exponents reach.
template <class T>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a)
{
    typedef typename T::raw raw;
    extern __shared__ __align__(16) unsigned char dynamic[];
    uint4 *buf = reinterpret_cast<uint4 *>(dynamic);
    __shared__ Shared sh;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x / size;
    const Row<T> row(a.in, r);
    const Part p = part_of(row, rank, size);
    const float weight = a.weight ? a.weight[r] : 1.0f;
    raw *g = static_cast<raw *>(a.grad.data);
    if (g)
        g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
    const bool aligned = g && same_phase(row, g);
    if (weight == 0.0f) {   // the same in all CTAs of the cluster
        if (rank == 0 && tid == 0 && a.loss)
            a.loss[r] = 0.0f;
        for (int i = tid; g && i < p.n; i += kThreads) {
            const int at = p.v0 + i;
            if (aligned && at >= row.full0 && at < row.full1)
                store_stream(g + row.id(at, 0), make_uint4(0, 0, 0, 0));
            else
                store_edge<T>(g, row, at, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(&sh.bar)) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    start_part<T>(row, p, buf, &sh.bar);
    if (tid >= kThreads - 32)
        read_teacher(sh.t, a.teacher, r, row.vocab);
    __syncthreads();
    // the entry of this thread, if its token is in the part
    const int k = a.teacher.k;
    int place = -1;       // in the part's elements
    bool first = false;
    float q_all = 0.0f, x_entry = 0.0f;
    if (tid < k) {
        const int32_t id = sh.t.ids[tid];
        if (id >= 0 && id < row.vocab) {
            const int at = id + row.phase - p.v0 * T::kPerVec;
            if (at >= 0 && at < p.n * T::kPerVec) {
                place = at;
                q_all = merged_q(sh.t, k, tid, first);
            }
        }
    }
    const bool arrived = wait_part(&sh.bar);
    if (tid < FO_MAX_TOP_K) {
        Stat l = {-kInf, 0.0f, 0.0f};
        if (place >= 0) {
            x_entry = T::widen(reinterpret_cast<const raw *>(buf)[place]);
            if (first && x_entry != -kInf) {
                l.z = x_entry - x_entry == 0.0f ? 1.0f : x_entry - x_entry;   // NaN for NaN and +inf
                l.m = x_entry == x_entry ? x_entry : l.m;
            }
        }
        l = warp_join<false>(l, a.in);
        if ((tid & 31) == 0)
            sh.listed[tid >> 5] = l;
    }
    __syncthreads();
    if (first)
        reinterpret_cast<raw *>(buf)[place] = T::narrow(-kInf);
    Stat listed = sh.listed[0];
#pragma unroll
    for (int i = 1; i < kEntryWarps; ++i)
        listed = join<false>(listed, sh.listed[i], a.in);
    if (tid < FO_MAX_TOP_K) {
        const bool use = place >= 0 && sh.t.q[tid] > 0.0f;
        float q = use ? sh.t.q[tid] : 0.0f;
        double dot = use ? (double)q * ((double)x_entry - (double)safe_max(listed.m)) : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            q += __shfl_xor_sync(~0u, q, o);
            dot += __shfl_xor_sync(~0u, dot, o);
        }
        if ((tid & 31) == 0) {
            sh.q[tid >> 5] = q;
            sh.dot[tid >> 5] = dot;
        }
    }
    __syncthreads();

    Running<T, false> run;
#pragma unroll 2
    for (int i = tid; i < p.n; i += kThreads)
        run.add(buf[i], a.in);
    Stat rest = run.stat(a.in);
    if (!arrived)
        rest.z = __int_as_float(0x7fffffff);
    rest = block_join<false, kWarps>(rest, sh.part, a.in);
    float qs = (sh.q[0] + sh.q[1]) + (sh.q[2] + sh.q[3]);
    double dot = (sh.dot[0] + sh.dot[1]) + (sh.dot[2] + sh.dot[3]);
    if (size > 1) {
        if (tid == 0)
            sh.mine = PartSums{rest, listed, qs, dot};
        cluster_arrive();
        cluster_wait();
        const uint32_t from = (tid & 7) % size;
        rest = warp_join<false>(ld_cluster_stat(map_shared(&sh.mine.rest, from)), a.in, size);
        listed = warp_join<false>(ld_cluster_stat(map_shared(&sh.mine.listed, from)), a.in, size);
        if (rank == 0 && tid < 32) {
            qs = 0.0f;
            dot = 0.0;
            for (uint32_t i = 0; i < size; ++i) {
                const float pq = ld_cluster_f32(map_shared(&sh.mine.q, i));
                if (pq == 0.0f)
                    continue;
                const double pm = safe_max(ld_cluster_f32(map_shared(&sh.mine.listed, i)));
                qs += pq;
                dot += ld_cluster_f64(map_shared(&sh.mine.dot, i)) + (double)pq * (pm - (double)safe_max(listed.m));
            }
        }
        cluster_arrive();   // what was read here is free to go; the wait is at the end
    }
    const Stat s = join<false>(rest, listed, a.in);
    const float inv_z = s.z == 0.0f ? 0.0f : 1.0f / s.z;
    const float sum = sh.t.sum, q_rest = sh.t.rest, m = safe_max(s.m), m_rest = safe_max(rest.m);
    // an unlisted token: p - q_rest p / p_rest, by 2^((x - m_rest) c)
    const float f = __fsub_rn(exp2_approx(distance(rest.m, m, a.in) * a.in.c) * (sum * inv_z), rest.z == 0.0f ? 0.0f : q_rest / rest.z);
    if (rank == 0 && tid < 32 && (a.loss || a.stats)) {
        // KL = sum q ln q - sum q s + (sum q) ln Z, and the rest's term
        float ql = 0.0f;
#pragma unroll
        for (int i = 0; i < kEntryWarps; ++i) {
            const float q = sh.t.q[tid + 32 * i];
            ql += q > 0.0f ? q * sh.t.logq[tid + 32 * i] : 0.0f;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            ql += __shfl_xor_sync(~0u, ql, o);
        if (tid == 0) {
            const double ln_z = logf(s.z), inv_t = a.in.inv_t;
            double kl = 0.0;
            if (qs != 0.0f)
                kl = s.z == 0.0f ? (double)kInf
                                 : (double)ql - (dot + (double)qs * ((double)safe_max(listed.m) - (double)m)) * inv_t + (double)qs * ln_z;
            if (q_rest > 0.0f)
                kl += rest.z == 0.0f ? (double)kInf
                                     : (double)q_rest * ((double)logf(q_rest) - (((double)m_rest - (double)m) * inv_t + (double)logf(rest.z) - ln_z));
            if (sum != sum || s.z != s.z)
                kl = __int_as_float(0x7fffffff);
            if (a.loss)
                a.loss[r] = (float)(kl * (double)weight);
            if (a.stats)
                a.stats[r] = make_float4(s.m, s.z, rest.m, f);
        }
    }
    if (g) {
        const float scale = weight * a.in.inv_t;
        const f2 nm = splat(-m_rest), ff = splat(f * (scale / T::kShift));
        for (int i = tid; i < p.n; i += kThreads) {
            const int at = p.v0 + i;
            const uint4 d = grad_vec<T>(buf[i], nm, ff, a.in);
            if (aligned && at >= row.full0 && at < row.full1)
                store_stream(g + row.id(at, 0), d);
            else
                store_edge<T>(g, row, at, d);
        }
        __syncthreads();
        if (first)
            g[sh.t.ids[tid]] = T::narrow(s.z == 0.0f ? 0.0f : grad_listed<T>(x_entry, m, q_all, sum, inv_z, scale, a.in));
    }
    if (!arrived)
        wait_part(&sh.bar);   // its copies are not left behind
    if (size > 1)
        cluster_wait();       // no CTA leaves while another reads its shared memory
}

// The gradient from saved statistics.
template <class T, int kVecs>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(DistillGradArgs a, int chunks)
{
    typedef typename T::raw raw;
    __shared__ Entries t;
    const int64_t r = blockIdx.x / (unsigned)chunks;
    const int v0 = (int)(blockIdx.x % (unsigned)chunks) * (kVecs * kThreads);
    const Row<T> row(a.in, r);
    raw *g = static_cast<raw *>(a.out.data) + row_offset(a.in, r, a.out.row_stride, a.out.outer_stride);
    const int tid = threadIdx.x;
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = v0 + i * kThreads + tid;
        if (at < row.vecs)
            v[i] = load_vec(row, at);
    }
    if (tid < 32)
        read_teacher(t, a.teacher, r, row.vocab);
    const float gl = a.g_loss[r];
    const float4 st = gl == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : a.stats[r];
    __syncthreads();
    const float inv_z = st.y == 0.0f ? 0.0f : 1.0f / st.y, scale = gl * a.in.inv_t;
    const bool zero = st.y == 0.0f;
    bool entry = false;
    float entry_value = 0.0f;
    if (!zero && tid < a.teacher.k) {
        const int32_t id = t.ids[tid];
        if (id >= max(0, row.id(v0, 0)) && id < min(row.vocab, row.id(v0 + kVecs * kThreads, 0))) {
            const float q = merged_q(t, a.teacher.k, tid, entry);
            entry_value = grad_listed<T>(T::widen(row.x[id]), safe_max(st.x), q, t.sum, inv_z, scale, a.in);
        }
    }
    __syncthreads();   // the entries' logits are read before a gradient in their place is written
    const bool aligned = same_phase(row, g);
    const f2 nm = splat(-safe_max(st.z)), f = splat(st.w * (scale / T::kShift));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = v0 + i * kThreads + tid;
        if (at >= row.vecs)
            break;
        const uint4 d = zero ? make_uint4(0, 0, 0, 0) : grad_vec<T>(v[i], nm, f, a.in);
        if (aligned && at >= row.full0 && at < row.full1)
            store_stream(g + row.id(at, 0), d);
        else
            store_edge<T>(g, row, at, d);
    }
    __syncthreads();
    if (entry)
        g[t.ids[tid]] = T::narrow(entry_value);
}

template <class T>
cudaError_t launch(const DistillArgs &a, cudaStream_t stream)
{
    // the smallest cluster whose parts are at most kPartBytes (three such CTAs
    // share an SM, so that one computes while the others load); larger while
    // the grid would leave SMs without a CTA and parts stay above 8 KB
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw);
    int size = 1;
    while (size < kMaxCluster && (bytes > size * kPartBytes || (a.in.rows * size < 2 * sm_count() && bytes > size * 8192)))
        size *= 2;
    return launch_cluster(distill_kernel<T>, a, a.in.rows, size, part_vecs(bytes, size) * 16, kThreads, stream);
}

template <class T>
cudaError_t launch(const DistillGradArgs &a, cudaStream_t stream)
{
    const int64_t vecs = a.in.vocab / T::kPerVec + 2;
    if (vecs * a.in.rows >= (int64_t)sm_count() * 8 * kThreads * 8) {
        const int64_t chunks = (vecs + 8 * kThreads - 1) / (8 * kThreads);
        distill_grad_kernel<T, 8><<<(unsigned)(chunks * a.in.rows), kThreads, 0, stream>>>(a, (int)chunks);
    } else {
        const int64_t chunks = (vecs + kThreads - 1) / kThreads;
        distill_grad_kernel<T, 1><<<(unsigned)(chunks * a.in.rows), kThreads, 0, stream>>>(a, (int)chunks);
    }
    count_launch();
    return cudaGetLastError();
}

template <class A>
cudaError_t by_type(int dtype, const A &a, cudaStream_t stream)
{
    return dtype == 0 ? launch<Bf16>(a, stream) : dtype == 1 ? launch<F32>(a, stream) : launch<F16>(a, stream);
}

}  // namespace

cudaError_t launch_distill(int dtype, const DistillArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }
cudaError_t launch_distill_grad(int dtype, const DistillGradArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }

}  // namespace fo
