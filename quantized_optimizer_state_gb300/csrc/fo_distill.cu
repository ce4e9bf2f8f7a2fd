// fo_distill.cu -- distillation from a teacher's top logits: loss, and its
// gradient in the same pass or from saved statistics.
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kStream = 256;                      // threads that walk over a row
constexpr int kWarps = kStream / 32;
constexpr int kThreads = kStream + 32;            // and a warp for the teacher's entries
constexpr int kGroup = 4;                         // vectors that a thread loads at once
constexpr int kGroupStep = kGroup * kStream;
constexpr int kGradThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int64_t kCacheBytes = 80 << 20;         // of the 129 MB L2 cache, for rows between their passes
constexpr int kSlots = FO_MAX_TOP_K / 32;         // entries of a lane of one warp that holds them all

// A teacher's row in one warp: entry lane + 32 i at place i.
struct TeacherRow {
    int32_t id[kSlots];          // -1: none
    float q[kSlots], logq[kSlots];
    float sum;                   // of q and of the rest; NaN where an id is out of range or q is not finite
    float rest;                  // the mass that is not listed (0 without tail)
};

// What it is made from, as loaded.
struct TeacherRaw {
    int32_t id[kSlots];
    float logit[kSlots], lse;
};

__device__ __forceinline__ TeacherRaw load_teacher(const Teacher &t, int64_t r)
{
    TeacherRaw w;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int e = (int)(threadIdx.x & 31) + 32 * i;
        w.id[i] = e < t.k ? t.ids[r * t.k + e] : -1;
        w.logit[i] = e < t.k ? load_dtype(t.logits, r * t.k + e, t.dtype) : 0.0f;
    }
    w.lse = t.lse ? t.lse[r] : 0.0f;
    return w;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__device__ __forceinline__ TeacherRow make_teacher(const Teacher &t, const TeacherRaw &w, int vocab)
{
    TeacherRow s;
    float m = -kInf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        s.id[i] = w.id[i];
        s.logq[i] = w.id[i] < 0 ? -kInf : w.logit[i] * t.inv_t;
        m = fmaxf(m, s.logq[i]);
        bad = bad || s.id[i] >= vocab;
    }
    float norm = w.lse, z = 1.0f;
    if (!t.tail) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        m = safe_max(m);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            z += expf(s.logq[i] - m);
        z = warp_sum(z);
        norm = z == 0.0f ? 0.0f : m + logf(z);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        s.logq[i] -= norm;
        s.q[i] = expf(s.logq[i]);
        sum += s.q[i];
    }
    sum = warp_sum(sum);
    bad = __any_sync(~0u, bad) || !(sum < kInf);
    s.rest = t.tail ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
    s.sum = bad ? __int_as_float(0x7fffffff) : t.tail ? fmaxf(1.0f, sum) : z == 0.0f ? 0.0f : 1.0f;
    return s;
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

// What a row's listed tokens in a CTA's part add to the row.
struct Listed {
    float m, z;     // their statistics
    float q, dot;   // sum of q over the entries, sum of q (x - m) / 4
};

struct Shared {
    Listed listed;
    Stat part[kWarps];
    Stat mine;                  // this CTA's sums, read by the others of the cluster
    float sum, rest, qlogq;     // of the teacher's row
    int32_t ids[FO_MAX_TOP_K];
    float q[FO_MAX_TOP_K];
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// m, z pairs joined over a warp: the largest m, and z at that.
__device__ __forceinline__ float2 join_pairs(float m, float z, const LogitRows &in)
{
    float top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    return make_float2(top, warp_sum(z * exp2_approx(distance(m, safe_max(top), in) * in.c)));
}

// The elements that `mask` has a bit for become -inf.
template <class T>
__device__ __forceinline__ uint4 without(uint4 v, uint32_t mask)
{
    typename T::raw *e = reinterpret_cast<typename T::raw *>(&v);
#pragma unroll
    for (int k = 0; k < T::kPerVec; ++k)
        if (mask >> k & 1)
            e[k] = T::narrow(-kInf);
    return v;
}

// All threads of the CTA, from different places in the code.
__device__ __forceinline__ void block_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// One row by a cluster of CTAs (one CTA for short rows). A first pass sums the
// exponentials, a second writes the gradient; it reads the row again, but from
// the L2 cache: the launch keeps the rows at work at once well below its size.
// With kTail the rest of the student's mass is summed over the tokens that are
// not listed, which a byte for each vector in shared memory marks: 1 - sum p
// would lose a small rest. That sum also keeps a reference of its own: it may
// lie further below the listed logits than FP32's exponents reach.
template <class T, bool kTail>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) distill_kernel(DistillArgs a)
{
    typedef typename T::raw raw;
    extern __shared__ __align__(16) unsigned char marks[];
    __shared__ __align__(16) Shared sh;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t r = blockIdx.x / size;
    const Row<T> row(a.in, r);
    const Part p = part_of(row, rank, size);
    const float weight = a.weight ? a.weight[r] : 1.0f;
    raw *g = static_cast<raw *>(a.grad.data);
    int lo = row.vecs, hi = 0;   // vectors that are stored whole
    if (g) {
        g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
        if (same_phase(row, g)) {
            lo = row.full0;
            hi = row.full1;
        }
    }
    if (weight == 0.0f) {   // the same in all CTAs of the cluster
        if (rank == 0 && tid == 0 && a.loss)
            a.loss[r] = 0.0f;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int i = p.v0 + tid; g && i < p.v0 + p.n; i += kThreads) {
            if (i >= lo && i < hi)
                store_stream(g + row.id(i, 0), zero);
            else
                store_edge<T>(g, row, i, zero);
        }
        return;
    }
    if (kTail) {
        for (int i = tid; i < (p.n + 15) / 16; i += kThreads)
            reinterpret_cast<uint4 *>(marks)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    const int end = p.v0 + p.n;
    int32_t mine[kSlots];   // entry warp: listed tokens in the part
    float x[kSlots];
    Stat s = {-kInf, 0.0f, 0.0f};
    if (tid >= kStream) {
        const TeacherRaw w = load_teacher(a.teacher, r);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            mine[i] = -1;
            x[i] = -kInf;
            if (w.id[i] < max(0, row.id(p.v0, 0)) || w.id[i] >= min(row.vocab, row.id(end, 0)))
                continue;
            mine[i] = w.id[i];
            x[i] = T::widen(row.x[w.id[i]]);
        }
        if (kTail) {
#pragma unroll
            for (int i = 0; i < kSlots; ++i)
                if (mine[i] >= 0) {
                    const int at = mine[i] + row.phase - p.v0 * T::kPerVec, byte = at / T::kPerVec;
                    atomicOr(reinterpret_cast<uint32_t *>(marks) + byte / 4, 1u << (byte % 4 * 8 + at % T::kPerVec));
                }
            block_barrier();
        }
        const TeacherRow t = make_teacher(a.teacher, w, row.vocab);
        float ql = 0.0f, m = -kInf;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            sh.ids[lane + 32 * i] = t.id[i];
            sh.q[lane + 32 * i] = t.q[i];
            ql += t.q[i] > 0.0f ? t.q[i] * t.logq[i] : 0.0f;
            m = fmaxf(m, x[i]);
        }
        __syncwarp();
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        Listed l = {m, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (mine[i] < 0)
                continue;
            if (t.q[i] > 0.0f) {
                l.q += t.q[i];
                l.dot = __fmaf_rn(t.q[i], quarter_distance(x[i], m), l.dot);
            }
            if (kTail) {   // each token once
                bool first = true;
                for (int j = 0; j < lane + 32 * i; ++j)
                    first = first && sh.ids[j] != mine[i];
                if (first)   // NaN for NaN and +inf
                    l.z += x[i] - x[i] == 0.0f || x[i] == -kInf ? exp2_approx(distance(x[i], safe_max(m), a.in) * a.in.c) : x[i] - x[i];
            }
        }
        l.z = warp_sum(l.z);
        l.q = warp_sum(l.q);
        l.dot = warp_sum(l.dot);
        ql = warp_sum(ql);
        if (lane == 0) {
            sh.listed = l;
            sh.sum = t.sum;
            sh.rest = t.rest;
            sh.qlogq = ql;
        }
    } else {
        if (kTail)
            block_barrier();
        Running<T, false> run;
        for (int i0 = p.v0; i0 < end; i0 += kGroupStep) {
            const int i = i0 + tid;
            if (i0 >= row.full0 && i0 + kGroupStep <= min(end, row.full1)) {
                uint4 v[kGroup];
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    v[j] = *row.vec(i + j * kStream);
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    if (kTail) {
                        const uint32_t mask = marks[i - p.v0 + j * kStream];
                        if (mask)
                            v[j] = without<T>(v[j], mask);
                    }
                    run.add(v[j], a.in);
                }
            } else {
#pragma unroll 1
                for (int j = i; j < min(end, i0 + kGroupStep); j += kStream)
                    run.add(without<T>(load_vec(row, j), kTail ? marks[j - p.v0] : 0u), a.in);
            }
        }
        s = warp_join<false>(run.stat(a.in), a.in);
        if (lane == 0)
            sh.part[tid >> 5] = s;
    }
    block_barrier();
    s = warp_join<false>(sh.part[lane % kWarps], a.in, kWarps);
    Listed l = sh.listed;
    if (size > 1) {
        if (tid == 0)
            sh.mine = s;
        cluster_arrive();
        cluster_wait();
        const uint32_t at = map_shared(&sh.mine, lane % size), from = map_shared(&sh.listed, lane % size);
        const bool once = lane < (int)size;
        const float2 v = join_pairs(ld_cluster_f32(at), once ? ld_cluster_f32(at + 4) : 0.0f, a.in);
        s = Stat{v.x, v.y, 0.0f};
        const float4 u = ld_cluster_f4(from);
        const float2 lz = join_pairs(u.x, once ? u.y : 0.0f, a.in);
        l.m = lz.x;
        l.z = lz.y;
        l.q = warp_sum(once ? u.z : 0.0f);
        l.dot = warp_sum(once && u.z != 0.0f ? __fmaf_rn(u.z, quarter_distance(u.x == -kInf ? 0.0f : u.x, l.m), u.w) : 0.0f);
        cluster_arrive();   // what was read here is free to go; the wait is at the end
    }
    // of all tokens (without tail the listed ones are in s already); m_rest and z_rest of those that are not listed
    const float m = kTail ? fmaxf(s.m, l.m) : s.m, mm = safe_max(m), m_rest = safe_max(s.m);
    const float down = exp2_approx(distance(s.m, mm, a.in) * a.in.c);
    const float z = kTail ? __fmaf_rn(s.z, down, l.z * exp2_approx(distance(l.m, mm, a.in) * a.in.c)) : s.z;
    const float inv_z = z == 0.0f ? 0.0f : 1.0f / z, sum = sh.sum, q_rest = sh.rest;
    // an unlisted token: p - q_rest p / p_rest, by 2^((x - m_rest) c)
    const float f = __fsub_rn(down * (sum * inv_z), !kTail || s.z == 0.0f ? 0.0f : q_rest / s.z);
    if (g) {
        const float scale = weight * a.in.inv_t;
        const f2 nm = splat(-m_rest), ff = splat(f * (scale / T::kShift));
        if (tid < kStream) {
            for (int i0 = p.v0; i0 < end; i0 += kGroupStep) {
                const int i = i0 + tid;
                if (i0 >= max(lo, row.full0) && i0 + kGroupStep <= min(end, hi)) {
                    uint4 v[kGroup];
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
                        v[j] = __ldcs(row.vec(i + j * kStream));
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
                        store_stream(g + row.id(i + j * kStream, 0), grad_vec<T>(v[j], nm, ff, a.in));
                } else {
#pragma unroll 1
                    for (int j = i; j < min(end, i0 + kGroupStep); j += kStream) {
                        const uint4 v = grad_vec<T>(load_vec(row, j), nm, ff, a.in);
                        if (j >= lo && j < hi)
                            store_stream(g + row.id(j, 0), v);
                        else
                            store_edge<T>(g, row, j, v);
                    }
                }
            }
        }
        block_barrier();
        if (tid >= kStream) {   // the listed tokens' places once more; the first of equal ids takes the weight of all
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                if (mine[i] < 0)
                    continue;
                float q = 0.0f;
                bool first = true;
                for (int j = 0; j < a.teacher.k; ++j)
                    if (sh.ids[j] == mine[i]) {
                        q += sh.q[j];
                        first = first && j >= lane + 32 * i;
                    }
                if (first)
                    g[mine[i]] = T::narrow(z == 0.0f ? 0.0f : grad_listed<T>(x[i], mm, q, sum, inv_z, scale, a.in));
            }
        }
    }
    if (rank == 0 && tid == 0) {
        // KL = sum q ln q - sum q s + (sum q) ln Z, and the rest's term
        const float ln_z = logf(z), four = 4.0f * a.in.inv_t;
        float kl = sh.qlogq;
        if (l.q != 0.0f)
            kl = __fmaf_rn(-four, __fmaf_rn(l.q, quarter_distance(l.m == -kInf ? 0.0f : l.m, m), l.dot), __fmaf_rn(l.q, ln_z, kl));
        if (z == 0.0f && sum != 0.0f)
            kl = kInf;
        if (kTail && q_rest > 0.0f)
            kl = s.z == 0.0f ? kInf : kl + q_rest * (logf(q_rest) - (__fmaf_rn(quarter_distance(s.m, m), four, logf(s.z)) - ln_z));
        if (sum != sum || z != z)
            kl = __int_as_float(0x7fffffff);
        if (a.loss)
            a.loss[r] = kl * weight;
        if (a.stats)
            a.stats[r] = make_float4(m, z, s.m, f);
    }
    if (size > 1)
        cluster_wait();   // no CTA leaves while another reads its shared memory
}

// The gradient from saved statistics.
template <class T, int kVecs>
__global__ void __launch_bounds__(kGradThreads) distill_grad_kernel(DistillGradArgs a, int chunks)
{
    typedef typename T::raw raw;
    __shared__ int32_t ids[FO_MAX_TOP_K];
    __shared__ float qs[FO_MAX_TOP_K], sum_q;
    const int64_t r = blockIdx.x / (unsigned)chunks;
    const int v0 = (int)(blockIdx.x % (unsigned)chunks) * (kVecs * kGradThreads);
    const Row<T> row(a.in, r);
    raw *g = static_cast<raw *>(a.out.data) + row_offset(a.in, r, a.out.row_stride, a.out.outer_stride);
    const int tid = threadIdx.x;
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = v0 + i * kGradThreads + tid;
        if (at < row.vecs)
            v[i] = load_vec(row, at);
    }
    if (tid < 32) {
        const TeacherRow t = make_teacher(a.teacher, load_teacher(a.teacher, r), row.vocab);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            ids[tid + 32 * i] = t.id[i];
            qs[tid + 32 * i] = t.q[i];
        }
        if (tid == 0)
            sum_q = t.sum;
    }
    const float gl = a.g_loss[r];
    const float4 st = gl == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : a.stats[r];
    __syncthreads();
    const float inv_z = st.y == 0.0f ? 0.0f : 1.0f / st.y, scale = gl * a.in.inv_t;
    const bool zero = st.y == 0.0f;
    bool entry = false;   // the first of equal ids takes the weight of all
    float entry_value = 0.0f;
    if (!zero && tid < a.teacher.k) {
        const int32_t id = ids[tid];
        if (id >= max(0, row.id(v0, 0)) && id < min(row.vocab, row.id(v0 + kVecs * kGradThreads, 0))) {
            float q = 0.0f;
            entry = true;
            for (int i = 0; i < a.teacher.k; ++i)
                if (ids[i] == id) {
                    q += qs[i];
                    entry = entry && i >= tid;
                }
            entry_value = grad_listed<T>(T::widen(row.x[id]), safe_max(st.x), q, sum_q, inv_z, scale, a.in);
        }
    }
    __syncthreads();   // the entries' logits are read before a gradient in their place is written
    const bool aligned = same_phase(row, g);
    const f2 nm = splat(-safe_max(st.z)), f = splat(st.w * (scale / T::kShift));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = v0 + i * kGradThreads + tid;
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
        g[ids[tid]] = T::narrow(entry_value);
}

template <class T>
cudaError_t launch(const DistillArgs &a, cudaStream_t stream)
{
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw), ctas = (int64_t)sm_count() * kCtasPerSm;
    // one CTA a row, or a cluster that shares it: while the rows at work at
    // once would not stay in the L2 cache between the passes, and while the
    // grid would leave SMs short of CTAs
    int size = 1;
    while (size < kMaxCluster && ((a.grad.data && bytes * (ctas / size) > kCacheBytes) || (a.in.rows * size < ctas && bytes > size * 8192)))
        size *= 2;
    if (a.teacher.tail)
        return launch_cluster(distill_kernel<T, true>, a, a.in.rows, size, (part_vecs(bytes, size) + 15) / 16 * 16, kThreads, stream);
    return launch_cluster(distill_kernel<T, false>, a, a.in.rows, size, 0, kThreads, stream);
}

template <class T>
cudaError_t launch(const DistillGradArgs &a, cudaStream_t stream)
{
    const int64_t vecs = a.in.vocab / T::kPerVec + 2;
    if (vecs * a.in.rows >= (int64_t)sm_count() * 8 * kGradThreads * 8) {
        const int64_t chunks = (vecs + 8 * kGradThreads - 1) / (8 * kGradThreads);
        distill_grad_kernel<T, 8><<<(unsigned)(chunks * a.in.rows), kGradThreads, 0, stream>>>(a, (int)chunks);
    } else {
        const int64_t chunks = (vecs + kGradThreads - 1) / kGradThreads;
        distill_grad_kernel<T, 1><<<(unsigned)(chunks * a.in.rows), kGradThreads, 0, stream>>>(a, (int)chunks);
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
