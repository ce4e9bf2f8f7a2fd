// fo_distill.cu -- distillation from a teacher's top logits: loss, and its
// gradient in the same pass or from saved statistics.
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kConsumers = 256;                   // threads that sum and write the gradient
constexpr int kWarps = kConsumers / 32;
constexpr int kFetcher = kWarps, kJoiner = kWarps + 1;   // two warps more: see distill_kernel
constexpr int kThreads = kConsumers + 64;
constexpr int kMaxBuffers = 3;
constexpr int kTurns = 4;                         // rows whose sums may be on their way
constexpr int kGradThreads = 256;
constexpr int64_t kPartBytes = 36 * 1024;
constexpr int64_t kSharedBytes = 212 * 1024;      // for parts, in one CTA
constexpr int kMaxRowsEach = 16;
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

// What the fetching warp hands over with a part.
struct Entries {
    int32_t id[FO_MAX_TOP_K];   // a listed token of the part, each once; -1: none
    float x[FO_MAX_TOP_K];      // its logit
    float q[FO_MAX_TOP_K];      // the weight of all entries that list it
    float part_q[FO_MAX_TOP_K]; // the weight of this entry, 0 outside the part
    float weight, sum, rest, qlogq;
};

// What the joining warp hands to those that write the gradient.
struct Coefficients {
    float m_rest, f;            // an unlisted token: f 2^((x - m_rest) c)
    float m, inv_z;             // a listed one: p = 2^((x - m) c) inv_z
};

struct Shared {
    uint64_t full[kMaxBuffers], ready[kMaxBuffers], empty[kMaxBuffers];
    uint64_t stats[kTurns], joined[kTurns], written;
    Listed listed[kTurns][kMaxCluster];               // of all CTAs of the cluster,
    float2 rest[kTurns][kMaxCluster * kWarps];        // m, z of their warps: written by each CTA into all
    Coefficients co[kTurns];
    Entries entries[kMaxBuffers];
    int32_t ids[FO_MAX_TOP_K];                        // for rows that list an id twice
    float q[FO_MAX_TOP_K];
};

// A buffer of a ring and how often it has been used, modulo 2.
struct Cursor {
    int at = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++at == n) {
            at = 0;
            turn ^= 1;
        }
    }
};

// The listed tokens of a part that has arrived: their logits are replaced by
// -inf, so that what is summed after is the rest alone. By one warp.
template <class T>
__device__ __forceinline__ void take_entries(const Row<T> &row, const Part &p, uint4 *buf, const TeacherRow &t, int k, Shared &sh, Entries &out)
{
    typedef typename T::raw raw;
    raw *e = reinterpret_cast<raw *>(buf);
    const int lane = threadIdx.x & 31;
    int place[kSlots];
    float x[kSlots], q[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        place[i] = -1;
        x[i] = 0.0f;
        q[i] = t.q[i];
        if (t.id[i] < 0 || t.id[i] >= row.vocab)
            continue;
        const int at = t.id[i] + row.phase - p.v0 * T::kPerVec;
        if (at >= 0 && at < p.n * T::kPerVec) {
            place[i] = at;
            x[i] = T::widen(e[at]);
        }
    }
    __syncwarp();
    // one entry of each token: whoever's number stands in the token's place
    constexpr bool k16 = sizeof(raw) == 2;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
        if (place[i] >= 0) {
            if (k16)
                reinterpret_cast<uint16_t *>(e)[place[i]] = (uint16_t)(lane + 32 * i);
            else
                reinterpret_cast<uint32_t *>(e)[place[i]] = (uint32_t)(lane + 32 * i);
        }
    __syncwarp();
    bool mine[kSlots], twice = false;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        mine[i] = place[i] >= 0 && (k16 ? reinterpret_cast<uint16_t *>(e)[place[i]] : reinterpret_cast<uint32_t *>(e)[place[i]]) ==
                                       (uint32_t)(lane + 32 * i);
        twice = twice || (place[i] >= 0 && !mine[i]);
    }
    if (__any_sync(~0u, twice)) {   // q of equal ids is added up in their order
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            sh.ids[lane + 32 * i] = t.id[i];
            sh.q[lane + 32 * i] = t.q[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (mine[i]) {
                q[i] = 0.0f;
                for (int j = 0; j < k; ++j)
                    if (sh.ids[j] == t.id[i])
                        q[i] += sh.q[j];
            }
    }
    __syncwarp();
    float ql = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (mine[i])
            e[place[i]] = T::narrow(-kInf);
        out.id[lane + 32 * i] = mine[i] ? t.id[i] : -1;
        out.x[lane + 32 * i] = x[i];
        out.q[lane + 32 * i] = q[i];
        out.part_q[lane + 32 * i] = place[i] >= 0 ? t.q[i] : 0.0f;
        ql += t.q[i] > 0.0f ? t.q[i] * t.logq[i] : 0.0f;
    }
    ql = warp_sum(ql);
    if (lane == 0) {
        out.sum = t.sum;
        out.rest = t.rest;
        out.qlogq = ql;
    }
}

// The sums over the entries in a part, in every lane of a warp.
__device__ __forceinline__ Listed sum_entries(const Entries &en, const LogitRows &in)
{
    const int lane = threadIdx.x & 31;
    float x[kSlots], m = -kInf;
    bool mine[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        x[i] = en.x[lane + 32 * i];
        mine[i] = en.id[lane + 32 * i] >= 0;
        if (mine[i])
            m = fmaxf(m, x[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    Listed l = {m, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const float q = en.part_q[lane + 32 * i];
        if (mine[i])   // NaN for NaN and +inf
            l.z += x[i] - x[i] == 0.0f || x[i] == -kInf ? exp2_approx(distance(x[i], safe_max(m), in) * in.c) : x[i] - x[i];
        if (q > 0.0f) {
            l.q += q;
            l.dot = __fmaf_rn(q, quarter_distance(x[i], m), l.dot);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        l.z += __shfl_xor_sync(~0u, l.z, o);
        l.q += __shfl_xor_sync(~0u, l.q, o);
        l.dot += __shfl_xor_sync(~0u, l.dot, o);
    }
    return l;
}

// Rows by a cluster of CTAs, each holding a part of a row in shared memory:
// logits are read from device memory once, for the loss and the gradient. In
// each CTA
//   - a warp fetches parts, by bulk copies, ahead of the others, and takes the
//     listed tokens out of them;
//   - eight warps sum the rest and send their sums to all CTAs of the cluster;
//     then they write the gradient of the row before from shared memory, whose
//     sums have been joined meanwhile;
//   - a warp sends the listed tokens' sums, joins all, and writes the loss.
// The rest is summed, not taken as 1 - sum p, which would lose a small one;
// and it keeps a reference of its own: it may lie further below the listed
// logits than FP32's exponents reach.
template <class T>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(DistillArgs a)
{
    typedef typename T::raw raw;
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ Shared sh;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = (int64_t)(blockIdx.x / size) * a.rows_each, last = min(a.in.rows, first + a.rows_each);
    uint4 *const parts = reinterpret_cast<uint4 *>(dynamic);
    if (tid == 0) {
        for (int i = 0; i < kMaxBuffers; ++i) {
            barrier_init(&sh.full[i], 1);
            barrier_init(&sh.ready[i], 1);
            barrier_init(&sh.empty[i], kWarps + 1);
        }
        for (int i = 0; i < kTurns; ++i) {
            barrier_init(&sh.stats[i], size * (kWarps + 1));
            barrier_init(&sh.joined[i], 1);
        }
        barrier_init(&sh.written, kWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (size > 1) {   // the barriers are there before another CTA's sums come
        cluster_arrive();
        cluster_wait();
    } else
        __syncthreads();

    bool ok = true;   // false: a wait ran out
    if (warp == kFetcher) {
        Cursor c;
        uint32_t full_turn = 0;   // a bit for each buffer
        float weight = a.weight ? a.weight[first] : 1.0f;
        TeacherRaw raw_teacher = load_teacher(a.teacher, first);
        for (int64_t r = first; r < last && ok; ++r, c.next(a.buffers)) {
            uint4 *const buf = parts + c.at * a.buffer_vecs;
            const Row<T> row(a.in, r);
            const Part p = part_of(row, rank, size);
            ok = warp_wait(&sh.empty[c.at], c.turn ^ 1);
            const bool use = weight != 0.0f && ok;
            if (use) {
                // the last row's stores to this buffer come before the copies of this one
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                load_part<T>(row, p, buf, &sh.full[c.at]);
            }
            const float this_weight = weight;
            const TeacherRaw w = raw_teacher;
            if (r + 1 < last) {   // on their way while this row's logits come
                weight = a.weight ? a.weight[r + 1] : 1.0f;
                raw_teacher = load_teacher(a.teacher, r + 1);
            }
            if (use) {
                const TeacherRow t = make_teacher(a.teacher, w, row.vocab);
                ok = warp_wait(&sh.full[c.at], (full_turn >> c.at) & 1);
                full_turn ^= 1u << c.at;
                __syncwarp();
                take_entries<T>(row, p, buf, t, a.teacher.k, sh, sh.entries[c.at]);
            }
            if (lane == 0)
                sh.entries[c.at].weight = this_weight;
            __syncwarp();
            if (lane == 0 && ok)
                barrier_arrive(&sh.ready[c.at]);
        }
        if (!ok)   // copies that are still on their way are not left behind
            for (int i = 0; i < a.buffers; ++i)
                barrier_wait(&sh.full[i], (full_turn >> i) & 1);
    } else if (warp == kJoiner) {
        Cursor c;
        uint32_t active = 0;   // rows whose sums have been exchanged
        for (int64_t r = first; r < last; ++r, c.next(a.buffers)) {
            const Entries &en = sh.entries[c.at];
            ok = ok && warp_wait(&sh.ready[c.at], c.turn);
            const float weight = en.weight;
            const bool writes = (uint32_t)r % size == rank && lane == 0;   // the loss, in turn
            if (!ok || weight == 0.0f) {   // the same in all CTAs of the cluster
                if (writes && a.loss)
                    a.loss[r] = ok ? 0.0f : __int_as_float(0x7fffffff);
            } else {
                const int turn = active % kTurns;
                const Listed own = sum_entries(en, a.in);
                if (size == 1) {
                    if (lane == 0) {
                        sh.listed[turn][0] = own;
                        barrier_arrive(&sh.stats[turn]);
                    }
                } else if (lane < (int)size) {
                    const uint32_t at = map_shared(&sh.listed[turn][rank], lane);
                    st_cluster(at, own.m, own.z);
                    st_cluster(at + 8, own.q, own.dot);
                    fence_cluster();
                    arrive_cluster(map_shared(&sh.stats[turn], lane));
                }
                ok = warp_wait(&sh.stats[turn], (active / kTurns) & 1);
                if (size > 1)
                    fence_cluster();
                ++active;
                // the rest: two of the warps' sums a lane, of one reference first
                float2 u = make_float2(-kInf, 0.0f), v = u;
                if (lane < (int)size * kWarps)
                    u = sh.rest[turn][lane];
                if (lane + 32 < (int)size * kWarps)
                    v = sh.rest[turn][lane + 32];
                const Listed l = lane < (int)size ? sh.listed[turn][lane] : Listed{-kInf, 0.0f, 0.0f, 0.0f};
                float mr = fmaxf(u.x, v.x), ml = l.m;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    mr = fmaxf(mr, __shfl_xor_sync(~0u, mr, o));
                    ml = fmaxf(ml, __shfl_xor_sync(~0u, ml, o));
                }
                const float m = fmaxf(mr, ml), mm = safe_max(m), mrr = safe_max(mr);
                // exponentials of -160 powers of two and less are 0
                float zr = u.y * exp2_approx(distance(u.x, mrr, a.in) * a.in.c) + v.y * exp2_approx(distance(v.x, mrr, a.in) * a.in.c);
                float zl = l.z * exp2_approx(distance(l.m, mm, a.in) * a.in.c);
                float qs = l.q, dot = l.q != 0.0f ? __fmaf_rn(l.q, quarter_distance(l.m == -kInf ? 0.0f : l.m, m), l.dot) : 0.0f;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    zr += __shfl_xor_sync(~0u, zr, o);
                    zl += __shfl_xor_sync(~0u, zl, o);
                    qs += __shfl_xor_sync(~0u, qs, o);
                    dot += __shfl_xor_sync(~0u, dot, o);
                }
                const float down = exp2_approx(distance(mr, mm, a.in) * a.in.c);
                const float z = __fmaf_rn(zr, down, zl), inv_z = z == 0.0f ? 0.0f : 1.0f / z;
                const float sum = ok ? en.sum : __int_as_float(0x7fffffff), q_rest = en.rest;
                // an unlisted token: p - q_rest p / p_rest, by 2^((x - m_rest) c)
                const float f = __fsub_rn(down * (sum * inv_z), zr == 0.0f ? 0.0f : q_rest / zr);
                if (lane == 0) {
                    sh.co[turn] = Coefficients{mrr, f, mm, inv_z};
                    barrier_arrive(&sh.joined[turn]);
                }
                if (writes) {
                    // KL = sum q ln q - sum q s + (sum q) ln Z, and the rest's term
                    const float ln_z = logf(z);
                    float kl = en.qlogq;
                    if (qs != 0.0f)
                        kl = __fmaf_rn(dot, -4.0f * a.in.inv_t, __fmaf_rn(qs, ln_z, kl));
                    if (z == 0.0f && sum != 0.0f)
                        kl = kInf;
                    if (q_rest > 0.0f)
                        kl = zr == 0.0f ? kInf : kl + q_rest * (logf(q_rest) - (__fmaf_rn(quarter_distance(mr, m), 4.0f * a.in.inv_t, logf(zr)) - ln_z));
                    if (sum != sum || z != z)
                        kl = __int_as_float(0x7fffffff);
                    if (a.loss)
                        a.loss[r] = kl * weight;
                    if (a.stats)
                        a.stats[r] = make_float4(m, z, mr, f);
                }
            }
            __syncwarp();
            if (lane == 0)
                barrier_arrive(&sh.empty[c.at]);
        }
    } else {
        Cursor c, d;                            // of the row that is summed, of the one whose gradient is written
        uint32_t summed = 0, done = 0, full_turn = 0;
        const bool has_grad = a.grad.data != nullptr;
        const int lag = a.buffers > 1 && has_grad ? 1 : 0;
        for (int64_t r = first; r < last + lag; ++r) {
            if (r < last) {
                const uint4 *const buf = parts + c.at * a.buffer_vecs;
                const Part p = part_of(Row<T>(a.in, r), rank, size);
                ok = ok && warp_wait(&sh.ready[c.at], c.turn);
                if (ok && sh.entries[c.at].weight != 0.0f) {
                    ok = warp_wait(&sh.full[c.at], (full_turn >> c.at) & 1);
                    full_turn ^= 1u << c.at;
                    Running<T, false> run;
#pragma unroll 2
                    for (int i = tid; i < p.n; i += kConsumers)
                        run.add(buf[i], a.in);
                    const Stat part = warp_join<false>(run.stat(a.in), a.in);
                    const int turn = summed++ % kTurns, slot = rank * kWarps + warp;
                    if (size == 1) {
                        if (lane == 0) {
                            sh.rest[turn][slot] = make_float2(part.m, part.z);
                            barrier_arrive(&sh.stats[turn]);
                        }
                    } else if (lane < (int)size) {
                        st_cluster(map_shared(&sh.rest[turn][slot], lane), part.m, part.z);
                        fence_cluster();
                        arrive_cluster(map_shared(&sh.stats[turn], lane));
                    }
                }
                if (!has_grad) {
                    __syncwarp();
                    if (lane == 0)
                        barrier_arrive(&sh.empty[c.at]);
                }
                c.next(a.buffers);
            }
            if (!has_grad || r < first + lag)
                continue;
            const uint4 *const buf = parts + d.at * a.buffer_vecs;
            const Entries &en = sh.entries[d.at];
            const Row<T> row(a.in, r - lag);
            const Part p = part_of(row, rank, size);
            raw *const g = static_cast<raw *>(a.grad.data) + row_offset(a.in, r - lag, a.grad.row_stride, a.grad.outer_stride);
            const bool aligned = same_phase(row, g);
            if (ok && en.weight == 0.0f) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int i = tid; i < p.n; i += kConsumers) {
                    const int at = p.v0 + i;
                    if (aligned && at >= row.full0 && at < row.full1)
                        store_stream(g + row.id(at, 0), zero);
                    else
                        store_edge<T>(g, row, at, zero);
                }
            } else if (ok) {
                const int turn = done % kTurns;
                ok = warp_wait(&sh.joined[turn], (done / kTurns) & 1);
                const Coefficients co = sh.co[turn];
                const float scale = en.weight * a.in.inv_t;
                const f2 nm = splat(-co.m_rest), f = splat(co.f * (scale / T::kShift));
#pragma unroll 2
                for (int i = tid; i < p.n; i += kConsumers) {
                    const int at = p.v0 + i;
                    const uint4 v = grad_vec<T>(buf[i], nm, f, a.in);
                    if (aligned && at >= row.full0 && at < row.full1)
                        store_stream(g + row.id(at, 0), v);
                    else
                        store_edge<T>(g, row, at, v);
                }
                // the listed tokens' places once more, after the vectors
                __syncwarp();
                if (lane == 0)
                    barrier_arrive(&sh.written);
                if (warp < kSlots)
                    ok = warp_wait(&sh.written, done & 1) && ok;
                ++done;
                if (tid < FO_MAX_TOP_K && en.id[tid] >= 0)
                    g[en.id[tid]] = T::narrow(co.inv_z == 0.0f ? 0.0f : grad_listed<T>(en.x[tid], co.m, en.q[tid], en.sum, co.inv_z, scale, a.in));
            }
            __syncwarp();
            if (lane == 0)
                barrier_arrive(&sh.empty[d.at]);
            d.next(a.buffers);
        }
    }
    if (size > 1) {   // no CTA leaves while another may write to it
        cluster_arrive();
        cluster_wait();
    }
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
cudaError_t launch(const DistillArgs &args, cudaStream_t stream)
{
    DistillArgs a = args;
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw), sms = sm_count();
    // the smallest cluster whose parts are at most kPartBytes (three buffers of
    // which leave room for two CTAs on an SM); larger while the grid would
    // leave SMs without a CTA and parts stay above 8 KB
    int size = 1;
    while (size < kMaxCluster && (bytes > size * kPartBytes || (a.in.rows * size < 2 * sms && bytes > size * 8192)))
        size *= 2;
    a.buffer_vecs = (int)part_vecs(bytes, size);
    const int64_t part = a.buffer_vecs * 16;
    a.buffers = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxBuffers, kSharedBytes / part));
    // rows in turn by one cluster, so that fetching runs ahead, as far as the
    // clusters that fit on the GPU at once still get several such groups each
    const int64_t resident = std::max<int64_t>(1, sms * std::min<int64_t>(3, (kSharedBytes + sizeof(Shared)) / (a.buffers * part + sizeof(Shared))) / size);
    a.rows_each = (int)std::min<int64_t>(kMaxRowsEach, std::max<int64_t>(1, a.in.rows / (4 * resident)));
    a.buffers = std::min(a.buffers, a.rows_each);
    const int64_t clusters = (a.in.rows + a.rows_each - 1) / a.rows_each;
    return launch_cluster(distill_kernel<T>, a, clusters, size, a.buffers * part, kThreads, stream);
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
