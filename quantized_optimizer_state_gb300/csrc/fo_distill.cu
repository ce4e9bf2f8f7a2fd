// fo_distill.cu -- distillation from a teacher's top logits: loss, and its
// gradient in the same pass or from saved statistics.
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

// distill_kernel's shape, by measurement on 8192 x 128256 BF16, 8192 x 50257
// BF16 with a tail and 1001 x 128256 FP32 with one, loss with gradient (us): 3
// CTAs an SM of 8 walking warps with 4 stages of 16 KB. 4 CTAs (48 registers,
// spills) with 3 such stages: 809 / 393 / 214 against 709 / 358 / 203 at the
// same rows in turn; 8 stages of 8 KB: 761 / 383 / 224 against 749 / 358 / 202;
// 2 CTAs of 16 warps: 813 / 493 / 212 against 778 / 393 / 225. (Each pair is of
// one build; what came later took 667 / 283 / 194.) Two rows in turn against 1
// and 4: 687 / 279 / 196 against 733 / 287 / 201 and 689 / 282 / 197: the
// fetching runs on into the second row, and short turns spread the grid's end.
constexpr int kLong = 8, kShort = 2;              // warps that walk over a row: see launch
constexpr int kStages = 4;                        // copies of four vectors a thread, in flight or in use
constexpr int kCtasPerSm = 3;                     // of kLong warps; of kShort ones kShortPerSm
constexpr int kShortPerSm = 8;
constexpr int64_t kMaxRowsEach = 2;
// Of the 129 MB L2 cache, for the rows at work between their passes. 78 MB are
// too many: 8192 x 128256 BF16 692 us against 672 in clusters of two (59 MB), 1001
// x 128256 FP32 with a tail 206 in clusters of two against 191 of four; 73 MB are
// not (4096 x 120000 BF16 336 against 354).
constexpr int64_t kCacheBytes = 70 << 20;
constexpr int64_t kOneTurn = 800 << 20;           // bytes of all rows and gradients
constexpr int64_t kShortRow = 32 * 1024;
constexpr int64_t kMaxPart = 146 * 1024;          // bytes of a part: its marks, a 16th of that, leave room for three CTAs
constexpr int64_t kMinPart = 16 * 1024;           // bytes of a row that are worth a CTA of their own
constexpr int kGradThreads = 256;
constexpr float kLn2High = 0x1.62e4p-1f;          // 15 bits of ln 2
constexpr float kLn2Low = (float)(0.69314718055994531 - 0x1.62e4p-1);
// Log probabilities that add up to 1 leave a rest of up to 2^-18 by their own
// roundings (and one at the size of lse), although the list holds all that a
// mask has left. Where the student's rest is 0, in 64 bits too (e^-746), KL would
// be infinite, or as large as the mask's value, for that.
constexpr float kNoRest = 0x1p-16f, kNoLogRest = -746.0f;
constexpr float kNan = __builtin_nanf("");
constexpr int kSlots = FO_MAX_TOP_K / 32;         // entries of a lane of one warp that holds them all

// A teacher's row in one warp: entry lane + 32 i at place i.
struct TeacherRow {
    int32_t id[kSlots];          // -1: none
    float q[kSlots], logq[kSlots];
    float sum;                   // of q and of the rest; NaN where an id is out of range or q is not finite
    float rest;                  // the mass that is not listed (0 without tail)
};

// What it is made from, as loaded: nothing here waits for a load, so that all
// of a row's are on their way at once (places beyond k repeat the first).
struct TeacherRaw {
    int32_t id[kSlots];
    uint32_t bits[kSlots];   // of the logits
    float lse;
};

__device__ __forceinline__ TeacherRaw load_teacher(const Teacher &t, int64_t r)
{
    TeacherRaw w;
    int64_t at[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int e = (int)(threadIdx.x & 31) + 32 * i;
        at[i] = r * t.k + (e < t.k ? e : 0);
        w.id[i] = t.ids[at[i]];
    }
    if (t.dtype == FO_LOGITS_F32) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            w.bits[i] = static_cast<const uint32_t *>(t.logits)[at[i]];
    } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            w.bits[i] = static_cast<const uint16_t *>(t.logits)[at[i]];
    }
    w.lse = t.lse ? t.lse[r] : 0.0f;
    return w;
}

// The id of place i: -1 for none.
__device__ __forceinline__ int32_t id_at(const Teacher &t, const TeacherRaw &w, int i)
{
    return (int)(threadIdx.x & 31) + 32 * i < t.k ? w.id[i] : -1;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// v / T - minus, for the teacher's T: 1 / T has two parts and the difference is
// fused with the product, so that the result is rounded at its own size and not
// at that of v.
__device__ __forceinline__ float over_temperature(const Teacher &t, float v, float minus)
{
    const float d = __fmaf_rn(v, t.inv_t, -minus);
    return fabsf(v) < kInf ? __fmaf_rn(v, t.inv_t_lo, d) : d;   // -inf times the lower part may be +inf
}

// The largest logit is subtracted before anything is rounded: a softmax does not
// depend on where its logits lie, and neither does the precision of q.
__device__ __forceinline__ TeacherRow make_teacher(const Teacher &t, const TeacherRaw &w, int vocab)
{
    TeacherRow s;
    float m = -kInf, logit[kSlots];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        s.id[i] = id_at(t, w, i);
        const float x = t.dtype == FO_LOGITS_F32    ? __uint_as_float(w.bits[i])
                        : t.dtype == FO_LOGITS_BF16 ? Bf16::widen((uint16_t)w.bits[i])
                                                    : F16::widen((uint16_t)w.bits[i]);
        logit[i] = s.id[i] < 0 ? -kInf : x;
        m = fmaxf(m, logit[i]);
        bad = bad || s.id[i] >= vocab;
    }
    float sum = 0.0f, z = 1.0f;
    if (t.tail) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s.logq[i] = over_temperature(t, logit[i], w.lse);
            s.q[i] = expf(s.logq[i]);
            sum += s.q[i];
        }
        sum = warp_sum(sum);
    } else {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        m = safe_max(m);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s.logq[i] = over_temperature(t, logit[i] - m, 0.0f);
            s.q[i] = expf(s.logq[i]);
            z += s.q[i];
        }
        z = warp_sum(z);
        const float ln_z = z == 0.0f ? 0.0f : logf(z), inv_z = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s.logq[i] -= ln_z;
            s.q[i] *= inv_z;
        }
        sum = z;
    }
    bad = __any_sync(~0u, bad) || !(sum < kInf);
    s.rest = t.tail ? fmaxf(0.0f, 1.0f - sum) : 0.0f;
    s.sum = bad ? kNan : t.tail ? fmaxf(1.0f, sum) : z == 0.0f ? 0.0f : 1.0f;
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
    uint64_t full[kStages], empty[kStages];                   // of a stage: copied; used
    uint64_t marked, summed, joined, written;                 // of a row
    uint64_t cluster[2];                                      // all CTAs' sums have come
    float4 sums[2][kMaxCluster];                              // written by each CTA into all: listed m, z, q, dot,
    float2 rests[2][kMaxCluster];                             // and the streamed m, z
    float2 part[kLong];                                       // m, z of the warps
    float m, f;                                               // the gradient: f 2^((x - m) c)
    __align__(16) int32_t ids[FO_MAX_TOP_K];
    float q[FO_MAX_TOP_K];
};

// m, z pairs joined over a warp: the largest m, and z at that.
__device__ __forceinline__ float2 join_pairs(float m, float z, const LogitRows &in)
{
    float top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    return make_float2(top, warp_sum(z * exp2_approx(distance(m, safe_max(top), in) * in.c)));
}

// A byte in shared memory for each vector of a part, with a bit for each of
// its elements that is a listed token.
template <class T>
__device__ __forceinline__ uint32_t mark_bit(const Row<T> &row, const Part &p, int32_t id, int &word)
{
    const int at = id + row.phase - p.v0 * T::kPerVec, byte = at / T::kPerVec;
    word = byte / 4;
    return 1u << (byte % 4 * 8 + at % T::kPerVec);
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

// For lists with a token in two entries, which is rare: the first stands for
// all. q_all: its weight, that of all. By one warp.
__device__ __forceinline__ uint32_t merge_twice(Shared &sh, const TeacherRow &t, int k, const int32_t (&mine)[kSlots], float (&q_all)[kSlots])
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        sh.ids[lane + 32 * i] = t.id[i];
        sh.q[lane + 32 * i] = t.q[i];
    }
    __syncwarp();
    uint32_t again = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        float q = 0.0f;
        for (int j = 0; j < k; ++j)
            if (sh.ids[j] == mine[i]) {
                q += sh.q[j];
                again |= j < lane + 32 * i ? 1u << i : 0u;
            }
        q_all[i] = q;
    }
    return again;
}

// Rows by a cluster of CTAs (one CTA a row for short rows). A first pass over
// a row sums the exponentials, a second writes the gradient,
//   dKL/dx_j = (w/T) [ p_j (A - [j not listed] q_rest / p_rest) - q_j ];
// it reads the row again, but from the L2 cache: the launch keeps the rows at
// work at once well below its size, and the first pass asks it to keep their
// lines, the second to let them go (98 % of the second pass hits; device memory
// gives 1.02 times the logits). 8192 x 128256 BF16: 0.667 ms, 0.90 of the
// measured copy rate for one read and one write (an earlier build took 0.674, and
// 0.689 without these requests).
// It is bound by the mixed traffic: the second pass adds half as much again in
// the L2 cache, which moves 10.2 TB/s, and instructions issue in half of the
// cycles. Rows held in shared memory between the passes were slower (1.02 ms at
// best): their clusters are larger, and each row waits for the exchange of its
// sums with less in flight.
// In each CTA
//   - a warp keeps bulk copies in flight into a ring of stages, running ahead
//     over the passes and rows, so that the memory is not idle while sums are
//     joined;
//   - kWarps warps take the stages, sum, and write the gradient;
//   - a warp reads the teacher's row, joins the sums, in the CTA and over the
//     cluster, and writes the loss and, last, the gradient of the listed
//     tokens.
// With kTail the rest of the student's mass is summed over the tokens that are
// not listed: 1 - sum p would lose a small rest. That sum also keeps a
// reference of its own: it may lie further below the listed logits than FP32's
// exponents reach.
template <class T, bool kTail, int kWarps>
__global__ void __launch_bounds__(kWarps * 32 + 64, kWarps == kLong ? kCtasPerSm : kShortPerSm) distill_kernel(DistillArgs a)
{
    typedef typename T::raw raw;
    constexpr int kStream = kWarps * 32, kFetcher = kWarps, kTeacher = kWarps + 1, kThreads = kStream + 64;
    constexpr int kStageVecs = 4 * kStream;   // vectors that are copied at once
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ __align__(16) Shared sh;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = blockIdx.x / size, step = gridDim.x / size, rows = a.in.rows;   // this cluster's rows
    uint4 *const stages = reinterpret_cast<uint4 *>(dynamic);
    unsigned char *const mark_bytes = dynamic + kStages * kStageVecs * 16;
    uint32_t *const marks = reinterpret_cast<uint32_t *>(mark_bytes);
    for (int i = tid; i < a.mark_words; i += kThreads)
        marks[i] = 0;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            barrier_init(&sh.full[i], 2);
            barrier_init(&sh.empty[i], kWarps);
        }
        barrier_init(&sh.marked, 1);
        barrier_init(&sh.summed, kWarps);
        barrier_init(&sh.joined, 1);
        barrier_init(&sh.written, kWarps);
        for (int i = 0; i < 2; ++i)
            barrier_init(&sh.cluster[i], size);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (size > 1) {   // the barriers are there before another CTA's sums come
        cluster_arrive();
        cluster_wait();
    } else
        __syncthreads();

    const int passes = a.grad.data ? 2 : 1;
    // false: a wait ran out. What the warp has not done of its rows by then, of
    // their sums, losses, statistics and gradients, becomes NaN; the others' waits
    // for it run out in turn.
    bool ok = true;
    uint32_t active = 0;     // rows done with a weight other than 0
    float next_weight = a.weight ? a.weight[first] : 1.0f;
    if (warp == kFetcher) {
        Cursor<kStages> c;
        const uint64_t keep = keep_policy(), drop = drop_policy();
        for (int64_t r = first; r < rows && ok; r += step) {
            const float weight = next_weight;
            if (r + step < rows && a.weight)
                next_weight = a.weight[r + step];
            if (weight == 0.0f)
                continue;
            const Row<T> row(a.in, r);
            const Part p = part_of(row, rank, size);
            for (int pass = 0; pass < passes; ++pass)
                for (int i = 0; i < p.n && ok; i += kStageVecs, c.next()) {
                    ok = warp_wait(&sh.empty[c.at], c.turn ^ 1);
                    // what was stored to this stage comes before the copy to it
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (ok)
                        fill_stage<T>(row, p.v0 + i, p.v0 + min(p.n, i + kStageVecs), stages + c.at * kStageVecs, &sh.full[c.at], pass + 1 < passes ? keep : drop);
                }
        }
        // copies that are still on their way are not left behind
        for (int i = 0; i < kStages && !ok; ++i, c.next())
            barrier_wait(&sh.full[c.at], c.turn ^ 1);
    } else if (warp == kTeacher) {
        int32_t mine[kSlots];   // listed tokens in the part; -2: none
        raw x[kSlots];          // their logits
        bool twice = false;     // a token is in two entries
        const auto start = [&](int64_t r, const TeacherRaw &w) {
            const Row<T> row(a.in, r);
            const Part p = part_of(row, rank, size);
            const int id0 = max(0, row.id(p.v0, 0)), id1 = min(row.vocab, row.id(p.v0 + p.n, 0));
            twice = false;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int32_t id = id_at(a.teacher, w, i);
                mine[i] = id >= id0 && id < id1 ? id : -2;
                x[i] = row.x[max(mine[i], 0)];   // used where there is one
                if (mine[i] >= 0 && a.mark_words) {
                    int word;
                    const uint32_t bit = mark_bit(row, p, mine[i], word), old = atomicOr(marks + word, bit);
                    twice = twice || (old & bit);
                }
            }
            twice = __any_sync(~0u, twice);
            if (lane == 0)
                barrier_arrive(&sh.marked);
        };
        TeacherRaw next = load_teacher(a.teacher, first);
        if (next_weight != 0.0f)
            start(first, next);
        for (int64_t r = first; r < rows; r += step) {
            const float weight = next_weight;
            const TeacherRaw w = next;
            if (r + step < rows) {
                next = load_teacher(a.teacher, r + step);
                if (a.weight)
                    next_weight = a.weight[r + step];
            }
            const bool writes = (uint32_t)r % size == rank && lane == 0;   // the loss, in turn
            if (weight == 0.0f || !ok) {   // the same in all CTAs of the cluster
                if (writes && a.loss)
                    a.loss[r] = ok ? 0.0f : kNan;
                if (writes && a.stats && weight != 0.0f)
                    a.stats[r] = make_float4(kNan, kNan, kNan, kNan);
                if (r + step < rows && next_weight != 0.0f)
                    start(r + step, next);
                continue;
            }
            const TeacherRow t = make_teacher(a.teacher, w, (int)a.in.vocab);
            float q_all[kSlots];
            uint32_t again = 0;   // a bit for the entries beside the one that stands for their token
#pragma unroll
            for (int i = 0; i < kSlots; ++i)
                q_all[i] = t.q[i];
            if (twice)
                again = merge_twice(sh, t, a.teacher.k, mine, q_all);
            Listed l = {-kInf, 0.0f, 0.0f, 0.0f};
            float ql = 0.0f, xf[kSlots];
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                ql += t.q[i] > 0.0f ? t.q[i] * t.logq[i] : 0.0f;
                xf[i] = mine[i] < 0 ? -kInf : T::widen(x[i]);
                l.m = fmaxf(l.m, xf[i]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                l.m = fmaxf(l.m, __shfl_xor_sync(~0u, l.m, o));
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                if (mine[i] < 0)
                    continue;
                if (t.q[i] > 0.0f) {
                    l.q += t.q[i];
                    l.dot = __fmaf_rn(t.q[i], quarter_distance(xf[i], l.m), l.dot);
                }
                if (kTail && !(again >> i & 1))   // NaN for NaN and +inf
                    l.z += xf[i] - xf[i] == 0.0f || xf[i] == -kInf ? exp2_approx(distance(xf[i], safe_max(l.m), a.in) * a.in.c) : xf[i] - xf[i];
            }
            if (kTail)
                l.z = warp_sum(l.z);
            l.q = warp_sum(l.q);
            l.dot = warp_sum(l.dot);
            ql = warp_sum(ql);

            ok = warp_wait(&sh.summed, active & 1);
            float2 s = make_float2(-kInf, 0.0f);
            if (lane < kWarps)
                s = sh.part[lane];
            s = join_pairs(s.x, s.y, a.in);
            if (!ok)   // NaN for the row's other CTAs too
                s.y = kNan;
            if (size > 1) {
                const int turn = active & 1;
                if (lane < (int)size) {
                    const uint32_t at = map_shared(&sh.sums[turn][rank], lane);
                    st_cluster(at, l.m, l.z);
                    st_cluster(at + 8, l.q, l.dot);
                    st_cluster(map_shared(&sh.rests[turn][rank], lane), s.x, s.y);
                    fence_cluster();
                    arrive_cluster(map_shared(&sh.cluster[turn], lane));
                }
                ok = ok && warp_wait(&sh.cluster[turn], (active >> 1) & 1);
                fence_cluster();
                float4 v = make_float4(-kInf, 0.0f, 0.0f, 0.0f);
                s = make_float2(-kInf, 0.0f);
                if (lane < (int)size) {
                    v = sh.sums[turn][lane];
                    s = sh.rests[turn][lane];
                }
                s = join_pairs(s.x, s.y, a.in);
                const float2 lz = join_pairs(v.x, v.y, a.in);
                l.m = lz.x;
                l.z = lz.y;
                l.q = warp_sum(v.z);
                l.dot = warp_sum(v.z != 0.0f ? __fmaf_rn(v.z, quarter_distance(v.x == -kInf ? 0.0f : v.x, l.m), v.w) : 0.0f);
            }
            // s: what was streamed: with kTail the rest alone, else all tokens
            const float m = kTail ? fmaxf(s.x, l.m) : s.x, mm = safe_max(m), m_rest = safe_max(s.x);
            const float down = exp2_approx(distance(s.x, mm, a.in) * a.in.c);
            const float z = kTail ? __fmaf_rn(s.y, down, l.z * exp2_approx(distance(l.m, mm, a.in) * a.in.c)) : s.y;
            const float inv_z = z == 0.0f ? 0.0f : 1.0f / z, sum = ok ? t.sum : kNan;
            const auto ln_rest = [&](float ln_z) {   // ln p_rest
                return s.y == 0.0f ? -kInf : __fmaf_rn(quarter_distance(s.x, m), 4.0f * a.in.inv_t, logf(s.y)) - ln_z;
            };
            float q_rest = t.rest;
            if (kTail && q_rest <= kNoRest && ln_rest(logf(z)) < kNoLogRest)
                q_rest = 0.0f;
            // an unlisted token: p - q_rest p / p_rest, by 2^((x - m_rest) c)
            const float f = __fsub_rn(down * (sum * inv_z), !kTail || s.y == 0.0f ? 0.0f : q_rest / s.y);
            const float scale = weight * a.in.inv_t;
            if (lane == 0) {
                sh.m = m_rest;
                sh.f = f * (scale / T::kShift);
                barrier_arrive(&sh.joined);
            }
            if (writes) {
                // KL = sum q ln q - sum q s + (sum q) ln Z, and the rest's
                // term. ln Z is taken as its power of two, whose product with
                // the upper bits of ln 2 is exact, and a part below 0.41: it
                // cancels most of sum q s, and a rounding of ln Z itself would
                // show in a small loss.
                const float ln_z = logf(z), four = 4.0f * a.in.inv_t;
                float kl = ql;
                if (l.q != 0.0f) {
                    const int k = z > 0.0f && z < kInf ? ilogbf(z * 1.41421356f) : 0;
                    const float low = __fmaf_rn((float)k, kLn2Low, logf(ldexpf(z, -k)));
                    const float qs = four * __fmaf_rn(l.q, quarter_distance(l.m == -kInf ? 0.0f : l.m, m), l.dot);
                    kl = __fadd_rn(__fmaf_rn(l.q, (float)k * kLn2High, -qs), __fmaf_rn(l.q, low, kl));
                }
                if (z == 0.0f && sum != 0.0f)
                    kl = kInf;
                if (kTail && q_rest > 0.0f)
                    kl = s.y == 0.0f ? kInf : kl + q_rest * (logf(q_rest) - ln_rest(ln_z));
                if (sum != sum || z != z)
                    kl = kNan;
                if (a.loss)
                    a.loss[r] = kl * weight;
                if (a.stats)
                    a.stats[r] = make_float4(m, z, s.x, f);
            }
            int32_t done[kSlots];   // this row's, while the next is started
            const Row<T> row(a.in, r);
            const Part p = part_of(row, rank, size);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                done[i] = mine[i];
                if (mine[i] >= 0 && a.mark_words) {   // every warp has summed: the marks go
                    int word;
                    mark_bit(row, p, mine[i], word);
                    marks[word] = 0;
                }
            }
            __syncwarp();
            if (r + step < rows && next_weight != 0.0f)
                start(r + step, next);
            if (passes == 2) {
                ok = ok && warp_wait(&sh.written, active & 1);
                raw *const g = static_cast<raw *>(a.grad.data) + row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
#pragma unroll
                for (int i = 0; i < kSlots; ++i)   // the listed tokens' places once more, after the vectors
                    if (done[i] >= 0 && !(again >> i & 1))
                        g[done[i]] = T::narrow(!ok ? kNan : z == 0.0f ? 0.0f : grad_listed<T>(xf[i], mm, q_all[i], sum, inv_z, scale, a.in));
            }
            ++active;
        }
    } else {
        Cursor<kStages> c;
        for (int64_t r = first; r < rows; r += step) {
            const float weight = next_weight;
            if (r + step < rows && a.weight)
                next_weight = a.weight[r + step];
            const Row<T> row(a.in, r);
            const Part p = part_of(row, rank, size);
            raw *g = static_cast<raw *>(a.grad.data);
            int lo = row.vecs, hi = 0;   // vectors that are stored whole
            if (g) {
                g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
                if (same_phase(row, g)) {
                    lo = row.full0;
                    hi = row.full1;
                }
            }
            const auto write = [&](int i, const uint4 &v) {
                if (i >= lo && i < hi)
                    store_stream(g + row.id(i, 0), v);
                else
                    store_edge<T>(g, row, i, v);
            };
            if (weight == 0.0f) {
                for (int i = p.v0 + tid; g && i < p.v0 + p.n; i += kStream)
                    write(i, make_uint4(0, 0, 0, 0));
                continue;
            }
            if (kTail)
                ok = ok && warp_wait(&sh.marked, active & 1);
            Running<T, false> run;
            for (int i0 = 0; i0 < p.n && ok; i0 += kStageVecs, c.next()) {
                ok = warp_wait(&sh.full[c.at], c.turn);
                const uint4 *const stage = stages + c.at * kStageVecs;
                if (i0 + kStageVecs <= p.n) {
                    uint4 v[kStageVecs / kStream];
#pragma unroll
                    for (int j = 0; j < kStageVecs / kStream; ++j)
                        v[j] = stage[tid + j * kStream];
#pragma unroll
                    for (int j = 0; j < kStageVecs / kStream; ++j) {
                        const uint32_t mask = kTail ? mark_bytes[i0 + j * kStream + tid] : 0u;
                        if (kTail && mask)
                            v[j] = without<T>(v[j], mask);
                    }
                    run.add(v, a.in);
                } else
                    for (int i = tid; i < p.n - i0; i += kStream)
                        run.add(without<T>(stage[i], kTail ? mark_bytes[i0 + i] : 0u), a.in);
                __syncwarp();
                if (lane == 0)
                    barrier_arrive(&sh.empty[c.at]);
            }
            if (passes == 1 && active > 0)   // the last row's sums have been read
                ok = ok && warp_wait(&sh.joined, (active - 1) & 1);
            const Stat s = warp_join<false>(run.stat(a.in), a.in);
            if (lane == 0) {
                sh.part[warp] = make_float2(s.m, ok ? s.z : kNan);
                barrier_arrive(&sh.summed);
            }
            if (passes == 2) {
                ok = ok && warp_wait(&sh.joined, active & 1);
                const f2 nm = splat(-sh.m), f = splat(sh.f);
                for (int i0 = 0; i0 < p.n && ok; i0 += kStageVecs, c.next()) {
                    ok = warp_wait(&sh.full[c.at], c.turn);
                    const uint4 *const stage = stages + c.at * kStageVecs;
                    if (i0 + kStageVecs <= p.n && p.v0 + i0 >= lo && p.v0 + i0 + kStageVecs <= hi) {
                        uint4 v[kStageVecs / kStream];
#pragma unroll
                        for (int j = 0; j < kStageVecs / kStream; ++j)
                            v[j] = stage[tid + j * kStream];
                        raw *const to = g + row.id(p.v0 + i0 + tid, 0);
#pragma unroll
                        for (int j = 0; j < kStageVecs / kStream; ++j)
                            store_stream(to + j * kStream * T::kPerVec, grad_vec<T>(v[j], nm, f, a.in));
                    } else
                        for (int i = tid; i < min(kStageVecs, p.n - i0); i += kStream)
                            write(p.v0 + i0 + i, grad_vec<T>(stage[i], nm, f, a.in));
                    __syncwarp();
                    if (lane == 0)
                        barrier_arrive(&sh.empty[c.at]);
                }
                for (int i = p.v0 + tid; !ok && i < p.v0 + p.n; i += kStream)
                    write(i, make_uint4(0x7fffffff, 0x7fffffff, 0x7fffffff, 0x7fffffff));   // NaN in every type
                __syncwarp();
                if (lane == 0)
                    barrier_arrive(&sh.written);
            }
            ++active;
        }
    }
    if (size > 1) {   // no CTA leaves while another may write to it
        cluster_arrive();
        cluster_wait();
    }
}

// The gradient from saved statistics: one pass, each CTA a chunk of a row, no
// sums to wait for. Bound by the device memory: 2048 x 128256 BF16 152 us with
// one id, 166 us with 64 (1.02 and 0.93 of the measured copy rate).
template <class T, int kVecs>
__global__ void __launch_bounds__(kGradThreads, 4) distill_grad_kernel(DistillGradArgs a, int chunks)
{
    typedef typename T::raw raw;
    __shared__ int32_t ids[FO_MAX_TOP_K];
    __shared__ float qs[FO_MAX_TOP_K], sum_q;
    __shared__ uint32_t taken[kVecs * kGradThreads * T::kPerVec / 32];   // a bit for each element of the chunk
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
    for (int i = tid; i < kVecs * kGradThreads * T::kPerVec / 32; i += kGradThreads)
        taken[i] = 0;
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
    // this thread's entry, if its token is in the chunk
    bool entry = false, again = false;
    float q = 0.0f, x = 0.0f;
    if (!zero && tid < a.teacher.k) {
        const int32_t id = ids[tid];
        entry = id >= max(0, row.id(v0, 0)) && id < min(row.vocab, row.id(v0 + kVecs * kGradThreads, 0));
        if (entry) {
            q = qs[tid];
            x = T::widen(row.x[id]);
            again = claim(taken, id - row.id(v0, 0));
        }
    }
    // the entries' logits are read before a gradient in their place is written
    if (__syncthreads_or(again) && entry) {   // rare: the first of equal ids takes the weight of all
        q = 0.0f;
        again = false;
        for (int i = 0; i < a.teacher.k; ++i)
            if (ids[i] == ids[tid]) {
                q += qs[i];
                again = again || i < tid;
            }
    }
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
    if (entry && !again)
        g[ids[tid]] = T::narrow(grad_listed<T>(x, safe_max(st.x), q, sum_q, inv_z, scale, a.in));
}

template <class T, int kWarps>
cudaError_t launch(DistillArgs a, int size, bool marks, int64_t ctas, cudaStream_t stream)
{
    const int64_t vecs = part_vecs(a.in.vocab * (int64_t)sizeof(typename T::raw), size);
    a.mark_words = marks ? (int)(vecs + 3) / 4 : 0;
    // The CTAs that fit take all rows up to kOneTurn, a bound that lies between the
    // sizes measured faster so and those measured slower; above it a few rows
    // each, so that short turns spread the grid's end. In us with a few each / all: loss alone, 2048 x 50257 F16 44.1 / 39.5, 8192 x
    // 50257 BF16 133 / 124, 8192 x 1000 25.6 / 22.7, 8192 x 100000 236 / 253; with
    // gradient, 1400 x 80000 90.4 / 85.8, 4096 x 16000 61.5 / 58.0, 4096 x 64128
    // 170 / 188.
    const int64_t each = std::min(kMaxRowsEach, std::max<int64_t>(1, a.in.rows * size / (4 * ctas)));
    const int64_t moved = a.in.rows * a.in.vocab * (int64_t)sizeof(typename T::raw) * (a.grad.data ? 2 : 1);
    const bool all = size == 1 && moved <= kOneTurn;
    const int64_t clusters = all ? std::min(a.in.rows, ctas) : (a.in.rows + each - 1) / each;
    const size_t shared = (size_t)kStages * 4 * kWarps * 32 * 16 + (size_t)a.mark_words * 4;
    const int threads = kWarps * 32 + 64;
    if (a.teacher.tail)
        return launch_cluster<distill_kernel<T, true, kWarps>>(a, clusters, size, shared, threads, stream);
    return launch_cluster<distill_kernel<T, false, kWarps>>(a, clusters, size, shared, threads, stream);
}

template <class T>
cudaError_t launch(const DistillArgs &a, cudaStream_t stream)
{
    const bool marks = a.teacher.tail || a.grad.data;
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw);
    // Many rows too short for eight warps, each by two: the steps between the
    // passes are what a short row takes its time for, and more of them overlap.
    // Loss with gradient, BF16, 8 ids, 8 warps against 2 (us): 16384 x 1000
    // 138 / 56, 4096 x 8192 48 / 35, 8192 x 16000 119 / 105, 8192 x 32000
    // 174 / 210.
    int64_t ctas = (int64_t)sm_count() * kShortPerSm;
    if (bytes <= kShortRow && a.in.rows >= ctas)
        return launch<T, kShort>(a, 1, marks, ctas, stream);
    // One CTA a row, or a cluster that shares it:
    //   - while the rows at work at once would not stay in the L2 cache between
    //     the passes (kCacheBytes);
    //   - until half of the CTAs that fit are there. All of them measured slower,
    //     a second set of clusters waiting for the first: 64 x 50257 BF16 14.6 us
    //     against 9.3, 100 x 128256 BF16 19.3 against 13.7.
    // Not for room for the marks: where they leave two CTAs to an SM and not
    // three, clusters that bring back the third are slower (8192 x 80000 BF16 528
    // us against 444, 300 x 128256 44 against 35). (Loss with gradient, 64 ids.)
    const int64_t sms = sm_count();
    const auto fit = [&](int size) { return sms * (marks && bytes > size * kMaxPart ? kCtasPerSm - 1 : kCtasPerSm); };
    const auto at_work = [&](int size) { return std::min(a.in.rows, fit(size) / size) * bytes; };
    int size = 1;
    while (size < kMaxCluster && ((a.grad.data && at_work(size) > kCacheBytes) || (2 * a.in.rows * size < sms * kCtasPerSm && bytes > size * kMinPart)))
        size *= 2;
    ctas = fit(size);
    return launch<T, kLong>(a, size, marks, ctas, stream);
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
