// fo_policy.cu -- the clipped loss of policy training on sampled tokens, with a KL
// term, and its gradient in the same call. (The gradient from saved statistics is
// that of the token's log probability: fo_logprobs.cu.)
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

// policy_kernel's shape is distill_kernel's, whose two passes it makes; the
// measurements behind it stand there (fo_distill.cu). Clusters only where the cache
// or few rows ask for them: loss alone, 1001 x 50257 FP32 by one CTA a row 40 us,
// by two 51, by four 58.
constexpr int kLong = 8, kShort = 2;              // warps that walk over a row: see launch
constexpr int kStages = 4;                        // copies of four vectors a thread, in flight or in use
constexpr int kCtasPerSm = 3, kShortPerSm = 8;    // of kLong and of kShort warps
constexpr int64_t kMaxRowsEach = 2;
constexpr int64_t kCacheBytes = 70 << 20;         // of the L2 cache, for the rows at work between their passes
constexpr int64_t kOneTurn = 800 << 20;           // bytes of all rows and gradients
constexpr int64_t kShortRow = 32 * 1024;
constexpr int64_t kMinPart = 16 * 1024;           // bytes of a row that are worth a CTA of their own

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

// What a row's loss is formed from.
struct Sample {
    int64_t token;
    float weight;            // 0 for a row that is no position
    float old, adv, ref;
};
__device__ __forceinline__ Sample load_sample(const PolicyArgs &a, int64_t r, bool whole)
{
    Sample s = {a.tokens[r], a.weight ? a.weight[r] : 1.0f, 0.0f, 0.0f, 0.0f};
    if (whole) {
        s.old = a.old_logp[r];
        s.adv = a.advantages[r];
        s.ref = a.ref_logp ? a.ref_logp[r] : 0.0f;
    }
    s.weight = s.token < 0 ? 0.0f : s.weight;
    return s;
}

__device__ __forceinline__ RowLoss row_loss(const PolicyArgs &a, const Sample &s, float logp)
{
    RowLoss o = {0.0f, 0.0f};
    const float adv = s.adv;
    if (adv != 0.0f) {
        const float q = expf(__fsub_rn(logp, s.old));
        const bool inside = adv >= 0.0f ? q <= a.ratio_high : q >= a.ratio_low;
        o.loss = -__fmul_rn(inside ? q : adv >= 0.0f ? a.ratio_high : a.ratio_low, adv);
        o.slope = inside ? o.loss : 0.0f;
        if (adv != adv || q != q)
            o.loss = o.slope = kNan;
    }
    if (a.ref_logp) {
        const float k = __fsub_rn(s.ref, logp);
        o.loss = __fmaf_rn(a.kl_weight, exp_rest(k), o.loss);
        o.slope = __fmaf_rn(a.kl_weight, -expm1f(k), o.slope);
    }
    return o;
}

// What the gradient takes of it: w slope / T, of the token itself, and -1 / Z of
// that, of every probability. A slope beyond FP32 makes the row's gradient NaN,
// not infinities and NaN; a row without a distribution has none.
struct Scaled {
    float slope, f;
};
__device__ __forceinline__ Scaled scaled(float slope, float weight, float sum, const LogitRows &in)
{
    const float c = __fmul_rn(slope, weight);
    Scaled o = {0.0f, 0.0f};
    if (sum != 0.0f) {
        o.slope = fabsf(c) < kInf ? __fmul_rn(c, in.inv_t) : kNan;
        o.f = -o.slope * (1.0f / sum);
    }
    return o;
}

struct Shared {
    uint64_t full[kStages], empty[kStages];   // of a stage: copied; used
    uint64_t summed, joined, written;         // of a row
    uint64_t cluster[2];                      // all CTAs' sums have come
    float2 sums[2][kMaxCluster];              // m, z, written by each CTA into all
    float2 part[kLong];                       // m, z of the warps
    float m, f;                               // the gradient: f 2^((x - m) c)
};

// Rows by a cluster of CTAs (one CTA a row for short rows), as distill_kernel
// takes them: a first pass sums the exponentials, a second, from the L2 cache,
// writes the gradient,
//   dloss/dx_j = (w slope / T) ([j = token] - p_j).
// In each CTA a warp keeps bulk copies in flight into a ring of stages, running
// ahead over the passes and rows; kWarps warps take the stages, sum, and write
// the gradient; a warp joins the sums, forms the loss, and writes it and, last,
// the token's own gradient. 8192 x 128256 BF16, loss with gradient: 663 us, 0.90 of
// the measured copy rate for one read and one write (1067 by a CTA a row without
// the ring, with the row's two passes from its own loads); 8192 x 50257 261 us,
// 0.93; loss alone, 4096 x 128256, 167 us, 0.93. Device memory gives 1.02 times
// the logits.
template <class T, int kWarps>
__global__ void __launch_bounds__(kWarps * 32 + 64, kWarps == kLong ? kCtasPerSm : kShortPerSm) policy_kernel(PolicyArgs a)
{
    typedef typename T::raw raw;
    constexpr int kStream = kWarps * 32, kFetcher = kWarps, kJoiner = kWarps + 1;
    constexpr int kStageVecs = 4 * kStream;   // vectors that are copied at once
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ __align__(16) Shared sh;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = blockIdx.x / size, step = gridDim.x / size, rows = a.in.rows;   // this cluster's rows
    uint4 *const stages = reinterpret_cast<uint4 *>(dynamic);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            barrier_init(&sh.full[i], 2);
            barrier_init(&sh.empty[i], kWarps);
        }
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
    // false: a wait ran out. What the warp has not done of its rows by then becomes
    // NaN; the others' waits for it run out in turn.
    bool ok = true;
    uint32_t active = 0;   // rows done with a weight other than 0
    if (warp == kFetcher) {
        Cursor<kStages> c;
        const uint64_t keep = keep_policy(), drop = drop_policy();
        float next_weight = load_sample(a, first, false).weight;
        for (int64_t r = first; r < rows && ok; r += step) {
            const float weight = next_weight;
            if (r + step < rows)
                next_weight = load_sample(a, r + step, false).weight;
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
    } else if (warp == kJoiner) {
        // A row's sample and the token's logit are loaded a row ahead: before a
        // gradient in their place is written, which waits for this warp.
        const auto logit = [&](int64_t r, const Sample &s) {
            const Row<T> row(a.in, r);
            return row.x[s.weight != 0.0f && s.token < row.vocab ? s.token : 0];   // used where there is one
        };
        Sample next = load_sample(a, first, true);
        raw next_x = logit(first, next);
        for (int64_t r = first; r < rows; r += step) {
            const Sample s = next;
            const raw xr = next_x;
            if (r + step < rows) {
                next = load_sample(a, r + step, true);
                next_x = logit(r + step, next);
            }
            const bool writes = (uint32_t)r % size == rank && lane == 0;   // the loss, in turn
            if (s.weight == 0.0f || !ok) {   // the weight is the same in all CTAs of the cluster
                const float v = s.weight == 0.0f ? 0.0f : kNan;
                if (writes && a.loss)
                    a.loss[r] = v;
                if (writes && a.logp)
                    a.logp[r] = v;
                if (writes && a.stats)
                    a.stats[r] = make_float4(v, v, v, v);
                continue;
            }
            ok = warp_wait(&sh.summed, active & 1);
            float2 z = make_float2(-kInf, 0.0f);
            if (lane < kWarps)
                z = sh.part[lane];
            z = join_pairs(z.x, z.y, a.in);
            if (!ok)   // NaN for the row's other CTAs too
                z.y = kNan;
            if (size > 1) {
                const int turn = active & 1;
                if (lane < (int)size) {
                    st_cluster(map_shared(&sh.sums[turn][rank], lane), z.x, z.y);
                    fence_cluster();
                    arrive_cluster(map_shared(&sh.cluster[turn], lane));
                }
                ok = ok && warp_wait(&sh.cluster[turn], (active >> 1) & 1);
                fence_cluster();
                z = make_float2(-kInf, 0.0f);
                if (lane < (int)size)
                    z = sh.sums[turn][lane];
                z = join_pairs(z.x, z.y, a.in);
            }
            const bool there = s.token < a.in.vocab;
            const float x = there ? T::widen(xr) : kNan, sum = ok && there ? z.y : kNan, mm = safe_max(z.x);
            const float logp = sum == 0.0f ? -kInf : sum != sum ? kNan : log_prob(x, z.x, sum, logf(sum), a.in.inv_t);
            const RowLoss o = row_loss(a, s, logp);
            const Scaled c = scaled(o.slope, s.weight, sum, a.in);
            const float slope = c.slope, f = c.f / T::kShift;
            if (lane == 0) {
                sh.m = mm;
                sh.f = f;
                barrier_arrive(&sh.joined);
            }
            if (writes) {
                if (a.loss)
                    a.loss[r] = __fmul_rn(o.loss, s.weight);
                if (a.logp)
                    a.logp[r] = logp;
                if (a.stats)
                    a.stats[r] = make_float4(z.x, sum, o.slope, 0.0f);
            }
            if (passes == 2) {
                ok = ok && warp_wait(&sh.written, active & 1);
                const Row<T> row(a.in, r);
                const Part p = part_of(row, rank, size);
                if (lane == 0 && s.token >= max(0, row.id(p.v0, 0)) && s.token < min(row.vocab, row.id(p.v0 + p.n, 0))) {
                    raw *const g = static_cast<raw *>(a.grad.data) + row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
                    float t;
                    g[s.token] = T::narrow(!ok ? kNan : sum == 0.0f ? 0.0f : __fmaf_rn(grad_exp<T>(distance(x, mm, a.in), a.in, t), f, slope));
                }
            }
            ++active;
        }
    } else {
        Cursor<kStages> c;
        float next_weight = load_sample(a, first, false).weight;
        for (int64_t r = first; r < rows; r += step) {
            const float weight = next_weight;
            if (r + step < rows)
                next_weight = load_sample(a, r + step, false).weight;
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
            Running<T, false> run;
            for (int i0 = 0; i0 < p.n && ok; i0 += kStageVecs, c.next()) {
                ok = warp_wait(&sh.full[c.at], c.turn);
                const uint4 *const stage = stages + c.at * kStageVecs;
                if (i0 + kStageVecs <= p.n) {
                    uint4 v[kStageVecs / kStream];
#pragma unroll
                    for (int j = 0; j < kStageVecs / kStream; ++j)
                        v[j] = stage[tid + j * kStream];
                    run.add(v, a.in);
                } else
                    for (int i = tid; i < p.n - i0; i += kStream)
                        run.add(stage[i], a.in);
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

// Rows short enough for the registers of a team of kTeam threads, kTeamVecs
// vectors each: read once, the next one's loads on their way while one is worked
// on. What a row of policy_kernel waits for, this one's neighbours on the SM hide.
// Bound by instructions: a row's sums are joined and its loss is formed by every
// lane, as much work as 32 elements of each.
constexpr int kTeamThreads = 256;
template <class T, int kTeam, int kTeamVecs, int kCtas>
__global__ void __launch_bounds__(kTeamThreads, kCtas) policy_rows_kernel(PolicyArgs a)
{
    typedef typename T::raw raw;
    constexpr int kTeams = kTeamThreads / kTeam;
    __shared__ Stat part[2][kTeamThreads / 32];
    const int tid = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
    const int64_t rows = a.in.rows, step = (int64_t)gridDim.x * kTeams;
    const uint32_t low = sizeof(raw) == 2 ? T::narrow(-kInf) * 0x10001u : __float_as_uint(-kInf);
    const uint4 none = make_uint4(low, low, low, low);
    uint4 next[kTeamVecs];
    raw next_x;
    const auto fetch = [&](int64_t r, const Sample &next_sample) {
        if (next_sample.weight == 0.0f)
            return;
        const Row<T> row(a.in, r);
        next_x = row.x[next_sample.token < row.vocab ? next_sample.token : 0];
#pragma unroll
        for (int k = 0; k < kTeamVecs; ++k)
            next[k] = tid + k * kTeam < row.vecs ? load_vec(row, tid + k * kTeam) : none;
    };
    // samples are loaded two rows ahead: which logit a row needs is known when its vectors are asked for
    int64_t r = (int64_t)blockIdx.x * kTeams + team;
    if (r >= rows)
        return;
    Sample next_sample = load_sample(a, r, true), later = load_sample(a, r + step < rows ? r + step : r, true);
    fetch(r, next_sample);
    for (int turn = 0; r < rows; r += step) {
        const Row<T> row(a.in, r);
        const Sample s = next_sample;
        const bool there = s.token < row.vocab;
        const float x = there ? T::widen(next_x) : kNan;
        uint4 v[kTeamVecs];
#pragma unroll
        for (int k = 0; k < kTeamVecs; ++k)
            v[k] = next[k];
        next_sample = later;
        if (r + 2 * step < rows)
            later = load_sample(a, r + 2 * step, true);
        if (r + step < rows)
            fetch(r + step, next_sample);
        raw *g = static_cast<raw *>(a.grad.data);
        if (g)
            g += row_offset(a.in, r, a.grad.row_stride, a.grad.outer_stride);
        float loss = 0.0f, logp = 0.0f, f = 0.0f, slope = 0.0f, mm = 0.0f;
        float4 stats = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const bool active = s.weight != 0.0f;   // the same in the team
        if (active) {
            Running<T, false> run;
            run.add(v, a.in);
            Stat z = warp_join<false>(run.stat(a.in), a.in);
            if constexpr (kTeam > 32) {
                if ((threadIdx.x & 31) == 0)
                    part[turn][threadIdx.x / 32] = z;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(kTeam) : "memory");
                z = warp_join<false>(part[turn][team * (kTeam / 32) + tid % (kTeam / 32)], a.in, kTeam / 32);
                turn ^= 1;   // one barrier a sum is enough for two sets in turn, of rows that have one
            }
            const float sum = there ? z.z : kNan;
            mm = safe_max(z.m);
            logp = sum == 0.0f ? -kInf : sum != sum ? kNan : log_prob(x, z.m, sum, logf(sum), a.in.inv_t);
            const RowLoss o = row_loss(a, s, logp);
            loss = __fmul_rn(o.loss, s.weight);
            const Scaled c = scaled(o.slope, s.weight, sum, a.in);
            slope = c.slope;
            f = c.f / T::kShift;
            stats = make_float4(z.m, sum, o.slope, 0.0f);
        }
        if (tid == 0) {
            if (a.loss)
                a.loss[r] = loss;
            if (a.logp)
                a.logp[r] = logp;
            if (a.stats)
                a.stats[r] = stats;
        }
        if (!g)
            continue;
        // the token's own gradient takes its place in the vector that holds it
        float t;
        const raw own = T::narrow(stats.y == 0.0f ? 0.0f : __fmaf_rn(grad_exp<T>(distance(x, mm, a.in), a.in, t), f, slope));
        const bool aligned = same_phase(row, g);
        const int at = active && there ? (int)s.token + row.phase : -1;
#pragma unroll
        for (int k = 0; k < kTeamVecs; ++k) {
            const int i = tid + k * kTeam;
            if (i >= row.vecs)
                break;
            uint4 d = active ? grad_vec<T>(v[k], splat(-mm), splat(f), a.in) : make_uint4(0, 0, 0, 0);
            if (at >= 0 && at / T::kPerVec == i) {
                raw *const e = reinterpret_cast<raw *>(&d);
#pragma unroll
                for (int j = 0; j < T::kPerVec; ++j)
                    e[j] = at % T::kPerVec == j ? own : e[j];
            }
            if (aligned && i >= row.full0 && i < row.full1)
                store_stream(g + row.id(i, 0), d);
            else
                store_edge<T>(g, row, i, d);
        }
    }
}

template <class T, int kTeam, int kTeamVecs, int kCtas>
cudaError_t launch_rows(const PolicyArgs &a, cudaStream_t stream)
{
    constexpr int kTeams = kTeamThreads / kTeam;
    const int64_t ctas = std::min((a.in.rows + kTeams - 1) / kTeams, (int64_t)sm_count() * kCtas);
    policy_rows_kernel<T, kTeam, kTeamVecs, kCtas><<<(unsigned)ctas, kTeamThreads, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <class T, int kWarps>
cudaError_t launch(const PolicyArgs &a, int size, int64_t ctas, cudaStream_t stream)
{
    const int64_t each = std::min(kMaxRowsEach, std::max<int64_t>(1, a.in.rows * size / (4 * ctas)));
    const int64_t moved = a.in.rows * a.in.vocab * (int64_t)sizeof(typename T::raw) * (a.grad.data ? 2 : 1);
    const bool all = size == 1 && moved <= kOneTurn;
    // Up to three turns: as few CTAs as take the rows in no more of them. They share the
    // memory's rate, and the last turn is as full as the others (loss alone, us, against
    // all CTAs: 1001 x 50257 FP32 37 / 39, 1001 x 128256 BF16 49 / 52, 600 x 128256 30 /
    // 34; with gradient 600 x 50257 29 / 31; but 2048 x 50257, five turns, 76 / 73).
    const int64_t turns = (a.in.rows + ctas - 1) / ctas;
    const int64_t even = turns <= 3 ? (a.in.rows + turns - 1) / turns : std::min(a.in.rows, ctas);
    const int64_t clusters = all ? even : (a.in.rows + each - 1) / each;
    return launch_cluster<policy_kernel<T, kWarps>>(a, clusters, size, (size_t)kStages * 4 * kWarps * 32 * 16, kWarps * 32 + 64, stream);
}

template <class T>
cudaError_t launch(const PolicyArgs &a, cudaStream_t stream)
{
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw), sms = sm_count(), vecs = row_vecs(bytes);
    // Loss with gradient, us, in registers / by two warps and the ring: 16384 x 1000
    // BF16 21 / 42, 8000 x 2000 19 / 27, 8000 x 4000 34 / 36, 10000 x 2000 FP32 36 /
    // 42, 8000 x 6000 BF16 57 / 45. (A warp with four vectors where they hold the row:
    // with eight 16384 x 1000 takes 27.)
    if (vecs <= 128)
        return launch_rows<T, 32, 4, 3>(a, stream);
    if (vecs <= 256)
        return launch_rows<T, 32, 8, 2>(a, stream);
    if (vecs <= 512)
        return launch_rows<T, 64, 8, 2>(a, stream);
    if (bytes <= kShortRow && a.in.rows >= sms * kShortPerSm)
        return launch<T, kShort>(a, 1, sms * kShortPerSm, stream);
    const int64_t ctas = sms * kCtasPerSm;
    const auto at_work = [&](int size) { return std::min(a.in.rows, ctas / size) * bytes; };
    int size = 1;
    while (size < kMaxCluster && ((a.grad.data && at_work(size) > kCacheBytes) || (2 * a.in.rows * size < ctas && bytes > size * kMinPart)))
        size *= 2;
    return launch<T, kLong>(a, size, ctas, stream);
}

}  // namespace

cudaError_t launch_policy(int dtype, const PolicyArgs &a, cudaStream_t stream)
{
    return dtype == 0 ? launch<Bf16>(a, stream) : dtype == 1 ? launch<F32>(a, stream) : launch<F16>(a, stream);
}

}  // namespace fo
