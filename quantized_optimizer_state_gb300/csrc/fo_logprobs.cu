// fo_logprobs.cu -- log probabilities of given tokens with entropy and top
// alternatives, and their gradient.
#include <algorithm>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr int kGradThreads = 256;
constexpr int kWide = 256, kMiddle = 128, kNarrow = 64;   // threads to a row: see launch
constexpr int kGroup = 4;                      // vectors of a thread that one maximum is kept for
constexpr int kThreadsPerSm = 1280;            // of resident rows
constexpr int64_t kMinPart = 32 * 1024;        // bytes of a row that are worth a CTA of their own
constexpr int kAheadBytes = 128;               // fetched ahead for each thread: see logprobs_kernel

// What the kN threads of a row share.
template <int kN>
struct Shared {
    static constexpr int kCandidates = kN == kWide ? 1024 : 512;
    static constexpr int kGroups = 2 * kN;
    Stat part[kN / 32];
    Stat mine;                                // this CTA's part, read by the others of the cluster
    int count, groups;                        // candidates found
    int sums[kN / 32 < kMaxCluster ? kMaxCluster : kN / 32];
    uint2 range[kN / 32];
    int counts[2][kN / 32];
    int group[kGroups];
    __align__(16) uint64_t list[kCandidates]; // candidates in any order; later the lists of the other CTAs
    uint64_t sorted[FO_MAX_TOP_K];            // this CTA's largest, descending
    int sorted_n;
};
static_assert(Shared<kWide>::kCandidates >= kMaxCluster * FO_MAX_TOP_K, "the lists of a cluster");

template <int kN>
__device__ __forceinline__ int block_sum(int v, Shared<kN> &sh)
{
    const int s = __reduce_add_sync(~0u, v);
    if ((threadIdx.x & 31) == 0)
        sh.sums[threadIdx.x >> 5] = s;
    barrier_among<kN>();
    int t = 0;
#pragma unroll
    for (int i = 0; i < kN / 32; ++i)
        t += sh.sums[i];
    barrier_among<kN>();
    return t;
}

// f(key, id) for every element of vector i of the row.
template <class T, class F>
__device__ __forceinline__ void each(const Row<T> &row, int i, const uint4 &v, F f)
{
    const typename T::raw *e = reinterpret_cast<const typename T::raw *>(&v);
#pragma unroll
    for (int k = 0; k < T::kPerVec; ++k) {
        const int id = row.id(i, k);
        if (id >= 0 && id < row.vocab)
            f(order_key(T::widen(e[k])), id);
    }
}

__device__ __forceinline__ uint64_t list_key(uint32_t key, int id) { return ((uint64_t)key << 32) | (0xffffffffu - (uint32_t)id); }

// The exact way for a part with very many candidates: most of it tied, as
// where a mask leaves fewer than k tokens, or its largest elements in few
// threads' hands. Finds the k-th largest value, then takes everything above it
// and, of the elements equal to it, those with the lowest ids, in the order of
// ids. `kth`: a value that at least k elements reach; if fewer than k are
// above it, as with ties, it is the k-th largest, else it is bisected for
// (a pass over the part, by now in the L2 cache, for each bit that values
// differ in, whatever the part holds).
template <class T, int kN>
__device__ __noinline__ void collect_exact(const Row<T> &row, const Part &p, uint32_t kth, int k, Shared<kN> &sh)
{
    constexpr uint32_t mask = T::kKeyBits;   // below it a key is all 0 or all 1
    const auto count = [&](uint32_t at) {
        int n = 0;
        for (int i = threadIdx.x; i < p.n; i += kN)
            each<T>(row, p.v0 + i, load_vec(row, p.v0 + i), [&](uint32_t key, int) { n += (key & mask) >= at; });
        return block_sum(n, sh);
    };
    constexpr uint32_t unit = mask & (0u - mask);
    if (kth != (0xffffffffu & mask) && count(kth + unit) >= k) {
        kth = 0;
        for (uint32_t bit = 0x80000000u; bit & mask; bit >>= 1)
            if (count(kth | bit) >= k)
                kth |= bit;
    }
    if (threadIdx.x == 0)
        sh.count = 0;
    barrier_among<kN>();
    for (int i = threadIdx.x; i < p.n; i += kN)
        each<T>(row, p.v0 + i, load_vec(row, p.v0 + i), [&](uint32_t key, int id) {
            if ((key & mask) > kth)
                sh.list[atomicAdd(&sh.count, 1)] = list_key(key, id);
        });
    barrier_among<kN>();
    int have = sh.count;   // below k
    for (int i0 = 0; i0 < p.n && have < k; i0 += kN) {
        const int i = i0 + threadIdx.x;
        uint4 v;
        int n = 0;
        if (i < p.n) {
            v = load_vec(row, p.v0 + i);
            each<T>(row, p.v0 + i, v, [&](uint32_t key, int) { n += (key & mask) == kth; });
        }
        // ties before this thread's
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int q = __shfl_up_sync(~0u, before, o);
            before += (threadIdx.x & 31) >= o ? q : 0;
        }
        if ((threadIdx.x & 31) == 31)
            sh.sums[threadIdx.x >> 5] = before;
        barrier_among<kN>();
        int all = 0;
        before -= n;
#pragma unroll
        for (int w = 0; w < kN / 32; ++w) {
            before += w < (int)(threadIdx.x >> 5) ? sh.sums[w] : 0;
            all += sh.sums[w];
        }
        if (n)
            each<T>(row, p.v0 + i, v, [&](uint32_t key, int id) {
                if ((key & mask) == kth && have + before < k)
                    sh.list[have + before++] = list_key(key, id);
            });
        have = min(k, have + all);
        barrier_among<kN>();
    }
    if (threadIdx.x == 0)
        sh.count = have;
    barrier_among<kN>();
}

template <class T>
__device__ __forceinline__ uint32_t largest_key(const Largest<T> &l) { return order_key(l.value_nan()); }

// The k-th largest of the threads' keys, cut to its upper 16 bits; 0 where
// fewer than k are not 0. Two bits a step, from the first that keys differ in.
template <int kN>
__device__ __forceinline__ uint32_t kth_key(uint32_t mine, int k, Shared<kN> &sh)
{
    constexpr int kWarps = kN / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t hi = __reduce_max_sync(~0u, mine), lo = __reduce_min_sync(~0u, mine);
    if (lane == 0)
        sh.range[warp] = make_uint2(lo, hi);
    barrier_among<kN>();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        lo = min(lo, sh.range[i].x);
        hi = max(hi, sh.range[i].y);
    }
    int bit = 31 - __clz((int)(((lo ^ hi) & 0xffff0000u) | 0x8000u));   // 15: they agree
    bit |= 1;                                                           // the upper of a pair
    uint32_t bound = bit >= 31 ? 0u : hi & (0xfffffffeu << bit);
    for (int step = 0; bit > 16; bit -= 2, ++step) {
        const uint32_t u = 1u << (bit - 1);
        const int n = __popc(__ballot_sync(~0u, mine >= bound + u)) | __popc(__ballot_sync(~0u, mine >= bound + 2 * u)) << 10 |
                      __popc(__ballot_sync(~0u, mine >= bound + 3 * u)) << 20;
        if (lane == 0)
            sh.counts[step & 1][warp] = n;
        barrier_among<kN>();
        int all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            all += sh.counts[step & 1][i];
        bound += (all >> 20) >= k ? 3 * u : (all >> 10 & 1023) >= k ? 2 * u : (all & 1023) >= k ? u : 0u;
    }
    return bound;
}

// A value that all elements with keys from `bound` on reach, NaN counting as
// the largest: !(x < floor). Where no number is it, a few more reach it.
__device__ __forceinline__ float key_floor(uint32_t bound)
{
    bound = min(bound, 0xff800000u);   // +inf
    return bound <= 0x007fffffu ? -kInf : __uint_as_float(bound & 0x80000000u ? bound & 0x7fffffffu : ~bound);
}

// A bit for each element of vector i that reaches the floor.
template <class T>
__device__ __forceinline__ uint32_t reached(const Row<T> &row, int i, const uint4 &v, float floor_)
{
    const typename T::raw *e = reinterpret_cast<const typename T::raw *>(&v);
    uint32_t found = 0;
#pragma unroll
    for (int k = 0; k < T::kPerVec; ++k)
        found |= T::widen(e[k]) < floor_ ? 0u : 1u << k;
    const int lo = max(0, -row.id(i, 0)), hi = min(T::kPerVec, row.vocab - row.id(i, 0));
    return found & ((1u << hi) - (1u << lo));
}

// Element k of a vector, k not known when it is compiled.
template <class T>
__device__ __forceinline__ float element(const uint4 &v, int k)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int at = k * 4 / T::kPerVec;
    const uint32_t word = at == 0 ? w[0] : at == 1 ? w[1] : at == 2 ? w[2] : w[3];
    return sizeof(typename T::raw) == 4 ? __uint_as_float(word) : T::widen((typename T::raw)(word >> k % 2 * 16));
}

// The part's largest elements (k, or all where it has fewer), descending, into
// sh.sorted. `mine` is the key of the largest element of this thread (0
// without elements): the k-th largest of the threads' maxima bounds the k-th
// largest element from below, and for spread-out values few elements besides
// the top k reach it. `maxima` holds a maximum for each kGroup vectors of a
// thread, so that only those groups are read again, from the L2 cache, that
// reach the bound.
template <class T, int kN>
__device__ __forceinline__ void find_top(const Row<T> &row, const Part &p, const Largest<T> *maxima, uint32_t mine, int k, Shared<kN> &sh)
{
    if (threadIdx.x == 0)
        sh.count = sh.groups = 0;
    const uint32_t bound = kth_key<kN>(mine, k, sh);
    const float floor_ = key_floor(bound);
    if (mine >= bound)
        for (int i = threadIdx.x; i < p.n; i += kGroup * kN) {
            const int at = i / (kGroup * kN) * kN + (int)threadIdx.x;
            if (!(maxima[at].value_nan() < floor_)) {
                const int n = atomicAdd(&sh.groups, 1);
                if (n < Shared<kN>::kGroups)
                    sh.group[n] = at;
            }
        }
    barrier_among<kN>();
    const int groups = sh.groups;
    if (groups <= Shared<kN>::kGroups)
        for (int j = threadIdx.x; j < groups; j += kN) {
            if (*(volatile int *)&sh.count > Shared<kN>::kCandidates)
                break;
            const int at = sh.group[j], i = at / kN * (kGroup * kN) + at % kN;
            uint4 v[kGroup];
#pragma unroll
            for (int q = 0; q < kGroup; ++q)
                if (i + q * kN < p.n)
                    v[q] = load_vec(row, p.v0 + i + q * kN);
            uint32_t found = 0;
#pragma unroll
            for (int q = 0; q < kGroup; ++q)
                if (i + q * kN < p.n)
                    found |= reached<T>(row, p.v0 + i + q * kN, v[q], floor_) << q * T::kPerVec;
            int n = found ? atomicAdd(&sh.count, __popc(found)) : 0;
            for (; found; found &= found - 1, ++n) {
                const int b = __ffs((int)found) - 1, q = b / T::kPerVec;
                if (n < Shared<kN>::kCandidates) {
                    const uint4 w = q == 0 ? v[0] : q == 1 ? v[1] : q == 2 ? v[2] : v[3];
                    sh.list[n] = list_key(order_key(element<T>(w, b % T::kPerVec)), row.id(p.v0 + i + q * kN, b % T::kPerVec));
                }
            }
        }
    barrier_among<kN>();
    if (groups > Shared<kN>::kGroups || sh.count > Shared<kN>::kCandidates) {
        barrier_among<kN>();
        collect_exact<T, kN>(row, p, bound & T::kKeyBits, k, sh);
    }
    const int n = sh.count;
    for (int i = threadIdx.x; i < n; i += kN) {   // no two keys are equal
        const uint64_t key = sh.list[i];
        int rank = 0;
#pragma unroll 2
        for (int j = 0; j + 1 < n; j += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&sh.list[j]);
            rank += (two.x > key) + (two.y > key);
        }
        rank += n % 2 && sh.list[n - 1] > key;
        if (rank < k)
            sh.sorted[rank] = key;
    }
    if (threadIdx.x == 0)
        sh.sorted_n = min(n, k);
    barrier_among<kN>();
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o == 0xffffffffu ? 0x7fffffffu : o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// What follows the pass over a part: the sums and top lists joined in the CTA
// and over the cluster, and the row's results. By the first kN threads; the
// cluster's barriers are passed once.
template <class T, int kN>
__device__ __forceinline__ void finish(const LogprobArgs &a, int64_t r, const Row<T> &row, const Part &p, const Running<T, true> &run,
                                       const Largest<T> *maxima, int64_t token, float token_x, Shared<kN> &sh)
{
    const uint32_t size = cluster_size(), rank = cluster_rank();
    Stat s = block_join<true, kN>(run.stat(a.in), sh.part, a.in);
    if (a.k)
        find_top<T, kN>(row, p, maxima, (int)threadIdx.x < p.n ? largest_key(run.top) : 0, a.k, sh);
    if (size > 1) {
        if (threadIdx.x == 0)
            sh.mine = s;
        cluster_arrive();
        cluster_wait();
        const uint32_t at = map_shared(&sh.mine, (threadIdx.x & 7) % size);
        s = warp_join<true>(Stat{ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)}, a.in, size);
    }
    const float ln_z = logf(s.z);
    if (rank == 0 && threadIdx.x == 0) {
        const float h = s.z == 0.0f ? 0.0f : ln_z - kLn2 * (s.w / s.z);
        if (a.logp)
            a.logp[r] = token < 0 ? 0.0f : token >= row.vocab ? __int_as_float(0x7fffffff) : log_prob(token_x, s.m, s.z, ln_z, a.in.inv_t);
        if (a.entropy)
            a.entropy[r] = h;
        if (a.stats)
            a.stats[r] = make_float4(s.m, s.z, h, 0.0f);
    }
    if (a.k == 0)
        return;
    // an element's place among all parts' lists: its own place and, for each
    // other list, how many of that are larger
    const int k = a.k;
    if (size > 1) {
        for (uint32_t i = threadIdx.x; i < size * k; i += kN) {
            const uint32_t from = i / k, j = i % k;
            sh.list[i] = ld_cluster_u64(map_shared(&sh.sorted[j], from));
        }
        if (threadIdx.x < size)
            sh.sums[threadIdx.x] = (int)__float_as_int(ld_cluster_f32(map_shared(&sh.sorted_n, threadIdx.x)));
        barrier_among<kN>();
    }
    for (int n = threadIdx.x; n < sh.sorted_n; n += kN) {
        const uint64_t key = sh.sorted[n];
        int place = n;
        for (uint32_t i = 0; i < size && size > 1; ++i) {
            if (i == rank)
                continue;
            int lo = 0, hi = sh.sums[i];   // the first place whose key is smaller
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sh.list[i * k + mid] > key)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            place += lo;
        }
        if (place < k) {
            a.top_ids[r * k + place] = (int32_t)entry_id(key);
            a.top_logp[r * k + place] = log_prob(key_value(key), s.m, s.z, ln_z, a.in.inv_t);
        }
    }
}

// Starts the way of a row's first bytes into the L2 cache.
template <class T>
__device__ __forceinline__ void fetch_ahead(const Row<T> &row, int bytes)
{
    const int n = min(row.full1 - row.full0, bytes / 16);
    if (n > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row.vec(row.full0)), "r"(n * 16) : "memory");
}

// The given token's logit, on its way while the row is walked over.
template <class T>
__device__ __forceinline__ float load_token(const LogprobArgs &a, int64_t r, const Row<T> &row, int64_t &token)
{
    token = -1;
    if (threadIdx.x != 0 || cluster_rank() != 0 || !a.logp)
        return 0.0f;
    token = a.tokens[r];
    return T::widen(row.x[token >= 0 && token < row.vocab ? token : 0]);
}

// One row by a cluster of CTAs of kN threads (one CTA where there are many
// rows): one pass over the row by plain loads, sums in registers. 4096 x 128256
// BF16: 166 us, 0.93 of the measured copy rate; it issues 6.7 instructions an
// element in half of the cycles. With alternatives (3001 x 50257 BF16, 64 of
// them: 76 us, 0.59) it is bound by the end of a row: the bound, the vectors
// read again and the ranking are chains of short steps, half as long as the
// pass. Meanwhile the CTA has the first bytes of the row that comes next to its
// place on its way into the L2 cache, 128 a thread (a.ahead rows on; 3001 x
// 50257 with 8 68.3 / 65.5 us, 4096 x 128256 with 64 225 / 213, without any 171
// / 166; twice as much 76.5 against 74.9 on the case above). Bulk copies into a
// ring that run ahead into the next row were slower (206 and 147 us): the same
// warps finish the row, and fewer of them fit.
template <class T, int kN>
__global__ void __launch_bounds__(kN, kThreadsPerSm / kN) logprobs_kernel(LogprobArgs a)
{
    extern __shared__ __align__(16) unsigned char dynamic[];
    Largest<T> *const maxima = reinterpret_cast<Largest<T> *>(dynamic);
    __shared__ Shared<kN> sh;
    constexpr int kStep = kGroup * kN;
    const uint32_t size = cluster_size();
    const int64_t r = blockIdx.x / size;
    const Row<T> row(a.in, r);
    const Part p = part_of(row, cluster_rank(), size);
    const int tid = threadIdx.x;
    int64_t token;
    const float token_x = load_token(a, r, row, token);
    Running<T, true> run;
    for (int i0 = 0; i0 < p.n; i0 += kStep) {
        const int i = p.v0 + i0 + tid;
        const Largest<T> before = run.top;
        run.top = Largest<T>::none();
        if (p.v0 + i0 >= row.full0 && i0 + kStep <= p.n && p.v0 + i0 + kStep <= row.full1) {
            uint4 v[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                v[j] = __ldcs(row.vec(i + j * kN));
            run.add(v, a.in);
        } else {
#pragma unroll 1
            for (int j = 0; j < kGroup; ++j)
                if (i0 + tid + j * kN < p.n)
                    run.add(load_vec(row, i + j * kN), a.in);
        }
        if (a.k && i0 + tid < p.n)
            maxima[i0 / kGroup + tid] = run.top;
        run.top = run.top.with(before);
    }
    if (a.ahead && tid == 0 && r + a.ahead < a.in.rows)
        fetch_ahead(Row<T>(a.in, r + a.ahead), kN * kAheadBytes);
    finish<T, kN>(a, r, row, p, run, maxima, token, token_x, sh);
    if (size > 1) {   // no CTA leaves while another reads its shared memory
        cluster_arrive();
        cluster_wait();
    }
}

// dx_j = (1/T) [ sum of the weights of entries at j - p_j (G + h (ln p_j + H)) ],
// G the sum of all entries' weights, the entries being the token and the top
// ids. With t = (x_j - m) c: dx_j = 2^t (alpha + beta t), plus the weights. One
// pass, each CTA a chunk of a row, no sums to wait for. Bound by the device
// memory: 2048 x 128256 BF16 158 us, 0.98 of the measured copy rate.
template <class T, int kVecs>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(LogprobGradArgs a, int chunks)
{
    typedef typename T::raw raw;
    __shared__ int64_t ids[FO_MAX_TOP_K + 1];
    __shared__ float weight[FO_MAX_TOP_K + 1], sum_weight;
    __shared__ bool any_weight;
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
    const float4 st = a.stats[r];
    const float m = safe_max(st.x), inv_z = st.y == 0.0f ? 0.0f : 1.0f / st.y, ln_z = logf(st.y);
    const float h = a.g_entropy ? a.g_entropy[r] : 0.0f;
    if (tid <= a.k) {
        const int i = tid - 1;
        ids[tid] = i < 0 ? (a.g_logp ? a.tokens[r] : -1) : a.top_ids[r * a.k + i];
        float w = i < 0 ? (a.g_logp ? a.g_logp[r] : 0.0f) : a.g_top[r * a.k + i];
        if (a.by_slope && w != 0.0f) {   // what is not finite makes the row NaN
            w = __fmul_rn(w, st.z);
            w = fabsf(w) < kInf ? w : kNan;
        }
        weight[tid] = w;
    }
    for (int i = tid; i < kVecs * kGradThreads * T::kPerVec / 32; i += kGradThreads)
        taken[i] = 0;
    __syncthreads();
    // the sum of the weights; NaN where an id is out of range
    if (tid < 32) {
        float part = 0.0f;
        bool any = false;
        for (int i = tid; i <= a.k; i += 32)
            if (ids[i] >= 0 && weight[i] != 0.0f) {
                any = true;
                part += ids[i] >= row.vocab ? __int_as_float(0x7fffffff) : weight[i];
            }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            part += __shfl_xor_sync(~0u, part, o);
        any = __any_sync(~0u, any);
        if (tid == 0) {
            sum_weight = part;
            any_weight = any;
        }
    }
    // this thread's entry, if its token is in the chunk
    bool entry = false, again = false;
    float w = 0.0f, x_entry = 0.0f;
    if (tid <= a.k) {
        const int64_t id = ids[tid];
        entry = id >= max(0, row.id(v0, 0)) && id < min(row.vocab, row.id(v0 + kVecs * kGradThreads, 0));
        if (entry) {
            w = weight[tid];
            x_entry = T::widen(row.x[id]);
            again = claim(taken, (int)id - row.id(v0, 0));
        }
    }
    // the entries' logits are read before a gradient in their place is written
    if (__syncthreads_or(again) && entry) {   // the first of equal ids takes the weight of all
        w = 0.0f;
        again = false;
        for (int i = 0; i <= a.k; ++i)
            if (ids[i] == ids[tid]) {
                w += weight[i];
                again = again || i < tid;
            }
    }
    const float sum = sum_weight;
    const bool zero = (!any_weight && h == 0.0f) || st.y == 0.0f;
    const float p_scale = inv_z * (a.in.inv_t / T::kShift);
    const float alpha = h == 0.0f ? -p_scale * sum : -p_scale * (sum + h * (st.z - ln_z));
    const float beta = h == 0.0f ? 0.0f : -p_scale * h * kLn2;
    const bool aligned = same_phase(row, g);
    const f2 nm = splat(-m), al = splat(alpha), be = splat(beta);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = v0 + i * kGradThreads + tid;
        if (at >= row.vecs)
            break;
        f2 x[T::kPerVec / 2];
        widen_vec<T>(v[i], x);
#pragma unroll
        for (int k = 0; k < T::kPerVec / 2; ++k) {
            float p, q;
            unpk(add2(x[k], nm), p, q);
            f2 t;
            const f2 e = grad_exp2<T>(pk(max_nan(p, a.in.d_min), max_nan(q, a.in.d_min)), a.in, t);
            x[k] = mul2(e, fma2(be, t, al));
        }
        const uint4 d = zero ? make_uint4(0, 0, 0, 0) : narrow_vec<T>(x);
        if (aligned && at >= row.full0 && at < row.full1)
            store_stream(g + row.id(at, 0), d);
        else
            store_edge<T>(g, row, at, d);
    }
    __syncthreads();
    if (entry && !again && !zero) {
        float t;
        const float e = grad_exp<T>(distance(x_entry, m, a.in), a.in, t);
        g[ids[tid]] = T::narrow(__fmaf_rn(w, a.in.inv_t, e * __fmaf_rn(beta, t, alpha)));
    }
}

template <class T, int kN>
cudaError_t launch(LogprobArgs a, int size, cudaStream_t stream)
{
    a.ahead = size == 1 ? sm_count() * (kThreadsPerSm / kN) : 0;
    const int64_t vecs = part_vecs(a.in.vocab * (int64_t)sizeof(typename T::raw), size);
    const int64_t groups = (vecs + kGroup * kN - 1) / (kGroup * kN);
    return launch_cluster<logprobs_kernel<T, kN>>(a, a.in.rows, size, a.k ? groups * kN * 4 : 0, kN, stream);
}

// Whether rows without alternatives are better off with kMiddle threads than
// with kWide. A last turn that is not full takes at least half of a full one's
// time, which costs long rows in few turns more than wide CTAs do: 2048 x 128256
// BF16 101 us with 128 threads, 91 with 256; 1700 x 50257 42.4 / 39.3; but 2700 x
// 128256 115 / 116, 8000 x 128256 311 / 318, 3100 x 32000 43.6 / 43.9.
bool fits_middle(int64_t rows, int64_t bytes)
{
    const auto time = [&](int threads) {
        const int64_t fit = (int64_t)sm_count() * (kThreadsPerSm / threads);
        const double rest = (double)(rows % fit) / (double)fit;
        return ((double)(rows / fit) + (rest == 0.0 ? 0.0 : std::max(rest, 0.5))) / threads;
    };
    return bytes <= 96 * 1024 || rows > 4 * sm_count() * (kThreadsPerSm / kMiddle) || time(kMiddle) <= time(kWide) * 1.03;
}

template <class T>
cudaError_t launch(const LogprobArgs &a, cudaStream_t stream)
{
    const int64_t bytes = a.in.vocab * (int64_t)sizeof(typename T::raw), ctas = (int64_t)sm_count() * (kThreadsPerSm / kWide);
    // More rows than CTAs of 256 threads fit: one CTA each, of as few threads as
    // the row and its list leave busy, so that more rows are on an SM at once and
    // their joins and lists overlap. A list of k wants 2 k threads: the bound is
    // the k-th of their maxima, and as the lowest of all it would let in more
    // candidates than there is room for (610 x 8192 BF16 with 64 alternatives,
    // 64 threads: 246 us, found the exact way, against 10). Measured at 256 / 128
    // / 64 threads: 16384 x 1000 BF16 54 / - / 18 us, with 20 alternatives 124 /
    // - / 53; 3001 x 50257 with 64 of them 91 / 81 / - us; 4096 x 128256 without
    // any 180 / 169 / -, with 64 of them 226 / 253 / -; 610 x 128256 30 / 40 / -.
    if (a.in.rows > ctas) {
        if (bytes <= 16 * 1024 && a.k <= kNarrow / 2)
            return launch<T, kNarrow>(a, 1, stream);
        if (a.k == 0 ? fits_middle(a.in.rows, bytes) : a.k <= 64 && bytes <= 128 * 1024)
            return launch<T, kMiddle>(a, 1, stream);
        return launch<T, kWide>(a, 1, stream);
    }
    // Few rows: a cluster shares one until there are two CTAs to an SM. Up to four
    // measured slower, where a second set of clusters waits for the first (100 x
    // 50257 BF16 13.5 / 8.0 us, 300 x 128256 FP32 35 / 26), and so did parts of
    // 8 KB against 32 KB (1 x 50257 with 64 alternatives 12.1 / 10.9, 64 x 50257
    // 16.6 / 12.6; without any, 4 x 50257, 5.6 / 6.6).
    int size = 1;
    while (size < kMaxCluster && a.in.rows * size < 2 * sm_count() && bytes > size * kMinPart)
        size *= 2;
    return launch<T, kWide>(a, size, stream);
}

template <class T>
cudaError_t launch(const LogprobGradArgs &a, cudaStream_t stream)
{
    const int64_t vecs = a.in.vocab / T::kPerVec + 2;
    if (vecs * a.in.rows >= (int64_t)sm_count() * 8 * kGradThreads * 8) {
        const int64_t chunks = (vecs + 8 * kGradThreads - 1) / (8 * kGradThreads);
        logprobs_grad_kernel<T, 8><<<(unsigned)(chunks * a.in.rows), kGradThreads, 0, stream>>>(a, (int)chunks);
    } else {
        const int64_t chunks = (vecs + kGradThreads - 1) / kGradThreads;
        logprobs_grad_kernel<T, 1><<<(unsigned)(chunks * a.in.rows), kGradThreads, 0, stream>>>(a, (int)chunks);
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

cudaError_t launch_token_logprobs(int dtype, const LogprobArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }
cudaError_t launch_token_logprobs_grad(int dtype, const LogprobGradArgs &a, cudaStream_t stream) { return by_type(dtype, a, stream); }

}  // namespace fo
