// top.hip -- the k largest logits of a row, in order, with the row's log-sum-exp.
//
// The row is read once for the threads' own maxima (and sums of exponentials).  Nothing below the threshold can be among
// the first k: every wavefront (whose lanes all have elements) takes the r-th largest of its lanes' maxima, r = k / wavefronts,
// and the least of those has k elements at or above it; for longer lists it is the k-th largest of the maxima of all groups of a
// thread's vectors.  The elements from there on are listed, from the few threads that have any, and sorted.
// Where they are too many, histograms over narrowing ranges of keys find the border first.
//
// Bound by memory for many rows, the VALU close behind: 2,048 rows of 131,328 bfloat16, 64 listed, 109 us (4.9 TB/s).  One
// such row, 20 listed, 15.2 us and 300 rows of 33,001 float32, 1,000 listed, 32 us: the steps of a workgroup, one after another.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace tt {
namespace {

constexpr uint32_t NONE = 0xFFFFFFFFu;
constexpr uint32_t LIST = 2048;      // listed elements
constexpr uint32_t BINS = 2048;
constexpr uint32_t QUICK_RANK = 16;    // of a wavefront's maxima

// The order of the logits as integers, -0 equal to +0; an element is its key and the complement of its ID, so that the larger
// of two comes first.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __builtin_bit_cast(float, key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t element(float x, uint32_t id) { return (uint64_t)key_of(x) << 32 | ~id; }

// Where sort_by_bins scatters to.
constexpr uint32_t CROWD = 64;   // elements of a bin, at most
struct Scatter {
    uint32_t bins[BINS + 1], part[16], low, high, crowded;
    uint64_t list[LIST];
};

// A thread's vectors in groups of DEPTH, the last of GROUPS with all that are left.  (256 threads have four vectors each.)
template <int THREADS> constexpr uint32_t GROUPS = THREADS == 256 ? 2 : 8;
template <class T> constexpr int DEPTH = sizeof(T) == 4 ? 2 : 4;

template <int THREADS> struct Lds {
    union {
        uint64_t list[LIST] __attribute__((aligned(16)));
        uint32_t bins[BINS];
    };
    union {
        float best[GROUPS<THREADS>][THREADS];      // the groups' largest logits
        Scatter scatter[THREADS == 1024];
    };
    uint16_t who[GROUPS<THREADS> * THREADS];   // groups with elements to list: group * THREADS + thread
    MaxSum sums[16];
    float bound[16];
    uint32_t part[16], counts[16];
    uint32_t count, threads, found_bin, found_before;
};

// At most the r-th largest of the wavefront's values: its upper 16 bits as a key, found bit by bit.
__device__ __forceinline__ float wave_rank(float v, uint32_t r)
{
    const uint32_t key = key_of(v);
    uint32_t at = 0;
#pragma unroll
    for (uint32_t bit = 0x80000000u; bit > 0x8000u; bit >>= 1) {
        const uint32_t up = at | bit;
        if (__popcll(__ballot(key >= up)) >= r) at = up;
    }
    return at <= key_of(NEG_INF) ? NEG_INF : logit_of(at);
}

// At most the r-th largest of all threads' values, of which thread t holds value(0) .. value(n - 1) as keys; the same way, with a
// count over the workgroup for each bit.
template <int THREADS, int N, class F> __device__ __forceinline__ float block_rank(uint32_t (&counts)[16], uint32_t r, F value)
{
    if (threadIdx.x < 16) counts[threadIdx.x] = 0;
    uint32_t key[N], at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = value(i);
    __syncthreads();
#pragma unroll 1
    for (uint32_t b = 0; b < 16; ++b) {
        const uint32_t up = at | 0x80000000u >> b;
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) n += __popcll(__ballot(key[i] >= up));
        if ((threadIdx.x & 63) == 0) atomicAdd(&counts[b], n);
        __syncthreads();
        if (counts[b] >= r) at = up;
    }
    return at <= key_of(NEG_INF) ? NEG_INF : logit_of(at);
}

// Sorts the first n (at most LIST) of list, descending; elements are all different.
//
// Few by their ranks, several threads counting for an element, two elements a read.  More by bins (below), or, by 256 threads
// and where most keys are the same, by a bitonic network over registers: element e * THREADS + thread, so that its steps are
// exchanges of lanes, of wavefronts (through the list) or of a thread's own.
typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
template <int THREADS> __device__ __forceinline__ void sort_by_rank(uint64_t *list, uint32_t n)
{
    const uint32_t even = (n + 1) & ~1u;
    uint32_t per = 1;   // threads of an element
    while (per < 16 && 2 * per * n <= THREADS) per *= 2;
    if (threadIdx.x == 0 && n < even) list[n] = 0;
    __syncthreads();
    const uint32_t e = threadIdx.x / per;
    const uint64_t own = e < n ? list[e] : 0;
    uint32_t rank = 0;
    if (e < n) {
#pragma unroll 4
        for (uint32_t i = 2 * (threadIdx.x & (per - 1)); i < even; i += 2 * per) {
            const u64x2 v = *(const u64x2 *)(list + i);
            rank += (v[0] > own) + (v[1] > own);
        }
    }
    for (uint32_t d = 1; d < per; d *= 2) rank += __shfl_xor(rank, d);
    __syncthreads();
    if (e < n && (threadIdx.x & (per - 1)) == 0) list[rank] = own;
    __syncthreads();
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, uint32_t d)
{
    return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), d) << 32 | (uint32_t)__shfl_xor((int)v, d);
}

template <int THREADS, int EACH> __device__ __forceinline__ void sort_by_network(uint64_t *list, uint32_t n)
{
    constexpr uint32_t ALL = THREADS * EACH;
    uint64_t v[EACH];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e) v[e] = e * THREADS + threadIdx.x < n ? list[e * THREADS + threadIdx.x] : 0;
#pragma unroll
    for (uint32_t size = 2; size <= ALL; size *= 2) {
#pragma unroll
        for (uint32_t d = size / 2; d; d /= 2) {
            if (d >= THREADS) {   // a thread's own: the larger at the lower index where the run descends
#pragma unroll
                for (uint32_t e = 0; e < EACH; ++e) {
                    const uint32_t o = e ^ (d / THREADS);
                    if (o < e) continue;
                    const bool down = (e * THREADS & size) == 0;
                    const uint64_t lo = v[e], hi = v[o];
                    v[e] = (lo > hi) == down ? lo : hi;
                    v[o] = (lo > hi) == down ? hi : lo;
                }
                continue;
            }
            if (d >= 64) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < EACH; ++e) list[e * THREADS + threadIdx.x] = v[e];
                __syncthreads();
            }
#pragma unroll
            for (uint32_t e = 0; e < EACH; ++e) {
                const uint32_t i = e * THREADS + threadIdx.x;
                const uint64_t o = d >= 64 ? list[i ^ d] : shfl_xor64(v[e], d);
                const bool larger = ((i & size) == 0) == ((i & d) == 0);   // this place keeps the larger of the two
                v[e] = (v[e] > o) == larger ? v[e] : o;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e) list[e * THREADS + threadIdx.x] = v[e];
    __syncthreads();
}

// More than a few by 1,024 threads: into bins by their keys, and in a bin by rank.  False, with the list as it was, where one
// bin gets more than CROWD of them.
template <int THREADS> __device__ __forceinline__ bool sort_by_bins(uint64_t *list, uint32_t n, Scatter &s)
{
    static_assert(THREADS == 1024 && LIST == 2 * THREADS && BINS == 2 * THREADS, "two of each a thread");
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
    uint64_t own[2];
    uint32_t low = ~0u, high = 0, at[2], bin[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        own[e] = e * THREADS + threadIdx.x < n ? list[e * THREADS + threadIdx.x] : 0;
        const uint32_t key = own[e] >> 32;
        if (own[e]) {
            low = key < low ? key : low;
            high = key > high ? key : high;
        }
        s.bins[e * THREADS + threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) {
        s.low = ~0u;
        s.high = s.crowded = 0;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t l = __shfl_xor(low, d), h = __shfl_xor(high, d);
        low = l < low ? l : low;
        high = h > high ? h : high;
    }
    __syncthreads();
    if (lane == 0) {
        atomicMin(&s.low, low);
        atomicMax(&s.high, high);
    }
    __syncthreads();
    high = s.high;
    const uint32_t range = high - s.low, shift = range < BINS ? 0 : 21 - __clz(range);   // BINS = 2^11
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!own[e]) continue;
        bin[e] = (high - (uint32_t)(own[e] >> 32)) >> shift;
        at[e] = atomicAdd(&s.bins[bin[e]], 1u);
        if (at[e] >= CROWD) s.crowded = 1;
    }
    __syncthreads();
    if (s.crowded) return false;
    const uint32_t c0 = s.bins[2 * threadIdx.x], c1 = s.bins[2 * threadIdx.x + 1];
    uint32_t run = c0 + c1;
#pragma unroll
    for (uint32_t d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    if (lane == 63) s.part[wave] = run;
    __syncthreads();
    uint32_t before = run - c0 - c1;
    for (uint32_t w = 0; w < wave; ++w) before += s.part[w];
    s.bins[2 * threadIdx.x] = before;
    s.bins[2 * threadIdx.x + 1] = before + c0;
    if (threadIdx.x == THREADS - 1) s.bins[BINS] = n;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (own[e]) s.list[s.bins[bin[e]] + at[e]] = own[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!own[e]) continue;
        const uint32_t first = s.bins[bin[e]], last = s.bins[bin[e] + 1];
        uint32_t to = first;
        for (uint32_t i = first; i < last; ++i) to += s.list[i] > own[e];
        list[to] = own[e];
    }
    __syncthreads();
    return true;
}

template <int THREADS> __device__ __forceinline__ void sort_list(uint64_t *list, uint32_t n, Scatter *scatter)
{
    if (n <= (THREADS < 384 ? THREADS : 384)) return sort_by_rank<THREADS>(list, n);
    if constexpr (THREADS == 1024) {
        if (sort_by_bins<THREADS>(list, n, *scatter)) return;
    }
    if (THREADS == 256 && n <= 512) sort_by_network<THREADS, 512 / 256>(list, n);
    else if (n <= 1024) sort_by_network<THREADS, 1024 / THREADS>(list, n);
    else sort_by_network<THREADS, 2048 / THREADS>(list, n);
}

// f(first element, elements, values) for the vectors of [begin, end), dealt out to the threads
template <class T, int THREADS, class F> __device__ __forceinline__ void each_vector(const T *x, uint32_t begin, uint32_t end, F f)
{
    for (uint32_t j = begin + threadIdx.x * VEC; j < end; j += THREADS * VEC) {
        float v[VEC];
        load_part(x + j, end - j, NEG_INF, v);
        f(j, v);
    }
}

// The thread's largest logit of [begin, end), and with SUM the sum of exponentials under it, DEPTH vectors at a time with the next
// ones on their way.  The powers are taken of x k - m k in one instruction: off by a rounding of m k, which lse = m / T + log(s)
// has anyway.  (2,048 rows of 131,328 bfloat16, 64 listed: 149 us with rows.h's vectors, two on their way and a power's argument
// in two instructions.)
template <class T, int THREADS, bool SUM> __device__ __forceinline__ MaxSum largest_of(const T *x, uint32_t begin, uint32_t end, float k2, float (&best)[GROUPS<THREADS>][THREADS])
{
    constexpr int D = DEPTH<T>;
    constexpr uint32_t STEP = THREADS * VEC;
    MaxSum a{NEG_INF, 0.f};
    float own = NEG_INF;   // of the group in work
    auto take = [&](const auto &v, auto n) {
        constexpr int N = decltype(n)::value;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = vec_at(v[i / VEC], i % VEC);
            own = e > own ? e : own;
        }
        const float m = own > a.m ? own : a.m;
        if constexpr (SUM) {
            float s[4] = {};
            const float from = m == NEG_INF ? 0.f : m * k2;   // nothing but -inf so far, or NaN: those are in the sums
            s[0] = a.s * (m == NEG_INF ? 1.f : exp_f(a.m - m, k2));   // exactly 1 where the maximum stays
            if (__builtin_fabsf(from) < 65536.f) {
#pragma unroll
                for (int i = 0; i < N; ++i) s[i & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(vec_at(v[i / VEC], i % VEC), k2, -from));
            } else {   // the rounding may be beyond a power's range, the product beyond the type's numbers
#pragma unroll
                for (int i = 0; i < N; ++i) s[i & 3] += exp_f(vec_at(v[i / VEC], i % VEC) - m, k2);
            }
            a.s = (s[0] + s[1]) + (s[2] + s[3]);
        }
        a.m = m;
    };
    uint32_t j = begin + threadIdx.x * VEC, group = 0, used = 0;
    auto close = [&] {   // a group ends, the last one goes on
        best[group][threadIdx.x] = own;
        used = group + 1;
        if (group + 1 < GROUPS<THREADS>) {
            ++group;
            own = NEG_INF;
        }
    };
    Vec<T> v[D];
    auto fetch = [&](uint32_t at) {
#pragma unroll
        for (int i = 0; i < D; ++i) v[i] = load_vec(x + at + i * STEP);
    };
    constexpr uint32_t REACH = (D - 1) * STEP + VEC;
    if (j + REACH <= end) fetch(j);
    for (; j + REACH <= end; j += D * STEP) {
        Vec<T> now[D];
#pragma unroll
        for (int i = 0; i < D; ++i) now[i] = v[i];
        if (j + D * STEP + REACH <= end) fetch(j + D * STEP);
        take(now, std::integral_constant<int, D * VEC>{});
        close();
    }
    if (j < end) {
        for (; j < end; j += STEP) {
            float e8[VEC];
            load_part(x + j, end - j, NEG_INF, e8);
            const Vec<T> one[1] = {to_vec<T>(e8)};
            take(one, std::integral_constant<int, VEC>{});
        }
        best[group][threadIdx.x] = own;
        used = group + 1;
    }
    for (; used < GROUPS<THREADS>; ++used) best[used][threadIdx.x] = NEG_INF;
    return a;
}

// The elements that may be among the first k, in sh.list, their number returned.  Too many: found by histograms.
template <class T, int THREADS>
__device__ __forceinline__ uint32_t list_by_histogram(const T *x, uint32_t begin, uint32_t end, uint32_t k, float least, float most, Lds<THREADS> &sh)
{
    uint32_t lo = key_of(least), hi = key_of(most), before = 0;   // `before` elements lie above hi
    lo = lo > key_of(NEG_INF) ? lo : key_of(NEG_INF) + 1;
    for (;;) {
        uint32_t shift = 0;
        while ((hi - lo) >> shift >= BINS) ++shift;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < BINS; i += THREADS) sh.bins[i] = 0;
        if (threadIdx.x == 0) sh.found_bin = NONE;
        __syncthreads();
        each_vector<T, THREADS>(x, begin, end, [&](uint32_t, const float (&v)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const uint32_t key = key_of(v[e]);
                if (v[e] == v[e] && key >= lo && key <= hi) atomicAdd(&sh.bins[(hi - key) >> shift], 1u);
            }
        });
        __syncthreads();
        // the bin in which the k-th lies: running sums, BINS / THREADS bins a thread
        constexpr uint32_t PER = BINS / THREADS;
        uint32_t own = 0;
        for (uint32_t i = 0; i < PER; ++i) own += sh.bins[threadIdx.x * PER + i];
        uint32_t run = own;
#pragma unroll
        for (uint32_t d = 1; d < 64; d *= 2) {
            const uint32_t o = __shfl_up(run, d);
            if ((threadIdx.x & 63) >= d) run += o;
        }
        if ((threadIdx.x & 63) == 63) sh.part[threadIdx.x >> 6] = run;
        __syncthreads();
        uint32_t at = before + run - own;
        for (uint32_t w = 0; w < (threadIdx.x >> 6); ++w) at += sh.part[w];
        for (uint32_t i = 0; i < PER; ++i) {
            const uint32_t c = sh.bins[threadIdx.x * PER + i];
            if (at < k && at + c >= k) {
                sh.found_bin = threadIdx.x * PER + i;
                sh.found_before = at;
                sh.count = at + c;
            }
            at += c;
        }
        __syncthreads();
        const uint32_t bin = sh.found_bin, upto = sh.count, above = sh.found_before;
        uint32_t low = lo;   // fewer than k in all: everything
        if (bin != NONE) {
            const uint32_t top = hi - (bin << shift);
            low = top - lo < (1u << shift) ? lo : top - ((1u << shift) - 1);
            if (upto > LIST && low < top) {   // narrower
                hi = top;
                lo = low;
                before = above;
                continue;
            }
        }
        __syncthreads();   // the bins make place for the list
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
        const bool equals = bin != NONE && upto > LIST;   // a border of more equals than the list holds: the first ones by ID
        each_vector<T, THREADS>(x, begin, end, [&](uint32_t j, const float (&v)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const uint32_t key = key_of(v[e]);
                if (v[e] == v[e] && key >= low && !(equals && key == low)) sh.list[atomicAdd(&sh.count, 1u)] = element(v[e], j + e);
            }
        });
        __syncthreads();
        if (!equals) return sh.count;
        uint32_t n = above;   // what is listed now
        for (uint32_t j0 = begin; j0 < end && n < k; j0 += THREADS) {
            const uint32_t j = j0 + threadIdx.x;
            const float v = j < end ? (float)x[j] : NEG_INF;
            const bool is = v == v && key_of(v) == low;
            const uint64_t mask = __ballot(is);
            if ((threadIdx.x & 63) == 0) sh.part[threadIdx.x >> 6] = __popcll(mask);
            __syncthreads();
            uint32_t to = n + __popcll(mask & ((1ull << (threadIdx.x & 63)) - 1));
            for (uint32_t w = 0; w < THREADS / 64; ++w) {
                if (w < (threadIdx.x >> 6)) to += sh.part[w];
                n += sh.part[w];
            }
            if (is && to < k) sh.list[to] = element(v, j);
            __syncthreads();
        }
        return n < k ? n : k;
    }
}

// The first k of [0, n), sorted in sh.list, and their number (fewer than k where there are no more), from the elements at or above
// `least` in the groups of vectors whose largest logits are in sh.best; address(group * THREADS + thread, i): where the group's i-th
// vector begins, NONE for no vector; i < per.
template <class T, int THREADS, class F>
__device__ __forceinline__ uint32_t list_of(const T *x, uint32_t n, uint32_t k, float least, float most, uint32_t per, Lds<THREADS> &sh, F address)
{
    for (uint32_t g = 0; g < GROUPS<THREADS>; ++g) {
        const float v = sh.best[g][threadIdx.x];
        if (v >= least && v > NEG_INF) sh.who[atomicAdd(&sh.threads, 1u)] = g * THREADS + threadIdx.x;
    }
    __syncthreads();
    const uint32_t loads = sh.threads * per;
    for (uint32_t i0 = threadIdx.x; i0 < loads; i0 += 4 * THREADS) {   // four loads in flight
        uint32_t at[4];
        Vec<T> x8[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t i = i0 + b * THREADS, j = i < loads ? address(sh.who[i / per], i % per) : NONE;
            at[b] = j < n ? j : NONE;
            if (at[b] != NONE) x8[b] = load_some(x + j, n - j);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (at[b] == NONE) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float v = vec_at(x8[b], e);
                if (v >= least && v > NEG_INF && at[b] + e < n) {
                    const uint32_t to = atomicAdd(&sh.count, 1u);
                    if (to < LIST) sh.list[to] = element(v, at[b] + e);
                }
            }
        }
    }
    __syncthreads();
    uint32_t listed = sh.count;
    if (listed > LIST) listed = list_by_histogram<T, THREADS>(x, 0, n, k, least, most, sh);
    sort_list<THREADS>(sh.list, listed, sh.scatter);
    return listed;
}

template <int THREADS> __device__ __forceinline__ float least_of(uint32_t k, Lds<THREADS> &sh)
{
    return block_rank<THREADS, GROUPS<THREADS>>(sh.counts, k, [&](uint32_t g) { return key_of(sh.best[g][threadIdx.x]); });
}

// Place i of the answer.
__device__ __forceinline__ void put(uint32_t i, uint32_t n, const uint64_t *list, uint32_t *ids, float *logits)
{
    ids[i] = i < n ? ~(uint32_t)list[i] : NONE;
    logits[i] = i < n ? logit_of(list[i] >> 32) : NEG_INF;
}

template <class T, int THREADS, bool SUM>
__global__ __launch_bounds__(THREADS, 8) void k_top(const T *logits, uint32_t n, uint64_t stride, uint32_t k, float inv_t, uint32_t *__restrict__ ids,
                                                 uint64_t ids_stride, float *__restrict__ out, uint64_t out_stride, float *__restrict__ lse)
{
    __shared__ Lds<THREADS> sh;
    constexpr uint32_t WAVES = THREADS / 64, STEP = THREADS * VEC;
    const uint64_t row = blockIdx.x;
    const T *x = logits + row * stride;
    const float k2 = LOG2E * inv_t;
    if (threadIdx.x == 0) sh.count = sh.threads = 0;
    const MaxSum a = largest_of<T, THREADS, SUM>(x, 0, n, k2, sh.best);
    // the wavefronts whose lanes all have elements
    const uint32_t whole = n / (64 * VEC) < WAVES ? n / (64 * VEC) : WAVES, rank = whole ? (k + whole - 1) / whole : 65;
    MaxSum all;
    float least;
    if (rank <= QUICK_RANK) {
        const float bound = (threadIdx.x >> 6) < whole ? wave_rank(a.m, rank) : -NEG_INF;
        if ((threadIdx.x & 63) == 0) sh.bound[threadIdx.x >> 6] = bound;
        all = block_join<THREADS>(a, sh.sums, k2);   // with the barrier that sh.bound needs
        least = sh.bound[0];
#pragma unroll
        for (uint32_t w = 1; w < WAVES; ++w) least = fminf(least, sh.bound[w]);
    } else {
        all = block_join<THREADS>(a, sh.sums, k2);
        least = least_of<THREADS>(k, sh);
    }
    // a group's vectors: as many as the last one may have
    const uint32_t vectors = (n + STEP - 1) / STEP;
    const uint32_t per = vectors > GROUPS<THREADS> * DEPTH<T> ? vectors - (GROUPS<THREADS> - 1) * DEPTH<T> : DEPTH<T>;
    const uint32_t listed = list_of<T, THREADS>(x, n, k, least, all.m, per, sh, [&](uint32_t who, uint32_t i) {
        const uint32_t g = who / THREADS;
        return g + 1 == GROUPS<THREADS> || i < DEPTH<T> ? ((g * DEPTH<T> + i) * THREADS + who % THREADS) * VEC : NONE;
    });
    for (uint32_t i = threadIdx.x; i < k; i += THREADS) put(i, listed, sh.list, ids + row * ids_stride, out + row * out_stride);
    if (SUM && threadIdx.x == 0) lse[row] = empty(all) ? NEG_INF : all.m * inv_t + log_of(all.s);
}

}  // namespace
}  // namespace tt

using namespace tt;

namespace {
// Nothing needs to be kept: a row is one workgroup's, few rows too.  (One row of 131,328 bfloat16 with its log-sum-exp, 20 listed, is 15.2 us;
// with its maxima and sums by 17 workgroups and the rest by one it was 17.5 us, with the pieces' own lists joined 19.4.)
constexpr uint64_t WORKSPACE = 256;
}  // namespace

extern "C" int toktier_top_logits_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint32_t k, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || k == 0 || k > TOKTIER_MAX_TOP)
        return TOKTIER_E_INVALID_ARG;
    *out_bytes = WORKSPACE;
    return TOKTIER_OK;
}

extern "C" int toktier_top_logits(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, uint32_t k, float temperature,
                                  uint32_t *out_ids, uint64_t out_ids_stride, float *out_logits, uint64_t out_logits_stride, float *lse,
                                  void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || k == 0 || k > TOKTIER_MAX_TOP ||
        !temperature_ok(temperature))
        return TOKTIER_E_INVALID_ARG;
    if (n_rows == 0) return TOKTIER_OK;
    if (!matrix_ok(logits, type, n_rows, n_vocab, stride) || !matrix_ok(out_ids, TOKTIER_F32, n_rows, k, out_ids_stride) ||
        !matrix_ok(out_logits, TOKTIER_F32, n_rows, k, out_logits_stride) || !aligned4(lse) || !workspace || ((uintptr_t)workspace & 255u))
        return TOKTIER_E_INVALID_ARG;
    if (workspace_bytes < WORKSPACE) return TOKTIER_E_CAPACITY;
    struct Area {
        const void *p;
        uint64_t n;
    };
    const Area in{logits, extent(type, n_rows, n_vocab, stride)};
    const Area out[] = {{workspace, WORKSPACE}, {out_ids, extent(TOKTIER_F32, n_rows, k, out_ids_stride)},
                        {out_logits, extent(TOKTIER_F32, n_rows, k, out_logits_stride)}, {lse, lse ? 4ull * n_rows : 0}};
    for (int i = 0; i < 4; ++i) {
        if (!apart(out[i].p, out[i].n, in.p, in.n)) return TOKTIER_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return TOKTIER_E_INVALID_ARG;
    }
    hipStream_t s = (hipStream_t)stream;
    const float inv_t = 1.f / temperature;
    with_type(type, [&](auto v) {
        using T = decltype(v);
        auto with_sum = [&](auto sum) {
            constexpr bool SUM = decltype(sum)::value;
            const T *x = (const T *)logits;
            auto launch = [&](auto threads) {
                constexpr int N = decltype(threads)::value;
                in_launches(n_rows, N, [&](uint64_t r, uint32_t rows) {
                    k_top<T, N, SUM><<<rows, N, 0, s>>>(x + r * stride, n_vocab, stride, k, inv_t, out_ids + r * out_ids_stride, out_ids_stride,
                                                           out_logits + r * out_logits_stride, out_logits_stride, lse ? lse + r : nullptr);
                });
            };
            if (n_vocab <= 256 * VEC * 4 && k <= 256) launch(std::integral_constant<int, 256>{});
            else launch(std::integral_constant<int, 1024>{});
        };
        if (lse) with_sum(std::true_type{});
        else with_sum(std::false_type{});
    });
    return hip_status(hipGetLastError());
}
