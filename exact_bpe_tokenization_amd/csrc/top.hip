// top.hip -- the k largest logits of a row, in order, with the row's log-sum-exp.
//
// The row is read once for the threads' own maxima (and sums of exponentials).  Nothing below the threshold can be among
// the first k: every wavefront takes the r-th largest of its lanes' maxima, r = k / wavefronts, and the least of those has
// k elements at or above it.  The elements from there on are listed, from the few threads that have any, and sorted.
// Where they are too many, histograms over narrowing ranges of keys find the border first.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace tt {
namespace {

constexpr uint32_t NONE = 0xFFFFFFFFu;
constexpr uint32_t LIST = 2048;      // listed elements
constexpr uint32_t BINS = 2048;
constexpr uint32_t MOST_RANK = 48;   // of a wavefront's maxima: below that too much is listed to try

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

struct Lds {
    union {
        uint64_t list[LIST];
        uint32_t bins[BINS];
    };
    uint16_t who[1024];
    MaxSum sums[16];
    float bound[16];
    uint32_t part[16];
    uint32_t count, threads, found_bin, found_before;
};

// Sorts the wavefront's values, descending over the lanes, and gives the one of rank r to all.
__device__ __forceinline__ float wave_rank(float v, uint32_t r)
{
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (uint32_t size = 2; size <= 64; size *= 2)
#pragma unroll
        for (uint32_t d = size / 2; d; d /= 2) {
            const float o = __shfl_xor(v, d);
            const bool up = (lane & size) != 0, low = (lane & d) == 0;
            v = (low != up) ? fmaxf(v, o) : fminf(v, o);
        }
    return __shfl(v, r);
}

// Sorts the first n (at most LIST) of list, descending; elements are all different.  Few by their ranks, each against all
// others, more by a bitonic network.
template <int THREADS> __device__ __forceinline__ void sort_list(uint64_t *list, uint32_t n)
{
    if (n <= 256 && n <= THREADS) {
        const uint64_t own = threadIdx.x < n ? list[threadIdx.x] : 0;
        uint32_t rank = 0;
        if (threadIdx.x < n)
            for (uint32_t i = 0; i < n; ++i) rank += list[i] > own;
        __syncthreads();
        if (threadIdx.x < n) list[rank] = own;
        __syncthreads();
        return;
    }
    uint32_t all = 512;
    while (all < n) all *= 2;
    for (uint32_t i = n + threadIdx.x; i < all; i += THREADS) list[i] = 0;
    for (uint32_t size = 2; size <= all; size *= 2)
        for (uint32_t d = size / 2; d; d /= 2) {
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < all / 2; i += THREADS) {
                const uint32_t lo = 2 * i - (i & (d - 1)), hi = lo + d;
                const uint64_t a = list[lo], b = list[hi];
                if ((a < b) == ((lo & size) == 0)) {
                    list[lo] = b;
                    list[hi] = a;
                }
            }
        }
    __syncthreads();
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

// The elements that may be among the first k, in sh.list, their number returned.  Too many: found by histograms.
template <class T, int THREADS>
__device__ __forceinline__ uint32_t list_by_histogram(const T *x, uint32_t begin, uint32_t end, uint32_t k, float least, float most, Lds &sh)
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

// The first k of [begin, end), sorted in sh.list; their number (fewer than k where there are no more) and the part's
// maximum and sum in `all`.
template <class T, int THREADS, int HELD, bool SUM>
__device__ __forceinline__ uint32_t top_of(const T *x, uint32_t begin, uint32_t end, uint32_t k, float k2, Lds &sh, MaxSum &all)
{
    constexpr uint32_t WAVES = THREADS / 64;
    if (threadIdx.x == 0) sh.count = sh.threads = 0;
    RowPart<T, THREADS, HELD> part{x, begin, end};
    MaxSum a{NEG_INF, 0.f};
    part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) {
        if constexpr (SUM) {
            add_vec(a, v, k2);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) a.m = v[e] > a.m ? v[e] : a.m;
        }
    });
    if (SUM && a.s != a.s) {   // a signaling NaN may have taken the place of the maximum (fmaxf), where a comparison passes it by
        a.m = NEG_INF;
        part.template each<false>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) a.m = v[e] > a.m ? v[e] : a.m;
        });
    }
    const float mine = a.m;
    const uint32_t rank = (k + WAVES - 1) / WAVES;
    const float bound = rank <= 64 ? wave_rank(mine, rank - 1) : NEG_INF;
    if ((threadIdx.x & 63) == 0) sh.bound[threadIdx.x >> 6] = bound;
    all = block_join<THREADS>(a, sh.sums, k2);   // with the barrier that sh.bound needs
    float least = sh.bound[0];
#pragma unroll
    for (uint32_t w = 1; w < WAVES; ++w) least = fminf(least, sh.bound[w]);

    const uint32_t vectors = (end - begin + THREADS * VEC - 1) / (THREADS * VEC);   // of a thread, at most
    uint32_t n = NONE;
    if (rank <= MOST_RANK || end - begin <= LIST) {
        if (mine >= least && mine > NEG_INF) sh.who[atomicAdd(&sh.threads, 1u)] = threadIdx.x;
        __syncthreads();
        const uint32_t threads = sh.threads;
        for (uint32_t i = threadIdx.x; i < threads * vectors; i += THREADS) {
            const uint32_t v = i / threads, j = begin + (v * THREADS + sh.who[i - v * threads]) * VEC;
            if (j >= end) continue;
            float e8[VEC];
            load_part(x + j, end - j, NEG_INF, e8);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e8[e] >= least && e8[e] > NEG_INF) {
                    const uint32_t to = atomicAdd(&sh.count, 1u);
                    if (to < LIST) sh.list[to] = element(e8[e], j + e);
                }
        }
        __syncthreads();
        n = sh.count;
    }
    if (n > LIST) n = list_by_histogram<T, THREADS>(x, begin, end, k, least, all.m, sh);
    sort_list<THREADS>(sh.list, n);
    return n;
}

// Place i of the answer.
__device__ __forceinline__ void put(uint32_t i, uint32_t n, const uint64_t *list, uint32_t *ids, float *logits)
{
    ids[i] = i < n ? ~(uint32_t)list[i] : NONE;
    logits[i] = i < n ? logit_of(list[i] >> 32) : NEG_INF;
}

template <class T, int THREADS, int HELD, bool SUM>
__global__ __launch_bounds__(THREADS) void k_top(const T *logits, uint32_t n_vocab, uint64_t stride, uint32_t k, float inv_t, uint32_t *__restrict__ ids,
                                                 uint64_t ids_stride, float *__restrict__ out, uint64_t out_stride, float *__restrict__ lse)
{
    __shared__ Lds sh;
    const uint64_t row = blockIdx.x;
    MaxSum a;
    const uint32_t n = top_of<T, THREADS, HELD, SUM>(logits + row * stride, 0, n_vocab, k, LOG2E * inv_t, sh, a);
    for (uint32_t i = threadIdx.x; i < k; i += THREADS) put(i, n, sh.list, ids + row * ids_stride, out + row * out_stride);
    if (SUM && threadIdx.x == 0) lse[row] = empty(a) ? NEG_INF : a.m * inv_t + log_of(a.s);
}

// Few long rows with a short list: every piece's first k, then the first k of those.
template <class T, bool SUM>
__global__ __launch_bounds__(PIECE_THREADS) void k_top_pieces(const T *logits, uint32_t n_vocab, uint64_t stride, uint32_t k, float inv_t,
                                                              uint64_t *__restrict__ lists, MaxSum *__restrict__ sums)
{
    __shared__ Lds sh;
    const uint64_t row = blockIdx.y, piece = row * gridDim.x + blockIdx.x;
    const uint32_t begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    MaxSum a;
    const uint32_t n = top_of<T, PIECE_THREADS, PIECE_HELD, SUM>(logits + row * stride, begin, end, k, LOG2E * inv_t, sh, a);
    for (uint32_t i = threadIdx.x; i < k; i += PIECE_THREADS) lists[piece * k + i] = i < n ? sh.list[i] : 0;
    if (SUM && threadIdx.x == 0) sums[piece] = a;
}

template <bool SUM>
__global__ __launch_bounds__(PIECE_THREADS) void k_top_join(const uint64_t *__restrict__ lists, const MaxSum *__restrict__ sums, uint32_t pieces,
                                                            uint32_t k, float inv_t, uint32_t *__restrict__ ids, uint64_t ids_stride,
                                                            float *__restrict__ out, uint64_t out_stride, float *__restrict__ lse)
{
    __shared__ Lds sh;
    const uint64_t row = blockIdx.x;
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < pieces * k; i += PIECE_THREADS) {
        const uint64_t e = lists[row * pieces * k + i];
        if (e) sh.list[atomicAdd(&sh.count, 1u)] = e;
    }
    MaxSum a{NEG_INF, 0.f};
    if (SUM && threadIdx.x < pieces) a = sums[row * pieces + threadIdx.x];
    if (SUM) a = block_join<PIECE_THREADS>(a, sh.sums, LOG2E * inv_t);
    __syncthreads();
    const uint32_t n = sh.count;
    sort_list<PIECE_THREADS>(sh.list, n);
    for (uint32_t i = threadIdx.x; i < k; i += PIECE_THREADS) put(i, n, sh.list, ids + row * ids_stride, out + row * out_stride);
    if (SUM && threadIdx.x == 0) lse[row] = empty(a) ? NEG_INF : a.m * inv_t + log_of(a.s);
}

// ---------------------------------------------------------------------------------------------
// host side

constexpr uint32_t MOST_SPLIT = 64;
struct Split {
    uint32_t pieces;   // 0: rows are not split
    uint64_t sums, total;
};
Split layout_of(uint32_t n_rows, uint32_t n_vocab, uint32_t k)
{
    Split L{0, 0, 256};
    const uint32_t pieces = (n_vocab + PIECE - 1) / PIECE;
    if (n_vocab < 8 * PIECE || n_rows > MOST_SPLIT || pieces * k > LIST) return L;
    L.pieces = pieces;
    L.sums = ((uint64_t)n_rows * pieces * k * 8 + 255) & ~255ull;
    L.total = L.sums + (((uint64_t)n_rows * pieces * sizeof(MaxSum) + 255) & ~255ull);
    return L;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int toktier_top_logits_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint32_t k, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || k == 0 || k > TOKTIER_MAX_TOP)
        return TOKTIER_E_INVALID_ARG;
    // what any call of up to n_rows rows, n_vocab IDs and k places needs: pieces * k <= LIST in all of them
    const uint64_t rows = std::clamp(n_rows, 1u, MOST_SPLIT), pieces = (n_vocab + PIECE - 1) / PIECE;
    *out_bytes = 256;
    if (n_vocab >= 8 * PIECE)
        *out_bytes = ((rows * std::min<uint64_t>(LIST, pieces * k) * 8 + 255) & ~255ull) + ((rows * pieces * sizeof(MaxSum) + 255) & ~255ull);
    return TOKTIER_OK;
}

extern "C" int toktier_top_logits(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, uint32_t k, float temperature,
                                  uint32_t *out_ids, uint64_t out_ids_stride, float *out_logits, uint64_t out_logits_stride, float *lse,
                                  void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || k == 0 || k > TOKTIER_MAX_TOP ||
        !(temperature > 0.f && temperature <= 3.4028234e38f && 1.f / temperature <= 3.4028234e38f))
        return TOKTIER_E_INVALID_ARG;
    if (n_rows == 0) return TOKTIER_OK;
    if (!matrix_ok(logits, type, n_rows, n_vocab, stride) || !matrix_ok(out_ids, TOKTIER_F32, n_rows, k, out_ids_stride) ||
        !matrix_ok(out_logits, TOKTIER_F32, n_rows, k, out_logits_stride) || !aligned4(lse) || !workspace || ((uintptr_t)workspace & 255u))
        return TOKTIER_E_INVALID_ARG;
    const Split L = layout_of(n_rows, n_vocab, k);
    if (workspace_bytes < L.total) return TOKTIER_E_CAPACITY;
    struct Area {
        const void *p;
        uint64_t n;
    };
    const Area in{logits, extent(type, n_rows, n_vocab, stride)};
    const Area out[] = {{workspace, L.total}, {out_ids, extent(TOKTIER_F32, n_rows, k, out_ids_stride)},
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
            if (L.pieces) {
                uint64_t *lists = (uint64_t *)workspace;
                MaxSum *sums = (MaxSum *)((uint8_t *)workspace + L.sums);
                k_top_pieces<T, SUM><<<dim3(L.pieces, n_rows), PIECE_THREADS, 0, s>>>(x, n_vocab, stride, k, inv_t, lists, sums);
                k_top_join<SUM><<<n_rows, PIECE_THREADS, 0, s>>>(lists, sums, L.pieces, k, inv_t, out_ids, out_ids_stride, out_logits,
                                                                 out_logits_stride, lse);
                return;
            }
            auto launch = [&](auto threads, auto held) {
                constexpr int N = decltype(threads)::value, H = decltype(held)::value;
                in_launches(n_rows, N, [&](uint64_t r, uint32_t rows) {
                    k_top<T, N, H, SUM><<<rows, N, 0, s>>>(x + r * stride, n_vocab, stride, k, inv_t, out_ids + r * out_ids_stride, out_ids_stride,
                                                           out_logits + r * out_logits_stride, out_logits_stride, lse ? lse + r : nullptr);
                });
            };
            if (n_vocab <= 256 * VEC * 4) launch(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
            else launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
        };
        if (lse) with_sum(std::true_type{});
        else with_sum(std::false_type{});
    });
    return hip_status(hipGetLastError());
}
