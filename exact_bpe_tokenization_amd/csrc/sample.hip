// sample.hip -- sampling of one ID per row: temperature, top-k, top-p, min-p, given random numbers.
//
// Every filter keeps a prefix of the order (logit descending, ID ascending), so the kept set is one pair: a
// logit (as an integer key of the same order) and how many of its equals, lowest IDs first.  Masses are
// sums of 64-bit integers, w = 2^y rounded to a multiple of 2^-S with y = (x - max) log2(e) / temperature in
// 64-bit floating point: exact in any order, so neither atomics nor the split of a row over threads can
// change an ID.
//
// One workgroup per row; a wavefront owns a contiguous segment of it, in registers where the row fits.
//   1. keys and the largest of them;
//   2. for top-k and top-p, a histogram over 4,095 bins of the key (sign, exponent, 7 mantissa bits) with
//      counts and masses; a scan from the top finds the bin where a filter ends, and a digit search over
//      that bin's keys the exact key and its equals (nothing to search for bfloat16, whose bins hold one key);
//   3. the ID by the running mass over IDs: per wavefront, then inside the one wavefront that holds it.
#include <type_traits>

#include "ops.h"

namespace tt {
namespace {

#define INLINE __attribute__((always_inline))   // of a lambda: the keys it sees stay in registers

constexpr uint32_t NO_ID = 0xFFFFFFFFu;
constexpr int BINS = 4096, HALF = BINS / 2 - 1;   // bins of a sign; bin 0 holds the largest keys
constexpr int DIGIT = 11, DIGITS = 1 << DIGIT;

// A key is the logit's sign and magnitude bits as an integer: the order of the logits, -0 equal to +0.
// Bins: magnitudes below 2^-9 share the middle one, those from 2^7 on the outermost, and between them a bin
// has 128 per octave.
template <class T> struct Keys;
template <> struct Keys<__bf16> {
    static constexpr int INF = 0x7F80, LOW = 0x3B00, SHIFT = 0;
    static __device__ __forceinline__ float value(int k)
    {
        const uint32_t m = (uint32_t)(k < 0 ? -k : k);
        return __builtin_bit_cast(float, m << 16 | ((uint32_t)k & 0x80000000u));
    }
};
template <> struct Keys<_Float16> {
    static constexpr int INF = 0x7C00, LOW = 0x1800, SHIFT = 3;
    static __device__ __forceinline__ float value(int k)
    {
        const uint32_t m = (uint32_t)(k < 0 ? -k : k);
        const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)m);
        return k < 0 ? -f : f;
    }
};
template <> struct Keys<float> {
    static constexpr int INF = 0x7F800000, LOW = 118 << 23, SHIFT = 16;
    static __device__ __forceinline__ float value(int k)
    {
        const uint32_t m = (uint32_t)(k < 0 ? -k : k);
        return __builtin_bit_cast(float, m | ((uint32_t)k & 0x80000000u));
    }
};

template <class T> __device__ __forceinline__ int bin_of(int k)
{
    using K = Keys<T>;
    const int sign = k >> 31, mag = (k ^ sign) - sign;
    int m = (mag - (K::LOW - (1 << K::SHIFT))) >> K::SHIFT;
    m = m < 0 ? 0 : m > HALF ? HALF : m;
    return HALF - ((m ^ sign) - sign);
}

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Eight keys: packed in pairs for the 16-bit types.
template <class T> struct Vec8 {
    u32x4 a;
    __device__ __forceinline__ s16x2 pair(int i) const
    {
        const uint32_t w = a[i];   // (a bit cast of the vector's element itself would read element 0)
        return __builtin_bit_cast(s16x2, w);
    }
    __device__ __forceinline__ int at(int e) const
    {
        return (e & 1) ? (int)a[e >> 1] >> 16 : (int)(int16_t)(a[e >> 1] & 0xFFFFu);
    }
    __device__ __forceinline__ int pick(int e) const   // at(), for an index known at run time only
    {
        const uint32_t w = e & 4 ? (e & 2 ? a[3] : a[2]) : (e & 2 ? a[1] : a[0]);
        return (e & 1) ? (int)w >> 16 : (int)(int16_t)(w & 0xFFFFu);
    }
    __device__ __forceinline__ void hide(int e) { a[e >> 1] = (e & 1) ? (a[e >> 1] & 0xFFFFu) | 0x80000000u : (a[e >> 1] & 0xFFFF0000u) | 0x8000u; }
    __device__ __forceinline__ int max() const
    {
        s16x2 m = pair(0);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, pair(i));
        return m.x > m.y ? m.x : m.y;
    }
    // logits to keys, in place
    __device__ __forceinline__ void order()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 b = pair(i), sign = b >> 15;
            const s16x2 m = __builtin_bit_cast(s16x2, a[i] & 0x7FFF7FFFu);
            a[i] = __builtin_bit_cast(uint32_t, (m ^ sign) - sign);
        }
    }
    __device__ __forceinline__ void bins(int (&b)[VEC]) const
    {
        using K = Keys<T>;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 k = pair(i), sign = k >> 15;
            const u16x2 mag = __builtin_bit_cast(u16x2, __builtin_elementwise_max(k, (s16x2)-k));
            u16x2 m = __builtin_elementwise_sub_sat(mag, (u16x2)(unsigned short)(K::LOW - (1 << K::SHIFT)));
            m = __builtin_elementwise_min((u16x2)(m >> K::SHIFT), (u16x2)(unsigned short)HALF);
            const s16x2 t = (s16x2)(short)HALF - ((__builtin_bit_cast(s16x2, m) ^ sign) - sign);
            b[2 * i] = t.x;
            b[2 * i + 1] = t.y;
        }
    }
};
template <> struct Vec8<float> {
    u32x4 a, b;
    __device__ __forceinline__ int at(int e) const { return e < 4 ? (int)a[e] : (int)b[e - 4]; }
    __device__ __forceinline__ int pick(int e) const
    {
        const uint32_t l = e & 2 ? (e & 1 ? a[3] : a[2]) : (e & 1 ? a[1] : a[0]);
        const uint32_t h = e & 2 ? (e & 1 ? b[3] : b[2]) : (e & 1 ? b[1] : b[0]);
        return (int)(e & 4 ? h : l);
    }
    __device__ __forceinline__ void set(int e, int v)
    {
        if (e < 4) a[e] = (uint32_t)v;
        else b[e - 4] = (uint32_t)v;
    }
    __device__ __forceinline__ void hide(int e) { set(e, (int)0x80000000); }
    __device__ __forceinline__ int max() const
    {
        int m = at(0);
#pragma unroll
        for (int e = 1; e < VEC; ++e) m = at(e) > m ? at(e) : m;
        return m;
    }
    __device__ __forceinline__ void order()
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int x = at(e), sign = x >> 31;
            set(e, ((x & 0x7FFFFFFF) ^ sign) - sign);
        }
    }
    __device__ __forceinline__ void bins(int (&out)[VEC]) const
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = bin_of<float>(at(e));
    }
};

// Keys of a bin: lo .. hi.
template <class T> __device__ __forceinline__ void bin_range(int b, int &lo, int &hi)
{
    using K = Keys<T>;
    const int s = HALF - b, m = s < 0 ? -s : s;
    const int a = m == 0 ? -(K::LOW - 1) : K::LOW + ((m - 1) << K::SHIFT);
    const int z = m == 0 ? K::LOW - 1 : m == HALF ? K::INF : K::LOW + (m << K::SHIFT) - 1;
    lo = s < 0 ? -z : a;
    hi = s < 0 ? -a : z;
}
// bfloat16: one key per bin, but for the middle and the outermost ones
template <class T> __device__ __forceinline__ bool bin_exact(int b)
{
    return __is_same(T, __bf16) && b != HALF && b != 0 && b != 2 * HALF;
}

// Weights of one row.  2^y = 2^n 2^f with n the nearest integer: 2^f on [-1/2, 1/2] by the polynomial of degree
// 10 that interpolates it at the Chebyshev nodes (relative error below 2^-51), the multiple of 2^-S by
// adding 2^(52 - S) and reading the low bits.
struct Weights {
    double c, max, magic;
    int max_key;

    __device__ __forceinline__ uint64_t one() const
    {
        return __builtin_bit_cast(uint64_t, 1.0 + magic) - __builtin_bit_cast(uint64_t, magic);
    }
    __device__ __forceinline__ uint64_t of(int key, float x) const
    {
        const double y = ((double)x - max) * c;
        const double n = __builtin_rint(y), f = y - n;
        double p = 7.072585949269224e-09;
        p = __builtin_fma(p, f, 1.0208690299958306e-07);
        p = __builtin_fma(p, f, 1.321544258792169e-06);
        p = __builtin_fma(p, f, 1.5252657260200837e-05);
        p = __builtin_fma(p, f, 0.0001540353044173605);
        p = __builtin_fma(p, f, 0.0013333558230164974);
        p = __builtin_fma(p, f, 0.009618129107606888);
        p = __builtin_fma(p, f, 0.05550410866444772);
        p = __builtin_fma(p, f, 0.24022650695910097);
        p = __builtin_fma(p, f, 0.69314718055995);
        p = __builtin_fma(p, f, 1.0);
        const double w = __builtin_amdgcn_ldexp(p, (int)n);
        const uint64_t q = __builtin_bit_cast(uint64_t, w + magic) - __builtin_bit_cast(uint64_t, magic);
        return key == max_key ? one() : y > -64.0 ? q : 0ull;   // the largest may be +inf; y may be -inf or NaN
    }
};

template <class V> __device__ __forceinline__ V wave_scan(V v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const V o = __shfl_up(v, d);
        if ((int)(threadIdx.x & 63) >= d) v += o;
    }
    return v;
}
template <class V> __device__ __forceinline__ V wave_sum(V v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

template <int WAVES> struct Shared {
    uint64_t mass[BINS];                                     // per bin; for the draw, the weight of its key
    union {
        uint32_t count[BINS];
        uint64_t digit[DIGITS];
    };
    uint64_t wave[WAVES];
    uint64_t above, inside;
    uint32_t found;
    int key;
};

// Sum over the threads below this one; total: over all.
template <int WAVES> __device__ __forceinline__ uint64_t block_before(uint64_t v, Shared<WAVES> &sh, uint64_t &total)
{
    const uint32_t wave = threadIdx.x >> 6;
    const uint64_t incl = wave_scan(v);
    if ((threadIdx.x & 63) == 63) sh.wave[wave] = incl;
    __syncthreads();
    uint64_t base = 0;
    total = 0;
#pragma unroll 4
    for (uint32_t w = 0; w < WAVES; ++w) {
        const uint64_t s = sh.wave[w];
        if (w < wave) base += s;
        total += s;
    }
    __syncthreads();
    return base + incl - v;
}

// The first of n bins (value(b), b ascending) at which the running sum reaches target(total), the sum before it
// and the bin's own value.  n / threads consecutive bins per thread.  False when the total is below target.
template <int N, int WAVES, class F, class G>
__device__ __forceinline__ bool find_bin(Shared<WAVES> &sh, F value, G target_of, uint32_t &bin, uint64_t &above,
                                         uint64_t &inside, uint64_t &target)
{
    constexpr int PER = N / (WAVES * 64);
    uint64_t v[PER], sum = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = value(threadIdx.x * PER + i);
        sum += v[i];
    }
    uint64_t run = block_before(sum, sh, total);
    target = target_of(total);
    if (target > total) return false;
    if (run < target && target <= run + sum) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (run < target && target <= run + v[i]) {
                sh.found = threadIdx.x * PER + i;
                sh.above = run;
                sh.inside = v[i];
            }
            run += v[i];
        }
    }
    __syncthreads();
    bin = sh.found;
    above = sh.above;
    inside = sh.inside;
    __syncthreads();
    return true;
}

// One row.  NV > 0: its keys stay in registers (NV vectors per thread at most); NV == 0: every pass reads them.
template <class T, int WAVES, int NV> struct Row {
    static constexpr int HELD = NV ? NV : 1;
    const T *x;
    const uint32_t *mask;
    uint32_t n, nv, first;   // elements, vectors per thread, this thread's first element
    bool nan;                // a positive NaN may be among the keys of a 16-bit type
    using V = Vec8<T>;
    V held[HELD];

    __device__ __forceinline__ uint32_t at(uint32_t i) const { return first + i * (64 * VEC); }

    __device__ __forceinline__ Vec8<T> raw(uint32_t j) const
    {
        Vec8<T> v;
        if (j + VEC <= n) {
            if constexpr (sizeof(T) == 4) {
                v.a = *(const u32x4_row *)(x + j);
                v.b = *(const u32x4_row *)(x + j + 4);
            } else {
                v.a = *(const u32x4_row *)(x + j);
            }
        } else {
            uint32_t e[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                if constexpr (sizeof(T) == 4) e[k] = j + k < n ? __builtin_bit_cast(uint32_t, x[j + k]) : 0xFF800000u;
                else e[k] = j + k < n ? (uint32_t)__builtin_bit_cast(uint16_t, x[j + k]) : 0x8000u | (uint32_t)Keys<T>::INF;
            }
            if constexpr (sizeof(T) == 4) {
                v.a = u32x4{e[0], e[1], e[2], e[3]};
                v.b = u32x4{e[4], e[5], e[6], e[7]};
            } else {
                v.a = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
            }
        }
        return v;
    }
    __device__ __forceinline__ void finish(Vec8<T> &v, uint32_t j) const
    {
        v.order();
        if (nan || sizeof(T) == 4) drop_nan(v);
        if (mask && j < n) {
            const uint32_t bits = mask[j >> 5] >> (j & 31u);
            if ((bits & 0xFFu) != 0xFFu) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (!((bits >> e) & 1u)) v.hide(e);
            }
        }
    }
    static __device__ __forceinline__ void drop_nan(Vec8<T> &v)
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (v.at(e) > Keys<T>::INF) v.hide(e);
    }
    __device__ __forceinline__ void load()
    {
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < (int)nv) held[i] = raw(at(i));
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < (int)nv) finish(held[i], at(i));
        }
    }
    // Keeps the compiler from carrying what it derived from the keys in one pass over to the next: those
    // values would need several times the registers of the keys themselves.
    static __device__ __forceinline__ void forget(V &v)
    {
        asm volatile("" : "+v"(v.a));
        if constexpr (sizeof(T) == 4) asm volatile("" : "+v"(v.b));
    }
    // f(index of the first element, keys) over this thread's vectors, ascending
    template <class F> __device__ __forceinline__ void each(F f)
    {
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < (int)nv) {
                    forget(held[i]);
                    f(at(i), held[i]);
                }
        } else {
            for (uint32_t i = 0; i < nv; ++i) {
                Vec8<T> v = raw(at(i));
                finish(v, at(i));
                f(at(i), v);
            }
        }
    }
};

// The index at which the running sum (over IDs) of the elements' measure exceeds target(total), and its key.
// sum(vector, index): a vector's, 0 at once where no lane has any; element(vector, index, e): one element's.
// Per wavefront first; then only the wavefront that holds it looks closer.
template <int WAVES, class R, class S, class E, class G>
__device__ __forceinline__ uint32_t locate(R &row, Shared<WAVES> &sh, S sum_of, E element, G target_of, uint64_t &total, int &key)
{
    const uint32_t wave = threadIdx.x >> 6;
    uint64_t sum = 0;
    row.each([&](uint32_t j, const auto &v) INLINE { sum += sum_of(v, j); });
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sh.wave[wave] = sum;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll 4
    for (uint32_t w = 0; w < WAVES; ++w) {
        const uint64_t s = sh.wave[w];
        if (w < wave) before += s;
        total += s;
    }
    const uint64_t target = target_of(total);
    if (before <= target && target < before + sum) {
        // by thread: the vector in which its share of the wavefront's running sum passes the target
        typename R::V hit{};
        uint64_t hit_at = 0, run = before;
        uint32_t hit_j = NO_ID;
        row.each([&](uint32_t j, const auto &v) INLINE {
            const uint64_t mine = sum_of(v, j);
            if (!__any(mine != 0)) return;
            const uint64_t incl = run + wave_scan(mine);
            if (incl - mine <= target && target < incl) {
                hit = v;
                hit_at = incl - mine;
                hit_j = j;
            }
            run = __shfl(incl, 63);
        });
        if (hit_j != NO_ID) {
#pragma unroll 1
            for (int e = 0; e < VEC; ++e) {
                hit_at += element(hit, hit_j, e);
                if (hit_at > target) {
                    sh.found = hit_j + e;
                    sh.key = hit.pick(e);
                    break;
                }
            }
        }
    }
    __syncthreads();
    const uint32_t id = sh.found;
    key = sh.key;
    __syncthreads();
    return id;
}

template <class T, int WAVES, int NV>
__global__ __launch_bounds__(WAVES * 64) void k_sample(const T *__restrict__ logits, uint32_t n_vocab, uint64_t stride,
                                                       const uint32_t *__restrict__ mask, uint64_t mask_stride,
                                                       const float *__restrict__ temperature,
                                                       const uint32_t *__restrict__ top_k, const float *__restrict__ top_p,
                                                       const float *__restrict__ min_p, const float *__restrict__ uniform,
                                                       uint32_t *__restrict__ out_ids, float *__restrict__ out_logprobs,
                                                       double magic)
{
    using K = Keys<T>;
    using V = Vec8<T>;
    constexpr int THREADS = WAVES * 64;
    constexpr bool TABLE = __is_same(T, __bf16);   // a weight per bin
    __shared__ Shared<WAVES> sh;
    const uint64_t r = blockIdx.x;
    Row<T, WAVES, NV> row;
    row.x = logits + r * stride;
    row.mask = mask ? mask + r * mask_stride : nullptr;
    row.n = n_vocab;
    row.nv = (n_vocab + THREADS * VEC - 1) / (THREADS * VEC);
    row.first = (threadIdx.x >> 6) * (row.nv * 64 * VEC) + (threadIdx.x & 63) * VEC;
    row.nan = false;
    row.load();
    const float temp = temperature ? temperature[r] : 1.f;
    const uint32_t k = top_k ? top_k[r] : 0;
    const float p = top_p ? top_p[r] : 1.f, mp = min_p ? min_p[r] : 0.f, u_in = uniform[r];

    // 1. the largest key, of each thread and of all
    int mine, top;
    for (;;) {
        mine = (int)0x80000000;
        row.each([&](uint32_t, const V &v) INLINE {
            const int m = v.max();
            mine = m > mine ? m : mine;
        });
        int m = mine;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const int o = __shfl_xor(m, d);
            m = o > m ? o : m;
        }
        if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = (uint32_t)m;
        __syncthreads();
        top = (int)(uint32_t)sh.wave[0];
#pragma unroll 4
        for (int w = 0; w < WAVES; ++w) top = (int)(uint32_t)sh.wave[w] > top ? (int)(uint32_t)sh.wave[w] : top;
        __syncthreads();
        if (sizeof(T) == 4 || top <= K::INF) break;
        row.nan = true;   // NaN of 16 bits: take them out and look again
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < (int)row.nv) row.drop_nan(row.held[i]);
        }
    }
    constexpr int LOWEST = -K::INF + 1;   // the smallest key in the choice
    if (top < LOWEST) {                   // nothing to choose from
        if (threadIdx.x == 0) {
            out_ids[r] = NO_ID;
            if (out_logprobs) out_logprobs[r] = -__builtin_inff();
        }
        return;
    }
    const bool first_alone = k == 1 || !(temp > 0.f);
    const Weights wt{1.4426950408889634 / (double)temp, (double)K::value(top), magic, top};
    auto weight = [&](int key) INLINE { return wt.of(key, K::value(key)); };

    // 2. kept so far: keys above key_f, and of those equal to it (count_f of them) the first `ties`
    int key_f = first_alone ? top : LOWEST;
    uint64_t ties = 1, count_f = first_alone ? 2 : 0;   // count_f 0: no filter so far, all are kept
    const bool need_k = !first_alone && k != 0 && k < n_vocab, need_p = !first_alone && p < 1.f;
    if (need_k || need_p) {
        int floor = LOWEST;
        bool found;
        uint32_t bin_k = BINS;
        uint64_t above, inside, target;
        auto count_of = [&](int i) INLINE { return (uint64_t)sh.count[i]; };
        auto target_k = [&](uint64_t) INLINE { return (uint64_t)k; };
        auto clear_counts = [&]() INLINE {
            for (int b = threadIdx.x; b < BINS; b += THREADS) sh.count[b] = 0;
            __syncthreads();
        };
        // Two rounds for a small k: k threads with a key >= f hold at least k such keys, so nothing below the
        // k-th largest of the threads' own largest keys (or its bin's lowest key) can be kept.
        for (int round = need_k && k <= THREADS / 2 ? 0 : 1;; ++round) {
            if (need_p && round)
                for (int b = threadIdx.x; b < BINS; b += THREADS) sh.mass[b] = 0;
            clear_counts();
            if (round == 0) {
                if (mine >= LOWEST) atomicAdd(&sh.count[bin_of<T>(mine)], 1u);
            } else {
                row.each([&](uint32_t, const V &v) INLINE {
                    if (!__any(v.max() >= floor)) return;
                    int b[VEC];
                    v.bins(b);
                    bool more = false;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (v.at(e) >= floor) {
                            atomicAdd(&sh.count[b[e]], 1u);
                            more |= !bin_exact<T>(b[e]);
                        }
                    if (need_p && __any(more)) {
#pragma unroll 1
                        for (int e = 0; e < VEC; ++e) {
                            const int key = v.pick(e), bin = bin_of<T>(key);
                            if (key >= floor && !bin_exact<T>(bin))
                                atomicAdd((unsigned long long *)&sh.mass[bin], (unsigned long long)weight(key));
                        }
                    }
                });
            }
            __syncthreads();
            found = need_k && find_bin<BINS>(sh, count_of, target_k, bin_k, above, inside, target);
            if (round) break;
            if (found) {
                int hi;
                bin_range<T>((int)bin_k, floor, hi);
                floor = floor < LOWEST ? LOWEST : floor;
            }
        }
        if (need_p && TABLE) {
#pragma unroll 1
            for (int b = threadIdx.x; b < BINS - 1; b += THREADS)
                if (bin_exact<T>(b) && sh.count[b]) {
                    int lo, hi;
                    bin_range<T>(b, lo, hi);
                    sh.mass[b] = sh.count[b] * weight(lo);
                }
            __syncthreads();
        }
        // Stage 0 by counts, stage 1 by masses: the bin where the filter ends, then the exact key in it, by the
        // running sum over the digits of hi - key, highest digit first (overwrites the counts).
        const bool cut_k = found;
        uint64_t excess = 0, mass_k = 0;   // mass of what lies beyond the ties of key_f; of the kept part of bin_k
        int from = LOWEST;
        for (int stage = cut_k ? 0 : 1; stage < (need_p ? 2 : 1); ++stage) {
            uint32_t bin = bin_k;
            if (stage) {
                find_bin<BINS>(sh, [&](int i) INLINE {
                    return !cut_k || i < (int)bin_k ? sh.mass[i] : i == (int)bin_k ? mass_k : 0ull;
                }, [&](uint64_t all) INLINE {
                    const double t = __builtin_ceil((double)p * (double)all);
                    const uint64_t q = t > 1.0 ? (uint64_t)t : 1ull;
                    return q < all ? q : all;
                }, bin, above, inside, target);
            }
            int lo, hi;
            bin_range<T>((int)bin, lo, hi);
            uint64_t left = target - above;   // to be reached inside the bin
            const int key_k = key_f;
            const bool last = stage && cut_k && bin == bin_k;
            if (last && from < key_k) from = key_k;
            key_f = lo;
            if (!bin_exact<T>((int)bin)) {
                const int bits = 32 - __builtin_clz((uint32_t)(hi - lo));
                int shift = (bits + DIGIT - 1) / DIGIT * DIGIT;
                uint32_t prefix = 0;
                while (shift > 0) {
                    const int up = shift;
                    shift -= DIGIT;
                    for (int b = threadIdx.x; b < DIGITS; b += THREADS) sh.digit[b] = 0;
                    __syncthreads();
                    auto add = [&](int key, uint64_t amount) INLINE {
                        const uint32_t d = (uint32_t)(hi - key);
                        if ((up < 32 ? d >> up : 0u) == prefix)
                            atomicAdd((unsigned long long *)&sh.digit[(d >> shift) & (DIGITS - 1)], (unsigned long long)amount);
                    };
                    row.each([&](uint32_t, const V &v) INLINE {
                        if (!__any(v.max() >= lo)) return;
#pragma unroll 1
                        for (int e = 0; e < VEC; ++e) {
                            const int key = v.pick(e);
                            if (key >= lo && key <= hi && key >= from) add(key, stage ? weight(key) : 1ull);
                        }
                    });
                    if (threadIdx.x == 0 && last && excess) add(key_k, 0ull - excess);
                    __syncthreads();
                    uint32_t digit;
                    uint64_t a, t;
                    find_bin<DIGITS>(sh, [&](int i) INLINE { return sh.digit[i]; }, [&](uint64_t) INLINE { return left; }, digit, a,
                                     inside, t);
                    left -= a;
                    prefix = prefix << DIGIT | digit;
                }
                key_f = hi - (int)prefix;
            }
            if (stage == 0) {
                ties = left;
                count_f = inside;
                if (need_p) {   // what its bin holds below key_f, and of its equals beyond the ties, is no longer kept
                    const uint64_t w = weight(key_f);
                    excess = (count_f - ties) * w;
                    mass_k = ties * w;
                    if (!bin_exact<T>((int)bin)) {
                        uint64_t part = 0;
                        row.each([&](uint32_t, const V &v) INLINE {
                            if (!__any(v.max() >= key_f)) return;
#pragma unroll 1
                            for (int e = 0; e < VEC; ++e) {
                                const int key = v.pick(e);
                                if (key >= key_f && key <= hi) part += weight(key);
                            }
                        });
                        block_before(part, sh, mass_k);
                        mass_k -= excess;
                    }
                }
            } else {
                const uint64_t w = weight(key_f), need = (left + w - 1) / w;
                if (last && key_f == key_k) {
                    ties = need < ties ? need : ties;
                } else {
                    count_f = inside / w;
                    ties = need;
                }
            }
        }
    }
    uint32_t id = NO_ID;   // the last index whose key may equal key_f
    uint64_t total;
    int key_at;
    if (ties < count_f)
        id = locate<WAVES>(row, sh, [&](const V &v, uint32_t) INLINE {
            uint64_t n = 0;
            if (__any(v.max() >= key_f)) {
                uint32_t c = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) c += v.at(e) == key_f;
                n = c;
            }
            return n;
        }, [&](const V &v, uint32_t, int e) INLINE { return (uint64_t)(v.pick(e) == key_f); },
        [&](uint64_t) INLINE { return ties - 1; }, total, key_at);
    if (first_alone) {
        if (threadIdx.x == 0) {
            out_ids[r] = id;
            if (out_logprobs) out_logprobs[r] = 0.f;
        }
        return;
    }

    // 3. the draw
    const uint32_t cut = id;
    const uint64_t one = wt.one();
    const uint64_t w_min = mp >= 1.f ? one : mp > 0.f ? (uint64_t)__builtin_ceil((double)mp * (double)one) : 0;
    const double u = u_in > 0.f ? (double)fminf(u_in, 0x1.fffffep-1f) : 0.0;
    if (TABLE) {   // the weights of the kept bins, so that no element needs its own exponential
        __syncthreads();
#pragma unroll 1
        for (int b = threadIdx.x; b < BINS - 1; b += THREADS) {
            int lo, hi;
            bin_range<T>(b, lo, hi);
            if (bin_exact<T>(b) && lo <= top) {
                const uint64_t w = lo >= key_f ? weight(lo) : 0;
                sh.mass[b] = w >= w_min ? w : 0;
            }
        }
        __syncthreads();
    }
    auto kept = [&](int key, uint32_t j) INLINE { return key > key_f || (key == key_f && j <= cut); };
    auto element = [&](const V &v, uint32_t j, int e) INLINE {
        const int key = v.pick(e);
        const uint64_t w = weight(key);
        return kept(key, j + e) && w >= w_min ? w : 0ull;
    };
    id = locate<WAVES>(row, sh, [&](const V &v, uint32_t j) INLINE {
        uint64_t sum = 0;
        if (!__any(v.max() >= key_f)) return sum;
        bool each = !TABLE;
        if (TABLE) {
            int b[VEC];
            v.bins(b);
            bool odd = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const bool in = kept(v.at(e), j + e);
                odd |= in && !bin_exact<T>(b[e]);
                if (in) sum += sh.mass[b[e]];
            }
            each = __any(odd);
            if (each) sum = 0;
        }
        if (each) {
#pragma unroll 1
            for (int e = 0; e < VEC; ++e) sum += element(v, j, e);
        }
        return sum;
    }, element, [&](uint64_t all) INLINE { return (uint64_t)(u * (double)all); }, total, key_at);
    if (threadIdx.x == 0) {
        out_ids[r] = id;
        if (out_logprobs) out_logprobs[r] = (float)log((double)weight(key_at) / (double)total);
    }
}

// S = 45 fraction bits keep the sum of up to 2^18 weights of at most one below 2^63; one bit less for every doubling.
double weight_magic(uint32_t n_vocab)
{
    int s = 45;
    for (uint32_t v = 1u << 18; v < n_vocab; v <<= 1) --s;
    return (double)(1ull << (52 - s));
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int toktier_sample_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu) return TOKTIER_E_INVALID_ARG;
    *out_bytes = 256;
    return TOKTIER_OK;
}

extern "C" int toktier_sample(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride,
                              const uint32_t *mask, uint64_t mask_stride, const float *temperature,
                              const uint32_t *top_k, const float *top_p, const float *min_p, const float *uniform,
                              uint32_t *out_ids, float *out_logprobs, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu) return TOKTIER_E_INVALID_ARG;
    if (n_rows == 0) return TOKTIER_OK;
    if (!matrix_ok(logits, type, n_rows, n_vocab, stride)) return TOKTIER_E_INVALID_ARG;
    if (!uniform || !out_ids) return TOKTIER_E_INVALID_ARG;
    if (!aligned4(mask) || !aligned4(temperature) || !aligned4(top_k) || !aligned4(top_p) || !aligned4(min_p) ||
        !aligned4(uniform) || !aligned4(out_ids) || !aligned4(out_logprobs))
        return TOKTIER_E_INVALID_ARG;
    const uint64_t words = (n_vocab + 31) / 32;
    if (mask && mask_stride != 0 && (mask_stride < words || mask_stride > (1ull << 40))) return TOKTIER_E_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
    if (workspace_bytes < 256) return TOKTIER_E_CAPACITY;
    const uint64_t lb = extent(type, n_rows, n_vocab, stride), ob = 4ull * n_rows;
    if (!apart(out_ids, ob, logits, lb) || (out_logprobs && (!apart(out_logprobs, ob, logits, lb) || !apart(out_logprobs, ob, out_ids, ob))))
        return TOKTIER_E_INVALID_ARG;
    const double magic = weight_magic(n_vocab);
    with_type(type, [&](auto t) {
        using T = decltype(t);
        auto launch = [&](auto waves, auto nv) {
            k_sample<T, decltype(waves)::value, decltype(nv)::value><<<n_rows, decltype(waves)::value * 64, 0, (hipStream_t)stream>>>(
                (const T *)logits, n_vocab, stride, mask, mask_stride, temperature, top_k, top_p, min_p, uniform, out_ids, out_logprobs,
                magic);
        };
        constexpr bool F32 = sizeof(T) == 4;
        const uint32_t nv = (n_vocab + 1024 * VEC - 1) / (1024 * VEC);
        if (n_vocab <= 256 * VEC * 4) launch(std::integral_constant<int, 4>{}, std::integral_constant<int, F32 ? 0 : 4>{});
        else if (!F32 && nv <= 5) launch(std::integral_constant<int, 16>{}, std::integral_constant<int, F32 ? 0 : 5>{});
        else launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 0>{});
    });
    return hip_status(hipGetLastError());
}
