// sample.hip -- sampling of one ID per row: temperature, top-k, top-p, min-p, given random numbers.
//
// Every filter keeps a prefix of the order (logit descending, ID ascending), so the kept set is one pair: a
// logit (as an integer key of the same order) and the last ID that may have it.  Masses are sums of 64-bit
// integers, w = 2^y rounded to a multiple of 2^-S with y = (x - max) log2(e) / temperature in 64-bit floating
// point: exact in any order, so neither atomics nor the split of a row over threads can change an ID.
//
// A row goes through four phases:
//   keys    the largest key, and a histogram of the keys over 6,143 bins (sign, exponent, 7 mantissa bits);
//   border  the bins in which top-k (by counts) and top-p (by masses) end;
//   cells   per cell of consecutive IDs, the mass of what lies above the border, and a list of what lies in it;
//   draw    the list sorted gives the exact border; the running mass over the cells, then inside one, gives the ID.
// A bin of bfloat16 holds one key, so that its mass is its count times one weight and its list is not needed.
// The least temperature, or k = 1, ends after the first phase; without top-k and top-p there is no border; a small k
// needs no histogram (list_first); rows that the phases do not fit (NaN, a border of thousands of equals) take
// general_row.
//
// A workgroup of 1,024 threads takes a row (256 threads up to 8,192 elements), so a row's time is the time of its chain of
// phases, and the rows of a batch of up to 256 run side by side.  131,328 bfloat16, one row and 256 of them (67 MB): first
// alone 8.5 and 16.3 us (4.1 TB/s), temperature with top-k 50 and top-p 0.95 18.3 and 28.5, top-k 1,000 with top-p 0.9 40 and
// 50, top-p 0.95 50 and 56, full distribution 29 and 40.  What bounds them: the loads of one CU in the keys phase without
// a histogram (5.8 us of a row); the LDS atomics of the histogram (the keys phase takes 16 us of a row alone, 20 in a
// batch of 256); in the cells phase VALU issue, some 100 instructions for a vector of eight (19 and 21 us); for float32
// and float16 the exponentials in 64 bits, 30 instructions each; else the latency of some ten barriers.  Every variant
// uses scratch: 128 VGPRs and 7 to 21 spilled ones (96 to 128 bytes a lane) at 16 wavefronts, 184 to 200 VGPRs and 64 bytes
// at four.  Not split over workgroups: a second launch costs 3 us, and a phase needs the one before from the whole row.
#include <type_traits>

#include "ops.h"

namespace tt {
namespace {

#define INLINE __attribute__((always_inline))   // of a lambda

constexpr uint32_t NO_ID = 0xFFFFFFFFu;
constexpr int BINS = 6144, HALF = BINS / 2 - 1;   // bins of a sign; bin 0 holds the largest keys
constexpr int DIGIT = 12, DIGIT_VALUES = 1 << DIGIT;
constexpr uint32_t LIST = 2048;                   // elements that a border may have to be sorted
constexpr uint32_t ODD = 512;                     // bfloat16: listed elements of bins with several keys
constexpr uint32_t MAX_CELLS = 256;               // of 8,192 elements

// A key is the logit's sign and magnitude bits as an integer: the order of the logits, -0 equal to +0.
// Bins: magnitudes below LOW (2^-13) share the middle one, those from 2^11 on (nearly) the outermost, and between
// them there are 128 per octave.
template <class T> struct Keys;
template <> struct Keys<__bf16> {
    static constexpr int INF = 0x7F80, LOW = (127 - 13) << 7, SHIFT = 0;
    static __device__ __forceinline__ float value(int k)
    {
        const uint32_t m = (uint32_t)(k < 0 ? -k : k);
        return __builtin_bit_cast(float, m << 16 | ((uint32_t)k & 0x80000000u));
    }
};
template <> struct Keys<_Float16> {
    static constexpr int INF = 0x7C00, LOW = (15 - 13) << 10, SHIFT = 3;
    static __device__ __forceinline__ float value(int k)
    {
        const uint32_t m = (uint32_t)(k < 0 ? -k : k);
        const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)m);
        return k < 0 ? -f : f;
    }
};
template <> struct Keys<float> {
    static constexpr int INF = 0x7F800000, LOW = (127 - 13) << 23, SHIFT = 16;
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
    const int s = b - HALF, m = s < 0 ? -s : s;
    return __is_same(T, __bf16) && (uint32_t)(m - 1) < (uint32_t)(HALF - 1);
}

// Whether weights come from a table of the bins: bfloat16 rows with more elements than bins.  (For shorter rows the table
// costs more than their own exponentials: 200 rows of 1,256, full distribution, 14.2 us with it, 8.9 us without.)
template <class T, int WAVES> constexpr bool TABLE_OF = __is_same(T, __bf16) && WAVES == 16;

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// All ones in the halves that are negative (in one instruction: the compiler makes compares and selects of it).
__device__ __forceinline__ uint32_t sign_pairs(uint32_t v)
{
    uint32_t r;
    asm("v_pk_ashrrev_i16 %0, 15, %1 op_sel_hi:[0,1]" : "=v"(r) : "v"(v));
    return r;
}

// The bins of eight elements.
struct Bins {
    u16x2 t[4];
    int least;   // the first of them
    bool odd;    // whether one is the first or the middle bin
    __device__ __forceinline__ int at(int e) const { return e & 1 ? t[e / 2].y : t[e / 2].x; }
    // how many are `bin`
    __device__ __forceinline__ uint32_t equals(int bin) const
    {
        u16x2 other = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            other += __builtin_elementwise_min((u16x2)(t[i] ^ (u16x2)(unsigned short)bin), (u16x2)(unsigned short)1);
        return VEC - other.x - other.y;
    }
};

// Eight keys: packed in pairs for the 16-bit types.
template <class T> struct Vec8 {
    u32x4 a;
    __device__ __forceinline__ s16x2 pair(int i) const
    {
        const uint32_t w = a[i];   // (a bit cast of the vector's element itself would read element 0)
        return __builtin_bit_cast(s16x2, w);
    }
    __device__ __forceinline__ int pick(int e) const   // e known at run time only
    {
        const uint32_t w = e & 4 ? (e & 2 ? a[3] : a[2]) : (e & 2 ? a[1] : a[0]);
        return (e & 1) ? (int)w >> 16 : (int)(int16_t)(w & 0xFFFFu);
    }
    __device__ __forceinline__ int at(int e) const
    {
        return (e & 1) ? (int)a[e >> 1] >> 16 : (int)(int16_t)(a[e >> 1] & 0xFFFFu);
    }
    __device__ __forceinline__ int max() const
    {
        s16x2 m = pair(0);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, pair(i));
        return m.x > m.y ? m.x : m.y;
    }
    // the bins of the logits (before order())
    __device__ __forceinline__ Bins bins() const
    {
        using K = Keys<T>;
        Bins r;
        u16x2 first = (u16x2)(unsigned short)BINS, zero = first;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 k = pair(i), sign = k >> 15;
            const u16x2 mag = __builtin_bit_cast(u16x2, a[i] & 0x7FFF7FFFu);
            u16x2 m = __builtin_elementwise_sub_sat(mag, (u16x2)(unsigned short)(K::LOW - (1 << K::SHIFT)));
            m = __builtin_elementwise_min((u16x2)(m >> K::SHIFT), (u16x2)(unsigned short)HALF);
            zero = __builtin_elementwise_min(zero, m);
            r.t[i] = __builtin_bit_cast(u16x2, (s16x2)((s16x2)(short)HALF - ((__builtin_bit_cast(s16x2, m) ^ sign) - sign)));
            first = __builtin_elementwise_min(first, r.t[i]);
        }
        r.least = first.x < first.y ? first.x : first.y;
        r.odd = (zero.x == 0) | (zero.y == 0) | (r.least == 0);
        return r;
    }
    // how many of the keys are `key`
    __device__ __forceinline__ uint32_t equals(int key) const
    {
        u16x2 other = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 d = pair(i) - (s16x2)(short)key;
            other += __builtin_elementwise_min(__builtin_bit_cast(u16x2, d), (u16x2)(unsigned short)1);
        }
        return VEC - other.x - other.y;
    }
    // logits to keys, in place; NaN becomes larger than +inf or smaller than -inf
    __device__ __forceinline__ void order()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 b = pair(i), sign = b >> 15;
            const s16x2 m = __builtin_bit_cast(s16x2, a[i] & 0x7FFF7FFFu);
            a[i] = __builtin_bit_cast(uint32_t, (m ^ sign) - sign);
        }
    }
    __device__ __forceinline__ void drop_nan()   // of keys
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const s16x2 left = __builtin_elementwise_sub_sat((s16x2)(short)Keys<T>::INF, pair(i));
            const uint32_t out = sign_pairs(__builtin_bit_cast(uint32_t, left));
            a[i] = (a[i] & ~out) | (0x80008000u & out);
        }
    }
    // elements whose bit is 0 out of the choice: the smallest key, or -inf as a logit
    template <bool RAW = false> __device__ __forceinline__ void allow(uint32_t bits)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t in = ((bits >> (2 * i) & 1u) ? 0xFFFFu : 0u) | ((bits >> (2 * i + 1) & 1u) ? 0xFFFF0000u : 0u);
            a[i] = (a[i] & in) | ((RAW ? 0x80008000u | (uint32_t)Keys<T>::INF * 0x10001u : 0x80008000u) & ~in);
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
    template <bool RAW = false> __device__ __forceinline__ void allow(uint32_t bits)
    {
        static_assert(!RAW, "keys");
#pragma unroll
        for (int e = 0; e < VEC; ++e) set(e, (bits >> e) & 1u ? at(e) : (int)0x80000000);
    }
    __device__ __forceinline__ uint32_t equals(int key) const
    {
        uint32_t n = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) n += at(e) == key;
        return n;
    }
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
    __device__ __forceinline__ void drop_nan()
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e) set(e, at(e) > Keys<float>::INF ? (int)0x80000000 : at(e));
    }
};

// p * f + c in one instruction: the compiler copies a constant addend to registers first, which doubles the work.
__device__ __forceinline__ double fma_const(double p, double f, double c)
{
    double r;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(p), "v"(f), "s"(c));
    return r;
}

// Weights of one row.  2^y = 2^n 2^f with n the nearest integer (y + 1.5 * 2^52 holds it in its low bits): 2^f on
// [-1/2, 1/2] by the polynomial of degree 10 that interpolates it at the Chebyshev nodes (relative error below
// 2^-51), the multiple of 2^-S by adding 2^(52 - S) and reading the low bits.
struct Weights {
    double c, max, magic;
    int max_key;

    static constexpr double HUGE_LOGIT = 1e300;   // in place of +inf, whose weight is one and all others' zero
    // At a temperature of +inf finite logits weigh the same, but nothing beside +inf: a scale too small for the former.
    static __device__ __forceinline__ double scale_of(float temp) { return __builtin_fmax(1.4426950408889634 / (double)temp, 1e-290); }

    // the weight as the low bits of a number whose high bits are those of `magic`; y below -80 gives zero
    __device__ __forceinline__ uint64_t raw(float x, bool in = true) const
    {
        const double d = __builtin_fmin((double)x, HUGE_LOGIT) - max;
        double y = __builtin_fmax(d * c, -80.0);
        y = in ? y : -80.0;
        const double t = y + 0x1.8p52, f = y - (t - 0x1.8p52);
        double p = 7.072585949269224e-09;
        p = fma_const(p, f, 1.0208690299958306e-07);
        p = fma_const(p, f, 1.321544258792169e-06);
        p = fma_const(p, f, 1.5252657260200837e-05);
        p = fma_const(p, f, 0.0001540353044173605);
        p = fma_const(p, f, 0.0013333558230164974);
        p = fma_const(p, f, 0.009618129107606888);
        p = fma_const(p, f, 0.05550410866444772);
        p = fma_const(p, f, 0.24022650695910097);
        p = fma_const(p, f, 0.69314718055995);
        p = fma_const(p, f, 1.0);
        const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, t);
        const uint64_t q = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(n << 20) << 32);
        return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, q) + magic);
    }
    __device__ __forceinline__ uint64_t zero() const { return __builtin_bit_cast(uint64_t, magic); }
    __device__ __forceinline__ uint64_t of(int, float x) const { return raw(x) - zero(); }
    __device__ __forceinline__ uint64_t one() const { return __builtin_bit_cast(uint64_t, 1.0 + magic) - zero(); }
};

// A kernel runs most of its code once per row, so fetching instructions costs more than issuing them: what is
// used in several places is a function of its own.
template <class T> __device__ __attribute__((noinline)) uint64_t weight_of(double c, double max, double magic, int max_key, int key)
{
    return Weights{c, max, magic, max_key}.of(key, Keys<T>::value(key));
}

// Inclusive sum over the wavefront's lanes, by DPP: no LDS round trips, which a shuffle would take.
template <int CTRL, int ROWS> __device__ __forceinline__ uint64_t dpp_add(uint64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, ROWS == 0xF);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, ROWS == 0xF);
    return v + ((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v)
{
    v = dpp_add<0x111, 0xF>(v);   // row_shr:1
    v = dpp_add<0x112, 0xF>(v);   // row_shr:2
    v = dpp_add<0x114, 0xF>(v);   // row_shr:4
    v = dpp_add<0x118, 0xF>(v);   // row_shr:8
    v = dpp_add<0x142, 0xA>(v);   // row_bcast:15
    v = dpp_add<0x143, 0xC>(v);   // row_bcast:31
    return v;
}
// Sums over the lanes of two or four values at once: halves, then rows of 16 lanes, change places between the
// registers, so that every addition is of two values' parts.  The last lane of each half or row has a sum.
__device__ __forceinline__ uint64_t halves(uint64_t a, uint64_t b)   // a in lanes 0..31, b in 32..63
{
    const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)b, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(a >> 32), (uint32_t)(b >> 32), false, false);
    return ((uint64_t)h[0] << 32 | l[0]) + ((uint64_t)h[1] << 32 | l[1]);
}
__device__ __forceinline__ uint64_t rows_of(uint64_t a, uint64_t b)   // a in the even rows, b in the odd ones
{
    const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)a, (uint32_t)b, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(a >> 32), (uint32_t)(b >> 32), false, false);
    return ((uint64_t)h[0] << 32 | l[0]) + ((uint64_t)h[1] << 32 | l[1]);
}
__device__ __forceinline__ uint64_t row_scan(uint64_t v)
{
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    return dpp_add<0x118, 0xF>(v);
}
__device__ __forceinline__ uint64_t wave_sums(const uint64_t (&v)[4])
{
    return row_scan(rows_of(halves(v[0], v[2]), halves(v[1], v[3])));
}
__device__ __forceinline__ uint64_t wave_sums(const uint64_t (&v)[2])
{
    return dpp_add<0x142, 0xA>(row_scan(halves(v[0], v[1])));
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, uint32_t lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), (int)lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, (int)lane);
}

template <int WAVES> struct Lds {
    uint64_t mass[BINS];         // masses, or weights, per bin; weights of the list
    union {
        uint32_t count[BINS];
        uint64_t list[LIST];     // key above, inverted ID below: the order is that of the numbers, descending
    };
    uint64_t cell[MAX_CELLS];    // mass of what is kept
    uint32_t border[MAX_CELLS];  // elements in the border's bins
    uint64_t wave[WAVES];
    uint64_t above, inside;
    uint32_t found, n_list, n_odd;
    int key;
    uint32_t odd[ODD];
};

// Sum over the threads below this one; total: over all.
typedef __attribute__((address_space(3))) uint64_t lds_u64;

template <int WAVES> __device__ __attribute__((noinline)) ulonglong2 block_sums(uint64_t v, lds_u64 *wave_sums)
{
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint64_t incl = wave_scan(v);
    if (lane == 63) wave_sums[wave] = incl;
    __syncthreads();
    const uint64_t sums = wave_scan(lane < WAVES ? wave_sums[lane] : 0);
    __syncthreads();
    const uint64_t base = wave ? lane_value(sums, wave - 1) : 0;
    return ulonglong2{base + incl - v, lane_value(sums, WAVES - 1)};
}

template <int WAVES> __device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t *wave_sums, uint64_t &total)
{
    const ulonglong2 r = block_sums<WAVES>(v, (lds_u64 *)wave_sums);
    total = r.y;
    return r.x;
}

// One row's logits, mask and settings.
template <class T> struct Row {
    using V = Vec8<T>;
    const T *x;
    const uint32_t *mask;
    uint32_t n;
    float temp, p, min_p, u;
    uint32_t k;

    __device__ __forceinline__ V raw(uint32_t j) const   // eight elements, all the row's
    {
        V v;
        v.a = *(const u32x4_row *)(x + j);
        if constexpr (sizeof(T) == 4) v.b = *(const u32x4_row *)(x + j + 4);
        return v;
    }
    __device__ __forceinline__ V part(uint32_t j) const   // what lies past the row's end is out of the choice
    {
        if (j + VEC <= n) return raw(j);
        V v;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if constexpr (sizeof(T) == 4) {
                v.set(e, j + e < n ? __builtin_bit_cast(int, x[j + e]) : (int)0xFF800000u);
            } else {
                const uint32_t h = j + e < n ? (uint32_t)__builtin_bit_cast(uint16_t, x[j + e]) : 0x8000u | (uint32_t)Keys<T>::INF;
                v.a[e >> 1] = (e & 1) ? v.a[e >> 1] | h << 16 : h;
            }
        }
        return v;
    }
    __device__ __forceinline__ void finish(V &v, uint32_t j) const
    {
        v.order();
        v.drop_nan();
        if (mask && j < n) v.allow(mask[j >> 5] >> (j & 31u));
    }
    __device__ __forceinline__ V fetch(uint32_t j) const;   // one vector, anywhere
    // f(index of the first element, keys, q) over the vectors of this thread, ascending: one of every `step` elements,
    // AHEAD loads in flight; q counts these, and after them g(index of their first element, how many they were).  (A
    // load under a condition would wait for those before it, so where fewer than AHEAD are left the last is loaded
    // again.)  Only the last step may pass the row's end.  Positive NaN are not taken out, and with RAW the logits are
    // not made keys.
    template <uint32_t AHEAD, bool RAW, class F, class G> __device__ __forceinline__ void each(uint32_t step, F f, G g) const
    {
        const uint32_t full = n / step, j0 = threadIdx.x * VEC;
#pragma unroll 1
        for (uint32_t i = 0; i < full; i += AHEAD) {
            V v[AHEAD];
            uint32_t word[AHEAD];
#pragma unroll
            for (uint32_t q = 0; q < AHEAD; ++q) v[q] = raw((i + q < full ? i + q : full - 1) * step + j0);
            if (mask) {
#pragma unroll
                for (uint32_t q = 0; q < AHEAD; ++q) word[q] = mask[((i + q < full ? i + q : full - 1) * step + j0) >> 5];
            }
#pragma unroll
            for (uint32_t q = 0; q < AHEAD; ++q)
                if (i + q < full) {
                    const uint32_t j = (i + q) * step + j0;
                    if (!RAW) v[q].order();
                    if (mask) v[q].template allow<RAW>(word[q] >> (j & 31u));
                    f(j, v[q], q);
                }
            g(i * step + j0, full - i < AHEAD ? full - i : AHEAD);
        }
        if (full * step < n) {
            const uint32_t j = full * step + j0;
            V v = part(j);
            if (!RAW) v.order();
            if (mask && j < n) v.template allow<RAW>(mask[j >> 5] >> (j & 31u));
            f(j, v, 0);
            g(j, 1);
        }
    }
};


template <class T> __device__ __attribute__((noinline)) Vec8<T> fetch_of(const T *x, const uint32_t *mask, uint32_t n, uint32_t j)
{
    Row<T> row;
    row.x = x;
    row.mask = mask;
    row.n = n;
    Vec8<T> v = row.part(j);
    row.finish(v, j);
    return v;
}
template <class T> __device__ __forceinline__ Vec8<T> Row<T>::fetch(uint32_t j) const { return fetch_of(x, mask, n, j); }

// Where the filters end.  Bins before lo are kept, bins after hi are not; those from lo to hi are the border.
struct Border {
    int lo, hi;
    bool hard;        // too many elements for the list: see general_row
    bool listed;      // the border's elements are sorted; else it is one key, of which the first `ties` of `count` are kept
    bool by_k, by_p;  // listed: limits on their number, on their mass
    uint64_t left_k, left_p;   // (left_p 0: top-p of what left_k keeps)
    int key;
    uint64_t ties, count;
};

// ---- keys: this thread's largest key and the vector where it first met it; HIST: with the
// counts of all keys per bin
template <class T, int WAVES, bool HIST>
__device__ __forceinline__ void scan_keys(const Row<T> &row, Lds<WAVES> &sh, int &mine, uint32_t &mine_j)
{
    using V = Vec8<T>;
    using K = Keys<T>;
    mine = (int)0x80000000;
    mine_j = 0;
    constexpr bool RAW = HIST && sizeof(T) == 2;
    row.template each<HIST || sizeof(T) == 4 ? 4 : 8, RAW>(WAVES * 64 * VEC, [&](uint32_t j, const V &logits, uint32_t) INLINE {
        V v = logits;
        Bins bins;
        bool odd = false;
        if constexpr (RAW) {
            bins = v.bins();
            odd = bins.odd;
            v.order();
        }
        const int m = v.max();
        mine_j = m > mine ? j : mine_j;
        mine = m > mine ? m : mine;
        if constexpr (HIST) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int key = v.at(e);
                int bin;
                if constexpr (RAW) bin = bins.at(e);
                else bin = bin_of<T>(key);
                if (key > -K::INF) atomicAdd(&sh.count[bin], 1u);
                if (TABLE_OF<T, WAVES>) odd |= (key > -K::INF) & (bin == 2 * HALF);
            }
            if (TABLE_OF<T, WAVES> && __any(odd)) {
#pragma unroll 1
                for (int e = 0; e < VEC; ++e) {
                    const int key = v.pick(e);
                    if ((key > -K::INF) & !bin_exact<T>(bin_of<T>(key))) {
                        const uint32_t at = atomicAdd(&sh.n_odd, 1u);
                        if (at < ODD) sh.odd[at] = (uint32_t)key;
                    }
                }
            }
        }
    }, [](uint32_t, uint32_t) INLINE {});
}

// Largest of the workgroup's values.
template <int WAVES> __device__ __forceinline__ uint32_t block_max(Lds<WAVES> &sh, uint32_t v)
{
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = v;
    __syncthreads();
    const uint32_t lane = threadIdx.x & 63;
    v = wave_max(lane < WAVES ? (uint32_t)sh.wave[lane] : 0u);
    __syncthreads();
    return v;
}

// The lowest index among the workgroup's largest keys.
template <class T, int WAVES>
__device__ __forceinline__ uint32_t first_of(const Row<T> &row, Lds<WAVES> &sh, int top, int mine, uint32_t mine_j)
{
    uint32_t at = 0;   // inverted index
    if (mine == top) {
        const Vec8<T> v = row.fetch(mine_j);
#pragma unroll
        for (int e = VEC - 1; e >= 0; --e)
            if (v.at(e) == top) at = ~(mine_j + e);
    }
    return ~block_max(sh, at);
}

// The first bin at which the running sum of value(bin) reaches target(total), the sum before it and its own;
// false where the total is below the target.
template <int WAVES, class F, class G>
__device__ __forceinline__ bool find_bin(Lds<WAVES> &sh, F value, G target_of, uint32_t &bin, uint64_t &before, uint64_t &inside,
                                         uint64_t &target)
{
    constexpr int PER = BINS / (WAVES * 64);
    const int b0 = threadIdx.x * PER;
    uint64_t sum = 0, total;
#pragma unroll 4
    for (int i = 0; i < PER; ++i) sum += value(b0 + i);
    uint64_t run = block_before<WAVES>(sum, sh.wave, total);
    target = target_of(total);
    if (target > total) return false;
    if (run < target && target <= run + sum) {
#pragma unroll 1
        for (int i = 0;; ++i) {
            const uint64_t v = value(b0 + i);
            if (target <= run + v) {
                sh.found = b0 + i;
                sh.above = run;
                sh.inside = v;
                break;
            }
            run += v;
        }
    }
    __syncthreads();
    bin = sh.found;
    before = sh.above;
    inside = sh.inside;
    __syncthreads();
    return true;
}

// ---- keys, for a small k: nothing below the k-th largest of the threads' own largest keys can be among the first
// k, since k threads hold one each.  So the list is filled from the threads that have a key that large (or as
// large as the lowest key of its bin, which is quicker to find), whose vectors are read again, by all.  False
// where they are too many.
template <class T, int WAVES>
__device__ __forceinline__ bool list_first(const Row<T> &row, Lds<WAVES> &sh, uint32_t cells, int mine, Border &b)
{
    using V = Vec8<T>;
    using K = Keys<T>;
    constexpr uint32_t THREADS = WAVES * 64, CELL = THREADS * VEC;
    const uint32_t tid = threadIdx.x;
    if (mine > -K::INF) atomicAdd(&sh.count[bin_of<T>(mine)], 1u);
    __syncthreads();
    uint32_t bin;
    uint64_t before, inside, target;
    int floor = -K::INF + 1, hi;
    b.lo = 0;
    b.hi = BINS - 1;
    if (find_bin<WAVES>(sh, [&](int i) INLINE { return (uint64_t)sh.count[i]; }, [&](uint64_t) INLINE { return (uint64_t)row.k; }, bin,
                        before, inside, target)) {
        bin_range<T>((int)bin, floor, hi);
        floor = floor > -K::INF ? floor : -K::INF + 1;
        b.hi = (int)bin;
    }
    uint32_t *holders = (uint32_t *)sh.mass;
    if (mine >= floor) holders[atomicAdd(&sh.n_odd, 1u)] = tid;
    __syncthreads();
    const uint32_t work = sh.n_odd * cells;
#pragma unroll 1
    for (uint32_t i = tid; i < work; i += THREADS) {
        const uint32_t j = i % cells * CELL + holders[i / cells] * VEC;
        const Vec8<T> v = row.fetch(j);
        if (v.max() >= floor) {
#pragma unroll 1
            for (int e = 0; e < VEC; ++e) {
                const int key = v.pick(e);
                if (key >= floor) {
                    const uint32_t at = atomicAdd(&sh.n_list, 1u);
                    if (at < LIST) sh.list[at] = (uint64_t)((uint32_t)key ^ 0x80000000u) << 32 | ~(j + e);
                }
            }
        }
    }
    __syncthreads();
    if (sh.n_list > LIST) return false;
    b.listed = b.by_k = true;
    b.by_p = row.p < 1.f;
    b.left_k = row.k;
    return true;
}

__device__ __forceinline__ uint64_t share_of(float p, uint64_t all)   // the mass that top-p has to reach, 1 .. all
{
    const double t = __builtin_ceil((double)p * (double)all);
    const uint64_t q = t > 1.0 ? (uint64_t)t : 1ull;
    return q < all ? q : all;
}

__device__ __forceinline__ uint64_t least_weight(const Weights &wt, float min_p)   // that min-p keeps
{
    const uint64_t one = wt.one();
    return min_p >= 1.f ? one : min_p > 0.f ? (uint64_t)__builtin_ceil((double)min_p * (double)one) : 0;
}
__device__ __forceinline__ uint64_t aim_of(float u, uint64_t total)   // the running mass that the ID has to exceed
{
    return (uint64_t)((u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0) * (double)total);
}

// ---- border, from sh.count; fill_masses() brings the masses into sh.mass where they are needed
template <class T, int WAVES, class W, class M>
__device__ __forceinline__ Border find_border(const Row<T> &row, Lds<WAVES> &sh, W weight, M fill_masses)
{
    Border r{};
    r.lo = r.hi = BINS;
    bool need_k = row.k != 0 && row.k < row.n;
    const bool need_p = row.p < 1.f;
    uint32_t bin_k = BINS, bin;
    uint64_t above_k = 0, count_k = 0, before, inside, target;
    const uint64_t k = row.k;
    if (need_k)
        need_k = find_bin<WAVES>(sh, [&](int b) INLINE { return (uint64_t)sh.count[b]; }, [&](uint64_t) INLINE { return k; }, bin_k,
                                 above_k, count_k, target);
    if (!need_k && !need_p) return r;
    const bool list_k = above_k + count_k <= LIST && !bin_exact<T>((int)bin_k);
    if (need_k && (list_k || !need_p)) {
        r.hi = (int)bin_k;
        r.by_k = true;
        if (list_k) {   // all that top-k may keep goes to the list
            r.lo = 0;
            r.listed = true;
            r.by_p = need_p;
            r.left_k = k;
            return r;
        }
        r.lo = r.hi;
        r.left_k = r.ties = k - above_k;
        r.count = count_k;
    } else {
        fill_masses(bin_k);
        uint64_t mass_k = 0;
        if (need_k) {
            if (!bin_exact<T>((int)bin_k)) {
                r.hard = true;
                return r;
            }
            int lo, hi;
            bin_range<T>((int)bin_k, lo, hi);
            mass_k = (k - above_k) * weight(lo);
        }
        find_bin<WAVES>(sh, [&](int b) INLINE { return b < (int)bin_k ? sh.mass[b] : b == (int)bin_k ? mass_k : 0ull; },
                        [&](uint64_t all) INLINE { return share_of(row.p, all); }, bin, before, inside, target);
        r.lo = r.hi = (int)bin;
        r.by_p = true;
        r.left_p = target - before;
        r.count = sh.count[bin];
    }
    int lo, hi;
    bin_range<T>(r.lo, lo, hi);
    r.key = lo;
    r.listed = !bin_exact<T>(r.lo);
    if (r.listed) {
        r.hard = r.count > LIST;
    } else if (r.by_p) {
        const uint64_t w = weight(lo);
        r.ties = (r.left_p + w - 1) / w;
    }
    __syncthreads();   // the counts have been read: the list may take their place
    return r;
}

// ---- cells: sh.cell, sh.border and sh.list
template <class T, int WAVES, class W>
__device__ __forceinline__ void scan_cells(const Row<T> &row, Lds<WAVES> &sh, const Weights &wt, const Border &b, uint64_t w_min,
                                           W weight)
{
    using V = Vec8<T>;
    using K = Keys<T>;
    constexpr bool TABLE = TABLE_OF<T, WAVES>;
    constexpr uint32_t AHEAD = sizeof(T) == 4 ? 2 : 4, CELL = WAVES * 64 * VEC;
    const uint32_t lane = threadIdx.x & 63;
    int lowest = -K::INF + 1, sure = -K::INF + 1;   // the lowest keys of the border, and above it
    const uint64_t raw_min = wt.zero() + w_min;
    const bool bordered = b.hi < BINS;
    if (b.hi < BINS) {
        int h;
        bin_range<T>(b.hi, lowest, h);
        lowest = lowest > -K::INF ? lowest : -K::INF + 1;
        bin_range<T>(b.lo, h, sure);
        ++sure;
    }
    if (TABLE) {   // the weights of the bins above the border, so that no element needs its own exponential
#pragma unroll 1
        for (int i = threadIdx.x; i < BINS - 1; i += WAVES * 64) {
            int l, h;
            bin_range<T>(i, l, h);
            uint64_t w = 0;
            if ((l >= sure) & (l <= wt.max_key) & bin_exact<T>(i)) w = weight(l);
            sh.mass[i] = w >= w_min ? w : 0;
        }
        __syncthreads();
    }
    uint64_t sums[AHEAD];   // a thread's, of the cells in flight
    row.template each<AHEAD, TABLE>(CELL, [&](uint32_t j, const V &logits, uint32_t q) INLINE {
        uint64_t &out = sums[q];
        out = 0;
        V v = logits;
        Bins bins;
        uint64_t sum = 0;
        if constexpr (TABLE) {
            bins = v.bins();
            if (!__any(bins.least <= b.hi)) return;
            if (__any(bins.least < b.lo)) {
                uint64_t w[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] = sh.mass[bins.at(e)];
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum += w[e];
            }
            if (__any(bins.odd) | b.listed) v.order();
            if (__any(bins.odd)) {
#pragma unroll 1
                for (int e = 0; e < VEC; ++e) {
                    const int key = v.pick(e);
                    const bool own = (key >= sure) & !bin_exact<T>(bin_of<T>(key));
                    if (!__any(own)) continue;
                    const uint64_t w1 = wt.of(key, K::value(key));
                    sum += own && w1 >= w_min ? w1 : 0;
                }
            }
        } else {
            const int most = v.max();
            if (!__any(most >= lowest)) return;
            if (__any(most >= sure)) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int key = v.at(e);
                    const uint64_t w = wt.raw(K::value(key), key >= sure);
                    sum += w < raw_min ? 0ull : w - wt.zero();
                }
            }
        }
        out = sum;
        // the border: elements from `lowest` up to `sure`, or equal to its one key
        if (!bordered) return;
        uint32_t in_border = 0;
        if (b.listed) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) in_border += (v.at(e) >= lowest) & (v.at(e) < sure);
        } else {
            in_border = TABLE ? bins.equals(b.hi) : v.equals(lowest);
        }
        if (__any(in_border != 0)) {
            const uint32_t incl = wave_incl_sum(in_border);
            if (!b.listed) {
                if (lane == 63) atomicAdd(&sh.border[j / CELL], incl);
            } else {
                uint32_t at = 0;
                if (lane == 63) at = atomicAdd(&sh.n_list, incl);
                at = (uint32_t)__builtin_amdgcn_readlane((int)at, 63) + incl - in_border;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int key = v.at(e);
                    if ((key >= lowest) & (key < sure)) {
                        if (at < LIST) sh.list[at] = (uint64_t)((uint32_t)key ^ 0x80000000u) << 32 | ~(j + e);
                        ++at;
                    }
                }
            }
        }
    }, [&](uint32_t j, uint32_t some) INLINE {
#pragma unroll
        for (uint32_t q = 0; q < AHEAD; ++q)
            if (q >= some) sums[q] = 0;
        uint64_t any = sums[0];
#pragma unroll
        for (uint32_t q = 1; q < AHEAD; ++q) any |= sums[q];
        if (!__any(any != 0)) return;
        const uint64_t all = wave_sums(sums);
        constexpr uint32_t LANES = 64 / AHEAD;
        if (lane % LANES == LANES - 1 && all) atomicAdd((unsigned long long *)&sh.cell[j / CELL + lane / LANES], (unsigned long long)all);
    });
}

// Sorts the first n (at most LIST) of sh.list, descending; they are all different.  Few by their ranks: each
// against all others, which takes fewer steps in a row; more by a bitonic network, a power of two of them padded with
// zeros.
template <int WAVES> __device__ __forceinline__ void sort_list(Lds<WAVES> &sh, uint32_t n)
{
    constexpr uint32_t FEW = WAVES * 16;   // four threads for each
    if (n <= FEW) {
        uint32_t *rank = (uint32_t *)sh.mass;
        const uint32_t i = threadIdx.x % FEW, part = threadIdx.x / FEW;
        if (part == 0) rank[i] = 0;
        __syncthreads();
        const uint64_t v = i < n ? sh.list[i] : 0;
        if (i < n) {
            uint32_t above = 0;
#pragma unroll 4
            for (uint32_t o = part; o < n; o += 4) above += sh.list[o] > v;
            atomicAdd(&rank[i], above);
        }
        __syncthreads();
        if (i < n && part == 0) sh.list[rank[i]] = v;
        __syncthreads();
        return;
    }
    uint32_t size = 2;
    while (size < n) size *= 2;
    for (uint32_t i = n + threadIdx.x; i < size; i += WAVES * 64) sh.list[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (uint32_t run = 2; run <= size; run *= 2)
#pragma unroll 1
        for (uint32_t stride = run / 2; stride; stride /= 2) {
#pragma unroll 1
            for (uint32_t t = threadIdx.x; t < size / 2; t += WAVES * 64) {
                const uint32_t i = 2 * t - (t & (stride - 1)), o = i + stride;
                const uint64_t a = sh.list[i], b = sh.list[o];
                if ((a < b) == ((i & run) == 0)) {
                    sh.list[i] = b;
                    sh.list[o] = a;
                }
            }
            // pairs less than 64 apart stay inside the 128 elements of one wavefront
            const uint32_t next = stride > 1 ? stride / 2 : run;
            if (stride >= 64 || next >= 64) __syncthreads();
            else wave_order();
        }
    __syncthreads();
}

// The cell, or the thread, at which the running sum exceeds the target: every thread brings its part and the sum
// of those before it.
template <int WAVES>
__device__ __forceinline__ uint32_t find_part(Lds<WAVES> &sh, uint64_t run, uint64_t part, uint64_t target, uint64_t &before)
{
    if (run <= target && target < run + part) {
        sh.found = threadIdx.x;
        sh.above = run;
    }
    __syncthreads();
    const uint32_t at = sh.found;
    before = sh.above;
    __syncthreads();
    return at;
}
template <int WAVES>
__device__ __forceinline__ uint32_t find_part(Lds<WAVES> &sh, uint64_t part, uint64_t target, uint64_t &before)
{
    uint64_t total;
    const uint64_t run = block_before<WAVES>(part, sh.wave, total);
    return find_part(sh, run, part, target, before);
}

// ---- draw
template <class T, int WAVES, class W>
__device__ __forceinline__ void draw(const Row<T> &row, Lds<WAVES> &sh, const Weights &wt, const Border &b, uint64_t w_min, W weight,
                                     uint32_t *out_id, float *out_logprob)
{
    using K = Keys<T>;
    using V = Vec8<T>;
    constexpr uint32_t THREADS = WAVES * 64, CELL = THREADS * VEC, CELL_SHIFT = __builtin_ctz(CELL);
    const uint32_t cells = (row.n + CELL - 1) / CELL, tid = threadIdx.x;
    int key_f = -K::INF + 1;
    uint32_t cut = NO_ID;
    auto kept_weight = [&](int key) INLINE {
        const uint64_t w = weight(key);
        return w >= w_min ? w : 0ull;
    };
    if (b.listed) {
        const uint32_t n = sh.n_list;
        sort_list(sh, n);
        // each thread's consecutive elements, their weights in sh.mass
        const uint32_t per = (n + THREADS - 1) / THREADS, i0 = tid * per;
        const uint32_t limit = b.by_k && b.left_k < n ? (uint32_t)b.left_k : n;
        uint64_t mine = 0, all;
#pragma unroll 1
        for (uint32_t i = i0; i < i0 + per && i < limit; ++i) {
            const uint64_t w = weight((int)((uint32_t)(sh.list[i] >> 32) ^ 0x80000000u));
            sh.mass[i] = w;
            mine += w;
        }
        uint64_t run = block_before<WAVES>(mine, sh.wave, all);
        const uint64_t target = !b.by_p ? ~0ull : b.left_p ? b.left_p : share_of(row.p, all);
        if (tid == 0) sh.found = 0;
        __syncthreads();
        uint32_t kept = 0;
#pragma unroll 1
        for (uint32_t i = i0; i < i0 + per && i < limit && run < target; ++i) {
            const uint64_t w = sh.mass[i];
            ++kept;
            run += w;
            if (w >= w_min) atomicAdd((unsigned long long *)&sh.cell[~(uint32_t)sh.list[i] >> CELL_SHIFT], (unsigned long long)w);
        }
        if (kept) atomicMax(&sh.found, i0 + kept);
        __syncthreads();
        const uint64_t last = sh.list[sh.found - 1];
        key_f = (int)((uint32_t)(last >> 32) ^ 0x80000000u);
        cut = ~(uint32_t)last;
        __syncthreads();
    } else if (b.hi < BINS) {
        key_f = b.key;
        const uint64_t w = kept_weight(key_f);
        uint64_t full = tid < cells ? sh.border[tid] : 0;
        if (b.ties < b.count) {   // the last of the equals that are kept: its cell, then its place there
            uint64_t before, before_thread;
            const uint32_t c = find_part(sh, full, b.ties - 1, before);
            const uint32_t j = c * CELL + tid * VEC;
            const Vec8<T> v = row.fetch(j);
            const uint32_t t = find_part(sh, (uint64_t)v.equals(key_f), b.ties - 1 - before, before_thread);
            if (tid == t) {
                uint64_t at = before + before_thread;
#pragma unroll 1
                for (int e = 0; e < VEC; ++e)
                    if (v.pick(e) == key_f && ++at == b.ties) sh.found = j + e;
            }
            __syncthreads();
            cut = sh.found;
            __syncthreads();
            full = tid < c ? full : tid == c ? b.ties - before : 0;
        }
        if (tid < cells) sh.cell[tid] += full * w;
        __syncthreads();
    }
    // the cell, the thread's vector in it, the element
    uint64_t total, before, before_thread;
    const uint64_t mass = tid < cells ? sh.cell[tid] : 0;
    const uint64_t before_cell = block_before<WAVES>(mass, sh.wave, total);
    uint64_t target = aim_of(row.u, total);
    const uint32_t c = find_part(sh, before_cell, mass, target, before), j = c * CELL + tid * VEC;
    target -= before;
    const Vec8<T> v = row.fetch(j);
    uint64_t sum = 0, w[VEC] = {};
    if (__any(v.max() >= key_f)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int key = v.at(e);
            const uint64_t x = wt.of(key, K::value(key));
            w[e] = ((key > key_f) | ((key == key_f) & (j + e <= cut))) & (x >= w_min) ? x : 0;
            sum += w[e];
        }
    }
    const uint32_t t = find_part(sh, sum, target, before_thread);
    if (tid == t) {
        uint64_t run = before_thread, own = 0;
        uint32_t id = NO_ID;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            run += w[e];
            if (id == NO_ID && run > target) {
                id = j + e;
                own = w[e];
            }
        }
        *out_id = id;
        if (out_logprob) *out_logprob = (float)log((double)own / (double)total);
    }
}

// Any row, by one search: histograms over bins and then over digits of the key, for counts and for masses, and
// the ID by running masses.  For borders with more elements than the list holds (float32 and float16 also where top-k ends past
// it and top-p follows), rows with a NaN of positive sign, and bfloat16 rows whose weights do not end at -2,047 (temperatures from about 64 on, or logits all below it).  An element at
// a time, in several passes.  131,328 elements, one row and 256: with a NaN, full distribution 91 and 105 us in bfloat16, 101
// and 115 in float16, 103 and 130 in float32, top-p 209 to 266 and 219 to 287; top-k 5,000 with top-p, float16 275 and 321,
// float32 330 and 379; top-p where all logits lie in a few bins (near -20), float16 567 and 578, float32 622 and 645; bfloat16
// at a temperature of 100, top-p 215 and 225.
template <class T, int WAVES>
__device__ __attribute__((noinline)) void general_row(const Row<T> &in, Lds<WAVES> &sh, double magic, uint32_t *out_id, float *out_logprob)
{
    using K = Keys<T>;
    using V = Vec8<T>;
    constexpr uint32_t THREADS = WAVES * 64;
    constexpr bool TABLE = __is_same(T, __bf16);   // a weight per bin
    const Row<T> row = in;
    const uint32_t n_vocab = row.n;
    const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    // a wavefront's segment: nv * 512 consecutive elements, a vector of each lane per step
    const uint32_t nv = (n_vocab + THREADS * VEC - 1) / (THREADS * VEC), first = wave * (nv * 64 * VEC) + lane * VEC;
    const float temp = row.temp, p = row.p, mp = row.min_p, u_in = row.u;
    const uint32_t k = row.k;

    // 1. the largest key, of each thread and of all
    int mine, top;
#pragma unroll 1
    for (;;) {
        constexpr uint32_t AHEAD = sizeof(T) == 4 ? 4 : 8;   // vectors of a thread in flight
        mine = (int)0x80000000;
#pragma unroll 1
        for (uint32_t i = 0; i < nv; i += AHEAD) {
            V v[AHEAD];
#pragma unroll
            for (uint32_t q = 0; q < AHEAD; ++q)
                if (i + q < nv) v[q] = row.part(first + (i + q) * (64 * VEC));
#pragma unroll
            for (uint32_t q = 0; q < AHEAD; ++q)
                if (i + q < nv) {
                    row.finish(v[q], first + (i + q) * (64 * VEC));
                    const int m = v[q].max();
                    mine = m > mine ? m : mine;
                }
        }
        int m = mine;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const int o = __shfl_xor(m, d);
            m = o > m ? o : m;
        }
        if (lane == 0) sh.wave[wave] = (uint32_t)m;
        __syncthreads();
        top = (int)0x80000000;
#pragma unroll 1
        for (int w = 0; w < WAVES; ++w) top = (int)(uint32_t)sh.wave[w] > top ? (int)(uint32_t)sh.wave[w] : top;
        __syncthreads();
        break;
    }
    constexpr int LOWEST = -K::INF + 1;   // the smallest key in the choice
    if (top < LOWEST) {                   // nothing to choose from
        if (tid == 0) {
            *out_id = NO_ID;
            if (out_logprob) *out_logprob = -__builtin_inff();
        }
        return;
    }
    const Weights wt{Weights::scale_of(temp), __builtin_fmin((double)K::value(top), Weights::HUGE_LOGIT), magic, top};
    auto weight = [&](int key) { return weight_of<T>(wt.c, wt.max, wt.magic, wt.max_key, key); };
    const bool first_alone = k == 1 || !(temp > 0.f);
    const bool need_k = !first_alone && k != 0 && k < n_vocab, need_p = !first_alone && p < 1.f;

    // Kept so far: keys above key_f, and of those equal to it (count_f of them) the first `ties`, which are those
    // up to index `cut`; count_f 0: no filter, all are kept.
    int key_f = first_alone ? top : LOWEST;
    uint64_t ties = 1, count_f = first_alone ? 2 : 0;
    uint32_t cut = NO_ID;
    // A step is one pass over elements lo <= key <= hi, each with an amount: 1, or its weight.
    enum { FLOOR, BIN, DIGITS, NTH, DRAW };
    int step = first_alone ? NTH : need_k ? (k <= THREADS / 2 ? FLOOR : BIN) : need_p ? BIN : DRAW;
    bool by_mass = !need_k;                            // of a search: top-p's
    int lo = first_alone ? top : LOWEST, hi = K::INF;  // of the pass
    int shift = 0, above_shift = 0;                    // of DIGITS: which digit of hi - key
    uint32_t prefix = 0;
    uint64_t target = 0, excess = 0;                   // excess: what the equals of top-k's key beyond its ties weigh
    int key_k = K::INF + 1;
    // of NTH and DRAW: 0 per wavefront, 1 per thread inside a wavefront's segment, 2 per element inside a thread's
    int level = 0;
    uint32_t begin = first, stride_v = 64 * VEC, count_v = nv, from = 0, until = n_vocab;
    uint64_t base = 0, total = 0;
    const uint64_t min_p_weight = mp >= 1.f ? wt.one() : mp > 0.f ? (uint64_t)__builtin_ceil((double)mp * (double)wt.one()) : 0;
#pragma unroll 1
    for (;;) {
        const bool hist = step <= DIGITS;
        const bool weighted = step == DRAW || (by_mass && (step == BIN || step == DIGITS));
        const uint64_t w_min = step == DRAW ? min_p_weight : 0;
        uint64_t sum = 0;
        int key_in = 0;
        if (hist || (TABLE && step == DRAW && level == 0)) {
#pragma unroll 1
            for (uint32_t b = tid; b < BINS; b += THREADS) {
                uint64_t w = 0;
                if (TABLE && !hist) {   // the draw takes the weights of bins with one key from a table
                    int l, h;
                    bin_range<T>((int)b, l, h);
                    if ((l >= key_f) & (l <= top)) w = weight(l);
                    w = w >= w_min ? w : 0;
                }
                sh.mass[b] = w;
            }
            __syncthreads();
        }
        if (step == FLOOR) {
            // k threads with a key >= f hold at least k such keys, so nothing below the k-th largest of the
            // threads' own largest keys (or its bin's lowest key) can be among the first k
            if (mine >= LOWEST) atomicAdd((unsigned long long *)&sh.mass[bin_of<T>(mine)], 1ull);
        } else {
            V next = row.part(begin);
#pragma unroll 1
            for (uint32_t i = 0; i < count_v; ++i) {
                const uint32_t j = begin + i * stride_v;
                V v = next;
                if (i + 1 < count_v) next = row.part(j + stride_v);
                row.finish(v, j);
                if (!__any(v.max() >= lo)) continue;
#pragma unroll 1
                for (int e = 0; e < VEC; ++e) {
                    const int key = v.pick(e);
                    const uint32_t at = j + e;
                    const bool in = (key >= lo) & (key <= hi) & ((key != key_f) | (at <= cut)) & (at >= from) & (at < until);
                    if (!__any(in)) continue;
                    const int b = bin_of<T>(key);
                    uint64_t amount = 1;
                    if (weighted) {
                        bool own = true;
                        if (TABLE) {
                            if (step == DRAW) amount = sh.mass[b];
                            own = in & !bin_exact<T>(b);   // (an exact bin's histogram holds counts until it is complete)
                        }
                        if (__any(own)) {
                            const uint64_t w = wt.of(key, K::value(key));
                            amount = own ? (w >= w_min ? w : 0) : amount;
                        }
                    }
                    if (hist) {
                        const uint32_t d = (uint32_t)(hi - key);
                        if (in & (step == BIN || (above_shift < 32 ? d >> above_shift : 0u) == prefix))
                            atomicAdd((unsigned long long *)&sh.mass[step == BIN ? (uint32_t)b : (d >> shift) & (DIGIT_VALUES - 1)],
                                      (unsigned long long)amount);
                    } else if (in) {
                        sum += amount;
                        key_in = key;
                    }
                }
            }
        }
        // sums in the order of the histogram's bins, or of the threads' elements
        constexpr uint32_t PER = BINS / THREADS;
        if (hist) {
            __syncthreads();
            if (weighted && excess && tid == 0) {
                const uint32_t d = (uint32_t)(hi - key_k);
                if (step == BIN) sh.mass[bin_of<T>(key_k)] -= TABLE && bin_exact<T>(bin_of<T>(key_k)) ? count_f - ties : excess;
                else if ((key_k >= lo) & (key_k <= hi) & ((above_shift < 32 ? d >> above_shift : 0u) == prefix))
                    sh.mass[(d >> shift) & (DIGIT_VALUES - 1)] -= excess;
            }
            __syncthreads();
#pragma unroll 1
            for (uint32_t q = 0; q < PER; ++q) {
                const uint32_t b = tid * PER + q;
                uint64_t c = sh.mass[b];
                if (TABLE && weighted && step == BIN && c && bin_exact<T>((int)b)) {
                    int l, h;
                    bin_range<T>((int)b, l, h);
                    c *= weight(l);
                    sh.mass[b] = c;
                }
                sum += c;
            }
        }
        const uint64_t incl = wave_scan(sum);
        if (lane == 63) sh.wave[wave] = incl;
        __syncthreads();
        uint64_t run = incl - sum, all = 0;
#pragma unroll 1
        for (uint32_t w = 0; w < WAVES; ++w) {
            const uint64_t s = sh.wave[w];
            run += w < wave ? s : 0;
            all += s;
        }
        if (hist) {
            if (step == FLOOR || step == BIN) {
                target = k;
                if (weighted) {
                    const double t = __builtin_ceil((double)p * (double)all);
                    target = t > 1.0 ? (uint64_t)t : 1ull;
                    target = target < all ? target : all;
                }
            }
            const bool enough = target <= all;   // else fewer than k are in the choice: the filter keeps all of them
            if (enough && run < target && target <= run + sum) {
#pragma unroll 1
                for (uint32_t q = 0;; ++q) {
                    const uint64_t c = sh.mass[tid * PER + q];
                    if (target <= run + c) {
                        sh.found = tid * PER + q;
                        sh.above = run;
                        sh.inside = c;
                        break;
                    }
                    run += c;
                }
            }
            __syncthreads();
            const uint32_t slot = sh.found;
            const uint64_t above = sh.above, inside = sh.inside;
            __syncthreads();
            bool done = !enough;   // with this search
            if (step == FLOOR) {
                if (enough) {
                    bin_range<T>((int)slot, lo, hi);
                    lo = lo < LOWEST ? LOWEST : lo;
                }
                hi = K::INF;
                step = BIN;
                continue;
            }
            int key = 0;
            if (enough) {
                target -= above;
                if (step == BIN) {
                    int l, h;
                    bin_range<T>((int)slot, l, h);
                    key = l;
                    done = bin_exact<T>((int)slot);
                    if (!done) {
                        const int bits = 32 - __builtin_clz((uint32_t)(h - l));
                        shift = (bits + DIGIT - 1) / DIGIT * DIGIT;
                        prefix = 0;
                        lo = l > lo ? l : lo;
                        hi = h;
                        step = DIGITS;
                    }
                } else {
                    prefix = prefix << DIGIT | slot;
                    key = hi - (int)prefix;
                    done = shift == 0;
                }
            }
            if (!done) {
                above_shift = shift;
                shift -= DIGIT;
                continue;
            }
            if (enough) {
                if (!by_mass) {
                    ties = target;
                    count_f = inside;
                    key_k = key;
                    if (need_p) excess = (count_f - ties) * weight(key);
                } else {
                    const uint64_t w = weight(key), need = (target + w - 1) / w;
                    if (key == key_k) {
                        ties = need < ties ? need : ties;
                    } else {
                        ties = need;
                        count_f = inside / w;
                    }
                }
                key_f = key;
            }
            hi = K::INF;
            lo = key_f;
            step = need_p && !by_mass ? BIN : ties < count_f ? NTH : DRAW;
            by_mass = true;
            if (step == NTH) hi = key_f;
        } else {
            if (level == 0) {
                total = all;
                target = ties - 1;
                if (step == DRAW) {
                    const double u = u_in > 0.f ? (double)fminf(u_in, 0x1.fffffep-1f) : 0.0;
                    target = (uint64_t)(u * (double)all);
                }
                // (the wavefront's sum, not the thread's: its elements alternate between the lanes)
                run -= incl - sum;
                sum = sh.wave[wave];
            }
            run += base;
            if ((level || lane == 0) && run <= target && target < run + sum) {
                sh.above = run;
                sh.found = level ? from : wave * (nv * 64 * VEC);
                sh.key = key_in;
            }
            __syncthreads();
            const uint32_t start = sh.found;
            base = sh.above;
            key_in = sh.key;
            __syncthreads();
            const uint32_t per = (nv + WAVES - 1) / WAVES;   // vectors per thread of a segment
            if (level == 0) {
                const uint32_t end = start + nv * 64 * VEC;
                from = start + tid * per * VEC;
                until = from + per * VEC < end ? from + per * VEC : end;
                until = until < n_vocab ? until : n_vocab;
                begin = from;
                stride_v = VEC;
                count_v = from < until ? per : 0;
            } else if (level == 1) {
                from = start + tid;
                until = from + 1;
                begin = from & ~(uint32_t)(VEC - 1);
                count_v = tid < per * VEC && from < n_vocab ? 1 : 0;
            } else {
                if (step == NTH && !first_alone) {   // now the draw
                    cut = start;
                    hi = K::INF;
                    step = DRAW;
                    level = 0;
                    begin = first;
                    stride_v = 64 * VEC;
                    count_v = nv;
                    from = 0;
                    until = n_vocab;
                    base = 0;
                    continue;
                }
                if (tid == 0) {
                    *out_id = start;
                    if (out_logprob) *out_logprob = first_alone ? 0.f : (float)log((double)weight(key_in) / (double)total);
                }
                return;
            }
            ++level;
        }
    }
}


template <class T>
__device__ __forceinline__ Row<T> row_of(const T *logits, uint32_t n_vocab, uint64_t stride, const uint32_t *mask, uint64_t mask_stride,
                                         const float *temperature, const uint32_t *top_k, const float *top_p, const float *min_p,
                                         const float *uniform, uint64_t r)
{
    return Row<T>{logits + r * stride, mask ? mask + r * mask_stride : nullptr, n_vocab, temperature ? temperature[r] : 1.f,
                  top_p ? top_p[r] : 1.f, min_p ? min_p[r] : 0.f, uniform[r], top_k ? top_k[r] : 0};
}

// One workgroup, all phases.
template <class T, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_sample(const T *__restrict__ logits, uint32_t n_vocab, uint64_t stride,
                                                       const uint32_t *__restrict__ mask, uint64_t mask_stride,
                                                       const float *__restrict__ temperature,
                                                       const uint32_t *__restrict__ top_k, const float *__restrict__ top_p,
                                                       const float *__restrict__ min_p, const float *__restrict__ uniform,
                                                       uint32_t *__restrict__ out_ids, float *__restrict__ out_logprobs,
                                                       double magic)
{
    using K = Keys<T>;
    constexpr uint32_t THREADS = WAVES * 64, CELL = THREADS * VEC;
    constexpr bool TABLE = TABLE_OF<T, WAVES>;
    __shared__ Lds<WAVES> sh;
    const uint64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x, cells = (n_vocab + CELL - 1) / CELL;
    const Row<T> row = row_of(logits, n_vocab, stride, mask, mask_stride, temperature, top_k, top_p, min_p, uniform, r);
    float *out_logprob = out_logprobs ? out_logprobs + r : nullptr;
    const bool first_alone = row.k == 1 || !(row.temp > 0.f);
    const bool filtered = !first_alone && ((row.k != 0 && row.k < n_vocab) || row.p < 1.f);

    for (int b = tid; b < BINS; b += THREADS) sh.count[b] = 0;
    if (tid < MAX_CELLS) {
        sh.cell[tid] = 0;
        sh.border[tid] = 0;
    }
    if (tid == 0) sh.n_list = sh.n_odd = 0;
    __syncthreads();
    int mine;
    uint32_t mine_j;
    const bool small_k = filtered && row.k != 0 && row.k <= THREADS / 4;
    if (filtered && !small_k) scan_keys<T, WAVES, true>(row, sh, mine, mine_j);
    else scan_keys<T, WAVES, false>(row, sh, mine, mine_j);
    const int top = (int)(block_max(sh, (uint32_t)mine ^ 0x80000000u) ^ 0x80000000u);
    if (top > K::INF) return general_row<T, WAVES>(row, sh, magic, out_ids + r, out_logprob);   // NaN
    if (top <= -K::INF || first_alone) {   // nothing to choose from, or the first alone
        uint32_t id = NO_ID;
        if (top > -K::INF) id = first_of(row, sh, top, mine, mine_j);
        if (tid == 0) {
            out_ids[r] = id;
            if (out_logprob) *out_logprob = top <= -K::INF ? -__builtin_inff() : 0.f;
        }
        return;
    }
    const Weights wt{Weights::scale_of(row.temp), __builtin_fmin((double)K::value(top), Weights::HUGE_LOGIT), magic, top};
    auto weight = [&](int key) INLINE { return weight_of<T>(wt.c, wt.max, wt.magic, wt.max_key, key); };
    const uint64_t w_min = least_weight(wt, row.min_p);
    Border b{};
    b.lo = b.hi = BINS;
    if (TABLE) {   // the last bin's keys (from -2,047 down) have no weight in the table: it has to be zero
        int lo, hi;
        bin_range<T>(2 * HALF, lo, hi);
        if (top <= hi || weight(hi) != 0) return general_row<T, WAVES>(row, sh, magic, out_ids + r, out_logprob);
    }
    bool listed = false;
    if (small_k) {
        listed = list_first<T, WAVES>(row, sh, cells, mine, b);
        if (!listed) return general_row<T, WAVES>(row, sh, magic, out_ids + r, out_logprob);
    } else if (filtered) {
        b = find_border<T, WAVES>(row, sh, weight, [&](uint32_t bin_k) INLINE {
            for (int i = tid; i < BINS; i += THREADS) {
                uint64_t m = 0;
                if (TABLE && i <= (int)bin_k && bin_exact<T>(i) && sh.count[i]) {
                    int lo, hi;
                    bin_range<T>(i, lo, hi);
                    m = sh.count[i] * weight(lo);
                }
                sh.mass[i] = m;
            }
            __syncthreads();
            const uint32_t n = sh.n_odd;
            if (TABLE && n <= ODD) {
                for (uint32_t i = tid; i < n; i += THREADS) {
                    const int key = (int)sh.odd[i];
                    atomicAdd((unsigned long long *)&sh.mass[bin_of<T>(key)], (unsigned long long)weight(key));
                }
            } else if (TABLE) {   // every element of these bins by itself
#pragma unroll 1
                for (uint32_t c = 0; c < cells; ++c) {
                    const Vec8<T> v = row.fetch(c * CELL + tid * VEC);
#pragma unroll 1
                    for (int e = 0; e < VEC; ++e) {
                        const int key = v.pick(e), bin = bin_of<T>(key);
                        if ((key > -K::INF) & !bin_exact<T>(bin))
                            atomicAdd((unsigned long long *)&sh.mass[bin], (unsigned long long)wt.of(key, K::value(key)));
                    }
                }
            } else {   // every element
                row.template each<2, false>(CELL, [&](uint32_t, const Vec8<T> &v, uint32_t) INLINE {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int key = v.at(e);
                        const uint64_t w = wt.raw(K::value(key), key > -K::INF) - wt.zero();
                        if (w) atomicAdd((unsigned long long *)&sh.mass[bin_of<T>(key)], (unsigned long long)w);
                    }
                }, [](uint32_t, uint32_t) INLINE {});
            }
            __syncthreads();
        });
        if (b.hard) return general_row<T, WAVES>(row, sh, magic, out_ids + r, out_logprob);
    }
    if (!listed) scan_cells<T, WAVES>(row, sh, wt, b, w_min, weight);
    __syncthreads();
    draw<T, WAVES>(row, sh, wt, b, w_min, weight, out_ids + r, out_logprob);
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
    if (mask && mask_stride != 0 && (mask_stride < words || mask_stride > (1ull << 46) / n_rows)) return TOKTIER_E_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
    if (workspace_bytes < 256) return TOKTIER_E_CAPACITY;
    const uint64_t lb = extent(type, n_rows, n_vocab, stride), ob = 4ull * n_rows;
    const uint64_t mb = 4 * (words + (mask_stride ? (n_rows - 1) * mask_stride : 0));
    auto alone = [&](const void *out) {   // an output beside all inputs
        return apart(out, ob, logits, lb) && apart(out, ob, uniform, ob) && (!mask || apart(out, ob, mask, mb)) &&
               (!temperature || apart(out, ob, temperature, ob)) && (!top_k || apart(out, ob, top_k, ob)) &&
               (!top_p || apart(out, ob, top_p, ob)) && (!min_p || apart(out, ob, min_p, ob));
    };
    if (!alone(out_ids) || (out_logprobs && (!alone(out_logprobs) || !apart(out_logprobs, ob, out_ids, ob)))) return TOKTIER_E_INVALID_ARG;
    const double magic = weight_magic(n_vocab);
    with_type(type, [&](auto t) {
        using T = decltype(t);
        auto launch = [&](auto waves) {
            constexpr int W = decltype(waves)::value;
            auto from = [](auto *p, uint64_t r) { return p ? p + r : p; };
            in_launches(n_rows, W * 64, [&](uint64_t r, uint32_t rows) {
                k_sample<T, W><<<rows, W * 64, 0, (hipStream_t)stream>>>(
                    (const T *)logits + r * stride, n_vocab, stride, from(mask, r * mask_stride), mask_stride, from(temperature, r),
                    from(top_k, r), from(top_p, r), from(min_p, r), uniform + r, out_ids + r, from(out_logprobs, r), magic);
            });
        };
        if (n_vocab <= 8192) launch(std::integral_constant<int, 4>{});
        else launch(std::integral_constant<int, 16>{});
    });
    return hip_status(hipGetLastError());
}
