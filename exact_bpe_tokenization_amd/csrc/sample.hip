// sample.hip -- sampling of one ID per row: temperature, top-k, top-p, min-p, given random numbers.
//
// Every filter keeps a prefix of the order (logit descending, ID ascending), so the kept set is one pair: a
// logit (as an order-preserving 32-bit key) and how many of its equals, lowest IDs first.  Counts find the
// top-k pair and masses the top-p pair, by the same search over histograms of key digits.  Masses are
// sums of 64-bit integers, w = 2^y rounded to a multiple of 2^-S with y = (x - max) log2(e) / temperature in
// 64-bit floating point: exact in any order, so neither atomics nor the split of a row over threads can
// change an ID.
#include "ops.h"

namespace tt {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr uint32_t SLAB = THREADS * VEC;                      // elements of one round of the workgroup's vectors
constexpr uint32_t MAX_SLABS = TOKTIER_MAX_VOCAB / SLAB;
constexpr uint32_t BINS = 2048;
constexpr uint32_t NO_ID = 0xFFFFFFFFu;

// Order-preserving key of a logit; 0 for one that is out of the choice (-inf, NaN).
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (!(x > -__builtin_inff())) return 0;
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);   // -0 and +0 are equals
    return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __builtin_bit_cast(float, (int32_t)k < 0 ? k & 0x7FFFFFFFu : ~k);
}

// Weights of one row.  2^y = 2^n 2^f with n the nearest integer: 2^f on [-1/2, 1/2] by the polynomial of degree
// 10 that interpolates it at the Chebyshev nodes (relative error below 2^-51), the multiple of 2^-S by
// adding 2^(52 - S) and reading the low bits.
struct Weights {
    double c, max, magic;
    uint32_t max_key;

    __device__ __forceinline__ uint64_t one() const
    {
        return __builtin_bit_cast(uint64_t, 1.0 + magic) - __builtin_bit_cast(uint64_t, magic);
    }
    __device__ __forceinline__ uint64_t of(uint32_t key) const
    {
        if (key == max_key) return one();
        const double y = ((double)key_logit(key) - max) * c;
        if (key == 0 || !(y > -64.0)) return 0;
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
        return __builtin_bit_cast(uint64_t, w + magic) - __builtin_bit_cast(uint64_t, magic);
    }
};

struct Shared {
    uint64_t hist[BINS];
    uint64_t slab[MAX_SLABS];
    uint64_t wave[WAVES];
    uint64_t found_above;
    uint32_t found;
    uint32_t found_key;
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

// Inclusive sum over the workgroup's threads; total: over all.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, Shared &sh, uint64_t &total)
{
    const uint32_t wave = threadIdx.x >> 6;
    v = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh.wave[wave] = v;
    __syncthreads();
    uint64_t base = 0;
    total = 0;
#pragma unroll
    for (uint32_t w = 0; w < WAVES; ++w) {
        const uint64_t s = sh.wave[w];
        if (w < wave) base += s;
        total += s;
    }
    return base + v;
}

template <class T> struct Row {
    const T *x;
    const uint32_t *mask;
    uint32_t n;

    // keys of the eight elements from j on (j a multiple of eight below n)
    __device__ __forceinline__ void keys(uint32_t j, uint32_t (&k)[VEC]) const
    {
        float v[VEC];
        load_part(x + j, n - j, -__builtin_inff(), v);
        const uint32_t bits = mask ? mask[j >> 5] >> (j & 31u) : 0xFFu;
#pragma unroll
        for (int e = 0; e < VEC; ++e) k[e] = (bits >> e) & 1u ? logit_key(v[e]) : 0u;
    }
};

// The bin of sh.hist where the sum from the highest bin down reaches `target` (1 .. the sum of all), and the
// sum above it.
__device__ __forceinline__ uint32_t find_bin(Shared &sh, uint64_t target, uint64_t &above)
{
    const uint32_t hi = BINS - 1 - 2 * threadIdx.x;
    const uint64_t a = sh.hist[hi], b = sh.hist[hi - 1];
    uint64_t total;
    const uint64_t incl = block_scan(a + b, sh, total), before = incl - a - b;
    if (before < target && target <= incl) {
        const bool second = before + a < target;
        sh.found = second ? hi - 1 : hi;
        sh.found_above = second ? before + a : before;
    }
    __syncthreads();
    above = sh.found_above;
    const uint32_t bin = sh.found;
    __syncthreads();
    return bin;
}

// The first index (ascending) at which the running sum of measure(key, index) exceeds `target`; the target is
// target(total of all).
template <class T, class M, class G>
__device__ __forceinline__ uint32_t locate(const Row<T> &row, Shared &sh, M measure, G target_of, uint64_t &total,
                                           uint32_t &key_at)
{
    const uint32_t slabs = (row.n + SLAB - 1) / SLAB;
    if (threadIdx.x < MAX_SLABS) sh.slab[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t s = 0; s < slabs; ++s) {
        const uint32_t j = s * SLAB + threadIdx.x * VEC;
        uint64_t sum = 0;
        if (j < row.n) {
            uint32_t k[VEC];
            row.keys(j, k);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += measure(k[e], j + e);
        }
        if (__ballot(sum != 0)) {
            sum = wave_scan(sum);
            if ((threadIdx.x & 63) == 63) atomicAdd((unsigned long long *)&sh.slab[s], (unsigned long long)sum);
        }
    }
    __syncthreads();
    uint64_t v = threadIdx.x < slabs ? sh.slab[threadIdx.x] : 0;
    uint64_t incl = block_scan(v, sh, total);
    const uint64_t target = target_of(total);
    if (incl - v <= target && target < incl) {
        sh.found = threadIdx.x;
        sh.found_above = incl - v;
    }
    __syncthreads();
    const uint32_t s = sh.found;
    const uint64_t base = sh.found_above;
    const uint32_t j = s * SLAB + threadIdx.x * VEC;
    uint32_t k[VEC] = {};
    v = 0;
    if (j < row.n) {
        row.keys(j, k);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v += measure(k[e], j + e);
    }
    uint64_t all;
    incl = base + block_scan(v, sh, all);
    if (incl - v <= target && target < incl) {
        uint64_t run = incl - v;
        uint32_t at = NO_ID, kk = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            run += measure(k[e], j + e);
            if (at == NO_ID && run > target) {
                at = j + e;
                kk = k[e];
            }
        }
        sh.found = at;
        sh.found_key = kk;
    }
    __syncthreads();
    const uint32_t r = sh.found;
    key_at = sh.found_key;
    __syncthreads();
    return r;
}

template <class T>
__global__ __launch_bounds__(THREADS) void k_sample(const T *__restrict__ logits, uint32_t n_vocab, uint64_t stride,
                                                    const uint32_t *__restrict__ mask, uint64_t mask_stride,
                                                    const float *__restrict__ temperature,
                                                    const uint32_t *__restrict__ top_k, const float *__restrict__ top_p,
                                                    const float *__restrict__ min_p, const float *__restrict__ uniform,
                                                    uint32_t *__restrict__ out_ids, float *__restrict__ out_logprobs,
                                                    double magic)
{
    __shared__ Shared sh;
    // levels of the key search: digits of 11, 11 and 10 bits; a 16-bit type has nothing below the second
    constexpr int LEVELS = sizeof(T) == 4 ? 3 : 2;
    const uint64_t r = blockIdx.x;
    const Row<T> row{logits + r * stride, mask ? mask + r * mask_stride : nullptr, n_vocab};
    const float temp = temperature ? temperature[r] : 1.f;

    // largest key with its lowest index, and how many are in the choice
    uint64_t best = 0;
    uint32_t valid = 0;
    for (uint32_t j = threadIdx.x * VEC; j < n_vocab; j += SLAB) {
        uint32_t k[VEC];
        row.keys(j, k);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            valid += k[e] != 0;
            const uint64_t b = (uint64_t)k[e] << 32 | ~(j + e);
            if (b > best) best = b;
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor(best, d);
        best = o > best ? o : best;
    }
    uint64_t total;
    block_scan(valid, sh, total);
    valid = (uint32_t)total;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = best;
    __syncthreads();
    for (int w = 0; w < WAVES; ++w) best = sh.wave[w] > best ? sh.wave[w] : best;
    __syncthreads();
    const uint32_t max_key = (uint32_t)(best >> 32);
    uint32_t k = top_k ? top_k[r] : 0;
    if (k == 0 || k > valid) k = valid;
    if (k <= 1 || !(temp > 0.f)) {   // nothing, or the first alone
        if (threadIdx.x == 0) {
            out_ids[r] = valid ? ~(uint32_t)best : NO_ID;
            if (out_logprobs) out_logprobs[r] = valid ? 0.f : -__builtin_inff();
        }
        return;
    }
    const Weights wt{1.4426950408889634 / (double)temp, (double)key_logit(max_key), magic, max_key};

    // kept so far: keys above key_f, and of those equal to it the first `ties`
    uint32_t key_f = 1, ties = 0xFFFFFFFFu, count_f = 0;   // (all)
    auto digit_shift = [](int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; };
    // One search: measure(key) summed per digit over the keys >= floor, level by level.  `floor_excess` is what
    // the equals of `floor` beyond its ties would add.
    auto search = [&](auto measure, uint32_t floor, uint64_t floor_excess, auto target_of, uint64_t &above_all,
                      uint64_t &target, uint64_t &in_bin) {
        uint32_t prefix = 0;
        above_all = 0;
        target = 0;
        for (int level = 0; level < LEVELS; ++level) {
            const int shift = digit_shift(level);
            const uint32_t dmask = level == 2 ? 1023u : 2047u;
            const int pshift = level == 0 ? 0 : digit_shift(level - 1);
            for (uint32_t b = threadIdx.x; b < BINS; b += THREADS) sh.hist[b] = 0;
            __syncthreads();
            for (uint32_t j = threadIdx.x * VEC; j < n_vocab; j += SLAB) {
                uint32_t kk[VEC];
                row.keys(j, kk);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (kk[e] >= floor && (level == 0 || kk[e] >> pshift == prefix))
                        atomicAdd((unsigned long long *)&sh.hist[(kk[e] >> shift) & dmask],
                                  (unsigned long long)measure(kk[e]));
            }
            __syncthreads();
            if (threadIdx.x == 0 && floor_excess && (level == 0 || floor >> pshift == prefix))
                sh.hist[(floor >> shift) & dmask] -= floor_excess;
            __syncthreads();
            if (level == 0) {
                uint64_t all;
                block_scan(sh.hist[2 * threadIdx.x] + sh.hist[2 * threadIdx.x + 1], sh, all);
                target = target_of(all);
                __syncthreads();
            }
            uint64_t above;
            const uint32_t bin = find_bin(sh, target - above_all, above);
            above_all += above;
            in_bin = sh.hist[bin];
            __syncthreads();
            prefix = level == 0 ? bin : prefix << (level == 2 ? 10 : 11) | bin;
        }
        // the digits below the last level are zeros, of a negative number ones
        const int low = digit_shift(LEVELS - 1);
        return low && !(prefix >> (31 - low)) ? prefix << low | ((1u << low) - 1u) : prefix << low;
    };

    uint64_t above, target, in_bin;
    uint64_t excess = 0;
    if (k < valid) {
        key_f = search([](uint32_t) { return 1ull; }, 1u, 0, [&](uint64_t) { return (uint64_t)k; }, above, target, in_bin);
        ties = k - (uint32_t)above;
        count_f = (uint32_t)in_bin;
        excess = (uint64_t)(count_f - ties) * wt.of(key_f);
    }
    const float p = top_p ? top_p[r] : 1.f;
    if (p < 1.f) {
        const uint32_t key_k = key_f;
        const uint32_t key = search([&](uint32_t kk) { return wt.of(kk); }, key_k, excess, [&](uint64_t all) {
            const double t = __builtin_ceil((double)p * (double)all);
            const uint64_t u = t > 1.0 ? (uint64_t)t : 1ull;
            return u < all ? u : all;
        }, above, target, in_bin);
        const uint64_t w = wt.of(key);
        const uint32_t need = (uint32_t)((target - above + w - 1) / w);
        if (key != key_k || count_f == 0) {
            count_f = (uint32_t)(in_bin / w);
            ties = need;
        } else {
            ties = need < ties ? need : ties;
        }
        key_f = key;
    }
    uint32_t cut = NO_ID;   // the last index whose key may equal key_f
    uint32_t dummy;
    if (ties < count_f) {
        uint64_t t;
        cut = locate(row, sh, [&](uint32_t kk, uint32_t) { return (uint64_t)(kk == key_f); },
                     [&](uint64_t) { return (uint64_t)ties - 1; }, t, dummy);
    }
    const float mp = min_p ? min_p[r] : 0.f;
    const uint64_t one = wt.one();
    const uint64_t w_min = mp >= 1.f ? one : mp > 0.f ? (uint64_t)__builtin_ceil((double)mp * (double)one) : 0;
    const float u_in = uniform[r];
    const double u = u_in > 0.f ? (double)fminf(u_in, 0x1.fffffep-1f) : 0.0;
    uint32_t key_at;
    const uint32_t id = locate(row, sh, [&](uint32_t kk, uint32_t j) {
        if (kk < key_f || (kk == key_f && j > cut)) return (uint64_t)0;
        const uint64_t w = wt.of(kk);
        return w >= w_min ? w : (uint64_t)0;
    }, [&](uint64_t all) { return (uint64_t)(u * (double)all); }, total, key_at);
    if (threadIdx.x == 0) {
        out_ids[r] = id;
        if (out_logprobs) out_logprobs[r] = (float)log((double)wt.of(key_at) / (double)total);
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
        k_sample<T><<<n_rows, THREADS, 0, (hipStream_t)stream>>>((const T *)logits, n_vocab, stride, mask, mask_stride, temperature, top_k,
                                                                 top_p, min_p, uniform, out_ids, out_logprobs, magic);
    });
    return hip_status(hipGetLastError());
}
