// rows.h -- rows of logits as workgroups read them: running maximum and sum of exponentials, vectors that stay in
// registers for a second pass, rows split into pieces (loss.hip, distill.hip, top.hip; sums also in linear_loss.hip).
#pragma once
#include "ops.h"

namespace tt {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
constexpr float NEG_INF = -__builtin_inff();

// exp(x), or exp(x / temperature) with k = log2(e) / temperature
__device__ __forceinline__ float exp_f(float x, float k = LOG2E) { return __builtin_amdgcn_exp2f(x * k); }

// Temperatures whose k is a positive number: with an infinite one a distance of 0 would be NaN.
inline bool temperature_ok(float t) { return t > 0.f && t <= 3.4028234e38f && LOG2E * (1.f / t) <= 3.4028234e38f; }

// Running maximum m and sum s of exp(x - m); an empty sum is (-inf, 0).  m is only ever -inf, finite or
// +inf; a NaN among the logits goes into s.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k = LOG2E)
{
    const float m = fmaxf(a.m, b.m);
    if (m == NEG_INF) return MaxSum{m, a.s + b.s};
    return MaxSum{m, a.s * exp_f(a.m - m, k) + b.s * exp_f(b.m - m, k)};
}

template <int THREADS> __device__ __forceinline__ MaxSum block_join(MaxSum v, MaxSum *lds, float k = LOG2E)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v = join(v, MaxSum{__shfl_xor(v.m, d), __shfl_xor(v.s, d)}, k);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll 4
    for (int w = 1; w < THREADS / 64; ++w) v = join(v, lds[w], k);
    return v;
}

__device__ __forceinline__ void add_vec(MaxSum &a, const float (&x)[VEC], float k = LOG2E)
{
    float m = a.m;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = fmaxf(m, x[i]);
    if (m == NEG_INF) {   // nothing but -inf so far, or NaN
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (x[i] != x[i]) a.s = x[i];
        return;
    }
    float s = a.s * exp_f(a.m - m, k);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += exp_f(x[i] - m, k);
    a = MaxSum{m, s};
}

// Elements [begin, end) of a row as a workgroup's vectors, the first HELD of each thread in registers, so that
// the second pass over them reads nothing.  The others are read again: from the caches, which hold the rows
// in work (two workgroups of 1,024 per CU) because the gradient is stored past them.
//
// 8,192 rows of 131,328 bfloat16 in 815 us (4.3 GB, 5.28 TB/s; a copy reaches 5.15), 4,096 of float32, of which half as
// much is held, in 1,011 us (4.26 TB/s); bfloat16 without registers 957 us
// with ordinary stores, 845 us with four held and streaming stores, 845 us with ten (64 VGPRs are used up at
// eight), 924 to 944 us with all seventeen (one workgroup per CU).
template <class T, int THREADS, int HELD> struct RowPart {
    static constexpr uint32_t STEP = THREADS * VEC;
    const T *x;
    uint32_t begin, end;
    Vec<T> held[HELD];

    template <class F> __device__ __forceinline__ void with(const Vec<T> &v, uint32_t j, F f) const
    {
        float x8[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) x8[k] = vec_at(v, k);
        f(j, (uint32_t)VEC, x8);
    }
    // brings what is held on its way; each<true> does so itself
    __device__ __forceinline__ void hold()
    {
        const uint32_t j0 = begin + threadIdx.x * VEC;
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (j0 + i * STEP + VEC <= end) held[i] = load_vec(x + j0 + i * STEP);
    }
    // f(index, elements, values): values past the row's end are `fill`
    template <bool FIRST, class F> __device__ __forceinline__ void each(float fill, F f)
    {
        const uint32_t j0 = begin + threadIdx.x * VEC;
        if constexpr (FIRST) hold();
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (j0 + i * STEP + VEC <= end) with(held[i], j0 + i * STEP, f);
        uint32_t j = j0 + HELD * STEP;
        for (; j + STEP + VEC <= end; j += 2 * STEP) {
            const Vec<T> v = load_vec(x + j), w = load_vec(x + j + STEP);
            with(v, j, f);
            with(w, j + STEP, f);
        }
        if (j + VEC <= end) with(load_vec(x + j), j, f);
        // the thread in whose vector the row ends
        const uint32_t tail = begin + (end - begin) / VEC * VEC;
        if (tail < end && (tail - begin) % STEP == threadIdx.x * VEC) {
            float x8[VEC];
            load_part(x + tail, end - tail, fill, x8);
            f(tail, end - tail, x8);
        }
    }
};

// A log-sum-exp so far from zero that its rounding, which is relative, would show in the probabilities (NaN too).
constexpr float FAR = 128.f;
__device__ __forceinline__ bool is_far(float lse) { return !(__builtin_fabsf(lse) < FAR); }

__device__ __forceinline__ bool empty(MaxSum a) { return a.m == NEG_INF && a.s == 0.f; }   // nothing but -inf
__device__ __forceinline__ float log_of(float s) { return LN2 * __builtin_amdgcn_logf(s); }

constexpr int PIECE_THREADS = 256, PIECE_HELD = 4;
constexpr uint32_t PIECE = PIECE_THREADS * PIECE_HELD * VEC;
constexpr uint32_t MAX_PIECES = TOKTIER_MAX_VOCAB / PIECE;

}  // namespace tt
