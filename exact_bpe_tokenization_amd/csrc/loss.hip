// loss.hip -- next-token cross entropy over the vocabulary and its gradient.
//
//   lse = m + log(s),  m = max_j x_j,  s = sum_j exp(x_j - m);  loss = (m - x_y) + log(s)
//   dx_j = c (exp(x_j - m) / s - [j == y])
//
// Bound by memory where rows are many and long: the logits are read and the gradient written, with one exponential per element.
// The loss alone of 1,500 x 33,001 float16, 29 us (3.4 TB/s), is bound by the VALU: 13.6 M wavefront
// instructions are three quarters of its issue at 2.4 GHz, and the exponentials among them take longer.
#include <algorithm>
#include <type_traits>

#include "ops.h"

namespace tt {
namespace {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
constexpr float NEG_INF = -__builtin_inff();

__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

// Running maximum m and sum s of exp(x - m); an empty sum is (-inf, 0).  m is only ever -inf, finite or
// +inf; a NaN among the logits goes into s.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b)
{
    const float m = fmaxf(a.m, b.m);
    if (m == NEG_INF) return MaxSum{m, a.s + b.s};
    return MaxSum{m, a.s * exp_f(a.m - m) + b.s * exp_f(b.m - m)};
}

template <int THREADS> __device__ __forceinline__ MaxSum block_join(MaxSum v, MaxSum *lds)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v = join(v, MaxSum{__shfl_xor(v.m, d), __shfl_xor(v.s, d)});
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll 4
    for (int w = 1; w < THREADS / 64; ++w) v = join(v, lds[w]);
    return v;
}

__device__ __forceinline__ void add_vec(MaxSum &a, const float (&x)[VEC])
{
    float m = a.m;
#pragma unroll
    for (int k = 0; k < VEC; ++k) m = fmaxf(m, x[k]);
    if (m == NEG_INF) {   // nothing but -inf so far, or NaN
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (x[k] != x[k]) a.s = x[k];
        return;
    }
    float s = a.s * exp_f(a.m - m);
#pragma unroll
    for (int k = 0; k < VEC; ++k) s += exp_f(x[k] - m);
    a = MaxSum{m, s};
}

// Gradient of one vector: x becomes c (exp(x - m) * r - [j == y]).
__device__ __forceinline__ void grad_vec(float (&x)[VEC], float m, float r, float c, uint32_t j, uint32_t y)
{
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[k] = c * (exp_f(x[k] - m) * r - (j + k == y ? 1.f : 0.f));
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
    // f(index, elements, values): values past the row's end are `fill`
    template <bool FIRST, class F> __device__ __forceinline__ void each(float fill, F f)
    {
        const uint32_t j0 = begin + threadIdx.x * VEC;
        if constexpr (FIRST) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (j0 + i * STEP + VEC <= end) held[i] = load_vec(x + j0 + i * STEP);
        }
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

// A row's gradient, once its maximum and sum are known.
template <class T, int THREADS, int HELD>
__device__ __forceinline__ void put_grad(RowPart<T, THREADS, HELD> &part, T *g, bool zero, MaxSum a, float c, uint32_t y)
{
    if (zero) {
        const float v[VEC] = {};
        for (uint32_t j = part.begin + threadIdx.x * VEC; j < part.end; j += THREADS * VEC) stream_part(g + j, part.end - j, v);
        return;
    }
    const float r = 1.f / a.s;
    part.template each<false>(0.f, [&](uint32_t j, uint32_t n, float (&v)[VEC]) {
        grad_vec(v, a.m, r, c, j, y);
        stream_part(g + j, n, v);
    });
}

__device__ __forceinline__ bool empty(MaxSum a) { return a.m == NEG_INF && a.s == 0.f; }   // nothing but -inf
__device__ __forceinline__ float log_of(float s) { return LN2 * __builtin_amdgcn_logf(s); }

// The loss comes from m - x_y, not from the rounded lse: at logits of 10,000 that is off by half a thousandth, in a row of
// the type's lowest value by all of the loss.
__device__ __forceinline__ void put_loss(MaxSum a, bool ignored, float target, float &loss, float &lse)
{
    const bool none = empty(a);
    const float log_s = log_of(a.s);
    lse = none ? NEG_INF : a.m + log_s;
    loss = ignored ? 0.f : none ? -NEG_INF : (a.m - target) + log_s;
}

template <class T, int THREADS, int HELD>
__global__ __launch_bounds__(THREADS, 8) void k_loss(const T *logits, uint32_t n_vocab, uint64_t stride,
                                                     const uint32_t *__restrict__ targets, float *__restrict__ loss,
                                                     float *__restrict__ lse_out, const float *__restrict__ grad_loss,
                                                     float grad_scale, T *grad, uint64_t gstride)
{
    __shared__ MaxSum lds[THREADS / 64];
    __shared__ float target;
    const uint64_t row = blockIdx.x;
    const uint32_t y = targets[row];
    RowPart<T, THREADS, HELD> part{logits + row * stride, 0, n_vocab};
    // (through LDS: the value is here before the barrier, the gradient may be written over it after)
    if (threadIdx.x == 0) target = y < n_vocab ? (float)part.x[y] : 0.f;
    MaxSum a{NEG_INF, 0.f};
    part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v); });
    a = block_join<THREADS>(a, lds);
    if (threadIdx.x == 0) put_loss(a, y >= n_vocab, target, loss[row], lse_out[row]);
    if (grad)
        put_grad(part, grad + row * gstride, empty(a) || y >= n_vocab, a, grad_scale * (grad_loss ? grad_loss[row] : 1.f), y);
}

// Few rows: each is split into pieces of one workgroup.  The first launch leaves the pieces' maxima and sums,
// and the target's logit; the second joins them, in the pieces' order, and writes the gradient.
constexpr int PIECE_THREADS = 256, PIECE_HELD = 4;
constexpr uint32_t PIECE = PIECE_THREADS * PIECE_HELD * VEC;
constexpr uint32_t MAX_PIECES = TOKTIER_MAX_VOCAB / PIECE;

template <class T>
__global__ __launch_bounds__(PIECE_THREADS) void k_loss_pieces(const T *logits, uint32_t n_vocab, uint64_t stride,
                                                               const uint32_t *__restrict__ targets,
                                                               MaxSum *__restrict__ sums, float *__restrict__ at_target)
{
    __shared__ MaxSum lds[PIECE_THREADS / 64];
    const uint64_t row = blockIdx.y;
    const uint32_t y = targets[row], begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    RowPart<T, PIECE_THREADS, PIECE_HELD> part{logits + row * stride, begin, end};
    if (threadIdx.x == 0 && y >= begin && y < end) at_target[row] = (float)part.x[y];
    MaxSum a{NEG_INF, 0.f};
    part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v); });
    a = block_join<PIECE_THREADS>(a, lds);
    if (threadIdx.x == 0) sums[row * gridDim.x + blockIdx.x] = a;
}

template <class T>
__global__ __launch_bounds__(PIECE_THREADS) void k_loss_join(const T *logits, uint32_t n_vocab, uint64_t stride, uint32_t pieces,
                                                             const uint32_t *__restrict__ targets,
                                                             const MaxSum *__restrict__ sums, const float *__restrict__ at_target,
                                                             float *__restrict__ loss, float *__restrict__ lse_out,
                                                             const float *__restrict__ grad_loss, float grad_scale, T *grad,
                                                             uint64_t gstride)
{
    __shared__ MaxSum lds[PIECE_THREADS / 64];
    const uint64_t row = blockIdx.y;
    const uint32_t y = targets[row], begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    static_assert(MAX_PIECES <= PIECE_THREADS, "a thread per piece");
    MaxSum a{NEG_INF, 0.f};
    if (threadIdx.x < pieces) a = sums[row * pieces + threadIdx.x];
    a = block_join<PIECE_THREADS>(a, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        put_loss(a, y >= n_vocab, y >= n_vocab ? 0.f : at_target[row], loss[row], lse_out[row]);
    if (!grad) return;
    RowPart<T, PIECE_THREADS, 1> part{logits + row * stride, begin, end};
    const float c = grad_scale * (grad_loss ? grad_loss[row] : 1.f), r = 1.f / a.s;
    const bool zero = empty(a) || y >= n_vocab;
    T *g = grad + row * gstride;
    part.template each<true>(0.f, [&](uint32_t j, uint32_t n, float (&v)[VEC]) {
        if (zero) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        } else {
            grad_vec(v, a.m, r, c, j, y);
        }
        stream_part(g + j, n, v);
    });
}

// The gradient from lse.  A rounding of lse is relative to it, so far from zero exp(x - lse) loses the digits that tell the
// probabilities (in a row of the type's lowest value each would be 1, not 1 / n).  From FAR on, where that would be as
// much as the power itself can be off (its exponent is rounded too, and reaches 104 before the power is zero), a row's
// maximum and sum are formed again.  One workgroup takes such a row whole, since in place the others would read
// what it has written.  (Two inputs in turn, 1,500 x 33,001 float16: 32 us, 51 with all rows far; 8,192 x 131,328 bfloat16: 767 and 1,216 us.)
constexpr float FAR = 128.f;

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void k_loss_backward(const T *logits, uint32_t n_vocab, uint64_t stride,
                                                              const uint32_t *__restrict__ targets,
                                                              const float *__restrict__ lse, const float *__restrict__ grad_loss,
                                                              float grad_scale, T *grad, uint64_t gstride)
{
    __shared__ MaxSum lds[THREADS / 64];
    const uint64_t row = blockIdx.y;
    const uint32_t y = targets[row], begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    const float z = lse[row], c = grad_scale * (grad_loss ? grad_loss[row] : 1.f);
    RowPart<T, THREADS, PIECE / (THREADS * VEC)> part{logits + row * stride, begin, end};
    T *g = grad + row * gstride;
    if (z == NEG_INF || y >= n_vocab) return put_grad(part, g, true, MaxSum{z, 1.f}, c, y);
    if (!(__builtin_fabsf(z) < FAR)) {   // NaN too
        if (blockIdx.x) return;
        part.end = n_vocab;
        MaxSum a{NEG_INF, 0.f};
        part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v); });
        a = block_join<THREADS>(a, lds);
        return put_grad(part, g, empty(a), a, c, y);
    }
    part.template each<true>(0.f, [&](uint32_t j, uint32_t n, float (&v)[VEC]) {
        grad_vec(v, z, 1.f, c, j, y);
        stream_part(g + j, n, v);
    });
}

}  // namespace
}  // namespace tt

using namespace tt;

namespace {

// The arguments that both entry points share.
int check_loss(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, const uint32_t *targets,
               const float *lse, const float *grad_loss, const void *grad, uint64_t gstride)
{
    if (!elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu) return TOKTIER_E_INVALID_ARG;
    if (n_rows == 0) return TOKTIER_OK;
    if (!matrix_ok(logits, type, n_rows, n_vocab, stride)) return TOKTIER_E_INVALID_ARG;
    if (!targets || !aligned4(targets) || !lse || !aligned4(lse) || !aligned4(grad_loss)) return TOKTIER_E_INVALID_ARG;
    if (grad) {
        if (!matrix_ok(grad, type, n_rows, n_vocab, gstride)) return TOKTIER_E_INVALID_ARG;
        const uint64_t gb = extent(type, n_rows, n_vocab, gstride), lb = extent(type, n_rows, n_vocab, stride);
        if (!(grad == logits && gstride == stride) && !apart(grad, gb, logits, lb)) return TOKTIER_E_INVALID_ARG;
        if (!apart(grad, gb, targets, 4ull * n_rows) || !apart(grad, gb, lse, 4ull * n_rows) ||
            (grad_loss && !apart(grad, gb, grad_loss, 4ull * n_rows)))
            return TOKTIER_E_INVALID_ARG;
    }
    return TOKTIER_OK;
}

}  // namespace

namespace {

// Few long rows are split: a second launch (3 us) buys the other CUs.  131,328 bfloat16 with gradient, split /
// whole: 1 row 10.4 / 22.3 us, 128 rows 20.0 / 24.9, 192 rows 30.0 / 27.9; of 33,024 elements 10.3 / 9.1 us and
// never better.
constexpr uint32_t MOST_SPLIT = 159;
bool split_rows(uint32_t n_rows, uint32_t n_vocab) { return n_vocab >= 8 * PIECE && n_rows <= MOST_SPLIT; }

struct LossLayout {
    uint32_t pieces;   // 0: rows are not split
    uint64_t at_target, total;
};

LossLayout loss_layout(uint32_t n_rows, uint32_t n_vocab)
{
    LossLayout L{0, 0, 256};
    if (!split_rows(n_rows, n_vocab)) return L;
    L.pieces = (n_vocab + PIECE - 1) / PIECE;
    L.at_target = ((uint64_t)n_rows * L.pieces * sizeof(MaxSum) + 255) & ~255ull;
    L.total = L.at_target + (((uint64_t)n_rows * 4 + 255) & ~255ull);
    return L;
}

}  // namespace

extern "C" int toktier_cross_entropy_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu) return TOKTIER_E_INVALID_ARG;
    // what any call of up to n_rows rows needs: the most of those whose rows are split
    *out_bytes = loss_layout(std::clamp(n_rows, 1u, MOST_SPLIT), n_vocab).total;
    return TOKTIER_OK;
}

extern "C" int toktier_cross_entropy(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride,
                                     const uint32_t *targets, float *loss, float *lse, const float *grad_loss,
                                     float grad_scale, void *grad_logits, uint64_t grad_stride, void *workspace,
                                     uint64_t workspace_bytes, void *stream)
{
    int rc = check_loss(logits, type, n_rows, n_vocab, stride, targets, lse, grad_loss, grad_logits, grad_stride);
    if (rc || n_rows == 0) return rc;
    if (!loss || !aligned4(loss) || !workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
    const LossLayout L = loss_layout(n_rows, n_vocab);
    if (workspace_bytes < L.total) return TOKTIER_E_CAPACITY;
    const uint64_t lb = extent(type, n_rows, n_vocab, stride), nb = 4ull * n_rows;
    if (!apart(workspace, L.total, logits, lb) || !apart(workspace, L.total, loss, nb) || !apart(workspace, L.total, lse, nb) ||
        !apart(workspace, L.total, targets, nb) || (grad_loss && !apart(workspace, L.total, grad_loss, nb)) ||
        !apart(loss, nb, lse, nb) || !apart(loss, nb, logits, lb) || !apart(lse, nb, logits, lb) || !apart(loss, nb, targets, nb) ||
        !apart(lse, nb, targets, nb) || (grad_loss && (!apart(loss, nb, grad_loss, nb) || !apart(lse, nb, grad_loss, nb))) ||
        (grad_logits && (!apart(grad_logits, extent(type, n_rows, n_vocab, grad_stride), loss, nb) ||
                         !apart(workspace, L.total, grad_logits, extent(type, n_rows, n_vocab, grad_stride)))))
        return TOKTIER_E_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    with_type(type, [&](auto t) {
        using T = decltype(t);
        constexpr int HELD = sizeof(T) == 4 ? 4 : 8;   // 32 VGPRs
        const T *x = (const T *)logits;
        T *g = (T *)grad_logits;
        if (L.pieces) {
            MaxSum *sums = (MaxSum *)workspace;
            float *at_target = (float *)((uint8_t *)workspace + L.at_target);
            // grid.y holds 65,535 rows at most; split_rows() has far fewer
            k_loss_pieces<T><<<dim3(L.pieces, n_rows), PIECE_THREADS, 0, s>>>(x, n_vocab, stride, targets, sums, at_target);
            k_loss_join<T><<<dim3(g ? L.pieces : 1, n_rows), PIECE_THREADS, 0, s>>>(x, n_vocab, stride, L.pieces, targets, sums, at_target,
                                                                                    loss, lse, grad_loss, grad_scale, g, grad_stride);
        } else {
            auto launch = [&](auto threads, auto held) {
                constexpr int N = decltype(threads)::value, H = decltype(held)::value;
                in_launches(n_rows, N, [&](uint64_t r, uint32_t rows) {
                    k_loss<T, N, H><<<rows, N, 0, s>>>(x + r * stride, n_vocab, stride, targets + r, loss + r, lse + r,
                                                       grad_loss ? grad_loss + r : nullptr, grad_scale,
                                                       g ? g + r * grad_stride : nullptr, grad_stride);
                });
            };
            if (n_vocab <= 256 * VEC * 4)   // short rows: more workgroups per CU
                launch(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
            else if (n_vocab <= 512 * VEC * 8)
                launch(std::integral_constant<int, 512>{}, std::integral_constant<int, HELD>{});
            else
                launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, HELD>{});
        }
    });
    return hip_status(hipGetLastError());
}

extern "C" int toktier_cross_entropy_backward(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride,
                                              const uint32_t *targets, const float *lse, const float *grad_loss,
                                              float grad_scale, void *grad_logits, uint64_t grad_stride, void *stream)
{
    if (n_rows && !grad_logits) return TOKTIER_E_INVALID_ARG;
    int rc = check_loss(logits, type, n_rows, n_vocab, stride, targets, lse, grad_loss, grad_logits, grad_stride);
    if (rc || n_rows == 0) return rc;
    const uint32_t pieces = (n_vocab + PIECE - 1) / PIECE;
    with_type(type, [&](auto t) {
        using T = decltype(t);
        for (uint32_t r = 0; r < n_rows; r += 65535) {   // grid.y
            const uint32_t rows = n_rows - r < 65535 ? n_rows - r : 65535;
            k_loss_backward<T, 256><<<dim3(pieces, rows), 256, 0, (hipStream_t)stream>>>(
                (const T *)logits + r * stride, n_vocab, stride, targets + r, lse + r, grad_loss ? grad_loss + r : nullptr, grad_scale,
                (T *)grad_logits + r * grad_stride, grad_stride);
        }
    });
    return hip_status(hipGetLastError());
}
