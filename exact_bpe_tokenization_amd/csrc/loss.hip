// loss.hip -- next-token cross entropy over the vocabulary and its gradient.
//
//   lse = m + log(s),  m = max_j x_j,  s = sum_j exp(x_j - m);  loss = lse - x_y
//   dx_j = c (exp(x_j - m) / s - [j == y])
//
// Bound by memory: the logits are read and the gradient written, with one exponential per element.
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
#pragma unroll
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

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_loss(const T *logits, uint32_t n_vocab, uint64_t stride,
                                                  const uint32_t *__restrict__ targets, float *__restrict__ loss,
                                                  float *__restrict__ lse_out, const float *__restrict__ grad_loss,
                                                  float grad_scale, T *grad, uint64_t gstride)
{
    __shared__ MaxSum lds[THREADS / 64];
    const uint64_t row = blockIdx.x;
    const T *x = logits + row * stride;
    const uint32_t y = targets[row];
    const float xy = y < n_vocab ? (float)x[y] : 0.f;
    MaxSum a{NEG_INF, 0.f};
    for (uint32_t j = threadIdx.x * VEC; j < n_vocab; j += THREADS * VEC) {
        float v[VEC];
        load_part(x + j, n_vocab - j, NEG_INF, v);
        add_vec(a, v);
    }
    a = block_join<THREADS>(a, lds);
    const bool none = a.m == NEG_INF && a.s == 0.f;
    const float lse = none ? NEG_INF : a.m + LN2 * __builtin_amdgcn_logf(a.s);
    if (threadIdx.x == 0) {
        lse_out[row] = lse;
        loss[row] = y >= n_vocab ? 0.f : none ? -NEG_INF : lse - xy;
    }
    if (!grad) return;
    const float c = grad_scale * (grad_loss ? grad_loss[row] : 1.f);
    const bool zero = none || y >= n_vocab;
    const float r = 1.f / a.s;
    for (uint32_t j = threadIdx.x * VEC; j < n_vocab; j += THREADS * VEC) {
        float v[VEC];
        if (zero) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        } else {
            load_part(x + j, n_vocab - j, 0.f, v);
            grad_vec(v, a.m, r, c, j, y);
        }
        store_part(grad + row * gstride + j, n_vocab - j, v);
    }
}

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_loss_backward(const T *logits, uint32_t n_vocab, uint64_t stride,
                                                           const uint32_t *__restrict__ targets,
                                                           const float *__restrict__ lse, const float *__restrict__ grad_loss,
                                                           float grad_scale, T *grad, uint64_t gstride)
{
    const uint64_t row = blockIdx.x;
    const uint32_t y = targets[row];
    const float z = lse[row], c = grad_scale * (grad_loss ? grad_loss[row] : 1.f);
    const bool zero = z == NEG_INF || y >= n_vocab;
    for (uint32_t j = threadIdx.x * VEC; j < n_vocab; j += THREADS * VEC) {
        float v[VEC];
        if (zero) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        } else {
            load_part(logits + row * stride + j, n_vocab - j, 0.f, v);
            grad_vec(v, z, 1.f, c, j, y);
        }
        store_part(grad + row * gstride + j, n_vocab - j, v);
    }
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

extern "C" int toktier_cross_entropy_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu) return TOKTIER_E_INVALID_ARG;
    *out_bytes = 256;
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
    if (workspace_bytes < 256) return TOKTIER_E_CAPACITY;
    with_type(type, [&](auto t) {
        using T = decltype(t);
        k_loss<T, 1024><<<n_rows, 1024, 0, (hipStream_t)stream>>>((const T *)logits, n_vocab, stride, targets, loss, lse, grad_loss,
                                                                  grad_scale, (T *)grad_logits, grad_stride);
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
    with_type(type, [&](auto t) {
        using T = decltype(t);
        k_loss_backward<T, 1024><<<n_rows, 1024, 0, (hipStream_t)stream>>>((const T *)logits, n_vocab, stride, targets, lse, grad_loss,
                                                                           grad_scale, (T *)grad_logits, grad_stride);
    });
    return hip_status(hipGetLastError());
}
