// linear_loss.h -- next-token cross entropy straight from hidden states and the table of the logits, and its gradients,
// without keeping the logits.
//
//   x = h W^T,  lse = log sum_v exp(x_v),  loss = lse - x_y
//   G = c (exp(x - lse) - [v == y]),  dh = G W,  dW = G^T h
//
// One product gives every tile's maximum and sum of exponentials per row, and, for as many IDs as a gibibyte holds, leaves
// the exponentials (in the operands' size), which become G once the rows' sums are known.  For the others the
// product is formed again, a piece of the vocabulary at a time.  G goes into dh (32-bit sums over the pieces) and into
// the pieces' rows of dW.  Positions whose target is no ID are left out of all products: the hidden states of the others
// are copied together first, into rows that the products need not check for their ends.
//
// Bound by the matrix cores from some 300 rows on, by the table's bytes below.  bfloat16, 8,192 rows x 131,328 x 4,096: loss 5.95 ms
// (1,480 TFLOP/s), with gradients 23.2 ms (half of the IDs' exponentials kept, 345 us to make them G, the others' product formed
// twice); 1,638 rows x 33,024 x 2,048: 184 and 655 us (as 1,638 that take part of 4,096: 690 to 706); 16 rows x 131,328 x 4,096: 218 us
// (4.9 TB/s) and 798.  float32, 2,048 rows x 33,024 x 1,024: 1.0 ms and 3.2 (130 TFLOP/s); 16 rows x 131,328 x 4,096: 468 us (4.6 TB/s) and
// 3,119.
//
// G is an operand of the type, as the matrix cores take no 32-bit one beside 16 bits: rounded once from 32 bits (and see keep_high).
// Gradients of 16 bits are so 2.1e-3 to 2.5e-3 (bfloat16) and 3.0e-4 (float16) from 64 bits, of which their own rounding is 1.7e-3 and 2.1e-4.
#pragma once
#include <algorithm>
#include <type_traits>

#include "product.h"
#include "rows.h"

namespace tt {

constexpr uint32_t PAD = 256;            // rows of the packed matrices come in this many

// What the calls leave for each other in the workspace.
struct Head {
    uint32_t count;       // rows that take part
    float scale, unscale; // G is kept times `scale`
    uint32_t far;         // whether some row's lse_in is far from zero
    uint32_t pad[60];
};

inline uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// What a workspace holds.  Every part grows with rows, IDs and columns.
//   Where gradients follow in the same call, exponentials of the first IDs are kept, up to KEEP_BYTES; G of the others is
//   formed again from the products, for a piece of the vocabulary of up to PIECE_BYTES (which the last-level cache
//   holds), of at least LEAST_IDS IDs.  A table whose rows are not whole steps of aligned 16-byte pieces is copied,
//   PIECE_BYTES at a time.
constexpr uint64_t KEEP_BYTES = 1ull << 30, PIECE_BYTES = 128ull << 20;
constexpr uint32_t LEAST_IDS = 4096;
constexpr uint32_t MOST_SHARES = 32;
constexpr uint64_t SHARE_FLOATS = 1ull << 25;
constexpr uint32_t MANY_TILES = 192;   // of 256 x 256, or of 128 x 128: enough for the CUs

struct Sizes {
    uint32_t n_pad, dim_pad, v_pad, elem;
    uint64_t rows, hidden, weight, sums, kept, g, shares;   // bytes of the parts
    uint64_t total;
};

inline Sizes sizes_of(uint32_t n_rows, uint32_t n_vocab, uint32_t dim, int type, bool grads)
{
    Sizes z{};
    z.elem = elem_size(type);
    z.n_pad = (uint32_t)up(std::max(n_rows, 1u), PAD);
    z.dim_pad = (uint32_t)up(dim, STEP_BYTES / z.elem);
    z.v_pad = (uint32_t)up(n_vocab, PAD);
    z.rows = sizeof(Head) + 6ull * 4 * z.n_pad;
    z.hidden = (uint64_t)z.n_pad * z.dim_pad * z.elem;
    const uint64_t row = (uint64_t)z.dim_pad * z.elem;
    z.weight = std::min(z.v_pad * row, std::max(PIECE_BYTES, PAD * row));
    // per wavefront of 128 IDs; those of 64, 32 and 16 are for fewer than MANY_TILES tiles of 256 x 256
    // or no more than PAD rows
    z.sums = 8 * std::max({(uint64_t)z.v_pad / 128 * z.n_pad, std::min((uint64_t)z.v_pad / 16 * z.n_pad, (uint64_t)16 * 256 * MANY_TILES),
                           (uint64_t)z.v_pad / 32 * PAD});
    if (grads) {
        z.kept = std::min((uint64_t)z.n_pad * z.v_pad * z.elem, KEEP_BYTES);
        z.g = z.elem * std::min((uint64_t)z.n_pad * z.v_pad, std::max(PIECE_BYTES / z.elem, (uint64_t)z.n_pad * LEAST_IDS));
        const uint64_t one = (uint64_t)z.n_pad * z.dim_pad;
        z.shares = 4 * (one + std::min((MOST_SHARES - 1) * one, SHARE_FLOATS));
    }
    for (uint64_t *p : {&z.rows, &z.hidden, &z.weight, &z.sums, &z.kept, &z.g, &z.shares}) z.total += *p = up(*p, 256);
    return z;
}

// A call's arguments, checked.
struct Call {
    const void *hidden, *weight;
    int type;
    uint32_t n_rows, n_vocab, dim;
    uint64_t hidden_stride, weight_stride;
    const uint32_t *targets;
    float *loss, *lse;
    const float *lse_in, *grad_loss;
    float grad_scale;
    void *grad_hidden;
    uint64_t grad_hidden_stride;
    void *grad_weight;
    int grad_weight_type;
    uint64_t grad_weight_stride;
    int accumulate;
};

// The launches (linear_loss_*.hip, one for every type, which take a while to compile).
template <class T> void linear_loss(const Call &c, const Sizes &z, uint8_t *ws, hipStream_t s);

namespace {

constexpr uint32_t NONE = 0xFFFFFFFFu;

struct Rows {             // of the packed rows
    Head *head;
    uint32_t *list;       // row of the caller's matrices, NONE for padding
    uint32_t *target;
    float *factor;        // c
    float *shift, *recip; // G = c (exp(x - shift) recip - [v == y])
    float *at_target;     // x_y
};

// ---------------------------------------------------------------------------------------------
// rows

// A row of n elements to one of n_pad, zeros behind it (or throughout), by the lanes of a wavefront, four vectors on their way.
template <class T> __device__ __forceinline__ void copy_row(T *__restrict__ to, const T *__restrict__ from, uint32_t n, uint32_t n_pad)
{
    uint32_t j = (threadIdx.x & 63) * VEC;
    for (; from && j + 3 * 64 * VEC + VEC <= n; j += 4 * 64 * VEC) {
        Vec<T> v[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) v[i] = load_vec(from + j + i * 64 * VEC);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) store_vec(to + j + i * 64 * VEC, v[i]);
    }
    for (; j < n_pad; j += 64 * VEC) {
        float x[VEC] = {};
        if (from && j < n) load_part(from + j, n - j, 0.f, x);
        store_vec(to + j, x);
    }
}

__device__ __forceinline__ float factor_of(const float *grad_loss, float grad_scale, uint32_t r)
{
    return grad_scale * (grad_loss ? grad_loss[r] : 1.f);
}

// Numbers the rows that take part, in order, copies their hidden states together, and clears what the others
// get.  Every workgroup counts through all targets, which saves a launch.
//
// float16's range does not hold c times a small probability: G is kept times the power of two that brings the largest |c| to
// 2^14..2^15, so that probabilities down to 2^-28 (2^-39 with fewer digits) keep their digits.
template <class T>
__global__ __launch_bounds__(256) void k_gather(const T *__restrict__ hidden, uint64_t stride, uint32_t dim, uint32_t dim_pad,
                                                const uint32_t *__restrict__ targets, uint32_t n_rows, uint32_t per, uint32_t n_vocab,
                                                const float *__restrict__ lse_in, const float *__restrict__ grad_loss, float grad_scale,
                                                float *loss, float *lse_out, Rows rows, T *__restrict__ packed, T *__restrict__ grad,
                                                uint64_t grad_stride)
{
    constexpr bool SCALED = __is_same(T, _Float16);
    __shared__ uint32_t part[4], befores[4], larges[4], fars[4], place[256];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, first = blockIdx.x * per, last = first + per < n_rows ? first + per : n_rows;
    uint32_t total = 0, before = 0, large = 0;
    bool far = false;
#pragma unroll 8
    for (uint32_t r = threadIdx.x; r < n_rows; r += 256) {
        const bool in = targets[r] < n_vocab;
        total += in;
        before += in && r < first;
        if constexpr (SCALED) {
            if (in) {
                const uint32_t size = __builtin_bit_cast(uint32_t, factor_of(grad_loss, grad_scale, r)) & 0x7FFFFFFFu;
                if (size < 0x7F800000u && size > large) large = size;
            }
        }
    }
    if (lse_in && blockIdx.x == 0) {   // (in the loop above it would cost the calls without it 5 us)
#pragma unroll 8
        for (uint32_t r = threadIdx.x; r < n_rows; r += 256) far |= targets[r] < n_vocab && lse_in[r] != NEG_INF && is_far(lse_in[r]);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        total += __shfl_xor(total, d);
        before += __shfl_xor(before, d);
        const uint32_t o = __shfl_xor(large, d);
        large = o > large ? o : large;
    }
    far = __any(far);
    if (lane == 0) {
        part[wave] = total;
        befores[wave] = before;
        larges[wave] = large;
        fars[wave] = far;
    }
    __syncthreads();
    total = part[0] + part[1] + part[2] + part[3];
    uint32_t at = befores[0] + befores[1] + befores[2] + befores[3];
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (int w = 0; w < 4; ++w) large = larges[w] > large ? larges[w] : large;
        const int e = (int)(large >> 23) - 127;   // the largest |c| is 2^e .. 2^(e + 1); subnormal ones count as 2^-127
        const float scale = large ? __builtin_amdgcn_ldexpf(1.f, 14 - e > 126 ? 126 : 14 - e) : 1.f;
        rows.head->count = total;
        rows.head->far = fars[0] | fars[1] | fars[2] | fars[3];
        rows.head->scale = scale;
        rows.head->unscale = 1.f / scale;
    }
    for (uint32_t r0 = first; r0 < last; r0 += 256) {
        const uint32_t r = r0 + threadIdx.x, y = r < last ? targets[r] : NONE;
        const bool in = r < last && y < n_vocab;
        const uint64_t mask = __ballot(in);
        __syncthreads();
        if (lane == 0) part[wave] = __popcll(mask);
        __syncthreads();
        uint32_t mine = at + __popcll(mask & ((1ull << lane) - 1));
        for (uint32_t w = 0; w < 4; ++w) {
            mine += w < wave ? part[w] : 0;
            at += part[w];
        }
        if (in) {
            float c = factor_of(grad_loss, grad_scale, r), shift = 0.f;
            if (lse_in) {
                shift = lse_in[r];
                if (shift == NEG_INF) c = shift = 0.f;   // nothing but -inf: no gradient
            }
            rows.list[mine] = r;
            rows.target[mine] = y;
            rows.factor[mine] = c;
            rows.shift[mine] = shift;
            rows.recip[mine] = 1.f;
        } else if (r < last && loss) {
            loss[r] = 0.f;
            lse_out[r] = 0.f;
        }
        place[threadIdx.x] = in ? mine : NONE;
        __syncthreads();
        for (uint32_t k = wave; k < 256 && r0 + k < last; k += 4) {
            const uint32_t to = place[k];
            if (to != NONE) {
                copy_row(packed + (uint64_t)to * dim_pad, hidden + (uint64_t)(r0 + k) * stride, dim, dim_pad);
            } else if (grad) {
                const float zero[VEC] = {};
                for (uint32_t j = lane * VEC; j < dim; j += 64 * VEC) store_part(grad + (uint64_t)(r0 + k) * grad_stride + j, dim - j, zero);
            }
        }
    }
    // up to the end of the last tile; what the product for dW reads in its last step as zeros
    const uint32_t end = (total + PAD - 1) / PAD * PAD, zeros = (total + STEP_K<T> - 1) / STEP_K<T> * STEP_K<T>;
    for (uint32_t i = total + blockIdx.x * 4 + wave; i < end; i += gridDim.x * 4) {
        if (i < zeros) copy_row(packed + (uint64_t)i * dim_pad, (const T *)nullptr, dim, dim_pad);
        if (lane == 0) {
            rows.list[i] = rows.target[i] = NONE;
            rows.factor[i] = rows.shift[i] = rows.recip[i] = 0.f;
        }
    }
}

// for_far: where it is not NULL, only if there are far rows
template <class T>
__global__ __launch_bounds__(256) void k_pack_weight(const T *__restrict__ weight, uint64_t stride, uint32_t ids, uint32_t dim, uint32_t dim_pad,
                                                     T *__restrict__ packed, const Head *__restrict__ for_far)
{
    if (for_far && !for_far->far) return;
    const uint64_t v = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (v < ids) copy_row(packed + v * dim_pad, weight + v * stride, dim, dim_pad);
}

// ---------------------------------------------------------------------------------------------
// logits

// What becomes of a tile of logits, vocabulary along m, rows along n.
enum Use {
    SUMS,    // each row's maximum and sum of exponentials over a wavefront's IDs (far_only: in tiles with far rows)
    KEPT,    // those, and the exponentials themselves, which k_scale turns into G
    G_AGAIN  // G
};
// How exponentials wait for their row's sum: beside a 16-bit type in 16 bits of their own, since they are rounded there and once
// more as G.  They lie in 0 .. 1, so that no bit goes to a sign and few to the exponent: of the 32-bit number the 16 bits from bit
// SHIFT on, beside bfloat16 seven of exponent and nine of fraction (any number down to 2^-126, off by 2^-10 where G is rounded by
// 2^-8), beside float16, times 2^-96, five and eleven (2^-12 where G is rounded by 2^-11; subnormal below 2^-30).  As numbers of the
// type they added a whole rounding to G: it was off by up to 2^-7 and 2^-10.  NaN comes out as a number, but its row's sum is NaN.
template <class T> constexpr int KEPT_SHIFT = __is_same(T, _Float16) ? 12 : 14;
template <class T> constexpr float KEPT_SCALE = __is_same(T, _Float16) ? 0x1p-96f : 1.f;

template <class T> __device__ __forceinline__ uint32_t keep_high(float e)   // in the upper half
{
    return (__builtin_bit_cast(uint32_t, e * KEPT_SCALE<T>) << (16 - KEPT_SHIFT<T>)) + 0x8000u;
}
// four neighbours
template <class T> __device__ __forceinline__ void keep4(T *to, const float (&e)[4])
{
    if constexpr (sizeof(T) == 4) {
        *(f32x4 *)to = f32x4{e[0], e[1], e[2], e[3]};
    } else {
        u32x2 v;
#pragma unroll
        for (int k = 0; k < 2; ++k) v[k] = keep_high<T>(e[2 * k]) >> 16 | (keep_high<T>(e[2 * k + 1]) & 0xFFFF0000u);
        *(u32x2 *)to = v;
    }
}
// element k of a vector of them, times KEPT_SCALE
template <class T> __device__ __forceinline__ float kept_at(const Vec<T> &v, int k)
{
    if constexpr (sizeof(T) == 4) return vec_at(v, k);
    const uint32_t w = v.a[k >> 1];
    return __builtin_bit_cast(float, ((k & 1) ? w >> 16 : w & 0xFFFFu) << KEPT_SHIFT<T>);
}

// Four neighbouring elements.
template <class T> __device__ __forceinline__ void store4(T *to, const float (&x)[4])
{
    if constexpr (sizeof(T) == 4) {
        *(f32x4 *)to = f32x4{x[0], x[1], x[2], x[3]};
    } else {
        u32x2 v;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * k]) | (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * k + 1]) << 16;
        *(u32x2 *)to = v;
    }
}

// first_id: the ID that the operand w and the columns of g begin with.
struct Logits {
    Operand w, h;
    uint32_t steps, first_id, n_vocab, n_pad;
    Rows rows;
    MaxSum *sums;
    bool far_only;
};

// Whether one of the tile's rows is far from zero; every wavefront looks at all of them.  (A reduction over the workgroup takes LDS,
// of which four of the smallest tiles for few rows leave none.)
template <class TILE> __device__ __forceinline__ bool far_in(const Rows &rows, uint32_t n0, uint32_t count)
{
    bool far = false;
    for (uint32_t r = threadIdx.x & 63; r < TILE::N; r += 64) far |= n0 + r < count && is_far(rows.shift[n0 + r]);
    return __any(far);
}

// Takes m off column j of the logits, before the product with log2(e): at the maximum the power is 1 itself, so that no loss is
// negative and a certain target's G is zero.  (In one instruction, x log2(e) - m log2(e), a power is off by the rounding of the second
// product: by 5e-6 at logits of 127, by any factor where they are large.)
template <class TILE> __device__ __forceinline__ void take_off(f32x4 (&acc)[TILE::TM][TILE::TN], int j, float m)
{
#pragma unroll
    for (int i = 0; i < TILE::TM; ++i) acc[i][j] -= m;
}

template <class T, class TILE, Use USE>
__device__ __forceinline__ void logits_tile(const Logits &a, uint32_t m0, uint32_t n0, uint32_t count, lds_u8 *lds, T *g, uint32_t g_cols)
{
    const uint32_t first_id = a.first_id, n_vocab = a.n_vocab, n_pad = a.n_pad;
    const Rows &rows = a.rows;
    MaxSum *sums = a.sums;
    f32x4 acc[TILE::TM][TILE::TN];
    product<T, TILE, false, false>(acc, lds, a.w, a.h, m0, n0, 0, a.steps, 0);

    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / TILE::WN, wn = wave % TILE::WN;
    const uint32_t m_wave = m0 + wm * TILE::TM * 16, m_lane = m_wave + (lane >> 4) * 4;   // the first in this wavefront, this lane
    const bool edge = first_id + m0 + TILE::M > n_vocab;
#pragma unroll
    for (int j = 0; j < TILE::TN; ++j) {
        const uint32_t n = n0 + (wn * TILE::TN + j) * 16 + (lane & 15);   // the packed rows reach that far
        const uint32_t y = rows.target[n] - (first_id + m_lane);          // target, from this lane's first ID
        if constexpr (USE != G_AGAIN) {
            float m = NEG_INF, at = 0.f;
            if (edge) {
#pragma unroll
                for (int i = 0; i < TILE::TM; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (first_id + m_lane + i * 16 + e >= n_vocab) acc[i][j][e] = NEG_INF;
            }
#pragma unroll
            for (int i = 0; i < TILE::TM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m = fmaxf(m, acc[i][j][e]);
                    at = y == (uint32_t)(i * 16 + e) ? acc[i][j][e] : at;
                }
            if (y < TILE::TM * 16 && (y & 15) < 4) rows.at_target[n] = at;
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (m != NEG_INF) take_off<TILE>(acc, j, m);   // nothing but -inf, or NaN, stays so
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < TILE::TM; ++i) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = exp_f(acc[i][j][e]);
                    s += x[e];
                }
                if constexpr (USE == KEPT) keep4(g + (uint64_t)n * g_cols + m_lane + i * 16, x);
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (lane < 16) sums[(uint64_t)((first_id + m_wave) / (TILE::TM * 16)) * n_pad + n] = MaxSum{m, s};
        } else {
            // padding, rows and IDs, is zeros whatever the products are: the other two products run over it
            const bool row = n < count;
            const float c = rows.factor[n] * rows.head->scale, r = rows.recip[n];
            take_off<TILE>(acc, j, rows.shift[n]);
            T *to = g + (uint64_t)n * g_cols + m_lane;
#pragma unroll
            for (int i = 0; i < TILE::TM; ++i) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp_f(acc[i][j][e]) * r;
                    x[e] = c * (p - (y == (uint32_t)(i * 16 + e) ? 1.f : 0.f));
                    x[e] = row ? x[e] : 0.f;
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = first_id + m_lane + i * 16 + e < n_vocab ? x[e] : 0.f;
                }
                store4(to + i * 16, x);
            }
        }
    }
}

template <class T, class TILE, Use USE>
__global__ __launch_bounds__(TILE::THREADS, 2) void k_logits(Logits a, uint32_t m_tiles, T *__restrict__ g, uint32_t g_cols)
{
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::LDS];
    if (USE == SUMS && a.far_only && !a.rows.head->far) return;
    // (of G every row up to a whole step of k is written: the product for dW reads it so)
    const uint32_t count = a.rows.head->count, reach = USE == G_AGAIN ? (count + STEP_K<T> - 1) / STEP_K<T> * STEP_K<T> : count;
    with_place<TILE>(m_tiles, a.w.count * a.w.stride, reach, [&](auto tile, uint32_t m0, uint32_t n0) {
        if (USE == SUMS && a.far_only && !far_in<decltype(tile)>(a.rows, n0, count)) return;
        logits_tile<T, decltype(tile), USE>(a, m0, n0, count, (lds_u8 *)shared, g, g_cols);
    });
}

// Eight kept exponentials of row n into G, in place: times c exp(m - shift) recip, m the maximum that each `span` of them was
// formed from; the target's element from its own logit, since p - 1 would show the rounding of p.  Rows and columns behind
// the last become zeros.  (A product for them again would cost 2 dim operations an element where this moves four bytes.)
struct Scaling {
    uint32_t n, count, span, n_pad, n_vocab, target;
    float c, shift, recip, at_target;
    const MaxSum *sums;
    template <class T> __device__ __forceinline__ void apply(T *g, uint32_t j) const
    {
        float x[VEC] = {};
        if (n < count) {
            const float f = c * exp_f(sums[(uint64_t)(j / span) * n_pad + n].m - shift) * recip * (1.f / KEPT_SCALE<T>);
            const Vec<T> v = load_vec(g + j);
            const uint32_t y = target - j;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = j + e < n_vocab ? kept_at(v, e) * f : 0.f;
            if (y < VEC) {
                const float own = c * (exp_f(at_target - shift) * recip - 1.f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = y == (uint32_t)e ? own : x[e];
            }
        }
        store_vec(g + j, x);
    }
};

// A row's loss and log-sum-exp from its maximum and sum (loss NULL: both are there), and what G is formed with.
__device__ __forceinline__ void put_row(MaxSum v, uint32_t n, const Rows &rows, float *loss, float *lse)
{
    const bool none = empty(v);
    if (loss) {
        const float log_s = log_of(v.s);
        const uint32_t r = rows.list[n];
        lse[r] = none ? NEG_INF : v.m + log_s;
        loss[r] = none ? -NEG_INF : (v.m - rows.at_target[n]) + log_s;
    }
    rows.shift[n] = none ? 0.f : v.m;
    rows.recip[n] = none ? 0.f : 1.f / v.s;
    if (none) rows.factor[n] = 0.f;
}

// Joins the maxima and sums over the vocabulary (`parts` of them): 16 rows a workgroup, 64 threads a row.  loss NULL: of the far
// rows.
__global__ __launch_bounds__(1024) void k_join(const MaxSum *__restrict__ sums, uint32_t parts, uint32_t n_pad, Rows rows,
                                               float *__restrict__ loss, float *__restrict__ lse)
{
    __shared__ MaxSum part[16][16];
    const uint32_t l = threadIdx.x & 15, n = blockIdx.x * 16 + l;
    if (blockIdx.x * 16 >= rows.head->count || (!loss && !rows.head->far)) return;
    MaxSum v{NEG_INF, 0.f};
    for (uint32_t t = threadIdx.x >> 4; t < parts; t += 64) v = join(v, sums[(uint64_t)t * n_pad + n]);
    v = join(v, MaxSum{__shfl_xor(v.m, 16), __shfl_xor(v.s, 16)});
    v = join(v, MaxSum{__shfl_xor(v.m, 32), __shfl_xor(v.s, 32)});
    if ((threadIdx.x & 63) < 16) part[threadIdx.x >> 6][l] = v;
    __syncthreads();
    if (threadIdx.x >= 16 || n >= rows.head->count || (!loss && !is_far(rows.shift[n]))) return;
    for (uint32_t i = 1; i < 16; ++i) v = join(v, part[i][l]);
    put_row(v, n, rows, loss, lse);
}

template <class T>
__global__ __launch_bounds__(256) void k_scale(T *__restrict__ g, uint32_t g_cols, uint32_t cols, uint32_t span, const MaxSum *__restrict__ sums,
                                               uint32_t n_pad, uint32_t n_vocab, Rows rows, uint32_t first_row)
{
    const uint32_t n = first_row + blockIdx.y, count = rows.head->count;
    if (n >= (count + PAD - 1) / PAD * PAD) return;
    const uint32_t j = (blockIdx.x * 256 + threadIdx.x) * VEC;
    if (j >= cols) return;
    const Scaling scaling{n, count, span, n_pad, n_vocab, rows.target[n], rows.factor[n] * rows.head->scale, rows.shift[n], rows.recip[n], rows.at_target[n], sums};
    scaling.apply(g + (uint64_t)n * g_cols, j);
}

// Both for up to PAD rows, a workgroup a row.
template <class T>
__global__ __launch_bounds__(1024) void k_join_scale(const MaxSum *__restrict__ sums, uint32_t parts, uint32_t n_pad, uint32_t n_vocab, Rows rows, float *__restrict__ loss,
                                                     float *__restrict__ lse, T *__restrict__ g, uint32_t g_cols, uint32_t cols, uint32_t span)
{
    __shared__ MaxSum part[16];
    const uint32_t n = blockIdx.x, count = rows.head->count;
    MaxSum v{NEG_INF, 0.f};
    if (n < count) {
        for (uint32_t t = threadIdx.x; t < parts; t += 1024) v = join(v, sums[(uint64_t)t * n_pad + n]);
        v = block_join<1024>(v, part);
        if (threadIdx.x == 0) put_row(v, n, rows, loss, lse);
    }
    const bool none = empty(v);
    const Scaling scaling{n, count, span, n_pad, n_vocab, rows.target[n], none ? 0.f : rows.factor[n] * rows.head->scale, none ? 0.f : v.m,
                          none ? 0.f : 1.f / v.s, rows.at_target[n], sums};
    for (uint32_t j = threadIdx.x * VEC; j < cols; j += 1024 * VEC) scaling.apply(g + (uint64_t)n * g_cols, j);
}

// ---------------------------------------------------------------------------------------------
// gradients

// The products for dh run over all IDs, which are split where the tiles are fewer than the workgroups that run at a time.
// How many rows take part only the device knows, so that the kernels work out the split.
struct Split {
    uint32_t m_tiles, n_rows_tile, blocks, most;   // tiles along m, rows of a tile, workgroups, shares at most
    uint32_t single;                               // one piece of the vocabulary is all
    __device__ __forceinline__ uint32_t n_tiles(uint32_t count) const { return (count + n_rows_tile - 1) / n_rows_tile; }
    __device__ __forceinline__ uint32_t shares(uint32_t count) const
    {
        const uint32_t tiles = m_tiles * n_tiles(count), s = tiles ? blocks / tiles : 1;
        return s < 1 ? 1 : s < most ? s : most;
    }
};

// dh: columns along m, rows along n, k over a share of the piece's IDs.  The sums go to `sums` ([share][n_pad][dim_pad], added
// to where the piece is not the first), or rounded to the caller's rows if one share of one piece is all.
template <class T, class TILE>
__global__ __launch_bounds__(TILE::THREADS, 2) void k_grad_hidden(Operand w, Operand g, uint32_t steps, uint32_t ids, Split split,
                                                                  uint32_t dim, uint32_t dim_pad, uint32_t n_pad, int add, Rows rows,
                                                                  float *__restrict__ sums, T *__restrict__ out, uint64_t stride)
{
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::LDS];
    const uint32_t count = rows.head->count, n_tiles = split.n_tiles(count), shares = split.shares(count);
    const uint32_t one = split.m_tiles * n_tiles, at = tile_of(blockIdx.x, one * shares);
    if (at == NONE) return;   // also where no row takes part, so that `one` is 0
    const uint32_t mine = at / one;
    uint32_t tm, tn;
    place_of(at % one, split.m_tiles, n_tiles, tm, tn);
    const uint32_t m0 = tm * TILE::M, n0 = tn * TILE::N, share = (steps + shares - 1) / shares;
    const uint32_t begin = mine * share < steps ? mine * share : steps, end = begin + share < steps ? begin + share : steps;
    if (!split.single || shares > 1) out = nullptr;
    f32x4 acc[TILE::TM][TILE::TN];
    product<T, TILE, true, false>(acc, (lds_u8 *)shared, w, g, m0, n0, begin, end, ids);
    const float unscale = rows.head->unscale;
    sums += (uint64_t)mine * n_pad * dim_pad;
    by_rows<TILE>(acc, (lds_u8 *)shared, [&](uint32_t n, uint32_t m, float (&x)[VEC]) {
        n += n0;
        m += m0;
        if (n >= count || m >= dim) return;
        if (out) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] *= unscale;
            return store_part(out + rows.list[n] * stride + m, dim - m, x);
        }
        float *to = sums + (uint64_t)n * dim_pad + m;   // whole vectors: dim_pad is a multiple of them
        if (add) {
            const Vec<float> v = load_vec(to);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] += vec_at(v, e);
        }
        store_vec(to, x);
    });
}

// The shares of dh summed, in order, and rounded.
template <class T>
__global__ __launch_bounds__(256) void k_finish_hidden(const float *__restrict__ sums, Split split, uint32_t n_pad, uint32_t dim,
                                                       uint32_t dim_pad, Rows rows, T *__restrict__ out, uint64_t stride)
{
    const uint32_t i = blockIdx.x, count = rows.head->count, shares = split.shares(count);
    if (i >= count || (split.single && shares == 1)) return;
    const uint32_t r = rows.list[i];
    const float unscale = rows.head->unscale;
    for (uint32_t j = threadIdx.x * VEC; j < dim; j += 256 * VEC) {
        float x[VEC] = {};
        for (uint32_t k = 0; k < shares; ++k) {
            const Vec<float> v = load_vec(sums + ((uint64_t)k * n_pad + i) * dim_pad + j);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] += vec_at(v, e);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] *= unscale;
        store_part(out + r * stride + j, dim - j, x);
    }
}

// dW of a piece: columns along m, IDs along n, k over the rows that take part.
struct Weights {
    Operand h, g;
    uint32_t ids, dim;
    int accumulate;
    Rows rows;
    uint64_t stride;
};

template <class T, class TILE, class OUT> __device__ __forceinline__ void weight_tile(const Weights &a, uint32_t m0, uint32_t n0, lds_u8 *lds, OUT *out)
{
    f32x4 acc[TILE::TM][TILE::TN];
    product<T, TILE, true, true>(acc, lds, a.h, a.g, m0, n0, 0, (a.rows.head->count + STEP_K<T> - 1) / STEP_K<T>, 0);
    const float unscale = a.rows.head->unscale;
    by_rows<TILE>(acc, lds, [&](uint32_t n, uint32_t m, float (&x)[VEC]) {
        n += n0;
        m += m0;
        if (n >= a.ids || m >= a.dim) return;
        OUT *to = out + n * a.stride + m;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] *= unscale;
        if (a.accumulate) {
            float was[VEC];
            load_part(to, a.dim - m, 0.f, was);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] += was[e];
        }
        // past the caches for 16 bits (into 131,328 x 4,096 bfloat16, 16 rows: 420 -> 335 us; a whole call of 128 rows 1,017 -> 916, 512 1,736 ->
        // 1,646, 2,048 5,402 -> 5,352, 8,192 as before, into 33,024 x 2,048 1,638 rows 670 -> 661; where it is added to, as before;
        // float32 loses, 128 rows into 33,024 x 1,024: 92 -> 115 us)
        if constexpr (sizeof(OUT) == 2) stream_part(to, a.dim - m, x);
        else store_part(to, a.dim - m, x);
    });
}

template <class T, class TILE, class OUT>
__global__ __launch_bounds__(TILE::THREADS, 2) void k_grad_weight(Weights a, uint32_t m_tiles, OUT *__restrict__ out)
{
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::LDS];
    with_place<TILE>(m_tiles, (uint64_t)a.rows.head->count * a.h.stride, a.ids,
                     [&](auto tile, uint32_t m0, uint32_t n0) { weight_tile<T, decltype(tile), OUT>(a, m0, n0, (lds_u8 *)shared, out); });
}

// ---------------------------------------------------------------------------------------------
// host side

// Big, 256 x 256: one workgroup a CU
typedef Tile<2, 2, 4, 4> Middle;   // 128 x 128: two
typedef Tile<2, 2, 2, 2> Small;    // 64 x 64: four

typedef Tile<2, 2, 1, 1> Tiny;     // 32 x 32

uint32_t tiles(uint64_t n, uint32_t of) { return (uint32_t)((n + of - 1) / of); }

// The largest tiles of which there are enough for the CUs.
template <class F> void with_tile(uint64_t m, uint64_t n, F f)
{
    if ((uint64_t)tiles(m, 256) * tiles(n, 256) >= MANY_TILES) f(Big{});
    else if ((uint64_t)tiles(m, 128) * tiles(n, 128) >= MANY_TILES) f(Middle{});
    else if ((uint64_t)tiles(m, 64) * tiles(n, 64) >= MANY_TILES) f(Small{});
    else f(Tiny{});
}

typedef Tile<4, 1, 2, 2> Thin;     // 128 x 32: four
typedef Tile<4, 1, 2, 4> Thicker;  // 128 x 64: three

// For the logits; of few rows, where the table's way through the CUs is what counts: tiles that are no wider, of which
// several run on a CU.
template <class F> void with_logits_tile(uint64_t m, uint64_t n, F f)
{
    if (n <= 32) f(Thin{});
    else if (n <= 64) f(Thicker{});
    else if (n <= 128) f(Middle{});
    else with_tile(m, n, f);
}

// For dh, whose k is split: the largest tiles whose shares fill most of the CUs.
template <class F> void with_split(uint32_t dim, uint32_t n_rows, uint32_t k_steps, uint64_t most, bool single, F f)
{
    auto of = [&](uint32_t size, uint32_t blocks) {
        Split s{tiles(dim, size), size, blocks, (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(k_steps / 8, most)), single};
        const uint64_t all = (uint64_t)s.m_tiles * tiles(n_rows, size), shares = std::clamp<uint64_t>(blocks / all, 1, s.most);
        return std::pair<Split, bool>(s, all * shares * 8 >= blocks * 5);
    };
    const auto big = of(256, 256), middle = of(128, 512), small = of(64, 1024), tiny = of(32, 1024);
    if (big.second) f(Big{}, big.first);
    else if (middle.second) f(Middle{}, middle.first);
    else if (small.second) f(Small{}, small.first);
    else f(Tiny{}, tiny.first);
}

// The IDs, in whole pads, whose tiles make up to 2^31 threads: a launch of 2^32 or more runs a part of them and reports success.
// Other launches are far smaller, as G and the columns are.
template <class TILE> uint32_t most_ids(uint32_t n_rows)
{
    const uint64_t ids = (1ull << 31) / TILE::THREADS / tiles(n_rows, TILE::N) * TILE::M;
    return (uint32_t)std::min<uint64_t>(1u << 30, ids / PAD * PAD);
}

template <class T> void enqueue(const Call &c, const Sizes &z, uint8_t *ws, hipStream_t s)
{
    Rows rows;
    rows.head = (Head *)ws;
    rows.list = (uint32_t *)(ws + sizeof(Head));
    rows.target = rows.list + z.n_pad;
    rows.factor = (float *)(rows.target + z.n_pad);
    rows.shift = rows.factor + z.n_pad;
    rows.recip = rows.shift + z.n_pad;
    rows.at_target = rows.recip + z.n_pad;
    T *hidden = (T *)(ws + z.rows), *packed = (T *)(ws + z.rows + z.hidden);
    MaxSum *sums = (MaxSum *)(ws + z.rows + z.hidden + z.weight);
    T *kept = (T *)((uint8_t *)sums + z.sums), *g = (T *)((uint8_t *)kept + z.kept);
    float *shares = (float *)((uint8_t *)g + z.g);
    const T *weight = (const T *)c.weight;
    const bool grads = c.grad_hidden || c.grad_weight, forward = c.loss != nullptr;

    const uint32_t per = std::max(4u, tiles(c.n_rows, 512));
    k_gather<T><<<std::max(32u, tiles(c.n_rows, per)), 256, 0, s>>>((const T *)c.hidden, c.hidden_stride, c.dim, z.dim_pad, c.targets, c.n_rows, per,
                                                                   c.n_vocab, c.lse_in, c.grad_loss, c.grad_scale, c.loss, c.lse, rows, hidden,
                                                                   (T *)c.grad_hidden, c.grad_hidden_stride);

    // The table as it lies: whole steps, aligned, a tile within 32-bit offsets.  Otherwise pieces of it are copied.
    const uint64_t w_bytes = c.weight_stride * z.elem;
    const bool as_is = c.dim == z.dim_pad && (uintptr_t)c.weight % 16 == 0 && w_bytes % 16 == 0 && w_bytes <= (1u << 22);
    const uint64_t row = (uint64_t)z.dim_pad * z.elem;
    const uint32_t most_packed = (uint32_t)std::min<uint64_t>(z.v_pad, z.weight / row / PAD * PAD);
    const uint32_t steps = z.dim_pad / STEP_K<T>;
    const Operand h{hidden, row, z.n_pad};
    bool copied = false;   // all of it, where that fits
    auto table = [&](uint32_t first, uint32_t ids, const Head *for_far = nullptr) {
        const T *from = weight + first * c.weight_stride;
        if (as_is) return Operand{from, w_bytes, ids};
        if (c.n_vocab > most_packed) {
            k_pack_weight<T><<<tiles(ids, 4), 256, 0, s>>>(from, c.weight_stride, ids, c.dim, z.dim_pad, packed, for_far);
            return Operand{packed, row, ids};
        }
        if (!copied) k_pack_weight<T><<<tiles(c.n_vocab, 4), 256, 0, s>>>(weight, c.weight_stride, c.n_vocab, c.dim, z.dim_pad, packed, nullptr);
        copied = true;
        return Operand{packed + (uint64_t)first * z.dim_pad, row, ids};
    };

    // What is kept: the exponentials of the first `keep` IDs (of a table that is copied in pieces, one piece's or none).
    uint32_t keep = 0;
    if (forward && grads) keep = (uint32_t)std::min<uint64_t>(z.v_pad, z.kept / z.elem / z.n_pad / PAD * PAD);
    if (!as_is && c.n_vocab > most_packed) keep = keep < most_packed ? 0 : most_packed;
    uint32_t span = 0;

    // Maxima and sums.  For gradients from lse of those rows whose lse is far from zero, which the device knows: launches that find
    // none take some 3 to 8 us (1,350 rows x 33,001 x 1,001 float16: 348 -> 355 us; with one far row 389, with all far 455).
    if ((forward || grads) && c.n_rows) {
        with_logits_tile(z.v_pad, c.n_rows, [&](auto t) {
            using TILE = decltype(t);
            span = TILE::TM * 16;
            for (uint32_t first = 0; first < c.n_vocab;) {
                uint32_t most = std::min((uint32_t)(as_is ? z.v_pad : most_packed), most_ids<TILE>(c.n_rows));
                if (first < keep) most = std::min(most, keep - first);
                const uint32_t ids = std::min(most, c.n_vocab - first), m_tiles = tiles(ids, TILE::M);
                const Operand w = table(first, ids, forward ? nullptr : rows.head);
                const uint32_t blocks = tile_blocks<TILE>(m_tiles, tiles(c.n_rows, TILE::N));
                const Logits a{w, h, steps, first, c.n_vocab, z.n_pad, rows, sums, !forward};
                if (first < keep) k_logits<T, TILE, KEPT><<<blocks, TILE::THREADS, 0, s>>>(a, m_tiles, kept + first, keep);
                else k_logits<T, TILE, SUMS><<<blocks, TILE::THREADS, 0, s>>>(a, m_tiles, nullptr, 0);
                first += most;
            }
        });
        const uint32_t parts = tiles(c.n_vocab, span), cols = (uint32_t)std::min<uint64_t>(keep, up(c.n_vocab, PAD));
        if (!forward) {
            k_join<<<z.n_pad / 16, 1024, 0, s>>>(sums, parts, z.n_pad, rows, nullptr, nullptr);
        } else if (c.n_rows <= PAD) {   // (of the loss alone: no columns)
            k_join_scale<T><<<grads ? PAD : c.n_rows, 1024, 0, s>>>(sums, parts, z.n_pad, c.n_vocab, rows, c.loss, c.lse, kept, keep, cols, span);
        } else {
            k_join<<<z.n_pad / 16, 1024, 0, s>>>(sums, parts, z.n_pad, rows, c.loss, c.lse);
            for (uint32_t first = 0; keep && first < z.n_pad; first += 32768)
                k_scale<T><<<dim3(tiles(cols, 256 * VEC), std::min(32768u, z.n_pad - first)), 256, 0, s>>>(kept, keep, cols, span, sums, z.n_pad, c.n_vocab, rows,
                                                                                                          first);
        }
    }
    if (!grads) return;

    // pieces of about the same size, whose G fits, after what is kept
    uint32_t piece = (uint32_t)std::min<uint64_t>(z.v_pad, z.g / z.elem / z.n_pad / PAD * PAD);
    if (!as_is) piece = std::min(piece, most_packed);
    const uint32_t rest = c.n_vocab > keep ? c.n_vocab - keep : 0, pieces = tiles(rest, piece);
    if (pieces) piece = (uint32_t)up(tiles(rest, pieces), PAD);
    const uint32_t all = pieces + (keep ? 1 : 0);
    Split finish{};
    uint32_t k_first = 0;
    for (uint32_t i = 0, first = 0; i < all; ++i) {
        const bool old = i == 0 && keep;
        const uint32_t width = old ? keep : piece, ids = std::min(width, c.n_vocab - first);
        const Operand w = c.n_rows ? table(first, ids) : Operand{};
        T *const go = old ? kept : g;
        if (!old && c.n_rows)
            with_logits_tile(ids, c.n_rows, [&](auto t) {
                using TILE = decltype(t);
                // every column of G up to the piece's width is written: the product for dh reads it in whole steps
                const uint32_t m_tiles = tiles(up(ids, PAD), TILE::M);
                k_logits<T, TILE, G_AGAIN><<<tile_blocks<TILE>(m_tiles, tiles(up(c.n_rows, STEP_K<T>), TILE::N)), TILE::THREADS, 0, s>>>(
                    Logits{w, h, steps, first, c.n_vocab, z.n_pad, rows, nullptr, false}, m_tiles, g, piece);
            });
        if (c.grad_hidden && c.n_rows) {
            const uint32_t k_steps = tiles(ids, STEP_K<T>);
            if (i == 0) k_first = k_steps;   // the pieces' sums meet in the same places: as many shares for all
            with_split(c.dim, c.n_rows, k_first, std::min<uint64_t>(MOST_SHARES, z.shares / 4 / ((uint64_t)z.n_pad * z.dim_pad)), all == 1,
                       [&](auto t, Split split) {
                using TILE = decltype(t);
                finish = split;
                const uint32_t blocks = std::max(tile_blocks<TILE>(split.m_tiles, tiles(c.n_rows, TILE::N)), split.blocks);
                k_grad_hidden<T, TILE><<<blocks, TILE::THREADS, 0, s>>>(
                    Operand{w.p, w.stride, z.dim_pad}, Operand{go, (uint64_t)width * z.elem, z.n_pad}, k_steps, ids, split, c.dim, z.dim_pad,
                    z.n_pad, i != 0, rows, shares, (T *)c.grad_hidden, c.grad_hidden_stride);
            });
        }
        if (c.grad_weight) {
            auto weights = [&](auto o) {
                using OUT = decltype(o);
                with_tile(c.dim, ids, [&](auto t) {
                    using TILE = decltype(t);
                    const uint32_t m_tiles = tiles(c.dim, TILE::M);
                    k_grad_weight<T, TILE, OUT><<<tile_blocks<TILE>(m_tiles, tiles(ids, TILE::N)), TILE::THREADS, 0, s>>>(
                        Weights{Operand{hidden, row, z.dim_pad}, Operand{go, (uint64_t)width * z.elem, width}, ids, c.dim, c.accumulate, rows,
                                c.grad_weight_stride},
                        m_tiles, (OUT *)c.grad_weight + first * c.grad_weight_stride);
                });
            };
            if (c.grad_weight_type == c.type) weights(T{});
            else weights(float{});
        }
        first += width;
    }
    if (c.grad_hidden && c.n_rows)
        k_finish_hidden<T><<<c.n_rows, 256, 0, s>>>(shares, finish, z.n_pad, c.dim, z.dim_pad, rows, (T *)c.grad_hidden, c.grad_hidden_stride);
}

}  // namespace
}  // namespace tt
