// distill.hip -- distillation from a teacher's top logits: loss and gradient over the vocabulary.
//
//   p = softmax(x / T);   q_k = exp(t_k / T - L),  L the listed log-sum-exp of t / T, or the teacher's own;   Q = sum_k q_k
//   loss = sum_k q_k (log q_k - log p_{id_k});   dx_j = (c / T) (Q p_j - sum of q_k over id_k = j)
//
// The row is read as for the cross entropy (rows.h), once where its vectors stay in registers; the gradient is written as
// if the list were empty, then the listed elements again, by the threads that hold the list's entries.  The row's loads and the
// list's go out together before the list is put into LDS, and both pairs of maximum and sum are joined behind one barrier.
//
// Bound by memory: 8,192 rows of 131,328 bfloat16, 64 listed, loss and gradient in one call: 833 us, 5.2 TB/s read and
// written (a large copy reaches 5.0); the loss alone 380 us.  1,500 rows of 33,001 float16, 100 listed: loss 33 us, gradient 39;
// with 1,000 listed 42 and 70, bound by the lists.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace tt {
namespace {

constexpr uint32_t NONE = 0xFFFFFFFFu;

struct Teacher {
    const uint32_t *ids;
    const float *top, *lse;   // lse: NULL where the listed ones are all there is
    uint64_t ids_stride, top_stride;
    uint32_t k;
};

// A row's list in LDS, and a hash table of its IDs that tells whether one is there twice.
struct List {
    uint32_t *id;      // NONE: no entry
    float *q, *x;      // q (the teacher's logit, to begin with); the row's own logit
    uint32_t *table, slots, *twice;

    __device__ __forceinline__ List(uint8_t *lds, uint32_t k, uint32_t n)
    {
        id = (uint32_t *)lds;
        q = (float *)(id + k);
        x = q + k;
        table = (uint32_t *)(x + k);
        slots = n;
        twice = table + n;
    }
};
inline uint32_t slots_of(uint32_t k)
{
    uint32_t n = 64;
    while (n < 2 * k) n *= 2;
    return n;
}
inline uint32_t list_bytes(uint32_t k) { return 12 * k + 4 * (slots_of(k) + 1); }

// This thread's entries of a row's list, on their way while something else is done.
template <int THREADS> struct Entries {
    static constexpr int EACH = (TOKTIER_MAX_TOP + THREADS - 1) / THREADS;
    uint32_t id[EACH];
    float top[EACH];
    __device__ __forceinline__ void load(const Teacher &t, uint64_t row)
    {
        const uint32_t *ids = t.ids + row * t.ids_stride;
        const float *tops = t.top + row * t.top_stride;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const uint32_t i = e * THREADS + threadIdx.x;
            id[e] = i < t.k ? ids[i] : NONE;
            top[e] = i < t.k ? tops[i] : NEG_INF;
        }
    }
};

template <int THREADS> __device__ __forceinline__ void clear_table(const List &list)
{
    for (uint32_t i = threadIdx.x; i < list.slots; i += THREADS) list.table[i] = NONE;
    if (threadIdx.x == 0) *list.twice = 0;
}

// Puts the list into LDS (its table has been cleared, and a barrier passed); this thread's part of maximum and sum over it.
// logit(entry, ID): the row's own.
template <int THREADS, class F>
__device__ __forceinline__ MaxSum read_list(const List &list, const Entries<THREADS> &own, uint32_t n, uint32_t n_vocab, float k, F logit)
{
    MaxSum b{NEG_INF, 0.f};
#pragma unroll
    for (int e = 0; e < Entries<THREADS>::EACH; ++e) {
        const uint32_t i = e * THREADS + threadIdx.x, id = own.id[e] < n_vocab ? own.id[e] : NONE;
        if (i >= n) continue;
        float v = NEG_INF, x = 0.f;
        if (id != NONE) {
            v = own.top[e];
            x = logit(i, id);
            uint32_t was = id + 1;
            for (uint32_t s = 0; s < list.slots && was != id && was != NONE; ++s)   // at most half of the slots are ever taken
                was = atomicCAS(&list.table[((id * 0x9E3779B1u >> 16) + s) & (list.slots - 1)], NONE, id);
            if (was == id) *list.twice = 1;
        }
        list.id[i] = id;
        list.q[i] = v;
        list.x[i] = x;
        if (v != v) b.s = v;
        else if (v > NEG_INF) b = join(b, MaxSum{v, 1.f}, k);
    }
    return b;
}

// Both joined over the workgroup, the wavefronts' by their first lanes.
template <int THREADS> __device__ __forceinline__ void block_join2(MaxSum &a, MaxSum &b, MaxSum (*lds)[THREADS / 64], float k)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        a = join(a, MaxSum{__shfl_xor(a.m, d), __shfl_xor(a.s, d)}, k);
        b = join(b, MaxSum{__shfl_xor(b.m, d), __shfl_xor(b.s, d)}, k);
    }
    if ((threadIdx.x & 63) == 0) {
        lds[0][threadIdx.x >> 6] = a;
        lds[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = lds[0][threadIdx.x & (THREADS / 64 - 1)];
    b = lds[1][threadIdx.x & (THREADS / 64 - 1)];
#pragma unroll
    for (int d = 1; d < THREADS / 64; d *= 2) {
        a = join(a, MaxSum{__shfl_xor(a.m, d), __shfl_xor(a.s, d)}, k);
        b = join(b, MaxSum{__shfl_xor(b.m, d), __shfl_xor(b.s, d)}, k);
    }
}

// This thread's entries of q; their sum, and with the row's maximum and sum their part of the loss.
template <int THREADS>
__device__ __forceinline__ void weigh_list(const List &list, const Teacher &t, uint64_t row, MaxSum b, MaxSum a, float inv_t, float &mass, float &loss)
{
    const float log_b = log_of(b.s), log_a = log_of(a.s);
    // a listed +inf is NaN with the teacher's own log-sum-exp too (asked where the list is read, it spills two registers)
    const float own = !t.lse ? 0.f : b.m == -NEG_INF ? __builtin_nanf("") : t.lse[row];
    const bool none = empty(a);
    mass = loss = 0.f;
    for (uint32_t i = threadIdx.x; i < t.k; i += THREADS) {
        const float v = list.q[i];
        const float log_q = t.lse ? v * inv_t - own : (v - b.m) * inv_t - log_b;
        const float q = v == NEG_INF ? 0.f : exp_f(log_q);
        list.q[i] = q;
        mass += q;
        if (q != 0.f) loss += none ? -NEG_INF : q * (log_q - ((list.x[i] - a.m) * inv_t - log_a));
    }
}

// Sums of the workgroup, in an order that its size fixes.
template <int THREADS> __device__ __forceinline__ float2 block_sum(float a, float b, float2 *lds)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
    }
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    float2 v = lds[threadIdx.x & (THREADS / 64 - 1)];
#pragma unroll
    for (int d = 1; d < THREADS / 64; d *= 2) {
        v.x += __shfl_xor(v.x, d);
        v.y += __shfl_xor(v.y, d);
    }
    return v;
}

// The gradient of a part of a row: c / T (mass exp((x - m) / T) r - q).
template <class T, int THREADS, int HELD, bool FIRST>
__device__ __forceinline__ void put_grad(RowPart<T, THREADS, HELD> &part, const List &list, uint32_t k, T *g, bool zero, float m, float r, float mass,
                                         float c, float k2)
{
    if (zero) {
        const float v[VEC] = {};
        for (uint32_t j = part.begin + threadIdx.x * VEC; j < part.end; j += THREADS * VEC) stream_part(g + j, part.end - j, v);
        return;
    }
    part.template each<FIRST>(0.f, [&](uint32_t j, uint32_t n, float (&v)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = c * (exp_f(v[e] - m, k2) * r * mass);
        stream_part(g + j, n, v);
    });
    __syncthreads();   // the listed elements come after the others
    const bool twice = *list.twice;
    for (uint32_t i = threadIdx.x; i < k; i += THREADS) {
        const uint32_t id = list.id[i];
        if (id < part.begin || id >= part.end) continue;
        float q = list.q[i];
        if (twice) {   // the first entry of an ID adds up all of them
            bool first = true;
            q = 0.f;
            for (uint32_t j = 0; j < k; ++j)
                if (list.id[j] == id) {
                    if (j < i) first = false;
                    q += list.q[j];
                }
            if (!first) continue;
        }
        g[id] = (T)(c * (exp_f(list.x[i] - m, k2) * r * mass - q));
    }
}

// Wavefronts of a SIMD: all eight have 64 registers each, in which 256 threads' parts of a list and of a row of 32 bits do not find room.
template <class T, int THREADS> constexpr int waves = sizeof(T) == 4 && THREADS == 256 ? 6 : 8;

template <class T, int THREADS, int HELD>
__global__ __launch_bounds__(THREADS, (waves<T, THREADS>)) void k_distill(const T *logits, uint32_t n_vocab, uint64_t stride, Teacher t, uint32_t slots, float inv_t,
                                                        float *__restrict__ loss, float *__restrict__ lse_out,
                                                        const float *__restrict__ grad_loss, float grad_scale, T *grad, uint64_t gstride)
{
    __shared__ MaxSum lds[2][THREADS / 64];
    __shared__ float2 lds_sum[THREADS / 64];
    extern __shared__ uint8_t dynamic[];
    const uint64_t row = blockIdx.x;
    const float k2 = LOG2E * inv_t;
    const List list(dynamic, t.k, slots);
    RowPart<T, THREADS, HELD> part{logits + row * stride, 0, n_vocab};
    Entries<THREADS> own_list;
    own_list.load(t, row);
    clear_table<THREADS>(list);
    __syncthreads();
    MaxSum a{NEG_INF, 0.f};
    part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v, k2); });
    MaxSum b = read_list<THREADS>(list, own_list, t.k, n_vocab, k2, [&](uint32_t, uint32_t id) { return (float)part.x[id]; });
    block_join2<THREADS>(a, b, lds, k2);
    float mass, own;
    weigh_list<THREADS>(list, t, row, b, a, inv_t, mass, own);
    const float2 sums = block_sum<THREADS>(mass, own, lds_sum);
    if (threadIdx.x == 0) {
        loss[row] = sums.y;
        lse_out[row] = empty(a) ? NEG_INF : a.m * inv_t + log_of(a.s);
    }
    if (grad)
        put_grad<T, THREADS, HELD, false>(part, list, t.k, grad + row * gstride, sums.x == 0.f || empty(a), a.m, 1.f / a.s, sums.x,
                                          grad_scale * (grad_loss ? grad_loss[row] : 1.f) * inv_t, k2);
}

// Few long rows: pieces of a row in workgroups of their own (rows.h).  The first launch leaves their maxima and sums and the
// list's own logits, since in place the second writes over them.
template <class T>
__global__ __launch_bounds__(PIECE_THREADS) void k_distill_pieces(const T *logits, uint32_t n_vocab, uint64_t stride, Teacher t, float inv_t,
                                                                  MaxSum *__restrict__ sums, float *__restrict__ kept)
{
    __shared__ MaxSum lds[PIECE_THREADS / 64];
    const uint64_t row = blockIdx.y;
    const uint32_t begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    RowPart<T, PIECE_THREADS, PIECE_HELD> part{logits + row * stride, begin, end};
    for (uint32_t i = threadIdx.x; i < t.k; i += PIECE_THREADS) {
        const uint32_t id = t.ids[row * t.ids_stride + i];
        if (id >= begin && id < end) kept[row * t.k + i] = (float)part.x[id];
    }
    MaxSum a{NEG_INF, 0.f};
    part.template each<true>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v, LOG2E * inv_t); });
    a = block_join<PIECE_THREADS>(a, lds, LOG2E * inv_t);
    if (threadIdx.x == 0) sums[row * gridDim.x + blockIdx.x] = a;
}

template <class T>
__global__ __launch_bounds__(PIECE_THREADS) void k_distill_join(const T *logits, uint32_t n_vocab, uint64_t stride, uint32_t pieces, Teacher t,
                                                                uint32_t slots, float inv_t, const MaxSum *__restrict__ sums,
                                                                const float *__restrict__ kept, float *__restrict__ loss,
                                                                float *__restrict__ lse_out, const float *__restrict__ grad_loss,
                                                                float grad_scale, T *grad, uint64_t gstride)
{
    __shared__ MaxSum lds[2][PIECE_THREADS / 64];
    __shared__ float2 lds_sum[PIECE_THREADS / 64];
    extern __shared__ uint8_t dynamic[];
    const uint64_t row = blockIdx.y;
    const float k2 = LOG2E * inv_t;
    const uint32_t begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    const List list(dynamic, t.k, slots);
    static_assert(MAX_PIECES <= PIECE_THREADS, "a thread per piece");
    Entries<PIECE_THREADS> own_list;
    own_list.load(t, row);
    clear_table<PIECE_THREADS>(list);
    __syncthreads();
    MaxSum b = read_list<PIECE_THREADS>(list, own_list, t.k, n_vocab, k2, [&](uint32_t i, uint32_t) { return kept[row * t.k + i]; });
    MaxSum a{NEG_INF, 0.f};
    if (threadIdx.x < pieces) a = sums[row * pieces + threadIdx.x];
    block_join2<PIECE_THREADS>(a, b, lds, k2);
    float mass, own;
    weigh_list<PIECE_THREADS>(list, t, row, b, a, inv_t, mass, own);
    const float2 all = block_sum<PIECE_THREADS>(mass, own, lds_sum);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        loss[row] = all.y;
        lse_out[row] = empty(a) ? NEG_INF : a.m * inv_t + log_of(a.s);
    }
    if (!grad) return;
    RowPart<T, PIECE_THREADS, PIECE_HELD> part{logits + row * stride, begin, end};
    put_grad<T, PIECE_THREADS, PIECE_HELD, true>(part, list, t.k, grad + row * gstride, all.x == 0.f || empty(a), a.m, 1.f / a.s, all.x,
                                                 grad_scale * (grad_loss ? grad_loss[row] : 1.f) * inv_t, k2);
}

// The gradient from lse.  From |lse| = FAR on a row's maximum and sum are formed again, by one workgroup, since in place the others
// would read what it has written.  So they are above a temperature of 2^120, where lse * temperature (the maximum that a sum of one
// would have) or a logit's distance from it might leave the range; below, a distance that does has no power.
constexpr float HOT = 0x1p120f;
// (Of float32 nine registers are spilled; with six wavefronts and none spilled 2,048 rows of 131,328 take 465 us in place of 419.)
template <class T, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void k_distill_backward(const T *logits, uint32_t n_vocab, uint64_t stride, Teacher t, uint32_t slots,
                                                                 float inv_t, float temperature, const float *__restrict__ lse,
                                                                 const float *__restrict__ grad_loss, float grad_scale, T *grad,
                                                                 uint64_t gstride)
{
    __shared__ MaxSum lds[2][THREADS / 64];
    __shared__ float2 lds_sum[THREADS / 64];
    extern __shared__ uint8_t dynamic[];
    const uint64_t row = blockIdx.y;
    const float k2 = LOG2E * inv_t, z = lse[row];
    const uint32_t begin = blockIdx.x * PIECE, end = n_vocab - begin < PIECE ? n_vocab : begin + PIECE;
    constexpr int HELD = PIECE / (THREADS * VEC);
    RowPart<T, THREADS, HELD> part{logits + row * stride, begin, end};
    const bool far = is_far(z) || temperature > HOT;   // -inf too: at a small temperature it may stand for a number beyond the range
    if (far) {
        if (blockIdx.x) return;
        part.end = n_vocab;
    }
    const List list(dynamic, t.k, slots);
    Entries<THREADS> own_list;
    own_list.load(t, row);
    part.hold();   // on its way while the list is read
    clear_table<THREADS>(list);
    __syncthreads();
    MaxSum b = read_list<THREADS>(list, own_list, t.k, n_vocab, k2,
                                  [&](uint32_t, uint32_t id) { return id >= part.begin && id < part.end ? (float)part.x[id] : 0.f; });
    b = block_join<THREADS>(b, lds[0], k2);
    MaxSum a{z * temperature, 1.f};   // the maximum that a sum of one would have
    float mass, own;
    weigh_list<THREADS>(list, t, row, b, a, inv_t, mass, own);
    const float2 sums = block_sum<THREADS>(mass, own, lds_sum);
    const float c = grad_scale * (grad_loss ? grad_loss[row] : 1.f) * inv_t;
    T *g = grad + row * gstride;
    if (far && sums.x != 0.f) {
        a = MaxSum{NEG_INF, 0.f};
        part.template each<false>(NEG_INF, [&](uint32_t, uint32_t, float (&v)[VEC]) { add_vec(a, v, k2); });
        a = block_join<THREADS>(a, lds[1], k2);
        return put_grad<T, THREADS, HELD, false>(part, list, t.k, g, empty(a), a.m, 1.f / a.s, sums.x, c, k2);
    }
    put_grad<T, THREADS, HELD, false>(part, list, t.k, g, sums.x == 0.f, a.m, 1.f, sums.x, c, k2);
}

// ---------------------------------------------------------------------------------------------
// host side

int check_distill(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, const Teacher &t, float temperature,
                  const float *lse, const float *grad_loss, const void *grad, uint64_t gstride)
{
    if (!elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || t.k == 0 || t.k > TOKTIER_MAX_TOP ||
        !temperature_ok(temperature))
        return TOKTIER_E_INVALID_ARG;
    if (n_rows == 0) return TOKTIER_OK;
    if (!matrix_ok(logits, type, n_rows, n_vocab, stride) || !matrix_ok(t.ids, TOKTIER_F32, n_rows, t.k, t.ids_stride) ||
        !matrix_ok(t.top, TOKTIER_F32, n_rows, t.k, t.top_stride) || !aligned4(t.lse) || !lse || !aligned4(lse) || !aligned4(grad_loss))
        return TOKTIER_E_INVALID_ARG;
    if (grad) {
        if (!matrix_ok(grad, type, n_rows, n_vocab, gstride)) return TOKTIER_E_INVALID_ARG;
        const uint64_t gb = extent(type, n_rows, n_vocab, gstride), nb = 4ull * n_rows;
        if (!(grad == logits && gstride == stride) && !apart(grad, gb, logits, extent(type, n_rows, n_vocab, stride))) return TOKTIER_E_INVALID_ARG;
        if (!apart(grad, gb, t.ids, extent(TOKTIER_F32, n_rows, t.k, t.ids_stride)) ||
            !apart(grad, gb, t.top, extent(TOKTIER_F32, n_rows, t.k, t.top_stride)) || !apart(grad, gb, lse, nb) ||
            (t.lse && !apart(grad, gb, t.lse, nb)) || (grad_loss && !apart(grad, gb, grad_loss, nb)))
            return TOKTIER_E_INVALID_ARG;
    }
    return TOKTIER_OK;
}

// Few long rows are split: the more CUs against a second launch, each row read twice and its list by every piece.  So fewer rows of 32
// bits are than of 16, and more where a row is so long that one workgroup keeps little of it.  With gradient, 64 listed, split / whole in
// us: 131,328 bfloat16 1 row 13.0 / 22.6, 96 rows 20.7 / 23.6, 128 25.4 / 24.8, 159 30.6 / 26.2; float32 64 rows 23.0 / 26.7, 96 33.6 / 30.8;
// 524,288 float32 64 rows 76 / 99, 128 134 / 133; 2,097,152 bfloat16 159 rows 362 / 462, float32 711 / 932; 65,536 bfloat16 16 rows 13.0 / 14.6
// (the loss alone 12.8 / 9.8, but its bits should not depend on whether a gradient is asked for).
constexpr uint32_t MOST_SPLIT = 159;
uint32_t most_split(uint32_t n_vocab, uint32_t elem) { return std::min(MOST_SPLIT, 256 / elem * std::max(1u, n_vocab >> 18)); }
bool split_rows(uint32_t n_rows, uint32_t n_vocab, uint32_t elem) { return n_vocab >= 8 * PIECE && n_rows <= most_split(n_vocab, elem); }

struct Split {
    uint32_t pieces;   // 0: rows are not split
    uint64_t kept, total;
};
Split layout_of(uint32_t n_rows, uint32_t n_vocab, uint32_t k, uint32_t elem)
{
    Split L{0, 0, 256};
    if (!split_rows(n_rows, n_vocab, elem)) return L;
    L.pieces = (n_vocab + PIECE - 1) / PIECE;
    L.kept = ((uint64_t)n_rows * L.pieces * sizeof(MaxSum) + 255) & ~255ull;
    L.total = L.kept + (((uint64_t)n_rows * k * 4 + 255) & ~255ull);
    return L;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int toktier_distill_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint32_t top_k, uint64_t *out_bytes)
{
    if (!out_bytes || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || n_rows > 0x7FFFFFFFu || top_k == 0 || top_k > TOKTIER_MAX_TOP)
        return TOKTIER_E_INVALID_ARG;
    // what any call of up to n_rows rows needs: the most of those whose rows are split, which are 16-bit ones
    *out_bytes = layout_of(std::clamp(n_rows, 1u, most_split(n_vocab, 2)), n_vocab, top_k, 2).total;
    return TOKTIER_OK;
}

extern "C" int toktier_distill(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, const uint32_t *top_ids,
                               uint64_t top_ids_stride, const float *top_logits, uint64_t top_logits_stride, uint32_t top_k,
                               const float *teacher_lse, float temperature, float *loss, float *lse, const float *grad_loss, float grad_scale,
                               void *grad_logits, uint64_t grad_stride, void *workspace, uint64_t workspace_bytes, void *stream)
{
    const Teacher t{top_ids, top_logits, teacher_lse, top_ids_stride, top_logits_stride, top_k};
    int rc = check_distill(logits, type, n_rows, n_vocab, stride, t, temperature, lse, grad_loss, grad_logits, grad_stride);
    if (rc || n_rows == 0) return rc;
    if (!loss || !aligned4(loss) || !workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
    const Split L = layout_of(n_rows, n_vocab, top_k, elem_size(type));
    if (workspace_bytes < L.total) return TOKTIER_E_CAPACITY;
    struct Area {
        const void *p;
        uint64_t n;
    };
    const uint64_t nb = 4ull * n_rows;
    const Area in[] = {{logits, extent(type, n_rows, n_vocab, stride)}, {top_ids, extent(TOKTIER_F32, n_rows, top_k, top_ids_stride)},
                       {top_logits, extent(TOKTIER_F32, n_rows, top_k, top_logits_stride)}, {teacher_lse, teacher_lse ? nb : 0},
                       {grad_loss, grad_loss ? nb : 0}};
    const Area out[] = {{workspace, L.total}, {loss, nb}, {lse, nb}};
    for (int i = 0; i < 3; ++i) {
        for (const Area &a : in)
            if (!apart(out[i].p, out[i].n, a.p, a.n)) return TOKTIER_E_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (!apart(out[i].p, out[i].n, out[k].p, out[k].n)) return TOKTIER_E_INVALID_ARG;
        if (grad_logits && !apart(out[i].p, out[i].n, grad_logits, extent(type, n_rows, n_vocab, grad_stride))) return TOKTIER_E_INVALID_ARG;
    }
    hipStream_t s = (hipStream_t)stream;
    const float inv_t = 1.f / temperature;
    const uint32_t slots = slots_of(top_k), lds = list_bytes(top_k);
    with_type(type, [&](auto v) {
        using T = decltype(v);
        constexpr int HELD = sizeof(T) == 4 ? 4 : 8;   // 32 VGPRs
        const T *x = (const T *)logits;
        T *g = (T *)grad_logits;
        if (L.pieces) {
            MaxSum *sums = (MaxSum *)workspace;
            float *kept = (float *)((uint8_t *)workspace + L.kept);
            k_distill_pieces<T><<<dim3(L.pieces, n_rows), PIECE_THREADS, 0, s>>>(x, n_vocab, stride, t, inv_t, sums, kept);
            k_distill_join<T><<<dim3(g ? L.pieces : 1, n_rows), PIECE_THREADS, lds, s>>>(x, n_vocab, stride, L.pieces, t, slots, inv_t, sums, kept,
                                                                                         loss, lse, grad_loss, grad_scale, g, grad_stride);
            return;
        }
        auto launch = [&](auto threads, auto held) {
            constexpr int N = decltype(threads)::value, H = decltype(held)::value;
            in_launches(n_rows, N, [&](uint64_t r, uint32_t rows) {
                Teacher part = t;
                part.ids += r * t.ids_stride;
                part.top += r * t.top_stride;
                if (part.lse) part.lse += r;
                k_distill<T, N, H><<<rows, N, lds, s>>>(x + r * stride, n_vocab, stride, part, slots, inv_t, loss + r, lse + r,
                                                        grad_loss ? grad_loss + r : nullptr, grad_scale, g ? g + r * grad_stride : nullptr,
                                                        grad_stride);
            });
        };
        if (n_vocab <= 256 * VEC * 4)   // short rows: more workgroups per CU
            launch(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
        else if (n_vocab <= 512 * VEC * 8)
            launch(std::integral_constant<int, 512>{}, std::integral_constant<int, HELD>{});
        else
            launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, HELD>{});
    });
    return hip_status(hipGetLastError());
}

extern "C" int toktier_distill_backward(const void *logits, int type, uint32_t n_rows, uint32_t n_vocab, uint64_t stride, const uint32_t *top_ids,
                                        uint64_t top_ids_stride, const float *top_logits, uint64_t top_logits_stride, uint32_t top_k,
                                        const float *teacher_lse, float temperature, const float *lse, const float *grad_loss,
                                        float grad_scale, void *grad_logits, uint64_t grad_stride, void *stream)
{
    if (n_rows && !grad_logits) return TOKTIER_E_INVALID_ARG;
    const Teacher t{top_ids, top_logits, teacher_lse, top_ids_stride, top_logits_stride, top_k};
    int rc = check_distill(logits, type, n_rows, n_vocab, stride, t, temperature, lse, grad_loss, grad_logits, grad_stride);
    if (rc || n_rows == 0) return rc;
    // Every piece reads the row's list; longer pieces, read by fewer, are slower all the same, since less of them is held
    // (8,192 rows of 131,328 bfloat16, 64 listed: 777 us, in whole rows 865; 1,500 of 33,001 float16, 100 listed: 39, in halves 38)
    const uint32_t slots = slots_of(top_k), lds = list_bytes(top_k), pieces = (n_vocab + PIECE - 1) / PIECE;
    with_type(type, [&](auto v) {
        using T = decltype(v);
        for (uint32_t r = 0; r < n_rows; r += 65535) {   // grid.y
            const uint32_t rows = n_rows - r < 65535 ? n_rows - r : 65535;
            Teacher part = t;
            part.ids += r * t.ids_stride;
            part.top += r * t.top_stride;
            if (part.lse) part.lse += r;
            k_distill_backward<T, 256><<<dim3(pieces, rows), 256, lds, (hipStream_t)stream>>>(
                (const T *)logits + r * stride, n_vocab, stride, part, slots, 1.f / temperature, temperature, lse + r,
                grad_loss ? grad_loss + r : nullptr, grad_scale, (T *)grad_logits + r * grad_stride, grad_stride);
        }
    });
    return hip_status(hipGetLastError());
}
