// embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
#include "ops.h"

namespace tt {
namespace {

// ---------------------------------------------------------------------------------------------
// lookup: out[t, :] = scale * table[ids[t], :]
//
// A copy with a gather in front: bound by the bytes read and written.  A workgroup takes L lanes per
// token (the row's vectors, a power of two up to 256) and 256 / L tokens per step, U steps whose loads
// are all in flight together.
template <class TI, class TO, int U>
__global__ __launch_bounds__(256) void k_embed(const TI *__restrict__ table, uint64_t tstride, uint32_t n_vocab,
                                               uint32_t dim, const uint32_t *__restrict__ ids, uint32_t n_tokens,
                                               float scale, TO *__restrict__ out, uint64_t ostride, uint32_t lshift)
{
    const uint32_t lane = threadIdx.x & ((1u << lshift) - 1u), sub = threadIdx.x >> lshift, step = 256u >> lshift;
    const uint32_t c = (blockIdx.y << lshift) * VEC + lane * VEC;
    if (c >= dim) return;
    const uint64_t t0 = (uint64_t)blockIdx.x * (U * step) + sub;
    const uint32_t n = dim - c;
    float x[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t t = t0 + (uint64_t)u * step;
        const uint32_t id = t < n_tokens ? ids[t] : 0xFFFFFFFFu;
        if (id < n_vocab) load_part(table + id * tstride + c, n, 0.f, x[u]);
        else
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[u][k] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t t = t0 + (uint64_t)u * step;
        if (t >= n_tokens) break;
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[u][k] *= scale;
        store_part(out + t * ostride + c, n, x[u]);
    }
}

// ---------------------------------------------------------------------------------------------
// gradient: tokens sorted by ID (stable, so equal IDs keep the token order), then one sum per run of
// equal IDs.
//
// Sort: least-significant-digit radix sort in one or two passes of up to 11 bits.  Each pass is a
// histogram per block and a stable scatter: a wavefront owns a contiguous part of its block, so the rank
// of an element is (block base + counts of the block's earlier wavefronts + the wavefront's own count so
// far + equal digits in lower lanes, from one ballot per digit bit).
constexpr int SORT_WAVES = 8, SORT_THREADS = SORT_WAVES * 64;
constexpr uint32_t SORT_MAX_BLOCKS = 128;
constexpr uint32_t MAX_BINS = 2048;

struct SortPlan {
    uint32_t bits, passes, dbits, bins, rounds, blocks;
};

SortPlan sort_plan(uint64_t n_tokens, uint32_t n_vocab)
{
    SortPlan p;
    p.bits = 32 - __builtin_clz(n_vocab);   // keys 0 .. n_vocab (n_vocab itself: no row)
    p.passes = p.bits <= 11 ? 1 : 2;
    p.dbits = (p.bits + p.passes - 1) / p.passes;
    p.bins = 1u << p.dbits;
    const uint64_t per = (uint64_t)SORT_THREADS * SORT_MAX_BLOCKS;
    p.rounds = (uint32_t)((n_tokens + per - 1) / per);
    if (p.rounds < 8) p.rounds = 8;
    p.blocks = (uint32_t)((n_tokens + (uint64_t)SORT_THREADS * p.rounds - 1) / ((uint64_t)SORT_THREADS * p.rounds));
    return p;
}

__device__ __forceinline__ uint32_t sort_key(const uint32_t *keys, bool first, uint32_t i, uint32_t n_vocab)
{
    const uint32_t k = keys[i];
    return first ? min(k, n_vocab) : k;
}

__global__ __launch_bounds__(SORT_THREADS) void k_sort_hist(const uint32_t *__restrict__ keys, int first, uint32_t n,
                                                            uint32_t n_vocab, uint32_t shift, uint32_t bins,
                                                            uint32_t rounds, uint32_t *__restrict__ hist)
{
    __shared__ uint32_t h[MAX_BINS];
    for (uint32_t b = threadIdx.x; b < bins; b += SORT_THREADS) h[b] = 0;
    __syncthreads();
    const uint64_t base = (uint64_t)blockIdx.x * (SORT_THREADS * rounds);
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint64_t i = base + (uint64_t)r * SORT_THREADS + threadIdx.x;
        if (i < n) atomicAdd(&h[(sort_key(keys, first, (uint32_t)i, n_vocab) >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += SORT_THREADS) hist[(uint64_t)blockIdx.x * bins + b] = h[b];
}

__global__ __launch_bounds__(SORT_THREADS) void k_sort_scatter(const uint32_t *__restrict__ keys,
                                                               const uint32_t *__restrict__ pos, int first, uint32_t n,
                                                               uint32_t n_vocab, uint32_t shift, uint32_t dbits,
                                                               uint32_t rounds, const uint32_t *__restrict__ hist,
                                                               uint32_t *__restrict__ keys_out,
                                                               uint32_t *__restrict__ pos_out)
{
    __shared__ uint32_t cnt[SORT_WAVES][MAX_BINS];   // per wavefront: counts, then next output places
    __shared__ uint32_t wsum[SORT_WAVES];
    const uint32_t bins = 1u << dbits, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    for (uint32_t b = lane; b < bins; b += 64) cnt[wave][b] = 0;
    __syncthreads();
    const uint64_t base = (uint64_t)blockIdx.x * (SORT_THREADS * rounds) + (uint64_t)wave * 64 * rounds;
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint64_t i = base + r * 64 + lane;
        if (i < n) atomicAdd(&cnt[wave][(sort_key(keys, first, (uint32_t)i, n_vocab) >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // first place of every bin in this block: all elements of lower bins, and of this bin in earlier blocks.
    // A thread owns up to four consecutive bins.
    uint32_t tot[MAX_BINS / SORT_THREADS], before[MAX_BINS / SORT_THREADS], sum = 0;
    constexpr uint32_t PER = MAX_BINS / SORT_THREADS;
#pragma unroll
    for (uint32_t q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        uint32_t all = 0, bef = 0;
        if (b < bins)
            for (uint32_t k = 0; k < gridDim.x; ++k) {
                const uint32_t v = hist[(uint64_t)k * bins + b];
                all += v;
                if (k < blockIdx.x) bef += v;
            }
        tot[q] = all;
        before[q] = bef;
        sum += all;
    }
    const uint32_t incl = wave_incl_sum(sum);
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    uint32_t at = incl - sum;
    for (uint32_t w = 0; w < wave; ++w) at += wsum[w];
#pragma unroll
    for (uint32_t q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        if (b < bins) {
            uint32_t place = at + before[q];
            for (int w = 0; w < SORT_WAVES; ++w) {
                const uint32_t c = cnt[w][b];
                cnt[w][b] = place;
                place += c;
            }
        }
        at += tot[q];
    }
    __syncthreads();
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint64_t i = base + r * 64 + lane;
        const bool in = i < n;
        const uint32_t key = in ? sort_key(keys, first, (uint32_t)i, n_vocab) : 0;
        const uint32_t d = (key >> shift) & (bins - 1);
        uint64_t same = __ballot(in);
        for (uint32_t b = 0; b < dbits; ++b) {
            const uint64_t one = __ballot((d >> b) & 1u);
            same &= (d >> b) & 1u ? one : ~one;
        }
        if (in) {
            const uint32_t rank = __popcll(same & ((1ull << lane) - 1ull)), count = __popcll(same);
            const uint32_t place = cnt[wave][d];
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) cnt[wave][d] = place + count;
            keys_out[place + rank] = key;
            pos_out[place + rank] = first ? (uint32_t)i : pos[i];
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Sums.  The sorted tokens are cut into chunks of C; a wavefront takes one chunk and 512 columns and adds
// up each run of equal IDs in registers.  A run inside a chunk is a finished row; one that crosses a
// chunk's border leaves a partial sum (slot 0: the run entered from the chunk before, slot 1: it starts
// here and goes on), joined in chunk order by k_embed_join.
constexpr uint32_t COLS = 64 * VEC;

template <class TT>
__device__ __forceinline__ void put_row(TT *__restrict__ row, uint32_t n, float scale, bool accumulate,
                                        const float (&acc)[VEC])
{
    float x[VEC];
    if (accumulate) {
        load_part(row, n, 0.f, x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] += scale * acc[k];
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] = scale * acc[k];
    }
    store_part(row, n, x);
}

constexpr int ZROWS = 16;   // table rows that a wavefront looks after when absent IDs get zeros

template <class TG, class TT>
__global__ __launch_bounds__(256) void k_embed_sum(const TG *__restrict__ grad, uint64_t gstride,
                                                   const uint32_t *__restrict__ keys, const uint32_t *__restrict__ pos,
                                                   uint32_t n, uint32_t n_vocab, uint32_t dim, uint32_t chunk,
                                                   uint32_t n_chunks, uint32_t ncb, float scale, int accumulate,
                                                   TT *__restrict__ table, uint64_t tstride, float *__restrict__ part,
                                                   uint32_t dpad)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t unit = __builtin_amdgcn_readfirstlane((uint32_t)(blockIdx.x * 4u + (threadIdx.x >> 6)));
    if (unit < (uint64_t)n_chunks * ncb) {
        const uint32_t ch = (uint32_t)(unit / ncb), c = (uint32_t)(unit % ncb) * COLS + lane * VEC;
        const uint32_t i0 = ch * chunk, len = min(chunk, n - i0);
        const uint32_t my = min(lane, len - 1);
        const uint32_t key_l = keys[i0 + my], pos_l = pos[i0 + my];
        const uint32_t live = __popcll(__ballot(lane < len && key_l < n_vocab));   // those without a row sort last
        if (live == 0) return;
        const bool enters = i0 > 0 && keys[i0 - 1] == (uint32_t)__builtin_amdgcn_readlane((int)key_l, 0);
        const bool leaves = i0 + len < n && keys[i0 + len] == (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)len - 1);
        const uint32_t m = c < dim ? dim - c : 0;
        float acc[VEC] = {};
        uint32_t run0 = 0;
        for (uint32_t i = 0; i < live; i += 4) {
            float x[4][VEC];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t p = (uint32_t)__builtin_amdgcn_readlane((int)pos_l, (int)min(i + u, live - 1));
                if (m) load_part(grad + p * gstride + c, m, 0.f, x[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t j = i + u;
                if (j >= live) break;
                const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)j);
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += x[u][k];
                const bool last = j + 1 == len;
                const uint32_t next = (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)min(j + 1, len - 1));
                if (last || next != key) {
                    const bool from = run0 == 0 && enters, on = last && leaves;
                    if (m) {
                        if (from || on) {
                            float *q = part + ((uint64_t)ch * 2 + (from ? 0 : 1)) * dpad + c;
                            store_vec(q, acc);
                        } else {
                            put_row(table + key * tstride + c, m, scale, accumulate, acc);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
                    run0 = j + 1;
                }
            }
        }
        return;
    }
    if (accumulate) return;
    // rows of absent IDs: a lane looks its row up in the sorted keys, then the wavefront writes zeros
    const uint64_t r0 = (unit - (uint64_t)n_chunks * ncb) * ZROWS;
    if (r0 >= n_vocab) return;
    const uint32_t row = (uint32_t)r0 + (lane % ZROWS);
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (keys[mid] < row) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = lane < ZROWS && row < n_vocab && (lo == n || keys[lo] != row);
    uint64_t todo = __ballot(absent);
    const float zero[VEC] = {};
    while (todo) {
        const uint32_t r = (uint32_t)r0 + (uint32_t)__builtin_ctzll(todo);
        todo &= todo - 1;
        for (uint32_t c = lane * VEC; c < dim; c += COLS) store_part(table + r * tstride + c, dim - c, zero);
    }
}

template <class TT>
__global__ __launch_bounds__(256) void k_embed_join(const uint32_t *__restrict__ keys, uint32_t n, uint32_t n_vocab,
                                                    uint32_t dim, uint32_t chunk, uint32_t n_chunks, uint32_t ncb,
                                                    float scale, int accumulate, TT *__restrict__ table,
                                                    uint64_t tstride, const float *__restrict__ part, uint32_t dpad)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t unit = __builtin_amdgcn_readfirstlane((uint32_t)(blockIdx.x * 4u + (threadIdx.x >> 6)));
    if (unit >= (uint64_t)n_chunks * ncb) return;
    const uint32_t ch = (uint32_t)(unit / ncb), c = (uint32_t)(unit % ncb) * COLS + lane * VEC;
    const uint32_t i0 = ch * chunk, end = i0 + chunk;
    if (end >= n) return;
    const uint32_t key = keys[end - 1];
    if (key >= n_vocab || keys[end] != key) return;                   // no run leaves this chunk
    if (keys[i0] == key && i0 > 0 && keys[i0 - 1] == key) return;     // it started in an earlier chunk
    if (c >= dim) return;
    float acc[VEC];
    load_part(part + ((uint64_t)ch * 2 + 1) * dpad + c, VEC, 0.f, acc);
    for (uint32_t h = ch + 1; h < n_chunks && keys[h * chunk] == key; ++h) {
        float x[VEC];
        load_part(part + (uint64_t)h * 2 * dpad + c, VEC, 0.f, x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += x[k];
    }
    put_row(table + key * tstride + c, dim - c, scale, accumulate, acc);
}

template <class TT>
__global__ __launch_bounds__(256) void k_zero_rows(TT *__restrict__ table, uint32_t n_vocab, uint32_t dim,
                                                   uint64_t tstride)
{
    const float zero[VEC] = {};
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += 256 * VEC)
        store_part(table + blockIdx.x * tstride + c, dim - c, zero);
}

constexpr uint32_t CHUNK = 64;

struct BackwardLayout {
    SortPlan sort;
    uint32_t n_chunks, ncb, dpad;
    uint64_t keys[2], pos[2], hist, part, total;
};

BackwardLayout backward_layout(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim)
{
    BackwardLayout L;
    L.sort = sort_plan(n_tokens, n_vocab);
    L.n_chunks = (uint32_t)((n_tokens + CHUNK - 1) / CHUNK);
    L.ncb = (dim + COLS - 1) / COLS;
    L.dpad = (dim + VEC - 1) / VEC * VEC;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += (bytes + 255) & ~255ull;
        return o;
    };
    for (int k = 0; k < 2; ++k) {
        L.keys[k] = take(4 * n_tokens);
        L.pos[k] = take(4 * n_tokens);
    }
    L.hist = take(4ull * L.sort.blocks * L.sort.bins);
    L.part = take(8ull * L.n_chunks * L.dpad);
    L.total = at < 256 ? 256 : at;
    return L;
}

bool sizes_ok(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim)
{
    return n_tokens < 0xFFFFFFFFull && n_vocab > 0 && n_vocab <= TOKTIER_MAX_VOCAB && dim > 0 && dim <= (1u << 24);
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int toktier_embed(const void *table, int table_type, uint32_t n_vocab, uint32_t dim, uint64_t table_stride,
                             const uint32_t *ids, uint64_t n_tokens, float scale, void *out, int out_type,
                             uint64_t out_stride, void *stream)
{
    if (!sizes_ok(n_tokens, n_vocab, dim)) return TOKTIER_E_INVALID_ARG;
    if (!elem_size(table_type) || !elem_size(out_type)) return TOKTIER_E_INVALID_ARG;
    if (n_tokens == 0) return TOKTIER_OK;
    if (!matrix_ok(table, table_type, n_vocab, dim, table_stride) || !matrix_ok(out, out_type, n_tokens, dim, out_stride) ||
        !ids || !aligned4(ids))
        return TOKTIER_E_INVALID_ARG;
    const uint64_t ob = extent(out_type, n_tokens, dim, out_stride);
    if (!apart(out, ob, table, extent(table_type, n_vocab, dim, table_stride)) || !apart(out, ob, ids, 4 * n_tokens))
        return TOKTIER_E_INVALID_ARG;
    const uint32_t nv = (dim + VEC - 1) / VEC;
    uint32_t lshift = 0;
    while (lshift < 8 && (1u << lshift) < nv) ++lshift;
    const uint32_t step = 256u >> lshift, gy = (nv + (1u << lshift) - 1) >> lshift;
    constexpr int U = 4;
    const uint64_t gx = (n_tokens + U * step - 1) / (U * step);
    if (gx > 0x7FFFFFFFull || gy > 65535) return TOKTIER_E_INVALID_ARG;
    with_type(table_type, [&](auto ti) {
        with_type(out_type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            k_embed<TI, TO, U><<<dim3((uint32_t)gx, gy), 256, 0, (hipStream_t)stream>>>(
                (const TI *)table, table_stride, n_vocab, dim, ids, (uint32_t)n_tokens, scale, (TO *)out, out_stride, lshift);
        });
    });
    return hip_status(hipGetLastError());
}

extern "C" int toktier_embed_backward_workspace_bytes(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim,
                                                      uint64_t *out_bytes)
{
    if (!out_bytes || !sizes_ok(n_tokens, n_vocab, dim)) return TOKTIER_E_INVALID_ARG;
    *out_bytes = backward_layout(n_tokens, n_vocab, dim).total;
    return TOKTIER_OK;
}

extern "C" int toktier_embed_backward(const void *grad_out, int grad_type, uint64_t grad_stride, const uint32_t *ids,
                                      uint64_t n_tokens, float scale, void *grad_table, int table_type,
                                      uint32_t n_vocab, uint32_t dim, uint64_t table_stride, int accumulate,
                                      void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(n_tokens, n_vocab, dim) || !elem_size(grad_type)) return TOKTIER_E_INVALID_ARG;
    if (!matrix_ok(grad_table, table_type, n_vocab, dim, table_stride)) return TOKTIER_E_INVALID_ARG;
    const uint64_t tb = extent(table_type, n_vocab, dim, table_stride);
    if (n_tokens) {
        if (!matrix_ok(grad_out, grad_type, n_tokens, dim, grad_stride) || !ids || !aligned4(ids)) return TOKTIER_E_INVALID_ARG;
        if (!workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
        const uint64_t gb = extent(grad_type, n_tokens, dim, grad_stride);
        if (!apart(grad_table, tb, grad_out, gb) || !apart(grad_table, tb, ids, 4 * n_tokens)) return TOKTIER_E_INVALID_ARG;
    }
    hipStream_t s = (hipStream_t)stream;
    if (n_tokens == 0) {
        if (accumulate) return TOKTIER_OK;
        with_type(table_type, [&](auto tt_) {
            using TT = decltype(tt_);
            k_zero_rows<TT><<<n_vocab, 256, 0, s>>>((TT *)grad_table, n_vocab, dim, table_stride);
        });
        return hip_status(hipGetLastError());
    }
    const BackwardLayout L = backward_layout(n_tokens, n_vocab, dim);
    if (workspace_bytes < L.total) return TOKTIER_E_CAPACITY;
    if (!apart(workspace, L.total, grad_table, tb) || !apart(workspace, L.total, ids, 4 * n_tokens) ||
        !apart(workspace, L.total, grad_out, extent(grad_type, n_tokens, dim, grad_stride)))
        return TOKTIER_E_INVALID_ARG;
    uint8_t *ws = (uint8_t *)workspace;
    const uint32_t n = (uint32_t)n_tokens;
    uint32_t *hist = (uint32_t *)(ws + L.hist);
    const uint32_t *keys = ids, *pos = nullptr;
    for (uint32_t p = 0; p < L.sort.passes; ++p) {
        const uint32_t shift = p * L.sort.dbits;
        uint32_t *ko = (uint32_t *)(ws + L.keys[p]), *po = (uint32_t *)(ws + L.pos[p]);
        k_sort_hist<<<L.sort.blocks, SORT_THREADS, 0, s>>>(keys, p == 0, n, n_vocab, shift, L.sort.bins, L.sort.rounds, hist);
        k_sort_scatter<<<L.sort.blocks, SORT_THREADS, 0, s>>>(keys, pos, p == 0, n, n_vocab, shift, L.sort.dbits,
                                                              L.sort.rounds, hist, ko, po);
        keys = ko;
        pos = po;
    }
    float *part = (float *)(ws + L.part);
    const uint64_t sums = (uint64_t)L.n_chunks * L.ncb, zeros = accumulate ? 0 : (n_vocab + ZROWS - 1) / ZROWS;
    const uint64_t blocks = (sums + zeros + 3) / 4, jblocks = (sums + 3) / 4;
    if (blocks > 0x3FFFFFFFull) return TOKTIER_E_INVALID_ARG;
    with_type(grad_type, [&](auto tg) {
        with_type(table_type, [&](auto tt_) {
            using TG = decltype(tg);
            using TT = decltype(tt_);
            k_embed_sum<TG, TT><<<(uint32_t)blocks, 256, 0, s>>>((const TG *)grad_out, grad_stride, keys, pos, n, n_vocab, dim, CHUNK,
                                                                 L.n_chunks, L.ncb, scale, accumulate, (TT *)grad_table,
                                                                 table_stride, part, L.dpad);
        });
    });
    with_type(table_type, [&](auto tt_) {
        using TT = decltype(tt_);
        k_embed_join<TT><<<(uint32_t)jblocks, 256, 0, s>>>(keys, n, n_vocab, dim, CHUNK, L.n_chunks, L.ncb, scale, accumulate,
                                                           (TT *)grad_table, table_stride, part, L.dpad);
    });
    return hip_status(hipGetLastError());
}
