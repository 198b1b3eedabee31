// embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
#include "ops.h"

#include <algorithm>
#include <type_traits>

namespace tt {
namespace {

// The first column of a vector: a row's last one is moved back so that it is whole (elements one by one take several times
// as long) where it may share columns with the vector before, whose lane then loads and stores the same values.
// A row that is added to needs both in one wavefront, its loads before its stores: see put_row.  (Gradient of 65,536 tokens, 33,024 x 2,047:
// 224 us with a last vector of seven, 156 us so.)
__device__ __forceinline__ uint32_t whole(uint32_t c, uint32_t dim, bool may)
{
    return may && c < dim && dim - c < VEC ? dim - VEC : c;
}

// ---------------------------------------------------------------------------------------------
// lookup: out[t, :] = scale * table[ids[t], :]
//
// A copy with a gather in front: bound by the bytes read and written.  A workgroup takes L lanes per
// token (the row's vectors, a power of two up to 256) and 256 / L tokens per step, U steps whose loads
// are all in flight together (16,384 rows of 4,096 bfloat16: 45 us with four steps, as with two, 54 with eight).  An output larger
// than the caches of the chip's parts is stored past them, so that it does not drive out table rows: 33.5 us,
// 5.7 TB/s.
constexpr uint64_t STREAM_BYTES = 32u << 20;

template <class TI, class TO, int U>
__global__ __launch_bounds__(256) void k_embed(const TI *__restrict__ table, uint64_t tstride, uint32_t n_vocab,
                                               uint32_t dim, const uint32_t *__restrict__ ids, uint32_t n_tokens,
                                               float scale, TO *__restrict__ out, uint64_t ostride, uint32_t lshift,
                                               bool stream)
{
    const uint32_t lane = threadIdx.x & ((1u << lshift) - 1u), sub = threadIdx.x >> lshift, step = 256u >> lshift;
    uint32_t c = (blockIdx.y << lshift) * VEC + lane * VEC;
    if (c >= dim) return;
    c = whole(c, dim, c > 0);
    const uint64_t t0 = (uint64_t)blockIdx.x * (U * step) + sub;
    const uint32_t n = dim - c;
    float x[U][VEC], by[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t t = t0 + (uint64_t)u * step;
        const uint32_t id = t < n_tokens ? ids[t] : 0xFFFFFFFFu;
        by[u] = id < n_vocab ? scale : 0.f;   // zeros stay zeros, whatever the scale
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
        for (int k = 0; k < VEC; ++k) x[u][k] *= by[u];
        if (stream) stream_part(out + t * ostride + c, n, x[u]);
        else store_part(out + t * ostride + c, n, x[u]);
    }
}

// ---------------------------------------------------------------------------------------------
// gradient: tokens sorted by ID (stable, so equal IDs keep the token order), then one sum per run of
// equal IDs.  Few tokens are not sorted: see k_embed_few.
//
// Sort: least-significant-digit radix sort in one or two passes of up to 11 bits.  A wavefront owns a
// contiguous part of its block, so the rank of an element is (places of lower digits and earlier blocks +
// counts of the block's earlier wavefronts + the wavefront's own count so far + equal digits in lower lanes,
// from one ballot per digit bit).  A pass is a histogram launch and a scatter launch.
//
// The launches of the sort leave most of the chip idle, so where rows of absent IDs have to become zeros and
// most of the rows are absent, the zeros are written by further blocks of these launches.
constexpr int SORT_WAVES = 8, SORT_THREADS = SORT_WAVES * 64;
// Elements per thread.  Two spread few tokens over more blocks (65,536 tokens, 33,024 IDs, 256 columns: the call takes 46 us,
// 48 with four, 56 with eight; 20,000: 35, 38, 48); for 600,000 it makes no difference.
constexpr int SORT_R = 2;
constexpr uint32_t MAX_BINS = 2048;

struct SortPlan {
    uint32_t bits, passes, dbits, bins, groups, blocks;   // a block sorts `groups` groups of 512 x SORT_R elements
};

SortPlan sort_plan(uint64_t n_tokens, uint32_t n_vocab)
{
    SortPlan p;
    p.bits = 32 - __builtin_clz(n_vocab);   // keys 0 .. n_vocab (n_vocab itself: no row)
    p.passes = p.bits <= 11 ? 1 : 2;
    p.dbits = std::max(2u, (p.bits + p.passes - 1) / p.passes);   // bins are taken four at a time
    p.bins = 1u << p.dbits;
    // every block reads all blocks' histograms, so there are at most 256 of them
    const uint64_t group = SORT_THREADS * SORT_R;
    p.groups = (uint32_t)((n_tokens + group * 256 - 1) / (group * 256));
    if (p.groups < 1) p.groups = 1;
    p.blocks = (uint32_t)((n_tokens + group * p.groups - 1) / (group * p.groups));
    return p;
}

// Rows of zeros: `rows` rows of row_bytes (a multiple of 2) from p, stride bytes apart, none of them past `end`.
struct Zeros {
    uint8_t *p;
    uint64_t row_bytes, stride, end;
    uint32_t rows, per_block, from;   // from: the launch's first row
};

template <bool STREAM> __device__ __forceinline__ void zero_rows(const Zeros &z, uint32_t block)
{
    const uint64_t r0 = z.from + (uint64_t)block * z.per_block;
    for (uint32_t q = 0; q < z.per_block && r0 + q < z.rows; ++q) {
        const uint64_t at = (r0 + q) * z.stride, left = z.end - at;
        const uint64_t n = z.row_bytes < left ? z.row_bytes : left;
        uint8_t *row = z.p + at;
        for (uint64_t c = threadIdx.x * 16ull; c < n; c += blockDim.x * 16ull) {
            if (c + 16 <= n) {
                if constexpr (STREAM) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, (u32x4_row *)(row + c));
                else *(u32x4_row *)(row + c) = u32x4{0, 0, 0, 0};
            } else {
                for (uint64_t d = c; d < n; d += 2) *(uint16_t *)(row + d) = 0;
            }
        }
    }
}
__device__ __forceinline__ void zero_block(const Zeros &z, uint32_t block)
{
    // past the caches where they are more than these hold: 538 MB in 22 us in each of four launches, 24 us through them
    if (z.end > STREAM_BYTES) zero_rows<true>(z, block);
    else zero_rows<false>(z, block);
}

struct SortLds {
    uint32_t cnt[SORT_WAVES][MAX_BINS];   // per wavefront: counts, then next output places
    uint32_t wsum[SORT_WAVES];
};

// One pass over this block's elements, `groups` groups of R per thread.  hist: the counts of every block ([blocks][bins]).
__global__ __launch_bounds__(SORT_THREADS) void k_sort_scatter(const uint32_t *__restrict__ keys,
                                                               const uint32_t *__restrict__ pos, int first, uint32_t n,
                                                               uint32_t n_vocab, uint32_t shift, uint32_t dbits,
                                                               uint32_t groups, uint32_t blocks,
                                                               const uint32_t *__restrict__ hist,
                                                               uint32_t *__restrict__ keys_out,
                                                               uint32_t *__restrict__ pos_out, Zeros z)
{
    __shared__ __align__(16) SortLds sh;
    if (blockIdx.x >= blocks) return zero_block(z, blockIdx.x - blocks);
    constexpr int R = SORT_R;
    const uint32_t block = blockIdx.x;
    const uint32_t bins = 1u << dbits, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint64_t base = ((uint64_t)block * SORT_WAVES + wave) * (64 * R) * groups + lane;
    uint32_t key[R];
    auto load = [&](uint32_t g) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t i = base + ((uint64_t)g * R + r) * 64;
            key[r] = i < n ? keys[i] : 0xFFFFFFFFu;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = min(key[r], n_vocab);   // an ID without a row; also what lies past the end
    };
    load(0);
    for (uint32_t b = lane * 4; b < bins; b += 256) *(u32x4 *)&sh.cnt[wave][b] = u32x4{0, 0, 0, 0};
    __syncthreads();
    for (uint32_t g = 0;;) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (base + ((uint64_t)g * R + r) * 64 < n)
                atomicAdd(&sh.cnt[wave][(key[r] >> shift) & (bins - 1)], 1u);
        if (++g == groups) break;
        load(g);
    }
    __syncthreads();
    // first place of every bin in this block: all elements of lower bins, and of this bin in earlier blocks and
    // wavefronts.  A thread owns four consecutive bins (`bins` is a multiple of 4).
    const uint32_t b0 = tid * 4;
    u32x4 all = 0, before = 0, sum;
    if (b0 < bins) {
#pragma unroll 8
        for (uint32_t k = 0; k < blocks; ++k) {
            const u32x4 v = *(const u32x4 *)&hist[(uint64_t)k * bins + b0];
            all += v;
            if (k < block) before += v;
        }
    }
    sum[0] = all[0];
    sum[1] = sum[0] + all[1];
    sum[2] = sum[1] + all[2];
    sum[3] = sum[2] + all[3];
    const uint32_t incl = wave_incl_sum(sum[3]);
    if (lane == 63) sh.wsum[wave] = incl;
    __syncthreads();
    uint32_t at = incl - sum[3];
#pragma unroll
    for (uint32_t w = 0; w < SORT_WAVES; ++w) at += w < wave ? sh.wsum[w] : 0;
    if (b0 < bins) {
        u32x4 place = before + at;
        place[1] += sum[0];
        place[2] += sum[1];
        place[3] += sum[2];
#pragma unroll
        for (int w = 0; w < SORT_WAVES; ++w) {
            const u32x4 c = *(u32x4 *)&sh.cnt[w][b0];
            *(u32x4 *)&sh.cnt[w][b0] = place;
            place += c;
        }
    }
    __syncthreads();
    for (uint32_t g = 0; g < groups; ++g) {
        if (groups > 1) load(g);
        uint32_t from[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t i = base + ((uint64_t)g * R + r) * 64;
            from[r] = first || i >= n ? (uint32_t)i : pos[i];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = base + ((uint64_t)g * R + r) * 64 < n;
            const uint32_t d = (key[r] >> shift) & (bins - 1);
            uint64_t same = __ballot(in);
            for (uint32_t b = 0; b < dbits; ++b) {
                const uint64_t one = __ballot((d >> b) & 1u);
                same &= (d >> b) & 1u ? one : ~one;
            }
            const uint32_t rank = __popcll(same & ((1ull << lane) - 1ull));
            const uint32_t place = sh.cnt[wave][d];
            wave_order();   // the bin's place is read by all its lanes before one moves it on
            if (in) {
                if (rank == 0) sh.cnt[wave][d] = place + __popcll(same);
                keys_out[place + rank] = key[r];
                pos_out[place + rank] = from[r];
            }
            wave_order();
        }
    }
}

__global__ __launch_bounds__(SORT_THREADS) void k_sort_hist(const uint32_t *__restrict__ keys, uint32_t n, uint32_t n_vocab,
                                                            uint32_t shift, uint32_t bins, uint32_t groups, uint32_t blocks,
                                                            uint32_t *__restrict__ hist, Zeros z)
{
    __shared__ uint32_t h[MAX_BINS];
    if (blockIdx.x >= blocks) return zero_block(z, blockIdx.x - blocks);
    for (uint32_t b = threadIdx.x; b < bins; b += SORT_THREADS) h[b] = 0;
    __syncthreads();
    const uint64_t base = (uint64_t)blockIdx.x * (SORT_THREADS * SORT_R) * groups + threadIdx.x;
    for (uint32_t g = 0; g < groups; ++g) {
        uint32_t key[SORT_R];
#pragma unroll
        for (int r = 0; r < SORT_R; ++r) {
            const uint64_t i = base + ((uint64_t)g * SORT_R + r) * SORT_THREADS;
            key[r] = i < n ? keys[i] : 0;
        }
#pragma unroll
        for (int r = 0; r < SORT_R; ++r)
            if (base + ((uint64_t)g * SORT_R + r) * SORT_THREADS < n)
                atomicAdd(&h[(min(key[r], n_vocab) >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += SORT_THREADS) hist[(uint64_t)blockIdx.x * bins + b] = h[b];
}

// Sums.  The sorted tokens are cut into chunks; a wavefront takes one chunk and 512 columns and adds up
// each run of equal IDs in registers, eight rows in flight.  A run inside a chunk is a finished row; one
// that crosses a chunk's border leaves a partial sum (slot 0: the run entered from the chunk before, slot 1:
// it starts here and goes on), joined in chunk order by k_embed_join.
// Bound by memory: 65,536 tokens of text added to 131,328 x 4,096 float32, 1.18 GB, in 227 us (5.2 TB/s; a copy reaches
// 5.15), and 29 us of sort before, 15 us of join after.  Sixteen rows in flight halve the
// wavefronts of a SIMD: the call takes 413 instead of 281 us.
constexpr uint32_t COLS = 64 * VEC;
constexpr int ROWS = 8, PARTS = 8;   // rows, and partial sums, of a wavefront in flight

template <class TT>
__device__ __forceinline__ void put_row(TT *__restrict__ row, uint32_t n, float scale, bool accumulate,
                                        const float (&acc)[VEC])
{
    float x[VEC];
    if (accumulate) {
        load_part(row, n, 0.f, x);
        wave_order();   // a neighbour may load, and store, some of the same columns
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] += scale * acc[k];
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] = scale * acc[k];
    }
    store_part(row, n, x);
}

constexpr int ZROWS = 16;   // table rows that a wavefront looks after when absent IDs get zeros here

// ONCE: gradients too large for any cache are loaded past them (537 MB added to a table of 131,328 x 4,096: 258 -> 242 us; 82 MB
// that the kernels before have left in the caches would take 156 instead of 121 us).
constexpr uint64_t ONCE_BYTES = 256u << 20;

template <class TG, class TT, bool ONCE>
__global__ __launch_bounds__(256) void k_embed_sum(const TG *__restrict__ grad, uint64_t gstride,
                                                   const uint32_t *__restrict__ keys, const uint32_t *__restrict__ pos,
                                                   uint32_t n, uint32_t n_vocab, uint32_t dim, uint32_t chunk,
                                                   uint32_t n_chunks, uint32_t ncb, float scale, int accumulate,
                                                   TT *__restrict__ table, uint64_t tstride, float *__restrict__ part,
                                                   uint32_t dpad, uint32_t absent_units, uint32_t first)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t unit = __builtin_amdgcn_readfirstlane((first + blockIdx.x) * 4u + (threadIdx.x >> 6)), sums = n_chunks * ncb;
    if (unit < sums) {
        const uint32_t ch = unit / ncb, c = whole(unit % ncb * COLS + lane * VEC, dim, lane > 0);
        const uint32_t i0 = ch * chunk, len = min(chunk, n - i0);
        const uint32_t my = min(lane, len - 1);
        const uint32_t key_l = keys[i0 + my], pos_l = pos[i0 + my];
        const uint32_t prev = i0 > 0 ? keys[i0 - 1] : 0xFFFFFFFFu, next_ch = i0 + len < n ? keys[i0 + len] : 0xFFFFFFFFu;
        const uint32_t live = __popcll(__ballot(lane < len && key_l < n_vocab));   // those without a row sort last
        if (live == 0) return;
        const bool enters = prev == (uint32_t)__builtin_amdgcn_readlane((int)key_l, 0);
        const bool leaves = next_ch == (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)len - 1);
        const uint32_t m = c < dim ? dim - c : 0;
        float acc[VEC] = {};
        uint32_t run0 = 0;
        for (uint32_t i = 0; i < live; i += ROWS) {
            Vec<TG> x[ROWS];
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const uint32_t p = (uint32_t)__builtin_amdgcn_readlane((int)pos_l, (int)min(i + u, live - 1));
                if (i + u < live && m) x[u] = ONCE ? load_once(grad + p * gstride + c, m) : load_some(grad + p * gstride + c, m);
            }
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const uint32_t j = i + u;
                if (j >= live) break;
                const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)j);
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += vec_at(x[u], k);
                const bool last = j + 1 == len;
                const uint32_t next = (uint32_t)__builtin_amdgcn_readlane((int)key_l, (int)min(j + 1, len - 1));
                if (last || next != key) {
                    const bool in = run0 == 0 && enters, on = last && leaves;
                    if (m) {
                        if (in || on) store_vec(part + ((uint64_t)ch * 2 + (in ? 0 : 1)) * dpad + c, acc);
                        else put_row(table + key * tstride + c, m, scale, accumulate, acc);
                    }
#pragma unroll
                    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
                    run0 = j + 1;
                }
            }
        }
        return;
    }
    // rows of absent IDs (launched where they are not zeros already): a lane looks its row up in the sorted
    // keys, then the wavefront writes zeros
    if (unit - sums >= absent_units) return;
    const uint64_t r0 = (uint64_t)(unit - sums) * ZROWS;
    const uint32_t row = (uint32_t)r0 + (lane % ZROWS);
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < row) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = lane < ZROWS && row < n_vocab && (lo == n || keys[lo] != row);
    uint64_t todo = __ballot(absent);
    const float zero[VEC] = {};
    while (todo) {
        const uint32_t r = (uint32_t)r0 + (uint32_t)__builtin_ctzll(todo);
        todo &= todo - 1;
        for (uint32_t c0 = lane * VEC; c0 < dim; c0 += COLS) {
            const uint32_t c = whole(c0, dim, c0 > 0);
            store_part(table + r * tstride + c, dim - c, zero);
        }
    }
}

// Adds up `count` partial sums, `step` elements apart, PARTS in flight.
__device__ __forceinline__ void add_parts(const float *__restrict__ p, uint64_t step, uint32_t count, float (&acc)[VEC])
{
    for (uint32_t q = 0; q < count; q += PARTS) {
        Vec<float> x[PARTS];
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
            if (q + u < count) x[u] = load_vec(p + (q + u) * step);
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
            if (q + u < count)
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += vec_at(x[u], k);
    }
}

// Runs that leave their chunk.  A wavefront looks after one chunk and 512 columns and joins a run that starts there
// and enters fewer than 64 chunks; a longer one is shared out between the workgroup's wavefronts, whose sums
// meet in LDS (40,000 tokens of text, 1,256 IDs, 320 columns: 38 us by one wavefront a run).
constexpr uint32_t JOIN_WAVES = 8, JOIN_THREADS = JOIN_WAVES * 64;

template <class TT>
__global__ __launch_bounds__(JOIN_THREADS) void k_embed_join(const uint32_t *__restrict__ keys, uint32_t n, uint32_t n_vocab,
                                                             uint32_t dim, uint32_t chunk, uint32_t n_chunks, uint32_t ncb,
                                                             float scale, int accumulate, TT *__restrict__ table,
                                                             uint64_t tstride, const float *__restrict__ part, uint32_t dpad,
                                                             uint32_t first, uint32_t blocks)
{
    __shared__ float sums[JOIN_WAVES][COLS];
    __shared__ uint32_t entered[JOIN_WAVES], any_long[JOIN_WAVES];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t units = n_chunks * ncb;
    // the columns of one run go to several workgroups
    auto unit = [&](uint32_t w) { return w * blocks + first + blockIdx.x; };
    // the chunks after ch whose first token is `key`, of 64 from h0 on
    auto heads = [&](uint32_t h0, uint32_t key) {
        const uint32_t h = h0 + lane;
        const uint64_t same = __ballot(h < n_chunks && keys[(uint64_t)min(h, n_chunks - 1) * chunk] == key);
        return ~same ? (uint32_t)__builtin_ctzll(~same) : 64u;
    };
    auto starts = [&](uint32_t ch, uint32_t &key) {   // whether a run starts in this chunk and leaves it
        const uint32_t i0 = ch * chunk;
        if (n - i0 <= chunk) return false;   // (i0 + chunk may be 2^32)
        const uint32_t end = i0 + chunk;
        const uint32_t prev = i0 > 0 ? keys[i0 - 1] : 0xFFFFFFFFu, head = keys[i0], next = keys[end];
        key = keys[end - 1];
        return key < n_vocab && next == key && !(head == key && prev == key);
    };
    uint32_t key;
    bool is_long = false;
    if (unit(wave) < units) {
        const uint32_t ch = unit(wave) / ncb, c = whole(unit(wave) % ncb * COLS + lane * VEC, dim, lane > 0);
        if (starts(ch, key)) {
            const uint32_t count = heads(ch + 1, key);
            is_long = count == 64;
            if (!is_long && c < dim) {
                float acc[VEC] = {};
                load_part(part + ((uint64_t)ch * 2 + 1) * dpad + c, VEC, 0.f, acc);
                add_parts(part + (uint64_t)(ch + 1) * 2 * dpad + c, 2ull * dpad, count, acc);
                put_row(table + key * tstride + c, dim - c, scale, accumulate, acc);
            }
        }
    }
    if (lane == 0) any_long[wave] = is_long;
    __syncthreads();
    for (uint32_t w = 0; w < JOIN_WAVES; ++w) {
        if (!any_long[w]) continue;
        const uint32_t ch = unit(w) / ncb, c = whole(unit(w) % ncb * COLS + lane * VEC, dim, lane > 0);
        starts(ch, key);
        uint32_t count = 0;
        for (uint32_t h0 = ch + 1;; h0 += JOIN_THREADS) {   // 64 chunks a wavefront
            const uint32_t mine = heads(h0 + wave * 64, key);
            if (lane == 0) entered[wave] = mine;
            __syncthreads();
            uint32_t all = 0;
            for (uint32_t o = 0; o < JOIN_WAVES && all == o * 64; ++o) all += entered[o];
            __syncthreads();
            count += all;
            if (all < JOIN_THREADS) break;
        }
        const uint32_t share = (count + JOIN_WAVES - 1) / JOIN_WAVES;
        const uint32_t from = min(wave * share, count), to = min(from + share, count);
        float acc[VEC] = {};
        if (c < dim) {
            if (wave == 0) load_part(part + ((uint64_t)ch * 2 + 1) * dpad + c, VEC, 0.f, acc);
            add_parts(part + (uint64_t)(ch + 1 + from) * 2 * dpad + c, 2ull * dpad, to - from, acc);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) sums[wave][k * 64 + lane] = acc[k];
        __syncthreads();
        if (wave == 0 && c < dim) {
#pragma unroll
            for (uint32_t o = 1; o < JOIN_WAVES; ++o)
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += sums[o][k * 64 + lane];
            put_row(table + key * tstride + c, dim - c, scale, accumulate, acc);
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(SORT_THREADS) void k_zero_rows(Zeros z) { zero_block(z, blockIdx.x); }

// Few tokens, in one launch without a sort: a workgroup per token looks through all IDs and lists the positions of its
// own.  The row's blocks of 512 columns are dealt out to the workgroups of the tokens with this ID, so a frequent ID
// brings the workgroups that its many rows need.  Up to 2 * ROWS rows a wavefront adds up by itself, in every
// eighth of the workgroup's blocks; more are shared out between the wavefronts, and their sums joined in LDS.  Further
// workgroups write the zeros of a small table, each for the rows that no ID names.
// The work grows with the square of the tokens, the sort's four to six launches hardly.  With the IDs of text (one in ten
// the most frequent), gradients of bfloat16 added to a float32 table of 33,024 x 2,048: 777 tokens 6.9 us (the call's own cost),
// 2,048 9.0 us, 26 us sorted, 4,096 17.6 and 31 us.  Tokens of one ID alone, which one workgroup per 512 columns then adds
// up, take longer: 777 18 us, 2,048 40 and 30 us, 4,096 80 and 40 us.
constexpr uint32_t FEW = 4096, FEW_WAVES = 8, FEW_THREADS = FEW_WAVES * 64;
constexpr uint64_t ZEROS_BESIDE = 32u << 20;       // larger tables are zeroed by a launch of their own (10 MB: 7.1 and 9.8 us)
constexpr uint32_t ZBYTES = 16384, ZMOST = 1024;   // of a workgroup that writes zeros: bytes (of at least a row), rows

// R: IDs of a thread
template <class TG, class TT, uint32_t R>
__global__ __launch_bounds__(FEW_THREADS) void k_embed_few(const TG *__restrict__ grad, uint64_t gstride,
                                                          const uint32_t *__restrict__ ids, uint32_t n, uint32_t n_vocab,
                                                          uint32_t dim, uint32_t ncb, float scale, int accumulate,
                                                          TT *__restrict__ table, uint64_t tstride, uint32_t zrows)
{
    __shared__ union {
        uint16_t list[R * FEW_THREADS];
        uint8_t present[ZMOST];
    } sh;
    __shared__ float sums[FEW_WAVES][COLS];
    __shared__ uint32_t counts[FEW_WAVES];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t block = blockIdx.x;
    const uint32_t seg = (n + FEW_THREADS - 1) / FEW_THREADS * 64, base = wave * seg + lane;   // each wavefront's part of the IDs
    uint32_t v[R];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) v[i] = ids[min(base + i * 64, n - 1)];
    if (block < n) {
        const uint32_t id = ids[block];
        if (id >= n_vocab) return;
        uint64_t same[R];
        uint32_t count = 0, before = 0;   // tokens with this ID; those before this one
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            const uint32_t at = base + i * 64;
            const bool is = (i * 64 < seg) & (at < n) & (v[i] == id);
            same[i] = __ballot(is);
            count += __popcll(same[i]);
            before += __popcll(__ballot(is & (at < block)));
        }
        if (lane == 0) counts[wave] = count | before << 16;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (uint32_t w = 0; w < FEW_WAVES; ++w) all += counts[w];
        all = __builtin_amdgcn_readfirstlane(all);
        const uint32_t total = all & 0xFFFFu, rank = all >> 16;
        if (rank >= ncb) return;
        uint32_t at = 0;
        for (uint32_t w = 0; w < wave; ++w) at += counts[w] & 0xFFFFu;
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            if (same[i] >> lane & 1u)
                sh.list[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(same[i] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same[i], 0))] =
                    (uint16_t)(base + i * 64);
            at += __popcll(same[i]);
        }
        __syncthreads();
        const bool shared = total > 2 * ROWS;
        const uint32_t share = shared ? (total + FEW_WAVES - 1) / FEW_WAVES : total;
        const uint32_t from = shared ? min(wave * share, total) : 0, to = min(from + share, total);
        for (uint32_t cb = rank + (shared ? 0 : total * wave); cb < ncb; cb += shared ? total : total * FEW_WAVES) {
            const uint32_t c = whole(cb * COLS + lane * VEC, dim, lane > 0), m = c < dim ? dim - c : 0;
            float acc[VEC] = {};
            for (uint32_t i = from; i < to; i += ROWS) {
                Vec<TG> x[ROWS];
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const uint32_t p = __builtin_amdgcn_readfirstlane(sh.list[min(i + u, to - 1)]);
                    if (i + u < to && m) x[u] = load_some(grad + p * gstride + c, m);
                }
#pragma unroll
                for (int u = 0; u < ROWS; ++u)
                    if (i + u < to)
#pragma unroll
                        for (int k = 0; k < VEC; ++k) acc[k] += vec_at(x[u], k);
            }
            if (shared) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) sums[wave][k * 64 + lane] = acc[k];
                __syncthreads();
                if (wave == 0)
#pragma unroll
                    for (uint32_t w = 1; w < FEW_WAVES; ++w)
#pragma unroll
                        for (int k = 0; k < VEC; ++k) acc[k] += sums[w][k * 64 + lane];
                __syncthreads();
                if (wave != 0) continue;
            }
            if (m) put_row(table + id * tstride + c, m, scale, accumulate, acc);
        }
        return;
    }
    block -= n;
    const uint32_t r0 = block * zrows, rows = min(zrows, n_vocab - r0);
    for (uint32_t i = tid; i < rows; i += FEW_THREADS) sh.present[i] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < R; ++i)
        if (v[i] >= r0 && v[i] - r0 < rows) sh.present[v[i] - r0] = 1;
    __syncthreads();
    const uint32_t vectors = (dim + VEC - 1) / VEC;
    const float zero[VEC] = {};
    for (uint32_t i = tid; i < rows * vectors; i += FEW_THREADS) {
        const uint32_t r = i / vectors, c0 = (i - r * vectors) * VEC, c = whole(c0, dim, c0 > 0);
        if (!sh.present[r]) store_part(table + (uint64_t)(r0 + r) * tstride + c, dim - c, zero);
    }
}

struct BackwardLayout {
    SortPlan sort;
    uint32_t chunk, n_chunks, ncb, dpad;
    uint64_t keys[2], pos[2], hist, part, total;
};

constexpr uint32_t LONG_CHUNK = 64, SHORT_CHUNK = 8, FULL_CHIP = 4096;   // tokens, tokens, wavefronts

uint64_t padded(uint64_t bytes) { return (bytes + 255) & ~255ull; }

BackwardLayout backward_layout(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim)
{
    BackwardLayout L;
    L.sort = sort_plan(n_tokens, n_vocab);
    L.ncb = (dim + COLS - 1) / COLS;
    L.dpad = (dim + VEC - 1) / VEC * VEC;
    // tokens per chunk: 64 (fewest partial sums), fewer where that would leave the chip with under 4,096
    // wavefronts, eight per CU and SIMD pair
    L.chunk = LONG_CHUNK;
    while (L.chunk > SHORT_CHUNK && n_tokens * L.ncb < (uint64_t)FULL_CHIP * L.chunk) L.chunk /= 2;
    L.n_chunks = (uint32_t)((n_tokens + L.chunk - 1) / L.chunk);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += padded(bytes);
        return o;
    };
    for (int k = 0; k < 2; ++k) {
        L.keys[k] = take(4 * n_tokens);
        L.pos[k] = take(4 * n_tokens);
    }
    L.hist = take(4ull * L.sort.blocks * L.sort.bins);
    L.part = take(8ull * L.n_chunks * L.dpad);
    L.total = n_tokens <= FEW ? 256 : at;   // few tokens need none
    return L;
}

// Bytes for every call of no more tokens, IDs and columns; single parts of the layout shrink as these grow.
// Histograms: of at most 256 blocks, and one digit of 11 bits from 1,024 IDs on.  Partial sums: chunks shorter than 64 are fewer
// than 2 FULL_CHIP / ncb, one more for the last, of at most ncb * COLS columns.
uint64_t backward_bytes(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim)
{
    if (n_tokens <= FEW) return 256;
    const uint64_t blocks = std::min<uint64_t>(256, (n_tokens + SORT_THREADS * SORT_R - 1) / (SORT_THREADS * SORT_R));
    const uint64_t bins = n_vocab >= MAX_BINS / 2 ? MAX_BINS : sort_plan(n_tokens, n_vocab).bins;
    const uint64_t dpad = (dim + VEC - 1) / VEC * VEC;
    const uint64_t brief = std::min<uint64_t>(n_tokens / SHORT_CHUNK * dpad, 2ull * FULL_CHIP * COLS);
    const uint64_t sums = std::max(n_tokens / LONG_CHUNK * dpad, brief) + dpad;
    return 4 * padded(4 * n_tokens) + padded(4 * blocks * bins) + padded(8 * sums);
}

// The rows of a table as zeros to write; contiguous rows are cut into pieces of 16 KiB, one per block
// (538 MB in one launch, through the caches: 88 us; in pieces of 64 KiB 96 us).
constexpr uint64_t PIECE = 16384;
// Blocks of a launch, beside those of a sort: 2^31 threads (tables over 68 GB take larger pieces).
constexpr uint32_t MOST_PIECES = (1u << 31) / SORT_THREADS;

Zeros zeros_of(void *table, uint32_t size, uint32_t n_vocab, uint32_t dim, uint64_t stride)
{
    Zeros z;
    z.p = (uint8_t *)table;
    z.row_bytes = (uint64_t)dim * size;
    z.stride = stride * size;
    z.end = z.stride * n_vocab;
    z.rows = n_vocab;
    if (z.row_bytes == z.stride) {
        z.row_bytes = z.stride = PIECE;
        z.rows = (uint32_t)((z.end + PIECE - 1) / PIECE);
    }
    z.per_block = z.row_bytes >= PIECE ? 1 : (uint32_t)(PIECE / z.row_bytes);
    while (z.rows / z.per_block >= MOST_PIECES) z.per_block *= 2;
    z.from = 0;
    return z;
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
    const uint64_t gx = (n_tokens + U * step - 1) / (U * step);   // gy is 8,192 at most
    with_type(table_type, [&](auto ti) {
        with_type(out_type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            in_launches(gx, 256, [&](uint64_t first, uint32_t blocks) {
                const uint64_t t = first * (U * step);
                k_embed<TI, TO, U><<<dim3(blocks, gy), 256, 0, (hipStream_t)stream>>>(
                    (const TI *)table, table_stride, n_vocab, dim, ids + t, (uint32_t)(n_tokens - t), scale, (TO *)out + t * out_stride,
                    out_stride, lshift, n_tokens * dim * sizeof(TO) > STREAM_BYTES);
            });
        });
    });
    return hip_status(hipGetLastError());
}

extern "C" int toktier_embed_backward_workspace_bytes(uint64_t n_tokens, uint32_t n_vocab, uint32_t dim,
                                                      uint64_t *out_bytes)
{
    if (!out_bytes || !sizes_ok(n_tokens, n_vocab, dim)) return TOKTIER_E_INVALID_ARG;
    *out_bytes = backward_bytes(n_tokens, n_vocab, dim);
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
    Zeros z = zeros_of(grad_table, elem_size(table_type), n_vocab, dim, table_stride);
    if (n_tokens == 0) {
        if (accumulate) return TOKTIER_OK;
        k_zero_rows<<<(z.rows + z.per_block - 1) / z.per_block, SORT_THREADS, 0, s>>>(z);
        return hip_status(hipGetLastError());
    }
    const BackwardLayout L = backward_layout(n_tokens, n_vocab, dim);
    if (workspace_bytes < L.total) return TOKTIER_E_CAPACITY;
    if (!apart(workspace, L.total, grad_table, tb) || !apart(workspace, L.total, ids, 4 * n_tokens) ||
        !apart(workspace, L.total, grad_out, extent(grad_type, n_tokens, dim, grad_stride)))
        return TOKTIER_E_INVALID_ARG;
    if (n_tokens <= FEW) {
        const uint32_t n = (uint32_t)n_tokens;
        const bool beside = !accumulate && (uint64_t)n_vocab * dim * elem_size(table_type) <= ZEROS_BESIDE;
        if (!accumulate && !beside) k_zero_rows<<<(z.rows + z.per_block - 1) / z.per_block, SORT_THREADS, 0, s>>>(z);
        const uint64_t row_bytes = (uint64_t)dim * elem_size(table_type);
        const uint32_t zrows = (uint32_t)std::clamp<uint64_t>(ZBYTES / row_bytes, 1, ZMOST);
        const uint32_t zb = beside ? (n_vocab + zrows - 1) / zrows : 0;
        with_type(grad_type, [&](auto tg) {
            with_type(table_type, [&](auto tt_) {
                using TG = decltype(tg);
                using TT = decltype(tt_);
                auto launch = [&](auto r) {
                    k_embed_few<TG, TT, decltype(r)::value><<<n + zb, FEW_THREADS, 0, s>>>(
                        (const TG *)grad_out, grad_stride, ids, n, n_vocab, dim, L.ncb, scale, accumulate, (TT *)grad_table,
                        table_stride, zrows);
                };
                if (n <= FEW / 2) launch(std::integral_constant<uint32_t, FEW / 2 / FEW_THREADS>{});
                else launch(std::integral_constant<uint32_t, FEW / FEW_THREADS>{});
            });
        });
        return hip_status(hipGetLastError());
    }
    const uint64_t sums = (uint64_t)L.n_chunks * L.ncb;
    if (sums > 0x7FFFFFFFull) return TOKTIER_E_INVALID_ARG;
    uint8_t *ws = (uint8_t *)workspace;
    const uint32_t n = (uint32_t)n_tokens;
    // fewer tokens than rows: all rows become zeros beside the sort, and those of present IDs are written
    // again; else only the absent ones, after it
    const bool early = !accumulate && n < n_vocab;
    uint32_t *hist = (uint32_t *)(ws + L.hist), *keys[2], *pos[2];
    for (int p = 0; p < 2; ++p) {
        keys[p] = (uint32_t *)(ws + L.keys[p]);
        pos[p] = (uint32_t *)(ws + L.pos[p]);
    }
    uint32_t zrows = z.rows;
    auto zero_blocks = [&](uint32_t launch, uint32_t launches) {   // this launch's share of the zeros
        if (!early) return 0u;
        const uint32_t share = (zrows + launches - 1) / launches;
        z.from = share * launch < zrows ? share * launch : zrows;
        z.rows = share < zrows - z.from ? z.from + share : zrows;
        return (z.rows - z.from + z.per_block - 1) / z.per_block;
    };
    const uint32_t last = L.sort.passes - 1;
    for (uint32_t p = 0; p <= last; ++p) {
        const uint32_t *ki = p ? keys[0] : ids, *pi = p ? pos[0] : nullptr, shift = p * L.sort.dbits, launches = 2 * L.sort.passes;
        const uint32_t zh = zero_blocks(2 * p, launches);
        k_sort_hist<<<L.sort.blocks + zh, SORT_THREADS, 0, s>>>(ki, n, n_vocab, shift, L.sort.bins, L.sort.groups, L.sort.blocks,
                                                                hist, z);
        const uint32_t zs = zero_blocks(2 * p + 1, launches);
        k_sort_scatter<<<L.sort.blocks + zs, SORT_THREADS, 0, s>>>(ki, pi, p == 0, n, n_vocab, shift, L.sort.dbits, L.sort.groups,
                                                                   L.sort.blocks, hist, keys[p], pos[p], z);
    }
    float *part = (float *)(ws + L.part);
    const uint64_t absent = accumulate || early ? 0 : (n_vocab + ZROWS - 1) / ZROWS;
    const uint32_t blocks = (uint32_t)((sums + absent + 3) / 4), jblocks = (uint32_t)((sums + JOIN_WAVES - 1) / JOIN_WAVES);
    with_type(grad_type, [&](auto tg) {
        with_type(table_type, [&](auto tt_) {
            using TG = decltype(tg);
            using TT = decltype(tt_);
            auto launch = [&](auto once) {
                in_launches(blocks, 256, [&](uint64_t first, uint32_t some) {
                    k_embed_sum<TG, TT, decltype(once)::value><<<some, 256, 0, s>>>(
                        (const TG *)grad_out, grad_stride, keys[last], pos[last], n, n_vocab, dim, L.chunk, L.n_chunks, L.ncb,
                        scale, accumulate, (TT *)grad_table, table_stride, part, L.dpad, (uint32_t)absent, (uint32_t)first);
                });
            };
            if ((uint64_t)n * dim * sizeof(TG) > ONCE_BYTES) launch(std::true_type{});
            else launch(std::false_type{});
        });
    });
    with_type(table_type, [&](auto tt_) {
        using TT = decltype(tt_);
        in_launches(jblocks, JOIN_THREADS, [&](uint64_t first, uint32_t some) {
            k_embed_join<TT><<<some, JOIN_THREADS, 0, s>>>(keys[last], n, n_vocab, dim, L.chunk, L.n_chunks, L.ncb, scale, accumulate,
                                                           (TT *)grad_table, table_stride, part, L.dpad, (uint32_t)first, jblocks);
        });
    });
    return hip_status(hipGetLastError());
}
