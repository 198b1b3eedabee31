// product.h -- matrix products on the matrix cores (gfx950) with an epilogue of the caller's: the tiles of
// linear_loss.hip.
//
//   out[n][m] = sum_k A(m, k) B(n, k)
//
// An operand is stored either along k ([row][k], "plain") or across it ([k][row], "turned").  All of them are aligned
// to 16 bytes and padded or clamped by the caller, so that the inner loop knows no edges.
#pragma once
#include <type_traits>
#include <utility>

#include "ops.h"

namespace tt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr uint32_t STEP_BYTES = 128;                                        // of k in a step, per row of an operand
template <class T> constexpr uint32_t STEP_K = STEP_BYTES / sizeof(T);      // 64 elements of 16 bits, 32 floats

// A workgroup's tile: WM x WN wavefronts, each with TM x TN tiles of 16 x 16.
template <int WM_, int WN_, int TM_, int TN_> struct Tile {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
    static constexpr int M = WM * TM * 16, N = WN * TN * 16, THREADS = WM * WN * 64;
    static constexpr uint32_t LDS_A = M * STEP_BYTES, LDS_B = N * STEP_BYTES, STAGE = LDS_A + LDS_B, LDS = 2 * STAGE;
};

__device__ __forceinline__ uint32_t lds_address(const lds_u8 *p) { return (uint32_t)(uintptr_t)p; }

// 16 bytes per lane from base + offset to LDS, at `to` + 16 * lane.  No register is written, and the caller waits
// (wait_loads) before a barrier; the compiler's own builtin would make every read of LDS wait for all of them.
__device__ __forceinline__ void load_to_lds(uint32_t to, const void *base, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "m0", "memory");
}
// until at most N of them are in flight
template <int N> __device__ __forceinline__ void wait_loads()
{
    static_assert(N < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The 16-byte pieces of an operand's rows in LDS change places within the row, so that the lanes of a read meet
// different banks: plain rows (128 bytes) by their number, turned ones so that the four (16-bit) or one (float) rows that
// a group of 16 lanes reads, and the groups beside it, lie apart.
template <class T, bool TURNED, int WIDTH> __device__ __forceinline__ uint32_t swizzle(uint32_t row)
{
    constexpr uint32_t PIECES = WIDTH * sizeof(T) / 16;   // of a turned row
    if constexpr (!TURNED) return row & 7;
    else if constexpr (sizeof(T) == 4) return (((row >> 2) & 3) << 2) & (PIECES - 1);
    else if constexpr (WIDTH >= 128) return ((row & 3) | ((row >> 3) & 1) << 2) << 1;
    else return ((((row >> 1) & 1) | ((row >> 3) & 1) << 1) << 1) & (PIECES - 1);
}

// One operand's way into LDS.  Every thread copies 16-byte pieces at fixed offsets from a base that advances with k.
template <class T, bool TURNED, int WIDTH, int THREADS> struct Loader {
    static constexpr uint32_t PER_ROW = TURNED ? WIDTH * sizeof(T) / 16 : STEP_BYTES / 16;
    static constexpr uint32_t PIECES = WIDTH * STEP_BYTES / 16;
    static constexpr int LOADS = PIECES / THREADS;
    static_assert(PIECES % THREADS == 0, "every wavefront has as many copies in flight");
    const uint8_t *base;
    uint64_t advance;     // bytes of a step
    uint32_t offset[LOADS];
    uint32_t wave;

    // rows of `stride` bytes; the operand's rows (plain) or columns (turned) from `first` on, `count` in all: the last one,
    // or the last 16 bytes, stand for those behind it, also where the whole tile lies there
    __device__ __forceinline__ void init(const T *p, uint64_t stride, uint32_t first, uint32_t count, uint32_t k_first)
    {
        constexpr uint32_t LEAST = TURNED ? 16 / sizeof(T) : 1;
        first = first < count - LEAST ? first : count - LEAST;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if constexpr (TURNED) {
            base = (const uint8_t *)p + (uint64_t)k_first * stride + (uint64_t)first * sizeof(T);
            advance = STEP_K<T> * stride;
        } else {
            base = (const uint8_t *)p + (uint64_t)first * stride + (uint64_t)k_first * sizeof(T);
            advance = STEP_BYTES;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t piece = i * THREADS + threadIdx.x, row = piece / PER_ROW;
            const uint32_t col = (piece % PER_ROW) ^ swizzle<T, TURNED, WIDTH>(row);
            if constexpr (TURNED) {
                const uint32_t last = (count - first) * sizeof(T) / 16 - 1;   // pieces of a row, of a count that fills them
                offset[i] = row * (uint32_t)stride + (col < last ? col : last) * 16;
            } else {
                const uint32_t last = count - first - 1;
                offset[i] = (row < last ? row : last) * (uint32_t)stride + col * 16;
            }
        }
    }
    // the i-th of this thread's LOADS copies of a step
    __device__ __forceinline__ void load(uint32_t lds, int i) const
    {
        load_to_lds(lds + (i * THREADS + wave * 64) * 16, base, offset[i]);
    }
    // the step in which only `rows` rows of k are there (turned): the last one stands for those behind it
    __device__ __forceinline__ void clamp(uint64_t stride, uint32_t rows)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t row = (i * THREADS + threadIdx.x) / PER_ROW;
            if (row >= rows) offset[i] -= (row - (rows - 1)) * (uint32_t)stride;
        }
    }
};

// A lane's part of a 16-row fragment, half `s` of a step, 16 bytes: of 16-bit types k = 8 (lane / 16) + 0..7 of
// 32, of floats k = 4 (lane / 16) + 0..3 of 16.
template <class T, bool TURNED, int WIDTH> __device__ __forceinline__ u32x4 fragment(const lds_u8 *lds, uint32_t tile, uint32_t s)
{
    const uint32_t lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    if constexpr (!TURNED) {
        const uint32_t row = tile * 16 + l;
        return *(const __attribute__((address_space(3))) u32x4 *)(lds + row * STEP_BYTES + (((4 * s + g) ^ (l & 7)) << 4));
    } else if constexpr (sizeof(T) == 4) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t k = 4 * (4 * s + g) + i, col = tile * 16 + l;
            v[i] = *(const __attribute__((address_space(3))) uint32_t *)(lds + k * (WIDTH * 4) + (((col >> 2) ^ swizzle<T, true, WIDTH>(k)) << 4) +
                                                                       ((col & 3) << 2));
        }
        return v;
    } else {
        // the transposing read: 16 lanes read four rows of 16 elements and each gets a column of them
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        u32x4 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = 32 * s + 8 * g + 4 * h + (l >> 2), piece = 2 * tile + ((l & 3) >> 1);
            const lds_u8 *at = lds + k * (WIDTH * 2) + ((piece ^ swizzle<T, true, WIDTH>(k)) << 4) + ((l & 1) << 3);
            const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
            v[2 * h] = w[0];
            v[2 * h + 1] = w[1];
        }
        return v;
    }
}

template <class T> __device__ __forceinline__ void multiply(u32x4 a, u32x4 b, f32x4 &acc)
{
    if constexpr (sizeof(T) == 4) {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], acc, 0, 0, 0);
    } else if constexpr (__is_same(T, __bf16)) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), acc, 0, 0, 0);
    } else {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), acc, 0, 0, 0);
    }
}

// f(0), f(1) .. f(N - 1) with constants as arguments: registers can only be told apart when the code is written.
template <class F, int... I> __device__ __forceinline__ void for_each(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void unrolled(F f) { for_each(f, std::make_integer_sequence<int, N>{}); }

// An operand as the host gives it: rows of `stride` bytes (a multiple of 16), of which `count` are there (plain) or
// `count` columns (turned).
struct Operand {
    const void *p;
    uint64_t stride;
    uint32_t count;
};

// The product of one tile, steps [begin, end) of k; `rows` > 0: rows of k that are there (turned A only, in the last step
// fewer than a step has).  After it all wavefronts are past their reads of LDS.
template <class T, class TILE, bool TURN_A, bool TURN_B>
__device__ __forceinline__ void product(f32x4 (&acc)[TILE::TM][TILE::TN], lds_u8 *lds, Operand a, Operand b, uint32_t m0, uint32_t n0,
                                        uint32_t begin, uint32_t end, uint32_t rows)
{
    const uint32_t wave = threadIdx.x >> 6, wm = wave / TILE::WN, wn = wave % TILE::WN;
#pragma unroll
    for (int i = 0; i < TILE::TM; ++i)
#pragma unroll
        for (int j = 0; j < TILE::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (begin >= end) return;
    Loader<T, TURN_A, TILE::M, TILE::THREADS> la;
    Loader<T, TURN_B, TILE::N, TILE::THREADS> lb;
    la.init((const T *)a.p, a.stride, m0, a.count, begin * STEP_K<T>);
    lb.init((const T *)b.p, b.stride, n0, b.count, begin * STEP_K<T>);
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(lds));
    constexpr int LOADS_A = decltype(la)::LOADS, LOADS = LOADS_A + decltype(lb)::LOADS;
    auto load = [&](int k, uint32_t place) {   // the k-th copy of a step
        if (k < LOADS_A) la.load(at + place, k);
        else lb.load(at + place + TILE::LDS_A, k - LOADS_A);
    };
    auto before = [&](uint32_t step) {
        if (TURN_A && rows && (step + 1) * STEP_K<T> > rows) la.clamp(a.stride, rows - step * STEP_K<T>);
    };
    auto after = [&] {
        la.base += la.advance;
        lb.base += lb.advance;
    };
    auto whole = [&](uint32_t step, uint32_t place) {
        before(step);
#pragma unroll
        for (int k = 0; k < LOADS; ++k) load(k, place);
        after();
    };
    // Half a step's fragments are read while the other half's are multiplied; a step's copies are in flight for the time of
    // one, from the barrier behind which no wavefront reads their place any more.  The matrix instructions take 16 cycles (of
    // 16 bits) and issue 4: the others stand between them, one at a time, in the order as it is written.
    u32x4 fa[2][TILE::TM], fb[2][TILE::TN];
    constexpr int CELLS = TILE::TM * TILE::TN;
    auto half = [&](auto cur, const lds_u8 *from, uint32_t s, auto between) {
        constexpr int C = decltype(cur)::value, X = C ^ 1, READS = TILE::TM + TILE::TN;
        unrolled<CELLS>([&](auto cell) {
            constexpr int c = decltype(cell)::value, i = c / TILE::TN, j = c % TILE::TN;
            multiply<T>(fa[C][i], fb[C][j], acc[i][j]);
            unrolled<READS>([&](auto read) {   // those that have their place here, B's first
                constexpr int r = decltype(read)::value;
                if constexpr (r * CELLS / READS != c) return;
                else if constexpr (r < TILE::TN) fb[X][r] = fragment<T, TURN_B, TILE::N>(from + TILE::LDS_A, wn * TILE::TN + r, s);
                else fa[X][r - TILE::TN] = fragment<T, TURN_A, TILE::M>(from, wm * TILE::TM + r - TILE::TN, s);
            });
            between(cell);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // (behind the last step the fragments are read from a place that holds another's: they are not used)
    auto body = [&](uint32_t step, auto loads) {
        const uint32_t place = ((step - begin) & 1) * TILE::STAGE;
        half(std::integral_constant<int, 0>{}, lds + place, 1, [](auto) {});
        wait_loads<0>();
        barrier();
        if (decltype(loads)::value) before(step + 2);
        half(std::integral_constant<int, 1>{}, lds + (place ^ TILE::STAGE), 0, [&](auto cell) {
            if constexpr (decltype(loads)::value)
                unrolled<LOADS>([&](auto copy) {
                    constexpr int k = decltype(copy)::value;
                    if constexpr ((2 * k + 1) * CELLS / (2 * LOADS) == decltype(cell)::value) load(k, place);
                });
        });
        if (decltype(loads)::value) after();
    };
    whole(begin, 0);
    if (begin + 1 < end) {
        whole(begin + 1, TILE::STAGE);
        wait_loads<LOADS>();
    } else {
        wait_loads<0>();
    }
    barrier();
#pragma unroll
    for (int j = 0; j < TILE::TN; ++j) fb[0][j] = fragment<T, TURN_B, TILE::N>(lds + TILE::LDS_A, wn * TILE::TN + j, 0);
#pragma unroll
    for (int i = 0; i < TILE::TM; ++i) fa[0][i] = fragment<T, TURN_A, TILE::M>(lds, wm * TILE::TM + i, 0);
    uint32_t step = begin;
    for (; step + 2 < end; ++step) body(step, std::true_type{});
    for (; step < end; ++step) body(step, std::false_type{});
    barrier();
}

// The tile by rows of n, eight neighbours along m at a time: f(n, m, values), through LDS, 16 rows of every column of
// wavefronts in turn.  (A lane holds four neighbours of one row, so that it would write 8 bytes in each of 16 rows, or, in
// rows that no 8 bytes fit, element by element.)
template <class TILE, class F> __device__ __forceinline__ void by_rows(const f32x4 (&acc)[TILE::TM][TILE::TN], lds_u8 *lds, F f)
{
    constexpr uint32_t STRIDE = TILE::M * 4 + 16, ROWS = TILE::WN * 16, PER_ROW = TILE::M / VEC;
    static_assert(ROWS * STRIDE <= TILE::LDS, "a turn's rows");
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / TILE::WN, wn = wave % TILE::WN;
    unrolled<TILE::TN>([&](auto turn) {
        constexpr int j = decltype(turn)::value;
#pragma unroll
        for (int i = 0; i < TILE::TM; ++i)
            *(lds_f32x4 *)(lds + (wn * 16 + (lane & 15)) * STRIDE + ((wm * TILE::TM + i) * 16 + (lane >> 4) * 4) * 4) = acc[i][j];
        barrier();
#pragma unroll
        for (uint32_t k = 0; k < (ROWS * PER_ROW + TILE::THREADS - 1) / TILE::THREADS; ++k) {
            const uint32_t v = k * TILE::THREADS + threadIdx.x, row = v / PER_ROW, m = v % PER_ROW * VEC;
            if (ROWS * PER_ROW % TILE::THREADS && row >= ROWS) break;
            const lds_u8 *from = lds + row * STRIDE + m * 4;
            const f32x4 a = *(const lds_f32x4 *)from, b = *(const lds_f32x4 *)(from + 16);
            float x[VEC] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            f((row / 16 * TILE::TN + j) * 16 + row % 16, m, x);
        }
        barrier();
    });
}

// Workgroups go round the eight XCDs, each with an L2 of its own; so that neighbours in a block of tiles share one, XCD x
// takes the tiles from x * (all / 8) on, in bands of GROUP tiles of m that go along n; all tiles of a share of k before
// the next.  (Bands of 4, 6, 8, 16: loss of 8,192 rows x 131,328 x 4,096 bfloat16 6.09, 6.14, 6.40, 6.72 ms; with gradients 23.6,
// 23.5, 23.6, 24.4.)
constexpr uint32_t XCDS = 8, GROUP = 6, CUS = 256;
__device__ __forceinline__ void place_of(uint32_t tile, uint32_t m_tiles, uint32_t n_tiles, uint32_t &tm, uint32_t &tn)
{
    const uint32_t band = tile / (GROUP * n_tiles), in = tile % (GROUP * n_tiles);
    const uint32_t high = m_tiles - band * GROUP < GROUP ? m_tiles - band * GROUP : GROUP;
    tm = band * GROUP + in % high;
    tn = in / high;
}
// The workgroup's tile among `all`, ~0 for none.
__device__ __forceinline__ uint32_t tile_of(uint32_t id, uint32_t all)
{
    const uint32_t per = (all + XCDS - 1) / XCDS, i = id % XCDS * per + id / XCDS;
    return id / XCDS < per && i < all ? i : ~0u;
}

// Tiles of 256 x 256, of which one workgroup runs on a CU.  Where the last ones along n would be half empty or more they are 128
// wide, and come after all others, to fill the last round, if the last-level cache still holds the operand along m then
// (loss of 1,638 rows x 33,024 x 2,048 bfloat16: 207 -> 191 us; 600 x 131,328 x 4,096: 694 -> 758, whence in their places there).
// Up to a quarter of a round that is left at the end is cut into strips of 64 along n, so that it takes the time of a strip.
typedef Tile<2, 4, 8, 4> Big;
typedef Tile<2, 4, 8, 2> Half;
typedef Tile<2, 4, 8, 1> Strip;
constexpr uint32_t STRIPS = Big::N / Strip::N;

constexpr uint64_t CACHED = 192ull << 20;   // bytes, of 256 MiB

// f(tile, m0, n0) for the workgroup's tile of m_tiles along m, whose operand has m_bytes, and as many as n take along n, if it
// has one.
template <class TILE, class F> __device__ __forceinline__ void with_place(uint32_t m_tiles, uint64_t m_bytes, uint32_t n, F f)
{
    uint32_t n_tiles = (n + TILE::N - 1) / TILE::N, tm, tn;
    if constexpr (__is_same(TILE, Big)) {
        const uint32_t rest = n % Big::N;
        const bool half = n > Big::N && rest && rest <= Half::N;
        const uint32_t halves = half && m_bytes <= CACHED ? m_tiles : 0;
        n_tiles -= halves ? 1 : 0;
        uint32_t all = m_tiles * n_tiles;
        const uint32_t left = all % CUS, strips = all > CUS && left * STRIPS <= CUS ? left * STRIPS : 0;
        all -= strips / STRIPS;
        const uint32_t first = (all + XCDS - 1) / XCDS * XCDS;   // of those that take halves, then strips
        if (blockIdx.x >= first) {
            uint32_t i = blockIdx.x - first;
            if (i < halves) return f(Half{}, i * Big::M, n_tiles * Big::N);
            i -= halves;
            if (i >= strips) return;
            place_of(all + i / STRIPS, m_tiles, n_tiles, tm, tn);
            return f(Strip{}, tm * Big::M, tn * Big::N + i % STRIPS * Strip::N);
        }
        const uint32_t tile = tile_of(blockIdx.x, all);
        if (tile == ~0u) return;
        place_of(tile, m_tiles, n_tiles, tm, tn);
        if (half && (tn + 1) * Big::N > n) return f(Half{}, tm * Big::M, tn * Big::N);
        return f(Big{}, tm * Big::M, tn * Big::N);
    }
    const uint32_t tile = tile_of(blockIdx.x, m_tiles * n_tiles);
    if (tile == ~0u) return;
    place_of(tile, m_tiles, n_tiles, tm, tn);
    f(TILE{}, tm * TILE::M, tn * TILE::N);
}
// workgroups of a launch of up to so many tiles (of Big: the rounding before halves, and strips)
template <class TILE> inline uint32_t tile_blocks(uint32_t m_tiles, uint32_t n_tiles)
{
    const uint32_t all = (m_tiles * n_tiles + XCDS - 1) / XCDS * XCDS;
    return all + (__is_same(TILE, Big) ? XCDS + (all > CUS ? CUS : 0) : 0);
}

}  // namespace tt
