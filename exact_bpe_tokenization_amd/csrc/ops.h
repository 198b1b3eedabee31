// ops.h -- shared parts of the token operators (embed.hip, loss.hip, sample.hip): element types,
// vectors of eight elements, reductions over a workgroup and the argument checks.
#pragma once
#include "../../include/toktier.h"
#include "internal.h"

namespace tt {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Rows start at any multiple of the element size: 16-byte accesses with the alignment of two bytes, which
// global memory takes on gfx950 (one global_load_dwordx4 / global_store_dwordx4 all the same).
typedef u32x4 u32x4_row __attribute__((aligned(2), may_alias));

constexpr int VEC = 8;   // elements of a vector: 16 bytes of a 16-bit type, 2 x 16 bytes of float

template <class T> struct Vec { u32x4 a; };
template <> struct Vec<float> { u32x4 a, b; };

template <class T> __device__ __forceinline__ Vec<T> load_vec(const T *p)
{
    Vec<T> v;
    v.a = *(const u32x4_row *)p;
    if constexpr (sizeof(T) == 4) v.b = *(const u32x4_row *)(p + 4);
    return v;
}

// Element k (a compile-time index after unrolling) of a vector, as float.
template <class T> __device__ __forceinline__ float vec_at(const Vec<T> &v, int k)
{
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(float, k < 4 ? v.a[k] : v.b[k - 4]);
    } else if constexpr (__is_same(T, __bf16)) {
        const uint32_t w = v.a[k >> 1];
        return __builtin_bit_cast(float, (k & 1) ? w & 0xFFFF0000u : w << 16);
    } else {
        const uint32_t w = v.a[k >> 1];
        return (float)__builtin_bit_cast(_Float16, (uint16_t)((k & 1) ? w >> 16 : w));
    }
}

// Eight floats rounded (to nearest even) to T.
template <class T> __device__ __forceinline__ Vec<T> to_vec(const float (&x)[VEC])
{
    Vec<T> v;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v.a[k] = __builtin_bit_cast(uint32_t, x[k]);
            v.b[k] = __builtin_bit_cast(uint32_t, x[k + 4]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v.a[k] = (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * k]) |
                     (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * k + 1]) << 16;
    }
    return v;
}

template <class T> __device__ __forceinline__ void store_vec(T *p, const Vec<T> &v)
{
    *(u32x4_row *)p = v.a;
    if constexpr (sizeof(T) == 4) *(u32x4_row *)(p + 4) = v.b;
}
template <class T> __device__ __forceinline__ void store_vec(T *p, const float (&x)[VEC]) { store_vec(p, to_vec<T>(x)); }

// Up to eight elements (n of them) where a row ends inside a vector.
template <class T> __device__ __forceinline__ void load_part(const T *p, uint32_t n, float fill, float (&x)[VEC])
{
    if (n >= VEC) {
        const Vec<T> v = load_vec(p);
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] = vec_at(v, k);
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[k] = k < (int)n ? (float)p[k] : fill;
}

// the same as a vector, zeros past the end
template <class T> __device__ __forceinline__ Vec<T> load_some(const T *p, uint32_t n)
{
    if (n >= VEC) return load_vec(p);
    float x[VEC];
    load_part(p, n, 0.f, x);
    return to_vec<T>(x);
}

// load_some past the caches, for what is read once
template <class T> __device__ __forceinline__ Vec<T> load_once(const T *p, uint32_t n)
{
    if (n < VEC) return load_some(p, n);
    Vec<T> v;
    v.a = __builtin_nontemporal_load((const u32x4_row *)p);
    if constexpr (sizeof(T) == 4) v.b = __builtin_nontemporal_load((const u32x4_row *)(p + 4));
    return v;
}

template <class T> __device__ __forceinline__ void store_part(T *p, uint32_t n, const float (&x)[VEC])
{
    if (n >= VEC) {
        store_vec(p, x);
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k)
        if (k < (int)n) p[k] = (T)x[k];
}

// store_part past the caches, for what no kernel of this call reads again
template <class T> __device__ __forceinline__ void stream_part(T *p, uint32_t n, const float (&x)[VEC])
{
    if (n < VEC) return store_part(p, n, x);
    Vec<T> v = to_vec<T>(x);
    __builtin_nontemporal_store(v.a, (u32x4_row *)p);
    if constexpr (sizeof(T) == 4) __builtin_nontemporal_store(v.b, (u32x4_row *)(p + 4));
}

// Every lane's accesses before this point come before every lane's after it.  A wavefront's lanes run in step, so this
// is no instruction; it keeps the compiler from moving an access of one lane past another lane's of the same place, which
// within a lane would change nothing.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------------------------
// host side

int hip_status(hipError_t e);   // TOKTIER_OK, or E_HIP with the text kept for toktier_last_hip_error

inline uint32_t elem_size(int type)
{
    return type == TOKTIER_F32 ? 4u : type == TOKTIER_F16 || type == TOKTIER_BF16 ? 2u : 0u;
}

// A matrix argument: known type, a pointer at a multiple of the element, rows that do not overlap and
// whose byte extent fits the address space.
inline bool matrix_ok(const void *p, int type, uint64_t rows, uint64_t cols, uint64_t stride)
{
    const uint64_t sz = elem_size(type);
    if (!p || !sz || ((uintptr_t)p & (sz - 1)) || stride < cols) return false;
    return rows == 0 || stride <= (1ull << 46) / rows;
}

inline uint64_t extent(int type, uint64_t rows, uint64_t cols, uint64_t stride)
{
    return rows ? ((rows - 1) * stride + cols) * elem_size(type) : 0;
}

inline bool apart(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return !na || !nb || x + na <= y || y + nb <= x;
}

inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// A dimension of a grid holds fewer than 2^32 threads; a launch of more reports success and runs what is left of the
// number modulo 2^32.  Calls f(first block, blocks) for launches of at most 2^31 threads that make up `blocks`.
template <class F> inline void in_launches(uint64_t blocks, uint32_t threads, F f)
{
    const uint64_t most = (1ull << 31) / threads;
    for (uint64_t first = 0; first < blocks; first += most) f(first, (uint32_t)(blocks - first < most ? blocks - first : most));
}

// Calls f with a value of the element type as its argument.
template <class F> inline void with_type(int type, F f)
{
    if (type == TOKTIER_F32) f(float{});
    else if (type == TOKTIER_F16) f(_Float16{});
    else f(__bf16{});
}

}  // namespace tt
