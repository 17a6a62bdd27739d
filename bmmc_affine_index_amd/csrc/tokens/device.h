// device.h -- typed vectors for the kernels on token rows (gfx950).
//
// Rows start at any element: an odd width or a view leaves them unaligned.
// Global memory takes 16-byte accesses at any address here, so the vectors
// below carry only their element's alignment, and one form serves aligned and
// unaligned rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bmmc {
namespace dev {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <typename T> struct Lanes {
    static constexpr int N = 16 / sizeof(T);  // elements of one 16-byte vector
};

template <typename T, int N> struct Vec {
    typedef T raw __attribute__((ext_vector_type(N)));
    typedef raw packed __attribute__((aligned(sizeof(T))));
    raw v;
};

template <int N> using Floats = float __attribute__((ext_vector_type(N)));

// NT: the data is streamed, past the caches' other lines (see by_hint).
template <typename T, int N, bool NT = true>
__device__ __forceinline__ Vec<T, N> load(const T *p) {
    const typename Vec<T, N>::packed *q = reinterpret_cast<const typename Vec<T, N>::packed *>(p);
    Vec<T, N> r;
    if constexpr (NT)
        r.v = __builtin_nontemporal_load(q);
    else
        r.v = *q;
    return r;
}

template <typename T, int N, bool NT = true>
__device__ __forceinline__ void store(T *p, const Vec<T, N> &x) {
    typename Vec<T, N>::packed *q = reinterpret_cast<typename Vec<T, N>::packed *>(p);
    if constexpr (NT)
        __builtin_nontemporal_store((typename Vec<T, N>::packed)x.v, q);
    else
        *q = x.v;
}

// body(streamed?) by a flag that all lanes share, for loads and stores that are
// streamed or not.  Streaming keeps what is read once out of the way, worth 5
// to 10% on arrays beyond the 256 MiB of the last cache.  Two things speak
// against it: data that was just written is read faster from the caches, and a
// line written in parts, as by rows that are not whole lines, is put together
// only in a cache.
//
// The empty statements keep the two bodies apart: the compiler takes loads that
// differ in nothing but the hint for the same, and drops it.
template <bool B> struct Flag {
    static constexpr bool value = B;
};
template <class F> __device__ __forceinline__ void by_hint(bool streamed, F body) {
    if (streamed) {
        asm volatile("");
        body(Flag<true>());
        asm volatile("");
    } else {
        body(Flag<false>());
    }
}

template <typename T, int N> __device__ __forceinline__ Floats<N> widen(const Vec<T, N> &x) {
    return __builtin_convertvector(x.v, Floats<N>);
}

// One rounding to nearest, ties to even.
template <typename T, int N> __device__ __forceinline__ Vec<T, N> narrow(const Floats<N> &x) {
    Vec<T, N> r;
    r.v = __builtin_convertvector(x, typename Vec<T, N>::raw);
    return r;
}

// Sum over the 64 lanes of a wave, the same in every lane (every lane active).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

}  // namespace dev
}  // namespace bmmc
