// elements.hpp -- elements of token rows (float32, float16, bfloat16) in accesses of
// 16 bytes, and reductions over lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rs {

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------
using bf16 = __bf16;
using f16 = _Float16;

template <class T, int N>
struct VecOf {
    // Only element alignment is assumed: gfx950 serves unaligned 16-byte
    // global accesses, so odd widths and strides take the same wide path.
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte access

template <class T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = static_cast<float>(*p);
    } else {
        const auto v = *reinterpret_cast<const typename VecOf<T, N>::type *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = static_cast<float>(v[i]);
    }
}

// Rounds to nearest even where T is narrower than float: the one rounding
// of a result, after its sum in float.
template <class T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[N]) {
    if constexpr (N == 1) {
        *p = static_cast<T>(f[0]);
    } else {
        typename VecOf<T, N>::type v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = static_cast<T>(f[i]);
        *reinterpret_cast<typename VecOf<T, N>::type *>(p) = v;
    }
}

// The N elements at p, of which only the first `have` exist (zeros beyond).
template <class T, int N>
__device__ __forceinline__ void load_some(const T *p, int have, float (&f)[N]) {
    if (have >= N) {
        load_vec<T, N>(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = i < have ? static_cast<float>(p[i]) : 0.0f;
    }
}

template <class T, int N>
__device__ __forceinline__ void store_some(T *p, int have, const float (&f)[N]) {
    if (have >= N) {
        store_vec<T, N>(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < have) p[i] = static_cast<T>(f[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Reductions over a group of 16, 32 or 64 consecutive lanes; every lane of the
// group gets the result.  All 64 lanes of the wave must be active.
// ---------------------------------------------------------------------------
// (CTRL permutes the lanes of a row of 16: every lane has a source.)
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xF, 0xF, true));
}

template <int G, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t x, F f) {
    static_assert(G == 16 || G == 32 || G == 64);
    x = f(x, dpp<0xB1>(x));   // quad_perm: lane ^ 1
    x = f(x, dpp<0x4E>(x));   // quad_perm: lane ^ 2
    x = f(x, dpp<0x141>(x));  // row_half_mirror: the other quad of 8
    x = f(x, dpp<0x140>(x));  // row_mirror: the other half of 16
    if constexpr (G == 32) x = f(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
    if constexpr (G == 64) {
        const uint32_t a = f(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 0)),
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 16)));
        const uint32_t b = f(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 32)),
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 48)));
        x = f(a, b);
    }
    return x;
}

template <int G>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int G>
__device__ __forceinline__ uint32_t group_min_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

template <int G>
__device__ __forceinline__ uint32_t group_sum_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a + b; });
}

// NaN if a lane's x is one.
template <int G>
__device__ __forceinline__ float group_max(float x) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__builtin_elementwise_maximum(__uint_as_float(a), __uint_as_float(b)));
    }));
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

}  // namespace rs
