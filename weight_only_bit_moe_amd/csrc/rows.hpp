// Loads, stores and arithmetic of the row kernels: eight elements of a row at
// a time, at any alignment of the element's own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wave.hpp"

namespace wna16 {

namespace {

// 8 consecutive elements with the element's own alignment: rows of odd length
// start anywhere, and gfx950 loads and stores 16 bytes at any address.  (Shared
// with those of a row's end, a load of 16 bytes falls into four: combine_tokens, T =
// 4096, k = 8, H = 4096 took 75 us instead of 64.)
template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Pack8 { T v[8]; };
struct __attribute__((packed, aligned(1))) Codes8 { uint32_t lo, hi; };

// Zeros past the row's end.
template <class T>
__device__ __forceinline__ Pack8<T> load_pack8(const T *p, int left)
{
    Pack8<T> t;
    if (left >= 8) {
        t = *reinterpret_cast<const Pack8<T> *>(p);
    } else {
        asm("" : "+v"(p));      // another address to the compiler: it would share the loads
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t.v[j] = j < left ? p[j] : T{};
    }
    return t;
}

template <class T>
__device__ __forceinline__ void load8(const T *p, int left, float (&f)[8])
{
    const Pack8<T> t = load_pack8(p, left);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = to_float(t.v[j]);
}

// 16 bytes at any element, past the caches' replacement order (NT): for outputs larger than they are.
typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store_past(void *p, Words4 v)
{
    __builtin_nontemporal_store(v, static_cast<Words4 *>(p));
}

template <bool NT = false, class T>
__device__ __forceinline__ void store8(T *p, int left, const float (&f)[8])
{
    if (left >= 8) {
        Pack8<T> t;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t.v[j] = from_float<T>(f[j]);
        if constexpr (!NT) {
            *reinterpret_cast<Pack8<T> *>(p) = t;
        } else {
            struct { Words4 w[sizeof(T) / 2]; } u = __builtin_bit_cast(decltype(u), t);
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k)
                store_past(reinterpret_cast<char *>(p) + 16 * k, u.w[k]);
        }
    } else {
        asm("" : "+v"(p));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left)
                p[j] = from_float<T>(f[j]);
    }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// sigmoid(x) to about 4 ulp.  exp(-x) = 2^t (1 + e ln 2): t = -x log2(e) rounded,
// and e its rounding error, which a large |x| would otherwise blow up.  Beyond
// 10^4 the result is 0 or 1 either way; the limit keeps e finite.
__device__ __forceinline__ float sigmoid(float x)
{
    constexpr float kLog2e = 1.44269502e+0f, kLow = 1.92596303e-8f, kLn2 = 0.693147181f;
    x = __builtin_amdgcn_fmed3f(x, -1e4f, 1e4f);
    const float t = -x * kLog2e;
    const float e = __builtin_fmaf(-x, kLow, __builtin_fmaf(-x, kLog2e, -t));
    const float p = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(e, kLn2, 1.f);
    return __builtin_amdgcn_rcpf(1.f + p);          // the hardware reciprocal (1 ulp; 1 / inf = 0)
}

}  // namespace

}  // namespace wna16
