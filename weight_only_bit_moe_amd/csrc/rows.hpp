// Loads, stores and arithmetic of the row kernels: eight elements of a row at
// a time, at any alignment of the element's own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wave.hpp"

namespace wna16 {

namespace {

// 8 consecutive elements with the element's own alignment: rows of odd length
// start anywhere, and gfx950 loads and stores 16 bytes at any address.
template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Pack8 { T v[8]; };
struct __attribute__((packed, aligned(1))) Codes8 { uint32_t lo, hi; };

template <class T>
__device__ __forceinline__ void load8(const T *p, int left, float (&f)[8])
{
    if (left >= 8) {
        const Pack8<T> t = *reinterpret_cast<const Pack8<T> *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = to_float(t.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = j < left ? to_float(p[j]) : 0.f;
    }
}

template <class T>
__device__ __forceinline__ void store8(T *p, int left, const float (&f)[8])
{
    if (left >= 8) {
        Pack8<T> t;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t.v[j] = from_float<T>(f[j]);
        *reinterpret_cast<Pack8<T> *>(p) = t;
    } else {
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
