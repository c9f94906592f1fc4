// Element types, wave-wide reductions and the launch shared by the operators'
// kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace wna16 {

namespace {

struct Bf16 { uint16_t u; };
struct Fp16 { uint16_t u; };

__device__ __forceinline__ float to_float(Bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float to_float(Fp16 v)
{
    return (float)__builtin_bit_cast(_Float16, v.u);
}
__device__ __forceinline__ float to_float(float v) { return v; }

// Rounded to nearest even.
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ Bf16 from_float<Bf16>(float v)
{
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)v)};
}
template <> __device__ __forceinline__ Fp16 from_float<Fp16>(float v)
{
    return Fp16{__builtin_bit_cast(uint16_t, (_Float16)v)};
}
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }

// Lane permutes without LDS (DPP).  The steps kXor1, kXor2, kHalfMirror,
// kMirror reduce a row of 16 lanes: after each, the lanes of a block of 2, 4, 8,
// 16 hold the same value, so a mirror serves where an exchange of halves would.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) { return (uint32_t)dpp<CTRL>((int)v); }
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp(uint64_t v)
{
    return (uint64_t)dpp<CTRL>((uint32_t)(v >> 32)) << 32 | dpp<CTRL>((uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    return __builtin_bit_cast(double, dpp<CTRL>(__builtin_bit_cast(uint64_t, v)));
}

__device__ __forceinline__ int lane_value(int v, int lane)
{
    return __builtin_amdgcn_readlane(v, lane);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane)
{
    return (uint32_t)lane_value((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __int_as_float(lane_value(__float_as_int(v), lane));
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane)
{
    return (uint64_t)lane_value((uint32_t)(v >> 32), lane) << 32 | lane_value((uint32_t)v, lane);
}
__device__ __forceinline__ double lane_value(double v, int lane)
{
    return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, v), lane));
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }

// Over the rows of 16 lanes, the first row's result on every lane; then over
// the wave.  All 64 lanes must be active.
template <class C>
__device__ __forceinline__ C each_row_max(C v)
{
    v = larger(v, dpp<kXor1>(v));
    v = larger(v, dpp<kXor2>(v));
    v = larger(v, dpp<kHalfMirror>(v));
    return larger(v, dpp<kMirror>(v));
}
template <class C>
__device__ __forceinline__ C each_row_sum(C v)
{
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    v += dpp<kHalfMirror>(v);
    return v + dpp<kMirror>(v);
}
template <class C>
__device__ __forceinline__ C row_max(C v) { return lane_value(each_row_max(v), 0); }
template <class C>
__device__ __forceinline__ C row_sum(C v) { return lane_value(each_row_sum(v), 0); }
template <class C>
__device__ __forceinline__ C wave_max(C v)
{
    v = each_row_max(v);
    if constexpr (std::is_same<C, uint32_t>::value) {
        // kept in scalar registers: what follows is then scalar too
        uint32_t a = larger(lane_value(v, 0), lane_value(v, 16));
        uint32_t b = larger(lane_value(v, 32), lane_value(v, 48));
        asm("" : "+s"(a), "+s"(b));
        uint32_t r = larger(a, b);
        asm("" : "+s"(r));
        return r;
    }
    return larger(larger(lane_value(v, 0), lane_value(v, 16)),
                  larger(lane_value(v, 32), lane_value(v, 48)));
}
template <class C>
__device__ __forceinline__ C wave_sum(C v)
{
    v = each_row_sum(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Launches kernel(args...), and returns this launch's own status: an error that
// an earlier call on the thread left behind is neither reported nor cleared.
template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, hipStream_t stream, P... args)
{
    void *p[] = {&args...};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, dim3((unsigned)threads), p,
                           0, stream);
}

}  // namespace

}  // namespace wna16
