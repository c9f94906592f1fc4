// Row kernels around the routed layer: residual addition + root-mean-square
// norm (+ 8-bit output), and SwiGLU with 8-bit output.
//
// Both are one pass over memory: a workgroup owns a row, every thread keeps
// its share of the row in registers between the reduction and the output, so
// each input is read once and each output written once.  They are bound by
// HBM for many rows and by the launch and one memory round trip for few.
// Kernel durations (in a captured graph, one call after another, 1 to 5 us more):
//   norm, bf16, H = 4096, residual, 16- and 8-bit outputs:
//     T = 8192  52 us = 5.8 TB/s;  T = 4  3.2 us
//   SwiGLU, bf16, I = 2048:  T = 8192  18.1 us = 4.6 TB/s;  T = 64  3.4 us
// (a copy of 2 GiB runs at 4.8 TB/s; part of these rows comes from the last-level
// cache).  In a graph, FP32: norm T = 8192 104 us = 5.5 TB/s, SwiGLU 30.1 us = 5.0.
//
// 8-bit rows.  With v the row before its norm's factor and m = max |v|:
//   q = rint(v * (127 / m)),  scale = m * rstd / 127.
// The norm's factor rstd is the same for the whole row, so it cancels from the
// codes and enters the scale only: the codes need the maximum, not the sum of
// squares, and both reductions share one exchange.  127 / m is rounded once
// per row to FP32; |v * (127 / m)| <= 127 * (1 + 2^-23), so rint stays in
// [-127, 127] and needs no clamp.  A row whose m is below 2^-100 gets zero
// codes and scale 0 (its 127 / m would overflow further down).  The maximum is
// taken over the magnitude bits as integers, where a NaN ranks above infinity:
// a row with either gets zero codes and a NaN scale, which the product that
// reads the row carries into its whole output row.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_wna16.h"
#include "ops.hpp"
#include "rows.hpp"
#include "wave.hpp"

namespace wna16 {

namespace {

// rint(f * mult) as bytes.  Adding 1.5 * 2^23 to a float of magnitude below
// 2^22 rounds it to an integer (nearest even, as rint does) that the low bits
// then hold in two's complement; two permutes a pair of bytes pack them.
__device__ __forceinline__ void store_codes(int8_t *p, int left, const float (&f)[8], float mult)
{
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v = f[j] * mult;
        asm("" : "+v"(v));      // two roundings: not to be fused into one
        b[j] = __float_as_uint(v + 12582912.f);
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000c0cu);
        w[k] = lo | hi;
    }
    if (left >= 8) {
        *reinterpret_cast<Codes8 *>(p) = Codes8{w[0], w[1]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left)
                p[j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
}

// Sum and maximum over the workgroup (up to 16 waves), the same on every thread.
__device__ __forceinline__ void reduce(float &sum, uint32_t &top, int waves)
{
    __shared__ float s[16];
    __shared__ uint32_t t[16];
    const int lane = threadIdx.x & 63;
    sum = wave_sum(sum);
    top = wave_max(top);
    if (waves == 1)
        return;
    if (lane == 0) {
        s[threadIdx.x >> 6] = sum;
        t[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    sum = row_sum(lane < waves ? s[lane & 15] : 0.f);
    top = row_max(lane < waves ? t[lane & 15] : 0u);
}

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = 0x0d800000u;   // 2^-100

// Multiplier of a row's codes from the bits of its largest magnitude.
__device__ __forceinline__ float code_mult(uint32_t top)
{
    return top < kTinyBits || top >= kInfBits ? 0.f : 127.f / __uint_as_float(top);
}
__device__ __forceinline__ float code_scale(uint32_t top, float rstd)
{
    if (top >= kInfBits)
        return __uint_as_float(0x7fc00000u);
    return top < kTinyBits ? 0.f : __uint_as_float(top) * rstd / 127.f;
}

// The workgroup owns a row, R chunks of 8 elements a thread.
template <class T, int R>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(NormArgs a)
{
    const int NT = a.threads;
    const int row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *w = static_cast<const T *>(a.weight);
    const long long at = (long long)row * a.H;
    float h[R][8];
    float sum = 0.f;
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * NT + (int)threadIdx.x) * 8;
        load8(x + c, a.H - c, h[i]);
    }
    // Every load before the first store: a store could alias the weight, and the
    // load behind it would be another round trip.  (Longer rows reload it.)
    constexpr bool kHold = R <= 2;
    float wt[kHold ? R : 1][8];
    if constexpr (kHold) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            load8(w + c, a.H - c, wt[i]);
        }
    }
    if (a.residual) {
        const T *r = static_cast<const T *>(a.residual) + row * a.r_stride;
        // The norm reads the sum as the residual stream stores it, so that the
        // next step, which starts from the stored sum, sees the same rows.
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            float f[8];
            load8(r + c, a.H - c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[i][j] = to_float(from_float<T>(h[i][j] + f[j]));
        }
    }
    if (a.residual_out) {
        T *o = static_cast<T *>(a.residual_out) + at;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            store8(o + c, a.H - c, h[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * NT + (int)threadIdx.x) * 8;
        if constexpr (!kHold)
            load8(w + c, a.H - c, wt[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum += h[i][j] * h[i][j];
            h[i][j] *= wt[kHold ? i : 0][j];    // v from here on
            top = larger(top, magnitude(h[i][j]));
        }
    }
    reduce(sum, top, NT >> 6);
    const float rstd = 1.f / sqrtf(sum / (float)a.H + a.eps);
    if (a.y) {
        T *o = static_cast<T *>(a.y) + at;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = h[i][j] * rstd;
            store8(o + c, a.H - c, f);
        }
    }
    if (a.q) {
        const float mult = code_mult(top);
        int8_t *o = a.q + row * a.q_stride;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            if (mult == 0.f) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    h[i][j] = 0.f;              // no inf * 0 in the codes
            }
            store_codes(o + c, a.H - c, h[i], mult);
        }
        if (threadIdx.x == 0)
            a.scale[row] = code_scale(top, rstd);
    }
}

// load8 with each conversion beside its load: a pass of perf/operators.py's T = 8192, I = 2048
// takes 60.7 us, with the conversions behind both kinds of loads 61.8.  (The norm gains from
// those: T = 8192, H = 1001 15.9 against 16.3 us.)
template <class T>
__device__ __forceinline__ void load8_each(const T *p, int left, float (&f)[8])
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

template <class T, int R>
__global__ void __launch_bounds__(1024) swiglu_quant_kernel(SwigluArgs a)
{
    const int NT = a.threads;
    const int row = blockIdx.x;
    const T *g = static_cast<const T *>(a.gu) + row * a.gu_stride;
    const T *u = g + a.I;
    const bool clamped = a.clamp < INFINITY;
    float v[R][8], f[R][8];
    float sum = 0.f;
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * NT + (int)threadIdx.x) * 8;
        load8_each(g + c, a.I - c, v[i]);
        load8_each(u + c, a.I - c, f[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float gc = v[i][j], uc = f[i][j];
            if (clamped) {      // comparisons that keep a NaN (fminf would drop it)
                gc = gc > a.clamp ? a.clamp : gc;
                uc = uc > a.clamp ? a.clamp : uc;
                uc = uc < -a.clamp ? -a.clamp : uc;
            }
            // past the row's end gate and up are 0, and so is the result
            v[i][j] = gc * sigmoid(a.alpha * gc) * (uc + a.beta);
            top = larger(top, magnitude(v[i][j]));
        }
    }
    reduce(sum, top, NT >> 6);
    const float mult = code_mult(top);
    int8_t *o = a.q + row * a.q_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * NT + (int)threadIdx.x) * 8;
        if (mult == 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.f;
        }
        store_codes(o + c, a.I - c, v[i], mult);
    }
    if (threadIdx.x == 0)
        a.scale[row] = code_scale(top, 1.f);
}

// Threads and chunks a thread for rows of n elements: one chunk a thread up to
// 1024 threads.  More waves with less each keep more loads in flight: T = 8192,
// H = 4096 takes 57 us with one chunk a thread, 63 us with two, 71 us with four (in
// a captured graph).
template <class F>
hipError_t with_shape(int n, F &&f)
{
    const int chunks = (n + 7) / 8;
    if (chunks <= 1024)
        return f((chunks + 63) / 64 * 64, std::integral_constant<int, 1>{});
    if (chunks <= 2048)
        return f(1024, std::integral_constant<int, 2>{});
    return f(1024, std::integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs &args, int dtype, hipStream_t stream)
{
    return with_shape(args.H, [&](int nt, auto r) {
        NormArgs a = args;
        a.threads = nt;
        constexpr int R = decltype(r)::value;
        if (dtype == MOE_WNA16_BF16)
            return launch(add_rmsnorm_kernel<Bf16, R>, dim3(a.T), nt, stream, a);
        if (dtype == MOE_WNA16_FP16)
            return launch(add_rmsnorm_kernel<Fp16, R>, dim3(a.T), nt, stream, a);
        return launch(add_rmsnorm_kernel<float, R>, dim3(a.T), nt, stream, a);
    });
}

hipError_t launch_swiglu_quant(const SwigluArgs &args, int dtype, hipStream_t stream)
{
    return with_shape(args.I, [&](int nt, auto r) {
        SwigluArgs a = args;
        a.threads = nt;
        constexpr int R = decltype(r)::value;
        if (dtype == MOE_WNA16_BF16)
            return launch(swiglu_quant_kernel<Bf16, R>, dim3(a.T), nt, stream, a);
        if (dtype == MOE_WNA16_FP16)
            return launch(swiglu_quant_kernel<Fp16, R>, dim3(a.T), nt, stream, a);
        return launch(swiglu_quant_kernel<float, R>, dim3(a.T), nt, stream, a);
    });
}

}  // namespace wna16
