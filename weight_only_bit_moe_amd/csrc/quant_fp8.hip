// Rows in 8-bit floating point (e4m3) with a power-of-two scale for each 128
// elements, of the rows themselves or of their SwiGLU.
//
// With m = max |v| of a block:
//   s = 2^ceil(log2(m / 448)),  q = v / s rounded to e4m3 (nearest even).
// 448 = 0.875 * 2^9 is the largest e4m3 value, so s is the smallest power of two
// under which the block fits.  Dividing by it is exact, and e4m3 has the same
// relative step at every exponent: a finer scale would change which bits are
// rounded away but not how many, and the only values that lose more are those
// below 2^-14 of the block's largest.  So a code has one rounding, of the
// value itself, and is defined bit for bit.  s comes from the bits of m: its
// exponent, one more where the mantissa is above 1.75.
//
// One pass over memory: 16 lanes hold a block, 8 elements each, and take its
// maximum by lane permutes; every input is read once and every output written
// once.  Memory bounds it: T = 8192, I = 2048 SwiGLU (84 MB) 20 us = 4.2 TB/s; T = 2047, K =
// 4096 (25 MB, most of it from the last-level cache or on its way there) 6.1 us with its
// launch = 4.1 TB/s.
#include <hip/hip_runtime.h>

#include "moe_wna16.h"
#include "expert_ops.hpp"
#include "rows.hpp"
#include "wave.hpp"

namespace wna16 {

namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// Biased exponent of a block's scale from the bits of its largest magnitude
// (finite): at least 1, so that the scale and its inverse are normal numbers.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top)
{
    const uint32_t e = (top + 0x1fffffu) >> 23;     // 1.75 = mantissa 0x600000: no carry up to it
    return e > 9u ? e - 8u : 1u;
}

// Eight values times mult as e4m3 codes, |value * mult| <= 448.
__device__ __forceinline__ Codes8 to_e4m3(const float (&v)[8], float mult)
{
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * mult, v[1] * mult, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * mult, v[3] * mult, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * mult, v[5] * mult, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * mult, v[7] * mult, hi, true);
    return Codes8{(uint32_t)lo, (uint32_t)hi};
}

template <class T, bool SWIGLU>
__global__ void __launch_bounds__(256) quant_fp8_kernel(QuantArgs a)
{
    // 16 lanes a block: those of a row's last block past its end hold zeros
    const uint32_t id = blockIdx.x * 16u + (threadIdx.x >> 4);
    const uint32_t row = id / (uint32_t)a.blocks, b = id - row * (uint32_t)a.blocks;
    if (row >= (uint32_t)a.T)
        return;                                     // whole rows of 16 lanes
    const int c = (int)b * 128 + (int)(threadIdx.x & 15) * 8, left = a.n - c;
    const T *x = static_cast<const T *>(a.x) + (long long)row * a.x_stride + c;
    float v[8];
    load8(x, left, v);
    if constexpr (SWIGLU) {
        float u[8];
        load8(x + a.n, left, u);
        const bool clamped = a.clamp < INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float gc = v[j], uc = u[j];
            if (clamped) {      // comparisons that keep a NaN (fminf would drop it)
                gc = gc > a.clamp ? a.clamp : gc;
                uc = uc > a.clamp ? a.clamp : uc;
                uc = uc < -a.clamp ? -a.clamp : uc;
            }
            v[j] = gc * sigmoid(a.alpha * gc) * (uc + a.beta);
        }
    }
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        top = larger(top, magnitude(v[j]));
    top = each_row_max(top);
    const bool fine = top < kInfBits;
    if (!fine) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = 0.f;
    }
    const uint32_t e = scale_exponent(fine ? top : 0u);
    const Codes8 q = to_e4m3(v, __uint_as_float((254u - e) << 23));
    uint8_t *o = a.q + (long long)row * a.q_stride + c;
    if (left >= 8) {
        *reinterpret_cast<Codes8 *>(o) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left)
                o[j] = (uint8_t)((j < 4 ? q.lo : q.hi) >> (8 * (j & 3)));
    }
    if ((threadIdx.x & 15) == 0)
        a.scale[(long long)row * a.s_stride + b] = __uint_as_float(fine ? e << 23 : 0x7fc00000u);
}

template <bool SWIGLU>
hipError_t launch_quant(const QuantArgs &a, int dtype, hipStream_t stream)
{
    const dim3 grid((unsigned)(((long long)a.T * a.blocks + 15) / 16));
    if (dtype == MOE_WNA16_BF16)
        return launch(quant_fp8_kernel<Bf16, SWIGLU>, grid, 256, stream, a);
    if (dtype == MOE_WNA16_FP16)
        return launch(quant_fp8_kernel<Fp16, SWIGLU>, grid, 256, stream, a);
    return launch(quant_fp8_kernel<float, SWIGLU>, grid, 256, stream, a);
}

}  // namespace

hipError_t launch_quant_fp8(const QuantArgs &args, bool swiglu, int dtype, hipStream_t stream)
{
    QuantArgs a = args;
    a.blocks = (a.n + 127) / 128;
    return swiglu ? launch_quant<true>(a, dtype, stream) : launch_quant<false>(a, dtype, stream);
}

}  // namespace wna16
