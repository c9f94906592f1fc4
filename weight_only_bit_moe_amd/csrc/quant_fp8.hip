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
// once.  Memory bounds it: T = 8192, I = 2048 SwiGLU (84 MB) 17.3 us = 4.9 TB/s; T = 2047, K =
// 4096 (25 MB) 6.2 us = 4.1 TB/s.  The SwiGLU's arithmetic is nearly as long: the vector
// units were 97 % busy at 19.1 us, when the clamps had a branch and took the detour that
// keeps a NaN; NaNs are now looked for beside them, into scalar masks.
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

// The larger of top, |a| and |b|, none of them a NaN that counts.
__device__ __forceinline__ float largest(float top, float a, float b)
{
    float r;
    asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(top), "v"(a), "v"(b));
    return r;
}

// One instruction, where fminf takes a second for signalling NaNs.
__device__ __forceinline__ float smaller(float a, float b)
{
    float r;
    asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// Where a block's elements, codes and scale are: elements from the start of x, q
// and scale.
struct Place {
    long long x, q, s;
    int c;                      // the lane's first element in its row
    bool here;
};

// A wave has four blocks in turn.  A row of four or more ends at most once among them:
// its place is worked out once for the wave, and a lane behind the end adds a stride.
__device__ __forceinline__ Place place_of(const QuantArgs &a)
{
    const int lane = threadIdx.x & 63;
    const uint32_t id0 =
        (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * 16u + (threadIdx.x >> 6) * 4u));
    const uint32_t n = (uint32_t)a.blocks, sub = (uint32_t)lane >> 4;
    Place p;
    if (n >= 4) {
        // id0 / n, as set by the launch
        const uint32_t row0 = __umulhi(id0, a.magic) >> a.shift, b0 = id0 - row0 * n;
        const bool next = b0 + sub >= n;
        const uint32_t b = b0 + sub - (next ? n : 0u);
        p.c = (int)b * 128 + (lane & 15) * 8;
        p.x = (long long)row0 * a.x_stride + (next ? a.x_stride : 0ll) + p.c;
        p.q = (long long)row0 * a.q_stride + (next ? a.q_stride : 0ll) + p.c;
        p.s = (long long)row0 * a.s_stride + (next ? a.s_stride : 0ll) + b;
        p.here = row0 + (next ? 1u : 0u) < (uint32_t)a.T;
    } else {
        const uint32_t row = (id0 + sub) / n, b = id0 + sub - row * n;
        p.c = (int)b * 128 + (lane & 15) * 8;
        p.x = (long long)row * a.x_stride + p.c;
        p.q = (long long)row * a.q_stride + p.c;
        p.s = (long long)row * a.s_stride + b;
        p.here = row < (uint32_t)a.T;
    }
    return p;
}

template <class T, bool SWIGLU>
__global__ void __launch_bounds__(256) quant_fp8_kernel(QuantArgs a)
{
    // 16 lanes a block: those of a row's last block past its end hold zeros
    const Place at = place_of(a);
    if (!at.here)
        return;                                     // whole rows of 16 lanes
    const int left = a.n - at.c;
    const T *x = static_cast<const T *>(a.x) + at.x;
    float v[8];
    load8(x, left, v);
    uint64_t odd = 0;                               // lanes with a NaN
    if constexpr (SWIGLU) {
        float u[8];
        load8(x + a.n, left, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            odd |= __ballot(__builtin_isunordered(v[j], u[j]));
            v[j] = smaller(v[j], a.clamp);          // these may drop a NaN
            u[j] = __builtin_amdgcn_fmed3f(u[j], -a.clamp, a.clamp);
            v[j] = v[j] * sigmoid(a.alpha * v[j]) * (u[j] + a.beta);
        }
    }
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        odd |= __ballot(__builtin_isunordered(v[j], v[j + 1]));
        most = largest(most, v[j], v[j + 1]);
    }
    const uint32_t top =
        each_row_max(__builtin_amdgcn_inverse_ballot_w64(odd) ? kInfBits : __float_as_uint(most));
    const bool fine = top < kInfBits;
    const uint32_t e = scale_exponent(fine ? top : 0u);
    Codes8 q = to_e4m3(v, __uint_as_float((254u - e) << 23));
    q.lo = fine ? q.lo : 0u;
    q.hi = fine ? q.hi : 0u;
    uint8_t *o = a.q + at.q;
    if (left >= 8) {
        *reinterpret_cast<Codes8 *>(o) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left)
                o[j] = (uint8_t)((j < 4 ? q.lo : q.hi) >> (8 * (j & 3)));
    }
    if ((threadIdx.x & 15) == 0)
        a.scale[at.s] = __uint_as_float(fine ? e << 23 : 0x7fc00000u);
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
    // id / blocks = id * magic / 2^(32 + shift): 2^shift < blocks <= 2^(shift + 1) and an
    // excess of magic * blocks over 2^(32 + shift) below blocks, so exact for id < 2^31
    while ((2 << a.shift) < a.blocks)
        ++a.shift;
    a.magic = (uint32_t)(((1ull << (32 + a.shift)) + a.blocks - 1) / a.blocks);
    return swiglu ? launch_quant<true>(a, dtype, stream) : launch_quant<false>(a, dtype, stream);
}

}  // namespace wna16
