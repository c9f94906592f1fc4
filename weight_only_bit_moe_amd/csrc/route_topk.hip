// Expert routing: router logits -> the expert ids and routing weights that
// the routed layer reads.
//
//   p = softmax(l) or sigmoid(l);  c = p + bias (the bias picks, it does not weigh)
//   groups: a group's score is the sum of its two largest c; only the experts
//           of the topk_groups best groups can be picked
//   ids:    the topk largest c, largest first, ties to the lower index
//   w_j = p[ids_j] / sum_i p[ids_i] * scale   (without the sum if not renormalised)
//
// An expert whose logit is -inf or NaN, or whose c is, is out: it is never
// picked.  When fewer than topk experts can be picked, the remaining slots get
// id -1 and weight 0, which the routed layer skips.  A logit of +inf counts as
// the largest finite one.
//
// Which of two nearly equal c is ahead decides which expert runs, so p, c and
// the groups' sums are carried in 64 bits: two experts swap only if they agree
// to about 2^-52.  Without bias and groups the order of c is the order of the
// logits, so no p is computed before the experts are picked.
//
// One wave owns a token; lane i holds experts [i*EPL, (i+1)*EPL).  Picking is
// topk rounds of a wave-wide maximum over order-preserving 64-bit keys, each
// round taking the lowest lane and slot that hold the maximum.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "moe_wna16.h"
#include "ops.hpp"

namespace wna16 {

namespace {

constexpr int kWaves = 4;   // tokens per workgroup

struct RBf16 { uint16_t u; };
struct RFp16 { uint16_t u; };
__device__ __forceinline__ float logit(RBf16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float logit(RFp16 v) { return (float)__builtin_bit_cast(_Float16, v.u); }
__device__ __forceinline__ float logit(float v) { return v; }

// Order-preserving map of the doubles above -inf to integers above 0; out
// (0) for -inf and NaN.  -0 and +0 get the same key.
__device__ __forceinline__ uint64_t key_of(double c)
{
    if (!(c > -(double)INFINITY))
        return 0;
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m)
{
    return __builtin_bit_cast(uint64_t, __shfl_xor(__builtin_bit_cast(double, v), m));
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = shfl_xor64(v, m);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        v += __shfl_xor(v, m);
    return v;
}

template <bool SOFTMAX>
__device__ __forceinline__ double score_of(float l, float top)
{
    if constexpr (SOFTMAX)
        return exp((double)l - (double)top);
    else
        return 1.0 / (1.0 + exp(-(double)l));
}

template <class T, int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(64 * kWaves) route_topk_kernel(RouteArgs a)
{
    // the groups' stage reads every c of the token: one row per wave
    __shared__ double s_c[kWaves][64 * EPL];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tok = blockIdx.x * kWaves + wave;
    if (tok >= a.T)
        return;                                     // waves share nothing: no barrier below
    const T *row = static_cast<const T *>(a.logits) + tok * a.stride;
    const int e0 = lane * EPL;
    float l[EPL];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        l[j] = e0 + j < a.E ? logit(row[e0 + j]) : -INFINITY;
        l[j] = l[j] > -INFINITY ? (l[j] > FLT_MAX ? FLT_MAX : l[j]) : -INFINITY;
        top = l[j] > top ? l[j] : top;
    }
    uint64_t key[EPL];
    const bool by_score = a.bias != nullptr || a.groups > 1;
    double sum = 1.0;
    if (SOFTMAX) {
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const float o = __shfl_xor(top, m);
            top = o > top ? o : top;
        }
    }
    if (by_score || (SOFTMAX && !a.renormalize)) {
        double p[EPL];
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            p[j] = l[j] > -INFINITY ? score_of<SOFTMAX>(l[j], top) : 0.0;
            part += p[j];
        }
        if (SOFTMAX)
            sum = wave_sum(part);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            double c = SOFTMAX ? p[j] / sum : p[j];
            if (a.bias && e0 + j < a.E)
                c += (double)a.bias[e0 + j];
            p[j] = l[j] > -INFINITY ? c : -(double)INFINITY;
            key[j] = key_of(p[j]);
        }
        if (a.groups > 1) {
            const int per = a.E / a.groups;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                s_c[wave][e0 + j] = key[j] ? p[j] : -(double)INFINITY;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            // lane g: the two largest of group g
            double one = -(double)INFINITY, two = -(double)INFINITY;
            if (lane < a.groups)
                for (int i = 0; i < per; ++i) {
                    const double c = s_c[wave][lane * per + i];
                    two = c > one ? one : (c > two ? c : two);
                    one = c > one ? c : one;
                }
            const double score = two > -(double)INFINITY ? one + two : one;
            int ahead = 0;
            for (int g = 0; g < a.groups; ++g) {
                const double o = __shfl(score, g);
                ahead += o > score || (o == score && g < lane) ? 1 : 0;
            }
            const uint64_t keep = __ballot(lane < a.groups && ahead < a.topk_groups);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e0 + j < a.E && !((keep >> ((e0 + j) / per)) & 1))
                    key[j] = 0;
        }
    }
    if (!by_score) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = key_of((double)l[j]);
    }
    // lane r keeps the r-th picked expert
    int mine = -1;
    for (int r = 0; r < a.topk; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            best = key[j] > best ? key[j] : best;
        const uint64_t all = wave_max(best);
        if (all == 0)
            break;
        const int win = __ffsll((unsigned long long)__ballot(best == all)) - 1;
        int at = 0;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
            at = key[j] == all ? j : at;
        at = __builtin_amdgcn_readlane(at, win);
        if (lane == r)
            mine = win * EPL + at;
        if (lane == win) {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                key[j] = j == at ? 0 : key[j];
        }
    }
    double p = 0.0;
    if (mine >= 0) {
        float x = logit(row[mine]);
        x = x > FLT_MAX ? FLT_MAX : x;
        p = score_of<SOFTMAX>(x, top);
    }
    // the softmax's own sum cancels when the weights are renormalised
    double w = p / (a.renormalize ? wave_sum(p) : sum) * (double)a.scale;
    if (!(p > 0.0))
        w = 0.0;
    if (lane < a.topk) {
        const long long o = (long long)tok * a.topk + lane;
        a.ids[o] = mine;
        a.weights[o] = (float)w;
    }
}

template <class T, bool SOFTMAX>
void launch_epl(const RouteArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
    const int epl = (a.E + 63) / 64;
    if (epl <= 1)
        route_topk_kernel<T, 1, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(a);
    else if (epl <= 2)
        route_topk_kernel<T, 2, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(a);
    else if (epl <= 4)
        route_topk_kernel<T, 4, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(a);
    else if (epl <= 8)
        route_topk_kernel<T, 8, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(a);
    else
        route_topk_kernel<T, 16, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs &a, int dtype, int score, hipStream_t stream)
{
    const bool softmax = score == MOE_WNA16_SOFTMAX;
    if (dtype == MOE_WNA16_BF16)
        softmax ? launch_epl<RBf16, true>(a, stream) : launch_epl<RBf16, false>(a, stream);
    else if (dtype == MOE_WNA16_FP16)
        softmax ? launch_epl<RFp16, true>(a, stream) : launch_epl<RFp16, false>(a, stream);
    else
        softmax ? launch_epl<float, true>(a, stream) : launch_epl<float, false>(a, stream);
    return hipGetLastError();
}

}  // namespace wna16
