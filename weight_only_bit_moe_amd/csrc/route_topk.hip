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
// Which of two nearly equal c is ahead decides which expert runs, so the order
// is that of 64-bit scores: two experts swap only if they agree to about 2^-52.
// Most tokens need no 64-bit score for it.  The scores are first taken in
// 32 bits, where they are off by less than 2^-19 (1 + |c|), and the token keeps
// that order if every comparison that mattered was wider than the two errors:
// consecutive picks, the last pick and the first expert left out, and any two
// groups.  Otherwise the wave repeats the picking in 64 bits.  Without bias and
// groups the order of c is the order of the logits, which is exact in 32 bits.
// The weights of the picked experts are always computed in 64 bits.
//
// One wave owns a token; lane i holds experts [i*EPL, (i+1)*EPL).  Picking is
// rounds of a wave-wide maximum (DPP, no LDS), each taking the lowest lane and
// slot that hold the maximum.  With one token the time is the chain of memory
// round trips and reductions; with many it is the VALU instructions per token.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "moe_wna16.h"
#include "ops.hpp"
#include "wave.hpp"

namespace wna16 {

namespace {

constexpr int kWaves = 4;   // tokens per workgroup

// exp(l - top) or sigmoid(l)
template <bool SOFTMAX>
__device__ __forceinline__ double score_of(float l, float top, double)
{
    if constexpr (SOFTMAX)
        return exp((double)l - (double)top);
    else
        return 1.0 / (1.0 + exp(-(double)l));
}
template <bool SOFTMAX>
__device__ __forceinline__ float score_of(float l, float top, float)
{
    constexpr float kLog2e = 1.44269504f;
    if constexpr (SOFTMAX)
        return __builtin_amdgcn_exp2f((l - top) * kLog2e);
    else
        return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l * -kLog2e));
}

// Whether two 32-bit scores may be in another order in 64 bits.  A sigmoid is
// off by less than 4 FP32 roundings; a softmax by up to 8 of its own and 22 of
// the sum (16 scores a lane, then 6 steps); adding the bias is one more.  So a
// score is off by less than 2^-19 (1 + |c|), a group's sum of two by twice that.
__device__ __forceinline__ bool too_near(float a, float b, float tolerance)
{
    return __builtin_fabsf(a - b) <= tolerance * (1.f + __builtin_fabsf(b));
}
__device__ __forceinline__ bool too_near(double, double, float) { return false; }

template <class C, int EPL>
__device__ __forceinline__ C top_of(const C (&c)[EPL])
{
    C v = c[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j)
        v = larger(v, c[j]);
    return v;
}

// Takes the experts outside the best groups out of c.  Returns whether two
// groups were too near to tell apart.
template <class C, int EPL>
__device__ __forceinline__ bool keep_groups(C (&c)[EPL], const RouteArgs &a, int lane, C *row)
{
    const C kOut = -(C)INFINITY;
    const int per = a.E / a.groups, span = per / EPL;
    bool near = false;
    // a group's two largest; with one expert left (or one in all) that one
    auto total = [&](C one, C two) { return two > kOut ? one + two : one; };
    auto count = [&](C score, int mine, auto &&of) {
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g) {
            const C o = of(g);
            ahead += o > score || (o == score && g < mine) ? 1 : 0;
            near |= g != mine && o > kOut && score > kOut && too_near(o, score, 0x1p-17f);
        }
        return ahead;
    };
    if (span * EPL == per && (span == 2 || span == 4 || span == 8 || span == 16)) {
        // groups are whole runs of lanes: merge the lanes' pairs by permutes
        C one = kOut, two = kOut;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            two = c[j] > one ? one : larger(two, c[j]);
            one = larger(one, c[j]);
        }
        auto merge = [&](C o1, C o2) {
            two = o1 > one ? larger(one, o2) : larger(two, o1);
            one = larger(one, o1);
        };
        merge(dpp<kXor1>(one), dpp<kXor1>(two));
        if (span >= 4)
            merge(dpp<kXor2>(one), dpp<kXor2>(two));
        if (span >= 8)
            merge(dpp<kHalfMirror>(one), dpp<kHalfMirror>(two));
        if (span >= 16)
            merge(dpp<kMirror>(one), dpp<kMirror>(two));
        const C score = total(one, two);
        const int mine = lane / span;
        const int ahead = count(score, mine, [&](int g) { return lane_value(score, g * span); });
        if (ahead >= a.topk_groups) {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                c[j] = kOut;
        }
        near = near && mine < a.groups;
    } else {
        // any other shape: lane g reads group g's scores
        const int e0 = lane * EPL;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            row[e0 + j] = c[j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        C one = kOut, two = kOut;
        if (lane < a.groups)
            for (int i = 0; i < per; ++i) {
                const C v = row[lane * per + i];
                two = v > one ? one : larger(two, v);
                one = larger(one, v);
            }
        const C score = total(one, two);
        const int ahead = count(score, lane, [&](int g) { return lane_value(score, g); });
        const uint64_t keep = __ballot(lane < a.groups && ahead < a.topk_groups);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e0 + j < a.E && !((keep >> ((e0 + j) / per)) & 1))
                c[j] = kOut;
        near = near && lane < a.groups;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    return __ballot(near) != 0;
}

// Picks the topk largest of c: lane r gets the r-th pick and its logit.
// Returns whether two that had to be told apart were too near.
template <class C, int EPL>
__device__ __forceinline__ bool pick(C (&c)[EPL], const float (&l)[EPL], int topk, bool check,
                                     int lane, int &mine, float &logit_of_mine)
{
    const C kOut = -(C)INFINITY;
    mine = -1;
    bool near = false;
    C last = (C)INFINITY;
    const int rounds = check ? topk + 1 : topk;     // one more: the first left out
    for (int r = 0; r < rounds; ++r) {
        const C best = top_of<C, EPL>(c);
        const C all = wave_max(best);
        if (!(all > kOut))
            break;
        near |= r > 0 && too_near(last, all, 0x1p-18f);
        last = all;
        if (r == topk)
            break;
        const int win = __ffsll((unsigned long long)__ballot(best == all)) - 1;
        int at = 0;
        float value = l[0];
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
            if (c[j] == all) {
                at = j;
                value = l[j];
            }
        const int won = __builtin_amdgcn_readlane(at, win);
        const float picked = lane_value(value, win);
        if (lane == r) {
            mine = win * EPL + won;
            logit_of_mine = picked;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            c[j] = lane == win && j == won ? kOut : c[j];
    }
    return near;
}

template <class T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Run { T v[N]; };

template <class T, int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(64 * kWaves) route_topk_kernel(RouteArgs a)
{
    __shared__ double s_row[kWaves][64 * EPL];      // one token's scores per wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tok = blockIdx.x * kWaves + wave;
    if (tok >= a.T)
        return;                                     // waves share nothing: no barrier below
    const T *row = static_cast<const T *>(a.logits) + tok * a.stride;
    const int e0 = lane * EPL;
    float l[EPL], b[EPL];
    if (e0 + EPL <= a.E) {
        const Run<T, EPL> t = *reinterpret_cast<const Run<T, EPL> *>(row + e0);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            l[j] = to_float(t.v[j]);
            b[j] = 0.f;
        }
        if (a.bias) {
            const Run<float, EPL> u = *reinterpret_cast<const Run<float, EPL> *>(a.bias + e0);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                b[j] = u.v[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            l[j] = e0 + j < a.E ? to_float(row[e0 + j]) : -INFINITY;
            b[j] = a.bias && e0 + j < a.E ? a.bias[e0 + j] : 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)                   // NaN counts as out
        l[j] = l[j] > -INFINITY ? (l[j] > FLT_MAX ? FLT_MAX : l[j]) : -INFINITY;
    float top = 0.f;
    if (SOFTMAX)
        top = wave_max(top_of<float, EPL>(l));
    int mine = -1;
    float picked = 0.f;
    double sum = 1.0;                               // softmax's own, where it does not cancel
    // scores of type C, groups, picking; true: two were too near to tell apart
    auto by_score = [&](auto zero) {
        using C = decltype(zero);
        C c[EPL], part = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            c[j] = l[j] > -INFINITY ? score_of<SOFTMAX>(l[j], top, zero) : (C)0;
            part += c[j];
        }
        if (SOFTMAX) {
            const C all = wave_sum(part);
            sum = (double)all;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                c[j] = c[j] / all;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const C v = c[j] + (C)b[j];
            c[j] = l[j] > -INFINITY && v > -(C)INFINITY ? v : -(C)INFINITY;
        }
        bool near = false;
        if (a.groups > 1)
            near = keep_groups<C, EPL>(c, a, lane, reinterpret_cast<C *>(s_row[wave]));
        return pick<C, EPL>(c, l, a.topk, sizeof(C) == 4, lane, mine, picked) || near;
    };
    if (a.bias || a.groups > 1) {
        if (by_score(0.f))
            by_score(0.0);
    } else {
        float c[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            c[j] = l[j];
        pick<float, EPL>(c, l, a.topk, false, lane, mine, picked);
    }
    if (SOFTMAX && !a.renormalize) {
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            part += l[j] > -INFINITY ? score_of<SOFTMAX>(l[j], top, 0.0) : 0.0;
        sum = wave_sum(part);
    }
    const double p = mine >= 0 ? score_of<SOFTMAX>(picked, top, 0.0) : 0.0;
    if (a.renormalize)
        sum = wave_sum(p);
    if (lane < a.topk) {
        const long long o = (long long)tok * a.topk + lane;
        a.ids[o] = mine;
        a.weights[o] = p > 0.0 ? (float)(p / sum * (double)a.scale) : 0.f;
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
        softmax ? launch_epl<Bf16, true>(a, stream) : launch_epl<Bf16, false>(a, stream);
    else if (dtype == MOE_WNA16_FP16)
        softmax ? launch_epl<Fp16, true>(a, stream) : launch_epl<Fp16, false>(a, stream);
    else
        softmax ? launch_epl<float, true>(a, stream) : launch_epl<float, false>(a, stream);
    return hipGetLastError();
}

}  // namespace wna16
