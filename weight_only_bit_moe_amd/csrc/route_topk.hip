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

// Order-preserving integers of the values above -inf; 0 for -inf (out).
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);    // -0 and +0 are equal
    return v > -INFINITY ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return v > -(double)INFINITY ? b ^ ((uint64_t)((int64_t)b >> 63) | 1ull << 63) : 0ull;
}
__device__ __forceinline__ double value_of(uint64_t k)
{
    return __builtin_bit_cast(double, k >> 63 ? k ^ 1ull << 63 : ~k);
}

// exp(l - top) or sigmoid(l), for picking
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

// The weights' arithmetic: good to about 2^-36, so that only the rounding to
// FP32 shows, at a fraction of the library functions' instructions.
__device__ __forceinline__ double reciprocal(double v)
{
    const double r = __builtin_amdgcn_rcp(v);
    return __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);      // one Newton step
}
__device__ __forceinline__ double exp_short(double x)
{
    // exp(x) = 2^n exp(r), |r| <= ln(2) / 2; Taylor to r^9 leaves r^10 / 10! < 2^-36
    x = x < -1000.0 ? -1000.0 : x;                              // 0 either way
    const double n = __builtin_rint(x * 1.4426950408889634);
    const double r = __builtin_fma(-n, 0.6931471805599453, x);
    double p = 1.0 / 362880;
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return ldexp(p, (int)n);
}
template <bool SOFTMAX>
__device__ __forceinline__ double weight_of(float l, float top)
{
    if constexpr (SOFTMAX)
        return exp_short((double)l - (double)top);
    else    // beyond 700 the exponential would overflow; the weight is 0 in FP32 from 104 on
        return reciprocal(1.0 + exp_short(l < -700.f ? 700.0 : -(double)l));
}

// Whether two 32-bit scores may be in another order in 64 bits.  A sigmoid is
// off by less than 4 FP32 roundings; a softmax by up to 8 of its own and 22 of
// the sum (16 scores a lane, then 6 steps); adding the bias is one more.  So a
// score is off by less than 2^-19 (1 + |c|), a group's sum of two by twice that.
__device__ __forceinline__ bool too_near(float a, float b, float tolerance)
{
    return __builtin_fabsf(a - b) <= tolerance * (1.f + __builtin_fabsf(b));
}

// Takes the experts outside the best groups out of c.  Returns whether two
// groups were too near to tell apart (32 bits).
template <class C, int EPL>
__device__ __forceinline__ bool keep_groups(C (&c)[EPL], const RouteArgs &a, int lane, C *row)
{
    const C kOut = -(C)INFINITY;
    const int per = a.per_group;
    int close = 0;                                  // groups within the error, itself included
    // a group's two largest; with one expert left (or one in all) that one
    auto total = [&](C one, C two) { return two > kOut ? one + two : one; };
    auto count = [&](C score, int mine, auto &&of) {
        int ahead = 0;
        if constexpr (sizeof(C) == 4) {
            // equal scores are near, so 64 bits decide them
            const float reach = 0x1p-17f * (1.f + __builtin_fabsf(score));
            for (int g = 0; g < a.groups; ++g) {
                const C o = of(g);
                ahead += o > score ? 1 : 0;
                close += __builtin_fabsf(o - score) <= reach ? 1 : 0;
            }
        } else {
            for (int g = 0; g < a.groups; ++g) {
                const C o = of(g);
                ahead += o > score || (o == score && g < mine) ? 1 : 0;
            }
        }
        if (!(score > kOut && score < (C)INFINITY))
            close = score > kOut ? 2 : 0;           // infinite scores go to 64 bits
        return ahead;
    };
    if (a.span > 0) {
        // groups are whole runs of `span` lanes: merge the lanes' pairs by permutes
        C one = kOut, two = kOut;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            two = c[j] > one ? one : (c[j] > two ? c[j] : two);
            one = c[j] > one ? c[j] : one;
        }
        auto merge = [&](C o1, C o2) {
            const C low = o1 > one ? one : o1, high = o1 > one ? o2 : two;
            two = high > low ? high : low;
            one = o1 > one ? o1 : one;
        };
        merge(dpp<kXor1>(one), dpp<kXor1>(two));
        if (a.span >= 4)
            merge(dpp<kXor2>(one), dpp<kXor2>(two));
        if (a.span >= 8)
            merge(dpp<kHalfMirror>(one), dpp<kHalfMirror>(two));
        if (a.span >= 16)
            merge(dpp<kMirror>(one), dpp<kMirror>(two));
        const C score = total(one, two);
        const int shift = __ffs(a.span) - 1;
        const int ahead = count(score, lane >> shift,
                                [&](int g) { return lane_value(score, g << shift); });
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            c[j] = ahead >= a.topk_groups ? kOut : c[j];
        return __ballot(close > 1) != 0;            // lanes past the experts have no score
    }
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
            two = v > one ? one : (v > two ? v : two);
            one = v > one ? v : one;
        }
    const C score = total(one, two);
    const int ahead = count(score, lane, [&](int g) { return lane_value(score, g); });
    const uint64_t keep = __ballot(lane < a.groups && ahead < a.topk_groups);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (e0 + j < a.E && !((keep >> ((e0 + j) / per)) & 1))
            c[j] = kOut;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return __ballot(close > 1) != 0;
}

// One lane's experts: keys, slots and logits, largest key first (ties: lower slot).
template <class K, int EPL>
struct Sorted {
    K key[EPL];
    int slot[EPL];
    float l[EPL];

    __device__ __forceinline__ void order(int i, int j)
    {
        const bool swap = key[j] > key[i] || (key[j] == key[i] && slot[j] < slot[i]);
        const K k = key[i];
        const int s = slot[i];
        const float x = l[i];
        key[i] = swap ? key[j] : k;
        key[j] = swap ? k : key[j];
        slot[i] = swap ? slot[j] : s;
        slot[j] = swap ? s : slot[j];
        l[i] = swap ? l[j] : x;
        l[j] = swap ? x : l[j];
    }
    // Batcher's odd-even merge sort
    __device__ __forceinline__ void sort()
    {
#pragma unroll
        for (int p = 1; p < EPL; p <<= 1)
#pragma unroll
            for (int k = p; k >= 1; k >>= 1)
#pragma unroll
                for (int j = k % p; j + k < EPL; j += 2 * k)
#pragma unroll
                    for (int i = 0; i < k; ++i)
                        if (i + j + k < EPL && (i + j) / (2 * p) == (i + j + k) / (2 * p))
                            order(i + j, i + j + k);
    }
    __device__ __forceinline__ void drop_first(bool me)
    {
#pragma unroll
        for (int j = 0; j + 1 < EPL; ++j) {
            key[j] = me ? key[j + 1] : key[j];
            slot[j] = me ? slot[j + 1] : slot[j];
            l[j] = me ? l[j + 1] : l[j];
        }
        key[EPL - 1] = me ? (K)0 : key[EPL - 1];
    }
};

// Picks the topk largest of c: lane r gets the r-th pick and its logit.  With
// CHECK (32-bit scores) returns whether two that had to be told apart were too
// near; one more round shows the first expert left out.
template <bool CHECK, class C, int EPL>
__device__ __forceinline__ bool pick(const C (&c)[EPL], const float (&l)[EPL], int topk, int lane,
                                     int &mine, float &picked)
{
    using K = decltype(key_of(c[0]));
    Sorted<K, EPL> s;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        s.key[j] = key_of(c[j]);
        s.slot[j] = j;
        s.l[j] = l[j];
    }
    s.sort();
    mine = -1;
    bool near = false;
    K last = 0;
    const int rounds = CHECK ? topk + 1 : topk;
    for (int r = 0; r < rounds; ++r) {
        const K all = wave_max(s.key[0]);
        if (all == 0)
            break;
        if constexpr (CHECK)
            near |= r > 0 && too_near(value_of(last), value_of(all), 0x1p-18f);
        last = all;
        const uint64_t who = __ballot(s.key[0] == all);
        const int win = __builtin_ctzll(who);
        const int id = win * EPL + lane_value(s.slot[0], win);
        const float x = lane_value(s.l[0], win);
        if (r < topk) {
            mine = lane == r ? id : mine;
            picked = lane == r ? x : picked;
        }
        s.drop_first(lane == win);
    }
    return near;
}

template <class T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Run { T v[N]; };

template <class T, int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(64 * kWaves) route_topk_kernel(RouteArgs a)
{
    __shared__ double s_row[kWaves][64 * EPL];      // one token's scores per wave
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    for (int j = 0; j < EPL; ++j) {                 // NaN counts as out
        const float x = __builtin_fminf(l[j], FLT_MAX);
        l[j] = l[j] > -INFINITY ? x : -INFINITY;
    }
    float top = 0.f;
    if (SOFTMAX) {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j)
            m = larger(m, l[j]);
        top = wave_max(m);
    }
    int mine = -1;
    float picked = 0.f;
    // scores of type C, groups, picking; true: two were too near to tell apart
    auto by_score = [&](auto zero) {
        using C = decltype(zero);
        C c[EPL], part = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            c[j] = score_of<SOFTMAX>(l[j], top, zero);
            c[j] = l[j] > -INFINITY ? c[j] : (C)0;
            part += c[j];
        }
        if (SOFTMAX) {
            const C all = wave_sum(part);
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
        return pick<sizeof(C) == 4, C, EPL>(c, l, a.topk, lane, mine, picked) || near;
    };
    if (a.bias || a.groups > 1) {
        if (by_score(0.f))
            by_score(0.0);
    } else {
        pick<false, float, EPL>(l, l, a.topk, lane, mine, picked);
    }
    double sum = 1.0;
    if (SOFTMAX && !a.renormalize) {                // softmax's own sum does not cancel
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            part += l[j] > -INFINITY ? weight_of<SOFTMAX>(l[j], top) : 0.0;
        sum = wave_sum(part);
    }
    const double p = mine >= 0 ? weight_of<SOFTMAX>(picked, top) : 0.0;
    if (a.renormalize)
        sum = wave_sum(p);
    if (lane < a.topk) {
        const long long o = (long long)tok * a.topk + lane;
        a.ids[o] = mine;
        // sums so small that their reciprocal would overflow weigh nothing in FP32 either
        const double w = sum > 0x1p-1000 ? p * reciprocal(sum) : 0.0;
        a.weights[o] = (float)(w * (double)a.scale);
    }
}

template <class T, bool SOFTMAX>
void launch_epl(const RouteArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
    auto go = [&](auto n) {
        constexpr int EPL = decltype(n)::value;
        RouteArgs b = a;
        b.per_group = a.E / a.groups;
        // groups that are whole power-of-two runs of at most 16 lanes merge by permutes
        const int span = b.per_group / EPL;
        b.span = span * EPL == b.per_group && span >= 2 && span <= 16 && (span & (span - 1)) == 0
                     ? span
                     : 0;
        route_topk_kernel<T, EPL, SOFTMAX><<<grid, 64 * kWaves, 0, stream>>>(b);
    };
    const int epl = (a.E + 63) / 64;
    if (epl <= 1)
        go(std::integral_constant<int, 1>{});
    else if (epl <= 2)
        go(std::integral_constant<int, 2>{});
    else if (epl <= 4)
        go(std::integral_constant<int, 4>{});
    else if (epl <= 8)
        go(std::integral_constant<int, 8>{});
    else
        go(std::integral_constant<int, 16>{});
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
