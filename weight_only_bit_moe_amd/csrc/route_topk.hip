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
// 32 bits, and the token keeps that order if every comparison that mattered was
// wider than the errors of both sides (kScoreError and kKeyError below):
// consecutive picks, the last pick and the first expert left out, and any two
// groups.  Otherwise the wave repeats the picking in 64 bits.  Without bias and
// groups the order of c is the order of the logits, which is exact in 32 bits.
// The weights of the picked experts are always computed in 64 bits.
//
// One wave owns a token, each lane EPL of its experts, sorted once.  Picking is
// rounds of a wave-wide maximum over the lanes' largest (DPP, no LDS); the lane
// that held it moves on to its next.  With few tokens the time is the launch and
// the chain of memory round trips and reductions (T = 4, E = 256, top-6 of 4 of 8
// groups: 3.5 us); with many it is the VALU instructions, about 500 a token
// (T = 8192, top-8: 11.3 us in a captured graph, of which the VALUs are busy 7; the
// logits alone take 2 us to read).  Everything in 64 bits took 25 us.
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
    else    // from 700 on a constant: below any FP32 number, next to a weight of 2^-100 too
        return reciprocal(1.0 + exp_short(l < -700.f ? 700.0 : -(double)l));
}
// Whether exp(l - top) or sigmoid(l) is above 0 in 64 bits.
template <bool SOFTMAX>
__device__ __forceinline__ bool has_weight(float l, float top)
{
    return SOFTMAX ? (double)l - (double)top > -745.1332191019412 : l > -709.7827f;
}

// Errors of a 32-bit score, in FP32 roundings of 1 + |c|: a sigmoid is off by
// less than 4, a softmax by up to 8 of its own and 22 of the sum (16 scores a
// lane, then 6 steps); adding the bias is one more.  A key that gives its lowest
// log2(EPL) bits to the slot moves by up to EPL - 1 units in its last place, each
// of at most two roundings of |c|, and two keys may move towards each other.  Two
// scores may be in another order in 64 bits if they differ by less than both
// errors, two groups' sums of two scores if they differ by less than all four.
template <bool SOFTMAX> constexpr float kScoreError = (SOFTMAX ? 31 : 5) * 0x1p-24f;
template <bool SOFTMAX, int EPL>
constexpr float kKeyError = kScoreError<SOFTMAX> + 2 * EPL * 0x1p-24f;   // of |c|

// Of a >= b, where |a| may be the larger: then a - b is larger still, and the
// unit that kKeyError counts beyond EPL - 1 covers it.
__device__ __forceinline__ bool too_near(float a, float b, float fixed, float relative)
{
    // two infinities differ by a NaN: too near as well
    return !(a - b > fixed + relative * __builtin_fabsf(b));
}

// Takes the experts outside the best groups out of c.  Returns whether two
// groups were too near to tell apart (32 bits).
template <class C, int EPL, bool SOFTMAX>
__device__ __forceinline__ bool keep_groups(C (&c)[EPL], const RouteArgs &a, int lane, C *row)
{
    const C kOut = -(C)INFINITY;
    const int per = a.per_group;
    int close = 0;                                  // groups within the error, itself included
    // a group's two largest; with one expert left (or one in all) that one
    auto total = [&](C one, C two) { return two > kOut ? one + two : one; };
    auto count = [&](C score, C one, C two, int mine, auto &&of) {
        int ahead = 0;
        if constexpr (sizeof(C) == 4) {
            // Equal scores are near, so 64 bits decide them.  The errors are those of the two
            // scores, which may cancel, and one rounding of their sum.  The group of the two
            // with the larger error reports the pair.
            const float reach = 2 * (kScoreError<SOFTMAX> + 0x1p-24f) *
                                (2.f + __builtin_fabsf(one) + (two > kOut ? __builtin_fabsf(two) : 0.f));
            for (int g = 0; g < a.groups; ++g) {
                const C o = of(g);
                ahead += o > score ? 1 : 0;
                close += __builtin_fabsf(o - score) <= reach ? 1 : 0;
            }
            // infinite scores, also of two finite ones, go to 64 bits; an empty group does not
            if (!(score > kOut && score < (C)INFINITY))
                close = one > kOut ? 2 : 0;
        } else {
            for (int g = 0; g < a.groups; ++g) {
                const C o = of(g);
                ahead += o > score || (o == score && g < mine) ? 1 : 0;
            }
        }
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
        const int ahead = count(score, one, two, lane >> shift,
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
    const int ahead =
        count(score, one, two, lane, [&](int g) { return lane_value(score, g); });
    const uint64_t keep = __ballot(lane < a.groups && ahead < a.topk_groups);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (e0 + j < a.E && !((keep >> ((e0 + j) / per)) & 1))
            c[j] = kOut;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return __ballot(close > 1) != 0;
}

// Batcher's odd-even merge sort of n values by order(i, j), i < j.
template <int N, class F>
__device__ __forceinline__ void sort_network(F &&order)
{
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p))
                        order(i + j, i + j + k);
}

// Picks by packed keys, largest first: lane r's `mine` is the r-th pick.
// Distinct keys, so a lane's are sorted by min and max alone.  With EXTRA, one
// more round shows the first expert left out.  id(key, lane) names the expert,
// near(last, key) whether two keys in a row were too near to tell apart.
template <bool EXTRA, class K, int EPL, class Id, class Near>
__device__ __forceinline__ bool pick(K (&key)[EPL], int topk, int lane, int &mine, Id &&id,
                                     Near &&near_to)
{
    sort_network<EPL>([&](int i, int j) {
        const K hi = larger(key[i], key[j]), lo = key[i] > key[j] ? key[j] : key[i];
        key[i] = hi;
        key[j] = lo;
    });
    mine = -1;
    K taken = 0, last = 0;                          // taken: lane r's the r-th picked key
    int n = 0;
    for (; n < topk; ++n) {
        const K all = wave_max(key[0]);
        if (all == 0)
            break;
        last = all;
        const int win = __builtin_ctzll(__ballot(key[0] == all));
        const int e = id(all, win);
        mine = lane == n ? e : mine;
        if constexpr (EXTRA)
            taken = lane == n ? all : taken;
        const bool me = lane == win;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const K own = key[j], next = j + 1 < EPL ? key[j + 1] : (K)0;
            key[j] = me ? next : own;
        }
    }
    if constexpr (EXTRA) {
        const K before = (K)__shfl_up((int)taken, 1);
        const K left = n == topk ? wave_max(key[0]) : 0;
        return __ballot(lane > 0 && lane < n && near_to(before, taken)) != 0 ||
               (left != 0 && near_to(last, left));
    }
    return false;
}

// The same by 64-bit scores, whose keys leave no room for the slot: a lane's
// equal keys are sorted by slot, and the wave takes the lowest lane.
template <int EPL>
__device__ __forceinline__ void pick_exact(const double (&c)[EPL], int topk, int lane, int &mine)
{
    uint64_t key[EPL];
    int slot[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        key[j] = key_of(c[j]);
        slot[j] = j;
    }
    sort_network<EPL>([&](int i, int j) {
        const bool swap = key[j] > key[i] || (key[j] == key[i] && slot[j] < slot[i]);
        const uint64_t k = key[i];
        const int s = slot[i];
        key[i] = swap ? key[j] : k;
        key[j] = swap ? k : key[j];
        slot[i] = swap ? slot[j] : s;
        slot[j] = swap ? s : slot[j];
    });
    mine = -1;
    for (int r = 0; r < topk; ++r) {
        const uint64_t all = wave_max(key[0]);
        if (all == 0)
            break;
        const int win = __builtin_ctzll(__ballot(key[0] == all));
        const int e = win * EPL + lane_value(slot[0], win);
        mine = lane == r ? e : mine;
        const bool me = lane == win;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint64_t own = key[j], next = j + 1 < EPL ? key[j + 1] : 0ull;
            const int here = slot[j], there = j + 1 < EPL ? slot[j + 1] : 0;
            key[j] = me ? next : own;
            slot[j] = me ? there : here;
        }
    }
}

template <class T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Run { T v[N]; };

// BY_SCORE: with a bias or groups, lane i holds experts [i*EPL, (i+1)*EPL), so
// that groups are runs of lanes.  Otherwise it holds experts i, i + 64, ..., so
// that the slot and then the lane order equal logits by expert.
template <class T, int EPL, bool SOFTMAX, bool BY_SCORE>
__global__ void __launch_bounds__(64 * kWaves) route_topk_kernel(RouteArgs a)
{
    __shared__ double s_row[kWaves][64 * EPL];      // one token's scores, then its logits
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tok = blockIdx.x * kWaves + wave;
    if (tok >= a.T)
        return;                                     // waves share nothing: no barrier below
    const T *row = static_cast<const T *>(a.logits) + tok * a.stride;
    const int e0 = BY_SCORE ? lane * EPL : lane;
    constexpr int kStep = BY_SCORE ? 1 : 64;
    float l[EPL], b[EPL];
    if (BY_SCORE && e0 + EPL <= a.E) {
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
            const int e = e0 + j * kStep;
            l[j] = e < a.E ? to_float(row[e]) : -INFINITY;
            b[j] = BY_SCORE && a.bias && e < a.E ? a.bias[e] : 0.f;
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
    // A 32-bit key gives its lowest bits to the slot (a lower slot counts as
    // more), which costs log2(EPL) of the 24 bits of a score.
    constexpr uint32_t kSlots = EPL - 1;
    auto packed = [&](float v, int j) {
        const uint32_t k = key_of(v);
        return k ? (k & ~kSlots) | (kSlots - j) : 0u;
    };
    if constexpr (BY_SCORE) {
        auto scores = [&](auto &c, auto zero) {
            using C = decltype(zero);
            C part = 0;
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
            return a.groups > 1 && keep_groups<C, EPL, SOFTMAX>(
                                       c, a, lane, reinterpret_cast<C *>(s_row[wave]));
        };
        float c[EPL];
        bool near = scores(c, 0.f);
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = packed(c[j], j);
        near |= pick<true>(
            key, a.topk, lane, mine,
            [&](uint32_t k, int win) { return win * EPL + (int)(kSlots - (k & kSlots)); },
            [&](uint32_t last, uint32_t k) {
                return too_near(value_of(last), value_of(k), 2 * kScoreError<SOFTMAX>,
                                2 * kKeyError<SOFTMAX, EPL>);
            });
        if (near) {
            double d[EPL];
            scores(d, 0.0);
            pick_exact<EPL>(d, a.topk, lane, mine);
        }
    } else {
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = packed(l[j], j);
        // 16-bit logits keep all their bits; FP32 logits that differ in the lost ones only
        // (or not at all) are picked again by 64-bit keys with all bits and the expert
        const bool near = pick<sizeof(T) == 4>(
            key, a.topk, lane, mine,
            [&](uint32_t k, int win) { return win + 64 * (int)(kSlots - (k & kSlots)); },
            [&](uint32_t last, uint32_t k) { return sizeof(T) == 4 && (last ^ k) <= kSlots; });
        if (near) {
            uint64_t full[EPL];
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const uint32_t k = key_of(l[j]);
                full[j] = k ? (uint64_t)k << 32 | (uint32_t)(1023 - (lane + 64 * j)) : 0ull;
            }
            pick<false>(
                full, a.topk, lane, mine,
                [&](uint64_t k, int) { return 1023 - (int)(uint32_t)k; },
                [&](uint64_t, uint64_t) { return false; });
        }
    }
    // the picked experts' logits
    float *held = reinterpret_cast<float *>(s_row[wave]);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        held[e0 + j * kStep] = l[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float picked = mine >= 0 ? held[mine] : 0.f;
    double sum = 1.0;
    if (SOFTMAX && !a.renormalize) {                // softmax's own sum does not cancel
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            part += l[j] > -INFINITY ? weight_of<SOFTMAX>(l[j], top) : 0.0;
        sum = wave_sum(part);
    }
    double p = mine >= 0 ? weight_of<SOFTMAX>(picked, top) : 0.0;
    if (a.renormalize) {
        sum = wave_sum(p);
        if (sum < 0x1p-100) {
            // Every picked score is tiny, but their ratios need not be: relative to the largest
            // one.  Both scores are exp(l) there, to 2^-100 (1 + exp(l) is 1).
            const bool any = mine >= 0 && has_weight<SOFTMAX>(picked, top);
            const float most = wave_max(any ? picked : -INFINITY);
            p = any ? exp_short((double)picked - (double)most) : 0.0;
            sum = wave_sum(p);
        }
    }
    if (lane < a.topk) {
        const long long o = (long long)tok * a.topk + lane;
        a.ids[o] = mine;
        const double w = sum > 0.0 ? p * reciprocal(sum) : 0.0;     // 0: nothing picked has a score
        a.weights[o] = (float)(w * (double)a.scale);
    }
}

template <class T, bool SOFTMAX>
hipError_t launch_epl(const RouteArgs &a, hipStream_t stream)
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
        if (a.bias || a.groups > 1)
            return launch(route_topk_kernel<T, EPL, SOFTMAX, true>, dim3(grid), 64 * kWaves, stream, b);
        return launch(route_topk_kernel<T, EPL, SOFTMAX, false>, dim3(grid), 64 * kWaves, stream, b);
    };
    const int epl = (a.E + 63) / 64;
    if (epl <= 1)
        return go(std::integral_constant<int, 1>{});
    if (epl <= 2)
        return go(std::integral_constant<int, 2>{});
    if (epl <= 4)
        return go(std::integral_constant<int, 4>{});
    if (epl <= 8)
        return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs &a, int dtype, int score, hipStream_t stream)
{
    const bool softmax = score == MOE_WNA16_SOFTMAX;
    if (dtype == MOE_WNA16_BF16)
        return softmax ? launch_epl<Bf16, true>(a, stream) : launch_epl<Bf16, false>(a, stream);
    if (dtype == MOE_WNA16_FP16)
        return softmax ? launch_epl<Fp16, true>(a, stream) : launch_epl<Fp16, false>(a, stream);
    return softmax ? launch_epl<float, true>(a, stream) : launch_epl<float, false>(a, stream);
}

}  // namespace wna16
