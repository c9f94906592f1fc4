// Tokens' rows in the order of their experts, and experts' rows back to their
// tokens, with the gradients.
//
// Sort: the slot of a (token, expert) pair is the number of pairs of lower experts,
// plus the number of earlier pairs of its own expert.  Up to kOneLaunch pairs
// every workgroup compares its own tokens' pairs with all ids: one launch, and
// the tokens' rows are on their way meanwhile.  More pairs are counted in chunks
// first; a workgroup then needs the counts of all chunks and the ids of its own.
// Past kManyChunks chunks a launch in between adds up the counts of the chunks before.
// No order of any atomic matters: they only count.
//
// The rows are the bulk: each token's row is read once, into registers, and
// written to its topk places, so memory's write rate bounds it.  T = 4096, k = 8, H =
// 4096 (302 MB) 68 us = 4.4 TB/s, of which the slots take 9 on their own; T = 65536, k =
// 8, H = 1024 (1.2 GB) 237 us = 5.1 TB/s; T = 64, k = 6, H = 4096 4 us, most of it the launch
// and one trip to memory for the ids and one for the rows.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_wna16.h"
#include "expert_ops.hpp"
#include "rows.hpp"
#include "wave.hpp"

namespace wna16 {

namespace {

// One launch against two, sort alone (256 experts): 4096 pairs 5.5 and 6.5 us, 8192 pairs 11.1
// and 6.9.
constexpr int kOneLaunch = 4096;        // pairs
constexpr int kOwn = 64;                // pairs placed by one workgroup, at least one token's
constexpr int kChunk = 1024;            // pairs of a counted chunk, about
// Two launches against three: 32 chunks (256 experts) 9.1 and 10.3 us, 64 (both 64 and 256)
// 11.4 either way, 128 20.0 and 12.4.
constexpr int kManyChunks = 64;
constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;

typedef uint32_t Row16 __attribute__((ext_vector_type(4), aligned(2)));  // at any element

__device__ __forceinline__ bool valid(int id, int E) { return (unsigned)id < (unsigned)E; }

// Exclusive prefix sums of c[0, n) in LDS, n <= 1024, by a workgroup of 256;
// returns the total.  Ends with a barrier.
__device__ __forceinline__ int exclusive_scan(int *c, int n)
{
    __shared__ int wave_total[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (int)threadIdx.x * 4 + i;
        v[i] = at < n ? c[at] : 0;
        sum += v[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d)
            incl += o;
    }
    if (lane == 63)
        wave_total[wave] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        before += w < wave ? wave_total[w] : 0;
        total += wave_total[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (int)threadIdx.x * 4 + i;
        if (at < n)
            c[at] = before;
        before += v[i];
    }
    __syncthreads();
    return total;
}

// Many pairs, first: each chunk's pairs of each expert.
__global__ void __launch_bounds__(kThreads) count_kernel(SortArgs a)
{
    __shared__ int count[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        count[e] = 0;
    __syncthreads();
    const long long first = (long long)blockIdx.x * a.chunk * a.topk, all = (long long)a.T * a.topk;
    const long long end = first + (long long)a.chunk * a.topk;
    for (long long p = first + threadIdx.x; p < (end < all ? end : all); p += kThreads) {
        const int id = a.ids[p];
        if (valid(id, a.E))
            atomicAdd(&count[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        a.counts[(size_t)blockIdx.x * a.E + e] = count[e];
}

// Then: each expert's counts -> the pairs of the chunks before, and all of them behind the
// last chunk's.  A workgroup has 64 experts, each one's chunks in 16 runs.  (All experts
// in one workgroup: T = 65536, k = 8 the sort alone took 40.7 us with 256 experts, 103 with
// 1024.)
__global__ void __launch_bounds__(1024) before_kernel(SortArgs a, int chunks)
{
    __shared__ int run[16][64];
    const int lane = threadIdx.x & 63, seg = threadIdx.x >> 6, e = (int)blockIdx.x * 64 + lane;
    const int per = (chunks + 15) / 16;
    const int c0 = seg * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    int sum = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c)
            sum += a.counts[(size_t)c * a.E + e];
    }
    run[seg][lane] = sum;
    __syncthreads();
    if (e >= a.E)
        return;
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        before += i < seg ? run[i][lane] : 0;
        all += run[i][lane];
    }
    if (seg == 0)
        a.counts[(size_t)chunks * a.E + e] = all;
    for (int c = c0; c < c1; c += 8) {                  // eight loads on their way at a time
        int n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = c + i < c1 ? a.counts[(size_t)(c + i) * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < c1)
                a.counts[(size_t)(c + i) * a.E + e] = before;
            before += n[i];
        }
    }
}

template <bool NT>
__device__ __forceinline__ void put(char *p, Row16 v)
{
    if constexpr (NT)
        store_past(p, Words4{v[0], v[1], v[2], v[3]});
    else
        *reinterpret_cast<Row16 *>(p) = v;
}

// Rows of a workgroup's tokens [t0, t0 + n), this workgroup's part of their columns,
// to the places slot[] (LDS).
template <bool NT>
__device__ __forceinline__ void copy_rows(const SortArgs &a, int t0, int n, const int *slot)
{
    const int chunks = a.row_bytes / 16, step = (int)gridDim.y * kThreads;
    const int c0 = (int)(blockIdx.y * kThreads + threadIdx.x);
    for (int i = 0; i < n; ++i) {
        const char *src = a.x + (long long)(t0 + i) * a.x_stride;
        for (int c = c0; c < chunks; c += 2 * step) {
            const bool two = c + step < chunks;
            const Row16 v = *reinterpret_cast<const Row16 *>(src + c * 16);
            const Row16 w = *reinterpret_cast<const Row16 *>(src + (two ? c + step : c) * 16);
            for (int j = 0; j < a.topk; ++j) {
                const int s = __builtin_amdgcn_readfirstlane(slot[i * a.topk + j]);
                if (s < 0)
                    continue;
                char *to = a.xs + s * a.xs_stride;
                put<NT>(to + c * 16, v);
                if (two)
                    put<NT>(to + (c + step) * 16, w);
            }
        }
        // the row's end, two bytes a thread
        const int b = chunks * 16 + (int)threadIdx.x * 2;
        if (blockIdx.y == 0 && b < a.row_bytes) {
            const uint16_t v = *reinterpret_cast<const uint16_t *>(src + b);
            for (int j = 0; j < a.topk; ++j) {
                const int s = slot[i * a.topk + j];
                if (s >= 0)
                    *reinterpret_cast<uint16_t *>(a.xs + s * a.xs_stride + b) = v;
            }
        }
    }
}

// One launch: up to 256 * PER pairs.  The workgroups behind the tokens' (one a part)
// write the offsets and mark the places behind the last pair.
template <int PER>
__global__ void __launch_bounds__(kThreads) sort_one_kernel(SortArgs a)
{
    __shared__ int own[kOwn], slot[kOwn], count[kMaxExperts];
    const int P = a.T * a.topk;
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int p = i * kThreads + (int)threadIdx.x;
        id[i] = p < P ? a.ids[p] : -1;
        id[i] = valid(id[i], a.E) ? id[i] : INT32_MAX;      // after all experts
    }
    const int t0 = blockIdx.x * a.per_group;
    if (t0 >= a.T) {                                        // the last workgroup of the row
        if (blockIdx.y != 0)
            return;
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            count[e] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (id[i] != INT32_MAX)
                atomicAdd(&count[id[i]], 1);
        __syncthreads();
        const int total = exclusive_scan(count, a.E);
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            a.offsets[e] = count[e];
        if (threadIdx.x == 0)
            a.offsets[a.E] = total;
        for (int p = total + (int)threadIdx.x; p < P; p += kThreads)
            a.tokens[p] = -1;
        return;
    }
    const int n_tokens = a.T - t0 < a.per_group ? a.T - t0 : a.per_group;
    const int p0 = t0 * a.topk, n = n_tokens * a.topk;
    if ((int)threadIdx.x < n) {
        const int e = a.ids[p0 + threadIdx.x];
        own[threadIdx.x] = valid(e, a.E) ? e : -1;
        slot[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int j = 0; j < n; ++j) {
        const int e = __builtin_amdgcn_readfirstlane(own[j]);
        if (e < 0)
            continue;
        int before = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool earlier = i * kThreads + (int)threadIdx.x < p0 + j;
            before += (int)__popcll(__ballot(id[i] < e + (earlier ? 1 : 0)));
        }
        if ((threadIdx.x & 63) == 0)
            atomicAdd(&slot[j], before);
    }
    __syncthreads();
    if ((int)threadIdx.x < n) {
        const int s = own[threadIdx.x] < 0 ? -1 : slot[threadIdx.x];
        slot[threadIdx.x] = s;                              // its own entry only
        if (blockIdx.y == 0) {
            a.slots[p0 + threadIdx.x] = s;
            if (s >= 0)
                a.tokens[s] = t0 + (int)threadIdx.x / a.topk;
        }
    }
    if (!a.x)
        return;
    __syncthreads();
    copy_rows<false>(a, t0, n_tokens, slot);
}

// Many pairs: a workgroup's tokens get their slots, and its part of their columns is
// copied.  BEFORE: before_kernel has added up the counts.
template <bool BEFORE, bool NT>
__global__ void __launch_bounds__(kThreads) place_kernel(SortArgs a, int chunks)
{
    __shared__ int base[kMaxExperts], earlier[kMaxExperts], own[kOwn], slot[kOwn];
    const int t0 = blockIdx.x * a.per_group;
    const int n_tokens = a.T - t0 < a.per_group ? a.T - t0 : a.per_group;
    const int P = a.T * a.topk, p0 = t0 * a.topk, n = n_tokens * a.topk;
    const int chunk = t0 / a.chunk, first = chunk * a.chunk * a.topk;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        if constexpr (BEFORE) {
            base[e] = a.counts[(size_t)chunks * a.E + e];
            earlier[e] = a.counts[(size_t)chunk * a.E + e];
        } else {
            int all = 0, mine = 0;
            for (int c = 0; c < chunks; c += 8) {           // eight loads on their way at a time
                int v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = c + i < chunks ? a.counts[(size_t)(c + i) * a.E + e] : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    all += v[i];
                    mine += c + i < chunk ? v[i] : 0;
                }
            }
            base[e] = all;
            earlier[e] = mine;
        }
    }
    if ((int)threadIdx.x < n)
        own[threadIdx.x] = a.ids[p0 + threadIdx.x];
    __syncthreads();
    for (int p = first + (int)threadIdx.x; p < p0; p += kThreads) {
        const int id = a.ids[p];
        if (valid(id, a.E))
            atomicAdd(&earlier[id], 1);
    }
    __syncthreads();
    const int total = exclusive_scan(base, a.E);
    if ((int)threadIdx.x < n) {
        const int id = own[threadIdx.x];
        int s = -1;
        if (valid(id, a.E)) {
            s = base[id] + earlier[id];
            for (int i = 0; i < (int)threadIdx.x; ++i)
                s += own[i] == id;
        }
        slot[threadIdx.x] = s;
        if (blockIdx.y == 0) {
            a.slots[p0 + threadIdx.x] = s;
            if (s >= 0)
                a.tokens[s] = t0 + (int)threadIdx.x / a.topk;
        }
    }
    if (blockIdx.y == 0) {
        if (blockIdx.x == 0) {
            for (int e = threadIdx.x; e < a.E; e += kThreads)
                a.offsets[e] = base[e];
            if (threadIdx.x == 0)
                a.offsets[a.E] = total;
        }
        // places behind the last sorted pair, this workgroup's share
        for (int p = total + (int)(blockIdx.x * kThreads + threadIdx.x); p < P;
             p += (int)gridDim.x * kThreads)
            a.tokens[p] = -1;
    }
    if (!a.x)
        return;
    __syncthreads();
    copy_rows<NT>(a, t0, n_tokens, slot);
}

// Rows that the last-level cache (256 MB) would not hold until they are read are
// written past it: T = 4096, k = 8, H = 4096 (268 MB) 60 us instead of 72; no
// difference at 67 MB.
bool past_caches(long long rows, long long row_bytes) { return rows * row_bytes > 128ll << 20; }

int tokens_a_chunk(int topk, int per_group)
{
    const int groups = kChunk / (topk * per_group);
    return per_group * (groups < 1 ? 1 : groups);
}
int tokens_a_group(int T, int topk)
{
    const int most = kOwn / topk < 1 ? 1 : kOwn / topk;     // topk <= kOwn
    const int even = (T + 1023) / 1024;                     // about 1024 workgroups
    return even < 1 ? 1 : even < most ? even : most;        // T = 0: one, without tokens
}

}  // namespace

size_t sort_workspace(int T, int topk, int E)
{
    if ((long long)T * topk <= kOneLaunch)
        return 0;
    const int per = tokens_a_chunk(topk, tokens_a_group(T, topk));
    return ((size_t)((T + per - 1) / per) + 1) * E * sizeof(int32_t);   // and all chunks' sums
}

hipError_t launch_sort_tokens(const SortArgs &args, hipStream_t stream)
{
    SortArgs a = args;
    const bool one = (long long)a.T * a.topk <= kOneLaunch;
    a.per_group = tokens_a_group(a.T, a.topk);
    a.chunk = tokens_a_chunk(a.topk, a.per_group);
    const int groups = a.T ? (a.T + a.per_group - 1) / a.per_group : 1;
    // few tokens: a row's columns over several workgroups
    int parts = 1;
    if (a.x)
        while (parts < 8 && groups * parts < 256 && parts * kThreads * 16 < a.row_bytes)
            parts *= 2;
    if (one) {
        const dim3 grid((unsigned)((a.T ? groups : 0) + 1), (unsigned)parts);
        const int P = a.T * a.topk;
        if (P <= 2 * kThreads)
            return launch(sort_one_kernel<2>, grid, kThreads, stream, a);
        if (P <= 8 * kThreads)
            return launch(sort_one_kernel<8>, grid, kThreads, stream, a);
        return launch(sort_one_kernel<kOneLaunch / kThreads>, grid, kThreads, stream, a);
    }
    const dim3 grid((unsigned)groups, (unsigned)parts);
    const int chunks = (a.T + a.chunk - 1) / a.chunk;
    hipError_t e = launch(count_kernel, dim3((unsigned)chunks), kThreads, stream, a);
    if (e != hipSuccess)
        return e;
    const bool nt = a.x && past_caches((long long)a.T * a.topk, a.row_bytes);
    if (chunks <= kManyChunks)
        return launch(nt ? place_kernel<false, true> : place_kernel<false, false>, grid, kThreads,
                      stream, a, chunks);
    e = launch(before_kernel, dim3((unsigned)((a.E + 63) / 64)), 1024, stream, a, chunks);
    if (e != hipSuccess)
        return e;
    return launch(nt ? place_kernel<true, true> : place_kernel<true, false>, grid, kThreads, stream, a,
                  chunks);
}

// ---------------------------------------------------------------------------
// Combine:  out[t] = sum_j w[t][j] y[slot[t][j]] + add[t], in FP32 in that
// order, rounded once.  A thread holds 8 columns of one token and has up to kRows
// rows on their way; the slots and weights are wave-uniform.  Four rows leave
// registers for more waves than eight: T = 8192, k = 8, H = 4096 116 us = 5.2 TB/s
// against 121 us (two thirds of the rows' bytes as T = 680, k = 6: 7.7 against 9.9).
// ---------------------------------------------------------------------------
namespace {

constexpr int kRows = 4;

template <class T>
__global__ void __launch_bounds__(1024) combine_kernel(CombineArgs a)
{
    const int t = blockIdx.x;
    const int c = (int)(blockIdx.y * a.threads + threadIdx.x) * 8, left = a.H - c;
    if (left <= 0)
        return;
    const int32_t *slots = a.slots + (long long)t * a.topk;
    const float *weights = a.weights ? a.weights + (long long)t * a.topk : nullptr;
    const T *y = static_cast<const T *>(a.y) + c;
    float acc[8] = {};
    float add[8];
    if (a.addend)
        load8(static_cast<const T *>(a.addend) + t * a.add_stride + c, left, add);
    for (int j0 = 0; j0 < a.topk; j0 += kRows) {
        float v[kRows][8];
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (j0 + j < a.topk) {
                const int s = slots[j0 + j];
                if ((unsigned)s < (unsigned)a.R)
                    load8(y + s * a.y_stride, left, v[j]);
            }
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (j0 + j < a.topk && (unsigned)slots[j0 + j] < (unsigned)a.R) {
                const float w = weights ? weights[j0 + j] : 1.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = __builtin_fmaf(w, v[j][i], acc[i]);
            }
    }
    if (a.addend) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] += add[i];
    }
    store8(static_cast<T *>(a.out) + t * a.out_stride + c, left, acc);
}

// The gradients:  dy[slot[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[slot[t][j]]>.
// A workgroup owns a token and holds its row of dout; each row of y is read and
// each row of dy written once.  Workgroups behind the tokens clear the rows of dy
// that no token has.  Bytes bound it: T = 4096, k = 8, H = 4096 (570 MB) 100 us = 5.7 TB/s;
// combine_kernel there (302 MB) 58 us = 5.2 TB/s.  The dot products are FP32: eight elements
// in order, then the rows' pieces, lanes and waves in a fixed order.
constexpr int kClearGroups = 256;

template <class T, int R, bool NT>
__global__ void __launch_bounds__(1024) combine_grad_kernel(CombineGradArgs a)
{
    __shared__ float part[64][16];
    const int threads = a.threads;
    // rows of dy from here on are cleared, and only that: a slot there gets nothing
    const int used = !a.used ? a.R : *a.used < 0 ? 0 : *a.used < a.R ? *a.used : a.R;
    if ((int)blockIdx.x >= a.T) {
        const float zero[8] = {};
        for (int s = used + (int)blockIdx.x - a.T; s < a.R; s += kClearGroups) {
            T *o = static_cast<T *>(a.dy) + s * a.dy_stride;
            for (int c = (int)threadIdx.x * 8; c < a.H; c += threads * 8)
                store8(o + c, a.H - c, zero);
        }
        return;
    }
    const int t = blockIdx.x;
    const int32_t *slots = a.slots + (long long)t * a.topk;
    const T *d = static_cast<const T *>(a.dout) + t * a.d_stride;
    float g[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * threads + (int)threadIdx.x) * 8;
        load8(d + c, a.H - c, g[i]);
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // lane j holds pair j's slot and weight: read before the first store, behind
    // which a load would wait for it
    const int slots_at = lane < a.topk ? slots[lane] : -1;
    const float weights_at =
        a.weights && lane < a.topk ? a.weights[(long long)t * a.topk + lane] : 1.f;
    auto slot = [&](int j) {
        const int s = __builtin_amdgcn_readlane(slots_at, j);
        return (unsigned)s < (unsigned)a.R ? s : -1;
    };
    // the next row of y is on its way while this one is multiplied
    Pack8<T> v[R], next[R];
    auto load = [&](int j, Pack8<T> (&to)[R]) {
        const int s = j < a.topk ? slot(j) : -1;
        if (s < 0)
            return;
        const T *y = static_cast<const T *>(a.y) + s * a.y_stride;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * threads + (int)threadIdx.x) * 8;
            to[i] = load_pack8(y + c, a.H - c);
        }
    };
    if (a.dw)
        load(0, v);
    for (int j = 0; j < a.topk; ++j) {
        const int s = slot(j);
        if (a.dw) {
            load(j + 1, next);
            float dot = 0.f;
            if (s >= 0) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dot = __builtin_fmaf(g[i][k], to_float(v[i].v[k]), dot);
            }
            dot = wave_sum(dot);
            if (lane == 0)
                part[j][wave] = dot;
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = next[i];
        }
        if (a.dy && s >= 0 && s < used) {
            const float w =
                __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weights_at), j));
            T *o = static_cast<T *>(a.dy) + s * a.dy_stride;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = (i * threads + (int)threadIdx.x) * 8;
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    f[k] = w * g[i][k];
                store8<NT>(o + c, a.H - c, f);
            }
        }
    }
    if (!a.dw)
        return;
    __syncthreads();
    if ((int)threadIdx.x < a.topk) {
        float sum = 0.f;
        for (int w = 0; w < threads >> 6; ++w)
            sum += part[threadIdx.x][w];
        a.dw[(long long)t * a.topk + threadIdx.x] = sum;
    }
}

template <class F>
hipError_t with_type(int dtype, F &&f)
{
    if (dtype == MOE_WNA16_BF16)
        return f(Bf16{});
    if (dtype == MOE_WNA16_FP16)
        return f(Fp16{});
    return f(0.f);
}

}  // namespace

hipError_t launch_combine_tokens(const CombineArgs &args, int dtype, hipStream_t stream)
{
    CombineArgs a = args;
    const int chunks = (a.H + 7) / 8;
    a.threads = chunks < 256 ? (chunks + 63) / 64 * 64 : 256;
    const dim3 grid((unsigned)a.T, (unsigned)((chunks + a.threads - 1) / a.threads));
    return with_type(dtype, [&](auto zero) {
        return launch(combine_kernel<decltype(zero)>, grid, a.threads, stream, a);
    });
}

hipError_t launch_combine_tokens_grad(const CombineGradArgs &args, int dtype, hipStream_t stream)
{
    CombineGradArgs a = args;
    const int chunks = (a.H + 7) / 8;
    const dim3 grid((unsigned)(a.T + (a.dy && a.used ? kClearGroups : 0)));
    auto run = [&](int threads, auto r) {
        a.threads = threads;
        constexpr int R = decltype(r)::value;
        return with_type(dtype, [&](auto zero) {
            using T = decltype(zero);
            return launch(past_caches(a.R, (long long)a.H * sizeof(T))
                              ? combine_grad_kernel<T, R, true>
                              : combine_grad_kernel<T, R, false>,
                          grid, threads, stream, a);
        });
    };
    if (chunks <= 1024)
        return run((chunks + 63) / 64 * 64, std::integral_constant<int, 1>{});
    if (chunks <= 2048)
        return run(1024, std::integral_constant<int, 2>{});
    return run(1024, std::integral_constant<int, 4>{});
}

}  // namespace wna16
