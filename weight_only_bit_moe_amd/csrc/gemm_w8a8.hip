// Product in 8-bit integers with scales for each token and channel:
//   out[t][n] = round( float(sum_k a[t][k] w[n][k]) * sa[t] * sw[n] + add[t][n] )
// The sum is exact in int32 (K <= 131071), whatever the order, so splitting K
// over waves or workgroups changes no result.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_wna16.h"
#include "ops.hpp"

namespace wna16 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

struct GBf16 { uint16_t u; };
struct GFp16 { uint16_t u; };
__device__ __forceinline__ float widen(GBf16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float widen(GFp16 v) { return (float)__builtin_bit_cast(_Float16, v.u); }
__device__ __forceinline__ float widen(float v) { return v; }
template <class T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ GBf16 narrow<GBf16>(float v)
{
    return GBf16{__builtin_bit_cast(uint16_t, (__bf16)v)};
}
template <> __device__ __forceinline__ GFp16 narrow<GFp16>(float v)
{
    return GFp16{__builtin_bit_cast(uint16_t, (_Float16)v)};
}
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }

template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Out4 { T v[4]; };

// Four consecutive outputs of one token, from column n.
template <class T>
__device__ __forceinline__ void emit4(const GemmArgs &g, int t, int n, const int (&acc)[4])
{
    if (t >= g.T || n >= g.N)
        return;
    const float sa = g.a_scale[t];
    const T *add = g.addend ? static_cast<const T *>(g.addend) + t * g.ld_add + n : nullptr;
    T *o = static_cast<T *>(g.out) + t * g.ldo + n;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = n + i < g.N ? (float)acc[i] * sa * g.w_scale[n + i] : 0.f;
    if (n + 4 <= g.N) {
        if (add) {
            const Out4<T> d = *reinterpret_cast<const Out4<T> *>(add);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] += widen(d.v[i]);
        }
        Out4<T> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.v[i] = narrow<T>(f[i]);
        *reinterpret_cast<Out4<T> *>(o) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < g.N)
                o[i] = narrow<T>(add ? f[i] + widen(add[i]) : f[i]);
    }
}

// 16 bytes from any address; gfx950 loads them unaligned.
struct __attribute__((packed, aligned(1))) Bytes16 { int v[4]; };
__device__ __forceinline__ v4i load16(const int8_t *p)
{
    const Bytes16 b = *reinterpret_cast<const Bytes16 *>(p);
    return v4i{b.v[0], b.v[1], b.v[2], b.v[3]};
}
// The first `left` of 16 bytes, zeros behind them.
__device__ __forceinline__ v4i load_tail(const int8_t *p, int left)
{
    if (left >= 16)
        return load16(p);
    v4i r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < left)
            r[i >> 2] |= (int)((uint32_t)(uint8_t)p[i] << (8 * (i & 3)));
    return r;
}

// ---------------------------------------------------------------------------
// Few tokens, and operands that no 16-byte copy can address.  A workgroup owns
// 16 channels and up to MT * 16 tokens; its waves split K and add their sums
// through LDS.  Both operands go from memory to the MFMA's registers directly:
// lane l holds 16 bytes of row l % 16 at K offset 16 * (l / 16), so a wave's
// load covers 64 consecutive bytes of 16 rows, and the next one the rest of the
// 128-byte lines.  Channels are the MFMA's rows, so a lane ends up with four
// consecutive channels of one token and stores them at once.
// ---------------------------------------------------------------------------
template <int MT, int NW>
__global__ void __launch_bounds__(64 * NW) gemm_rows_kernel(GemmArgs g, int out_dtype)
{
    __shared__ int part[NW][MT][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * (MT * 16);
    const int r = lane & 15, kc = (lane >> 4) * 16;
    const int nr = n0 + r < g.N ? n0 + r : g.N - 1;     // rows past the end repeat the last
    const int8_t *w = g.w + nr * g.ldw + kc;
    const int8_t *a[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int tr = t0 + m * 16 + r;
        a[m] = g.a + (tr < g.T ? tr : g.T - 1) * g.lda + kc;
    }
    v4i acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        acc[m] = v4i{0, 0, 0, 0};
    // steps of 64 K; a wave takes runs of two (whole 128-byte lines)
    constexpr int S = 2;
    int k = wave * (64 * S);
    for (; k + 64 * S <= g.K; k += NW * 64 * S) {
        v4i fw[S], fa[S][MT];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            fw[s] = load16(w + k + s * 64);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                fa[s][m] = load16(a[m] + k + s * 64);
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s], fa[s][m], acc[m], 0, 0, 0);
    }
    // what is left of K for this wave: less than one run
    for (; k < g.K && k < (g.K + 64 * S - 1) / (64 * S) * (64 * S); k += NW * 64 * S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int left = g.K - (k + s * 64 + kc);
            const v4i fw = load_tail(w + k + s * 64, left);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    fw, load_tail(a[m] + k + s * 64, left), acc[m], 0, 0, 0);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
        *reinterpret_cast<v4i *>(&part[wave][m][lane * 4]) = acc[m];
    __syncthreads();
    for (int m = wave; m < MT; m += NW) {
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NW; ++i)
            sum += *reinterpret_cast<const v4i *>(&part[i][m][lane * 4]);
        const int v[4] = {sum[0], sum[1], sum[2], sum[3]};
        const int t = t0 + m * 16 + r, n = n0 + (lane >> 4) * 4;
        if (out_dtype == MOE_WNA16_BF16)
            emit4<GBf16>(g, t, n, v);
        else if (out_dtype == MOE_WNA16_FP16)
            emit4<GFp16>(g, t, n, v);
        else
            emit4<float>(g, t, n, v);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

// LDS byte address of a __shared__ pointer.
__device__ __forceinline__ uint32_t lds_of(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)(p);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Lane l's 16 bytes at base + voff land at LDS address lds + l * 16.  base and
// lds are wave-uniform.  Inline asm, so that the compiler does not make every
// later LDS read wait for all copies in flight; the caller waits with vmcnt.
__device__ __forceinline__ void copy16_to_lds(const int8_t *base_in, uint32_t voff, uint32_t lds_in)
{
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_in);
    const uint64_t b = reinterpret_cast<uintptr_t>(base_in);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    const void *base = reinterpret_cast<const void *>(((uint64_t)hi << 32) | (uint64_t)lo);
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base),
                 "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Tile of BM tokens x BN channels, WM x WN waves, K in chunks of 128 bytes.
// Operand rows of 128 bytes sit in LDS as 8 pieces of 16 bytes; piece c of row
// r is stored at place c ^ ((r >> 1) & 7), so that the 16 rows that one MFMA
// operand read touches are spread over all banks.  Two stages: the copies of
// chunk i + 1 run while chunk i is multiplied.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile8 {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
    static constexpr int KC = 128;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr int STAGE = (BM + BN) * KC;
    static constexpr int COPIES = (BM + BN) / 8 / NW;     // 8 rows per copy
    static_assert((BM + BN) / 8 % NW == 0 && BM / 8 % NW == 0, "copies divide evenly");

    static __device__ __forceinline__ int place(int row, int c) { return c ^ ((row >> 1) & 7); }

    template <class T>
    static __device__ __forceinline__ void run(const GemmArgs &g, int t0, int n0, char *lds)
    {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds0 = lds_of(lds);
        // Copies: copy i of this wave brings rows [8 * (i * NW + wave), +8).
        // Rows past the end repeat the last row; their results are dropped.
        uint32_t off[COPIES];
        const int8_t *base[2] = {g.a + (long long)t0 * g.lda, g.w + (long long)n0 * g.ldw};
        const int crow = lane >> 3;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int row = (i * NW + wave) * 8 + crow;
            const bool is_a = i < BM / 8 / NW;
            const int rr = is_a ? row : row - BM;
            const int last = is_a ? g.T - 1 - t0 : g.N - 1 - n0;
            off[i] = (uint32_t)((rr < last ? rr : last) * (is_a ? g.lda : g.ldw)) +
                     (uint32_t)place(row, lane & 7) * 16;
        }
        // K past the end (a multiple of 16): the piece's first one is read
        // again and the channel operand's fragment is cleared below.
        auto copy = [&](int k, int stage) {
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
                const int row = (i * NW + wave) * 8 + crow;
                const int kk = k + place(row, lane & 7) * 16;
                const uint32_t o = kk < g.K ? off[i] + (uint32_t)k
                                            : off[i] - (uint32_t)place(row, lane & 7) * 16;
                copy16_to_lds(base[i < BM / 8 / NW ? 0 : 1], o,
                              lds0 + stage * STAGE + (i * NW + wave) * 1024);
            }
        };
        v4i acc[NT][MT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[n][m] = v4i{0, 0, 0, 0};
        const int r = lane & 15, kq = lane >> 4;
        const int arow = wm * (MT * 16) + r, brow = BM + wn * (NT * 16) + r;
        copy(0, 0);
        const int chunks = (g.K + KC - 1) / KC;
        for (int c = 0; c < chunks; ++c) {
            __builtin_amdgcn_s_waitcnt(0x0f70);        // vmcnt(0): this chunk has arrived
            __syncthreads();
            if (c + 1 < chunks)
                copy((c + 1) * KC, (c + 1) & 1);
            const char *st = lds + (c & 1) * STAGE;
            const bool tail = (c + 1) * KC > g.K;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                v4i fa[MT], fb[NT];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    fa[m] = *reinterpret_cast<const v4i *>(
                        st + (arow + m * 16) * KC + place(arow + m * 16, s * 4 + kq) * 16);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    fb[n] = *reinterpret_cast<const v4i *>(
                        st + (brow + n * 16) * KC + place(brow + n * 16, s * 4 + kq) * 16);
                if (tail && c * KC + s * 64 + kq * 16 >= g.K) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        fb[n] = v4i{0, 0, 0, 0};
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[n][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[n], fa[m], acc[n][m],
                                                                          0, 0, 0);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = t0 + arow + m * 16;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int v[4] = {acc[n][m][0], acc[n][m][1], acc[n][m][2], acc[n][m][3]};
                emit4<T>(g, t, n0 + wn * (NT * 16) + n * 16 + kq * 4, v);
            }
        }
    }
};

template <class C, class T>
__global__ void __launch_bounds__(64 * C::NW) gemm_tile_kernel(GemmArgs g, int tiles_m, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) char lds[2 * C::STAGE];
    // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of
    // tiles, so its L2 serves neighbours that share an operand.
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= total || (int)(blockIdx.x >> 3) >= per)
        return;
    const int tm = id / tiles_n, tn = id % tiles_n;
    C::template run<T>(g, tm * C::BM, tn * C::BN, lds);
}

template <class C>
hipError_t launch_tile(const GemmArgs &g, int out_dtype, hipStream_t stream)
{
    const int tm = (g.T + C::BM - 1) / C::BM, tn = (g.N + C::BN - 1) / C::BN;
    const unsigned grid = (unsigned)((tm * tn + 7) / 8 * 8);
    auto go = [&](auto kernel) {
        kernel<<<grid, 64 * C::NW, 0, stream>>>(g, tm, tn);
        return hipGetLastError();
    };
    if (out_dtype == MOE_WNA16_BF16)
        return go(gemm_tile_kernel<C, GBf16>);
    if (out_dtype == MOE_WNA16_FP16)
        return go(gemm_tile_kernel<C, GFp16>);
    return go(gemm_tile_kernel<C, float>);
}

template <int MT>
hipError_t launch_rows(const GemmArgs &g, int out_dtype, hipStream_t stream)
{
    constexpr int NW = 16;
    const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)((g.T + MT * 16 - 1) / (MT * 16)));
    gemm_rows_kernel<MT, NW><<<grid, 64 * NW, 0, stream>>>(g, out_dtype);
    return hipGetLastError();
}

bool aligned16(const GemmArgs &g)
{
    return (reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.w) |
            (uintptr_t)g.lda | (uintptr_t)g.ldw | (uintptr_t)g.K) % 16 == 0;
}

}  // namespace

GemmPlan gemm_plan(int T, int N, int K)
{
    (void)K;
    GemmPlan p{};
    p.split = 1;
    if (T <= 64) {
        p.variant = 0;
        p.bm = (T + 15) / 16 * 16;
        p.bn = 16;
    } else {
        p.variant = 1;
        const long long big = (long long)((T + 255) / 256) * ((N + 255) / 256);
        p.bm = p.bn = big >= 192 ? 256 : 128;
    }
    return p;
}

hipError_t launch_gemm_w8a8(const GemmArgs &g, const GemmPlan &p, int out_dtype,
                            hipStream_t stream)
{
    if (p.variant == 1 && aligned16(g)) {
        if (p.bm == 256)
            return launch_tile<Tile8<256, 256, 2, 4>>(g, out_dtype, stream);
        return launch_tile<Tile8<128, 128, 2, 2>>(g, out_dtype, stream);
    }
    if (g.T <= 16)
        return launch_rows<1>(g, out_dtype, stream);
    if (g.T <= 32)
        return launch_rows<2>(g, out_dtype, stream);
    return launch_rows<4>(g, out_dtype, stream);
}

}  // namespace wna16
