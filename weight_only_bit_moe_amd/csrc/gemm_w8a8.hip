// Product in 8-bit integers with scales for each token and channel:
//   out[t][n] = round( float(sum_k a[t][k] w[n][k]) * sa[t] * sw[n] + add[t][n] )
// The sum is exact in int32 (K <= 131071), whatever the order, so splitting K
// over waves or workgroups changes no result.
//
// Times in this file are those of calls one after another in a captured graph,
// bf16 out, codes distributed as activations' unless it says otherwise; a kernel
// trace gives 0.5 to 1 us less for the short ones.
//
// Up to 64 tokens the weights are streamed once through kernels that are bound
// by the launch, one memory round trip and HBM (T = 4, N = K = 4096: 5.5 us,
// 16.8 MB; T = 64, K = 2048: 5.9 us; N = 16384, T = 4: 14.8 us = 4.5 TB/s).  More
// tokens go through MFMA tiles (T = 8192, N = K = 4096: 118-126 us = 2.2-2.3
// POP/s, 131 us with uniform codes).  In a long run of the tile loop (K = 32768,
// 2.4 POP/s) the MFMAs are busy 72 % of the cycles, at a clock that has fallen to
// 1.5 GHz: power bounds it, the more bits of the operands change the more.  A
// library product of the same size takes 128 us.
// Operands whose rows do not all begin at multiples of 16 bytes go the same ways
// through registers (N = 4096, K = 4090 against 4096: T = 4 6.2 and 5.5 us, T = 64
// 11.4 and 8.5 us, T = 256 16.9 and 10.5 us, T = 8192 215 and 126 us): every such
// load touches two lines, and an LDS store follows it.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_wna16.h"
#include "ops.hpp"
#include "wave.hpp"

namespace wna16 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Out4 { T v[4]; };

// What four consecutive outputs of one token, from column n, need besides
// their sums: loaded while the operands are on their way.
template <class T>
struct Beside {
    float sa, sw[4];
    Out4<T> add;

    __device__ __forceinline__ void load(const GemmArgs &g, int t, int n)
    {
        add = Out4<T>{};
        if (t >= g.T || n >= g.N)
            return;
        sa = g.a_scale[t];
        const T *p = static_cast<const T *>(g.addend) + t * g.ld_add + n;
        if (n + 4 <= g.N) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sw[i] = g.w_scale[n + i];
            if (g.addend)
                add = *reinterpret_cast<const Out4<T> *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < g.N) {
                    sw[i] = g.w_scale[n + i];
                    if (g.addend)
                        add.v[i] = p[i];
                }
        }
    }
    __device__ __forceinline__ void emit(const GemmArgs &g, int t, int n, v4i acc) const
    {
        if (t >= g.T || n >= g.N)
            return;
        T *o = static_cast<T *>(g.out) + t * g.ldo + n;
        Out4<T> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = (float)acc[i] * sa * sw[i];
            r.v[i] = from_float<T>(g.addend ? f + to_float(add.v[i]) : f);
        }
        if (n + 4 <= g.N) {
            *reinterpret_cast<Out4<T> *>(o) = r;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < g.N)
                    o[i] = r.v[i];
        }
    }
};

// 16 bytes from any address; gfx950 loads them unaligned.
struct __attribute__((packed, aligned(1))) Bytes16 { int v[4]; };
__device__ __forceinline__ v4i load16(const int8_t *p)
{
    const Bytes16 b = *reinterpret_cast<const Bytes16 *>(p);
    return v4i{b.v[0], b.v[1], b.v[2], b.v[3]};
}
// Pieces of 16 bytes of which left(i) (any number) lie before the row's end,
// zeros behind it.  Of a piece that crosses the end the row's last 16 bytes are
// loaded and moved down; a row of fewer bytes is read one by one.
template <int N, class At, class Left>
__device__ __forceinline__ void load_ends(v4i (&to)[N], At &&at, Left &&left)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        to[i] = load16(left(i) >= 16 ? at(i) : at(i) + (left(i) - 16));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int gone = 16 - left(i);
        const unsigned __int128 u = __builtin_bit_cast(unsigned __int128, to[i]);
        if (gone > 0)
            to[i] = __builtin_bit_cast(v4i, gone < 16 ? u >> (8 * gone) : 0);
    }
}
template <int N, class At, class Left>
__device__ __forceinline__ void load_short(v4i (&to)[N], At &&at, Left &&left)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        unsigned __int128 u = 0;
        for (int b = left(i) - 1; b >= 0; --b)
            u = u << 8 | (uint8_t)at(i)[b];
        to[i] = __builtin_bit_cast(v4i, u);
    }
}

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

// Place of a row's 16-byte piece c among the 8 of its 128-byte LDS row: the 16
// rows that one MFMA operand read touches are spread over all banks.
__device__ __forceinline__ int place(int row, int c) { return c ^ ((row >> 1) & 7); }

template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Sums the waves' 16-channel x MT*16-token results; wave m writes tokens
// [t0 + 16m, +16), for which it holds `beside`.
template <class T, int MT, int NW>
__device__ __forceinline__ void join_waves(const GemmArgs &g, const v4i (&acc)[MT], int *part,
                                           int n0, int t0, const Beside<T> &beside)
{
    static_assert(MT <= NW, "a wave for every 16 tokens");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int m = 0; m < MT; ++m)
        *reinterpret_cast<v4i *>(part + ((wave * MT + m) * 64 + lane) * 4) = acc[m];
    __syncthreads();
    if (wave < MT) {
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NW; ++i)
            sum += *reinterpret_cast<const v4i *>(part + ((i * MT + wave) * 64 + lane) * 4);
        beside.emit(g, t0 + wave * 16 + (lane & 15), n0 + (lane >> 4) * 4, sum);
    }
}

// ---------------------------------------------------------------------------
// Few tokens (decode): the weights are streamed once.  A workgroup owns 16
// channels and all tokens (up to 8 * TC); its waves take the 128-byte chunks of
// K in turn and add their sums through LDS at the end.  Each wave copies its
// chunks into its own ring of R stages, so no barrier is needed before the
// join.  The way through LDS is for the addresses: an MFMA wants lane l to hold
// row l % 16, and a load in that order has every lane in another row, which the
// address unit takes one lane a cycle; the copies take eight lanes of one row
// in a row, four lanes a cycle.  ANY: operands at any address and any K, which
// no such copy can fetch: R chunks of a wave are held in registers instead, and
// pass through one stage.
// ---------------------------------------------------------------------------
template <class T, int TC, int NW, int R, bool ANY>
__global__ void __launch_bounds__(64 * NW) gemm_stream_kernel(GemmArgs g)
{
    constexpr int MT = TC < 2 ? 1 : TC / 2, ROWS = 16 + 8 * TC, STAGE = ROWS * 128;
    constexpr int COPIES = ROWS / 8, RING = NW * (ANY ? 1 : R) * STAGE, PART = NW * MT * 1024;
    __shared__ __attribute__((aligned(1024))) char lds[RING > PART ? RING : PART];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    char *ring = lds + wave * ((ANY ? 1 : R) * STAGE);
    const uint32_t ring0 = lds_of(ring);
    // copy i brings rows [8i, 8i + 8): channels first, then tokens; rows past
    // the end repeat the last one
    const int crow = lane >> 3;
    uint32_t off[COPIES];
    int cplace[2] = {place(crow, lane & 7) * 16, place(8 + crow, lane & 7) * 16};
    const int8_t *wbase = g.w + (long long)n0 * g.ldw;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int row = i < 2 ? i * 8 + crow : (i - 2) * 8 + crow;
        const int last = i < 2 ? g.N - 1 - n0 : g.T - 1;
        off[i] = (uint32_t)((row < last ? row : last) * (i < 2 ? g.ldw : g.lda)) +
                 (uint32_t)cplace[i & 1];
    }
    const int chunks = (g.K + 127) / 128;
    auto copy = [&](int c, int stage) {
        const bool part = (c + 1) * 128 > g.K;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            uint32_t o = off[i] + (uint32_t)(c * 128);
            // K past the end (a multiple of 16): the row's first piece is read
            // again, and the channels' registers are cleared below
            if (part && c * 128 + cplace[i & 1] >= g.K)
                o = off[i] - (uint32_t)cplace[i & 1];
            copy16_to_lds(i < 2 ? wbase : g.a, o, ring0 + stage * STAGE + i * 1024);
        }
    };
    const int r = lane & 15, kq = lane >> 4;
    Beside<T> beside;
    if (wave < MT)
        beside.load(g, wave * 16 + r, n0 + kq * 4);
    v4i acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        acc[m] = v4i{0, 0, 0, 0};
    // a chunk's products from its stage
    auto read = [&](const char *st, v4i (&fw)[2], v4i (&fa)[2][MT]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            fw[s] = *reinterpret_cast<const v4i *>(st + r * 128 + place(r, s * 4 + kq) * 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int row = TC == 1 ? 16 + (r & 7) : 16 + m * 16 + r;
                fa[s][m] = *reinterpret_cast<const v4i *>(st + row * 128 +
                                                          place(row, s * 4 + kq) * 16);
            }
        }
    };
    auto multiply = [&](const v4i (&fw)[2], const v4i (&fa)[2][MT]) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s], fa[s][m], acc[m], 0, 0, 0);
    };
    if constexpr (ANY) {
        v4i held[R][COPIES];
        auto load = [&](v4i (&to)[COPIES], int c) {
            auto at = [&](int i) { return (i < 2 ? wbase : g.a) + off[i] + (uint32_t)(c * 128); };
            auto left = [&](int i) { return g.K - c * 128 - cplace[i & 1]; };
            if ((c + 1) * 128 <= g.K) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    to[i] = load16(at(i));
            } else if (g.K >= 16) {
                load_ends(to, at, left);
            } else {
                load_short(to, at, left);
            }
        };
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (wave + i * NW < chunks)
                load(held[i], wave + i * NW);
        for (int c0 = wave; c0 < chunks; c0 += R * NW)
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int c = c0 + j * NW;
                if (c >= chunks)
                    break;
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    *reinterpret_cast<v4i *>(ring + i * 1024 + lane * 16) = held[j][i];
                if (c + R * NW < chunks)
                    load(held[j], c + R * NW);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                v4i fw[2], fa[2][MT];
                read(ring, fw, fa);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                multiply(fw, fa);
            }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (wave + i * NW < chunks)
                copy(wave + i * NW, i);
        for (int c = wave, stage = 0; c < chunks;
             c += NW, stage = stage + 1 == R ? 0 : stage + 1) {
            // the copies behind this chunk's stay in flight
            if (c + (R - 1) * NW < chunks)
                wait_copies<(R - 1) * COPIES>();
            else
                wait_copies<0>();
            v4i fw[2], fa[2][MT];
            read(ring + stage * STAGE, fw, fa);
            if ((c + 1) * 128 > g.K) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (c * 128 + s * 64 + kq * 16 >= g.K)
                        fw[s] = v4i{0, 0, 0, 0};
            }
            if (c + R * NW < chunks) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read
                copy(c + R * NW, stage);
            }
            multiply(fw, fa);
        }
    }
    __syncthreads();                                // every ring has been read
    join_waves<T, MT, NW>(g, acc, reinterpret_cast<int *>(lds), n0, 0, beside);
}

// ---------------------------------------------------------------------------
// Many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

// Tile of BM tokens x BN channels, WM x WN waves, K in chunks of 128 bytes
// (two MFMA steps).  Operand rows of 128 bytes sit in LDS as 8 pieces of 16
// bytes; piece c of row r is stored at place c ^ ((r >> 1) & 7), so that the
// 16 rows that one operand read touches cover all banks once.
//
// Pipeline, ST LDS stages and two sets of operand registers.  While the
// first step of chunk c is multiplied, the second step's operands are read;
// then one barrier: every wave holds all it needs of chunk c, and chunk c + 1
// has arrived; while the second step is multiplied, chunk c + ST is copied over
// chunk c and the first operands of chunk c + 1 are read.
//
// ANY: operands at any address and any K.  No 16-byte copy into LDS can fetch
// those, so a chunk goes through registers, and two stages are enough: chunk
// c + 3 is loaded (at any address) where the copy would be, and chunk c + 2,
// loaded one chunk before, is stored over chunk c.
template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Tile8 {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
    static constexpr int KC = 128, ST = ST_;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr int STAGE = (BM + BN) * KC;
    static constexpr int ACOPIES = BM / 8 / NW, COPIES = (BM + BN) / 8 / NW;   // 8 rows each
    static_assert((BM + BN) / 8 % NW == 0 && BM / 8 % NW == 0, "copies divide evenly");
    // epilogue: each wave stages rows of its BN / WN channels
    static constexpr int WCOLS = BN / WN, REGION = ST * STAGE / NW;

    struct Frag {
        v4i a[MT], b[NT];
    };
    // of the lane's tokens t + 16m and channels n + 16j .. + 3; past the end the last one's
    struct Scales {
        float sa[MT], sw[NT][4];

        __device__ __forceinline__ void load(const GemmArgs &g, int t, int n)
        {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = n + j * 16 + i;
                    sw[j][i] = g.w_scale[col < g.N ? col : g.N - 1];
                }
#pragma unroll
            for (int m = 0; m < MT; ++m)
                sa[m] = g.a_scale[t + m * 16 < g.T ? t + m * 16 : g.T - 1];
        }
    };

    // The tile's sums over the chunks [c0, c1) of K, written or left for the join.
    template <class T, bool ANY>
    static __device__ __forceinline__ void run(const GemmArgs &g, int t0, int n0, int c0, int c1,
                                               int tile, int slice, char *lds)
    {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds0 = lds_of(lds) + wave * 1024;
        // Copy i of this wave brings rows [8 * (i * NW + wave), +8).  Rows past
        // the end repeat the last row; their results are dropped.
        uint32_t off[COPIES];
        const int crow = lane >> 3;
        const int cplace = place(wave * 8 + crow, lane & 7) * 16;   // the same for every copy
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const bool is_a = i < ACOPIES;
            const int row = ((is_a ? i : i - ACOPIES) * NW + wave) * 8 + crow;
            const int last = is_a ? g.T - 1 - t0 : g.N - 1 - n0;
            off[i] = (uint32_t)((row < last ? row : last) * (is_a ? g.lda : g.ldw)) +
                     (uint32_t)cplace;
        }
        const int8_t *abase = g.a + (long long)t0 * g.lda, *wbase = g.w + (long long)n0 * g.ldw;
        const int r = lane & 15, kq = lane >> 4;
        const int arow = wm * (MT * 16) + r, brow = BM + wn * (NT * 16) + r;
        // place() of the lane's rows is the same for every 16-row step
        const char *at[2] = {lds + arow * KC + place(arow, kq) * 16,
                             lds + arow * KC + place(arow, 4 + kq) * 16};
        const char *bt[2] = {lds + brow * KC + place(brow, kq) * 16,
                             lds + brow * KC + place(brow, 4 + kq) * 16};
        // operand i of MT + NT of a step
        auto read_one = [&](Frag &f, int i, int stage, int s) {
            if (i < NT)
                f.b[i] = *reinterpret_cast<const v4i *>(bt[s] + stage * STAGE + i * 16 * KC);
            else
                f.a[i - NT] =
                    *reinterpret_cast<const v4i *>(at[s] + stage * STAGE + (i - NT) * 16 * KC);
        };
        auto read = [&](Frag &f, int stage, int s) {
#pragma unroll
            for (int i = 0; i < MT + NT; ++i)
                read_one(f, i, stage, s);
        };
        v4i acc[NT][MT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[n][m] = v4i{0, 0, 0, 0};
        // A step's products, with `count` actions spread between them: a wave
        // that issues its copies or reads in a row waits for the address unit
        // (16 cycles a copy, shared by the workgroup's waves) with idle MFMAs.
        auto multiply = [&](const Frag &f, auto count, auto &&act) {
            constexpr int N = MT * NT, C = decltype(count)::value;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int m = j / NT, n = j % NT;
                acc[n][m] =
                    __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[n], f.a[m], acc[n][m], 0, 0, 0);
#pragma unroll
                for (int i = j * C / N; i < (j + 1) * C / N; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    act(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        constexpr std::integral_constant<int, MT + NT> kReads{};
        constexpr std::integral_constant<int, MT + NT + COPIES> kReadsAndCopies{};
        constexpr std::integral_constant<int, 0> kNothing{};
        auto clear_past_k = [&](Frag &f, int k) {
            if (k + kq * 16 >= g.K) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    f.b[n] = v4i{0, 0, 0, 0};
            }
        };
        // Chunk c to its stage.  The loop's copies are whole chunks; the last
        // chunk of K may be a part.
        auto copy_whole = [&](int c) {
            const uint32_t st = lds0 + (c - c0) % ST * STAGE;
            const int8_t *a = abase + (long long)c * KC, *w = wbase + (long long)c * KC;
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                copy16_to_lds(i < ACOPIES ? a : w, off[i], st + i * NW * 1024);
        };
        auto copy_any = [&](int c) {
            if ((c + 1) * KC <= g.K) {
                copy_whole(c);
                return;
            }
            // K past the end (K is a multiple of 16): the row's first piece is
            // read again, and the channel operand's registers are cleared below
            const uint32_t st = lds0 + (c - c0) % ST * STAGE;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
                const bool in = c * KC + cplace < g.K;
                copy16_to_lds(i < ACOPIES ? abase : wbase,
                              in ? off[i] + (uint32_t)(c * KC) : off[i] - (uint32_t)cplace,
                              st + i * NW * 1024);
            }
        };
        Frag f0, f1;
        // The scales are on their way while the last chunks are multiplied, where
        // registers are left for them.
        constexpr bool kEarly = NT * MT < 32;
        Scales sc;
        if constexpr (ANY) {
            v4i held[COPIES];
            auto at = [&](int i, int c) {
                return (i < ACOPIES ? abase : wbase) + off[i] + (uint32_t)(c * KC);
            };
            auto load = [&](int c) {
                auto here = [&](int i) { return at(i, c); };
                auto left = [&](int) { return g.K - c * KC - cplace; };
                if ((c + 1) * KC <= g.K) {
#pragma unroll
                    for (int i = 0; i < COPIES; ++i)
                        held[i] = load16(here(i));
                } else if (g.K >= 16) {
                    load_ends(held, here, left);
                } else {
                    load_short(held, here, left);
                }
            };
            auto store_one = [&](int i, int stage) {
                *reinterpret_cast<v4i *>(lds + stage * STAGE + (i * NW + wave) * 1024 +
                                         lane * 16) = held[i];
            };
            auto store = [&](int stage) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    store_one(i, stage);
            };
#pragma unroll 1
            for (int i = 0; i < 3 && c0 + i < c1; ++i) {
                load(c0 + i);
                if (i < 2)
                    store(i);
            }
            __syncthreads();
            read(f0, 0, 0);
            int c = c0, stage = 0;
            const int whole = c1 * KC <= g.K ? c1 : c1 - 1;
            for (; c + 3 < whole; ++c, stage ^= 1) {
                multiply(f0, kReads, [&](int i) { read_one(f1, i, stage, 1); });
                __syncthreads();
                multiply(f1, kReadsAndCopies, [&](int i) {
                    if (i < MT + NT) {
                        read_one(f0, i, stage ^ 1, 0);
                    } else {
                        store_one(i - MT - NT, stage);
                        held[i - MT - NT] = load16(at(i - MT - NT, c + 3));
                    }
                });
            }
#pragma unroll 1
            for (; c < c1; ++c, stage ^= 1) {              // the last ones
                read(f1, stage, 1);
                multiply(f0, kNothing, [](int) {});
                __syncthreads();
                if (c + 2 < c1)
                    store(stage);
                if (c + 3 < c1)
                    load(c + 3);
                if (c + 1 < c1)
                    read(f0, stage ^ 1, 0);
                multiply(f1, kNothing, [](int) {});
            }
            if (kEarly)
                sc.load(g, t0 + wm * (MT * 16) + r, n0 + wn * WCOLS + kq * 4);
        } else {
#pragma unroll
            for (int i = 0; i < ST; ++i)
                if (c0 + i < c1)
                    copy_any(c0 + i);
            // the first chunk has arrived; the ones behind it stay in flight
            if (c1 - c0 >= ST)
                wait_copies<(ST - 1) * COPIES>();
            else
                wait_copies<0>();
            __syncthreads();
            read(f0, 0, 0);
            int c = c0, stage = 0;
            const int whole = c1 * KC <= g.K ? c1 : c1 - 1;
            for (; c + ST < whole; ++c) {
                const int next = stage + 1 == ST ? 0 : stage + 1;
                multiply(f0, kReads, [&](int i) { read_one(f1, i, stage, 1); });
                wait_copies<(ST - 2) * COPIES>();          // chunk c + 1 has arrived
                __syncthreads();
                const uint32_t st = lds0 + stage * STAGE;
                const int8_t *a = abase + (long long)(c + ST) * KC;
                const int8_t *w = wbase + (long long)(c + ST) * KC;
                multiply(f1, kReadsAndCopies, [&](int i) {
                    if (i < MT + NT)
                        read_one(f0, i, next, 0);
                    else
                        copy16_to_lds(i - MT - NT < ACOPIES ? a : w, off[i - MT - NT],
                                      st + (i - MT - NT) * NW * 1024);
                });
                stage = next;
            }
            if (kEarly)
                sc.load(g, t0 + wm * (MT * 16) + r, n0 + wn * WCOLS + kq * 4);
            for (; c < c1; ++c) {                          // the last ones
                const int next = stage + 1 == ST ? 0 : stage + 1;
                read(f1, stage, 1);
                clear_past_k(f0, c * KC);
                multiply(f0, kNothing, [](int) {});
                wait_copies<0>();
                __syncthreads();
                if (c + ST < c1)
                    copy_any(c + ST);                      // part of a chunk
                if (c + 1 < c1)
                    read(f0, next, 0);
                clear_past_k(f1, c * KC + 64);
                multiply(f1, kNothing, [](int) {});
                stage = next;
            }
        }
        if (!kEarly)
            sc.load(g, t0 + wm * (MT * 16) + r, n0 + wn * WCOLS + kq * 4);
        if (g.split == 1 || join(g, acc, tile, slice))
            epilogue<T>(g, t0 + wm * (MT * 16), n0 + wn * WCOLS, acc, sc, lds + wave * REGION);
    }

    // Split K: every workgroup of a tile leaves its int32 sums in the workspace
    // and counts itself; the last one adds the others' to its own and writes the
    // tile (true), so nobody waits, and since the sums are integers the order
    // changes nothing.  The sums are written past the XCDs' caches (agent
    // scope), and counted only when every wave's have arrived.
    static __device__ __forceinline__ bool join(const GemmArgs &g, v4i (&acc)[NT][MT], int tile,
                                                int slice)
    {
        __shared__ int s_count;
        constexpr int PER = NT * MT * 2 * 64 * NW;         // 8-byte words of a tile's sums
        uint64_t *sums = reinterpret_cast<uint64_t *>(g.partial) + (size_t)tile * g.split * PER;
        const int at = (int)(threadIdx.x >> 6) * (NT * MT * 2 * 64) + (int)(threadIdx.x & 63);
        uint64_t *own = sums + (size_t)slice * PER + at;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t v = (uint32_t)acc[n][m][2 * h] |
                                       (uint64_t)(uint32_t)acc[n][m][2 * h + 1] << 32;
                    __hip_atomic_store(own + ((n * MT + m) * 2 + h) * 64, v, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
                }
        wait_copies<0>();
        __syncthreads();
        if (threadIdx.x == 0) {
            int32_t *count = g.counters + tile;
            s_count = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (s_count == g.split - 1)
                __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (s_count != g.split - 1)
            return false;
        for (int i = 0; i < g.split; ++i) {
            if (i == slice)
                continue;
            const uint64_t *other = sums + (size_t)i * PER + at;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t v =
                            __hip_atomic_load(other + ((n * MT + m) * 2 + h) * 64, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
                        acc[n][m][2 * h] += (int)(uint32_t)v;
                        acc[n][m][2 * h + 1] += (int)(uint32_t)(v >> 32);
                    }
        }
        return true;
    }

    // A lane holds four consecutive channels of one token per 16 x 16 result:
    // written straight to memory, an instruction would touch 16 rows with 32
    // bytes each.  The wave's rows go through its own part of LDS instead (free:
    // the loop's last barrier is past every read), and leave as whole runs of
    // WCOLS elements, 16 bytes a lane.  Pieces of 16 bytes are swizzled as the
    // operands are.
    template <class T>
    static __device__ __forceinline__ void epilogue(const GemmArgs &g, int t0, int n0,
                                                    const v4i (&acc)[NT][MT], const Scales &sc,
                                                    char *region)
    {
        constexpr int ROW = WCOLS * sizeof(T), PIECES = ROW / 16, EPP = 16 / sizeof(T);
        constexpr int MP = MT < 2 ? MT : 2;   // 16-row steps a pass
        // rows of 4, 8 or 16 pieces are swizzled, others lie a piece further apart
        constexpr bool kSwizzled = (PIECES & (PIECES - 1)) == 0;
        constexpr int PITCH = kSwizzled ? ROW : ROW + 16;
        static_assert(MT % MP == 0 && PIECES >= 4 && MP * 16 * PITCH <= REGION, "passes fit");
        static_assert(MP * 16 * PIECES % 64 == 0, "whole stores");
        auto spread = [](int row) {
            return !kSwizzled ? 0 : PIECES >= 8 ? (row >> 1) & 7 : (row >> 2) & 3;
        };
        const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
#pragma unroll
        for (int p = 0; p < MT / MP; ++p) {
            Out4<T> add[MP][NT];
            if (g.addend) {
#pragma unroll
                for (int mm = 0; mm < MP; ++mm)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        add[mm][n] = load_addend<T>(g, t0 + (p * MP + mm) * 16 + r,
                                                    n0 + n * 16 + kq * 4);
            }
#pragma unroll
            for (int mm = 0; mm < MP; ++mm) {
                const int m = p * MP + mm, row = mm * 16 + r;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int byte = (n * 16 + kq * 4) * (int)sizeof(T);
                    char *at = region + row * PITCH + (((byte >> 4) ^ spread(row)) << 4) +
                               (byte & 15);
                    Out4<T> v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float f = (float)acc[n][m][i] * sc.sa[m] * sc.sw[n][i];
                        if (g.addend)
                            f += to_float(add[mm][n].v[i]);
                        v.v[i] = from_float<T>(f);
                    }
                    if constexpr (sizeof(T) == 4)
                        *reinterpret_cast<v4i *>(at) = __builtin_bit_cast(v4i, v);
                    else
                        *reinterpret_cast<uint64_t *>(at) = __builtin_bit_cast(uint64_t, v);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            constexpr int STEPS = MP * 16 * PIECES / 64;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int id = i * 64 + lane, row = id / PIECES, c = id % PIECES;
                const int t = t0 + p * MP * 16 + row, n = n0 + c * EPP;
                const v4i v = *reinterpret_cast<const v4i *>(region + row * PITCH +
                                                             ((c ^ spread(row)) << 4));
                store_piece<T>(g, t, n, v);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }

    template <class T>
    static __device__ __forceinline__ Out4<T> load_addend(const GemmArgs &g, int t, int n)
    {
        Out4<T> r{};
        if (t < g.T && n < g.N) {
            const T *p = static_cast<const T *>(g.addend) + t * g.ld_add + n;
            if (n + 4 <= g.N) {
                r = *reinterpret_cast<const Out4<T> *>(p);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < g.N)
                        r.v[i] = p[i];
            }
        }
        return r;
    }

    template <class T>
    static __device__ __forceinline__ void store_piece(const GemmArgs &g, int t, int n, v4i v)
    {
        constexpr int EPP = 16 / sizeof(T);
        if (t >= g.T || n >= g.N)
            return;
        struct __attribute__((packed, aligned(sizeof(T)))) Piece { T v[EPP]; };
        Piece x = __builtin_bit_cast(Piece, v);
        T *o = static_cast<T *>(g.out) + t * g.ldo + n;
        if (n + EPP <= g.N) {
            *reinterpret_cast<Piece *>(o) = x;
        } else {
#pragma unroll
            for (int i = 0; i < EPP; ++i)
                if (n + i < g.N)
                    o[i] = x.v[i];
        }
    }
};

constexpr int kBand = 8;

template <class C, class T, bool ANY>
__global__ void __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_tile_kernel(GemmArgs g, int tiles_m, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) char lds[C::ST * C::STAGE];
    // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of
    // tiles, so its L2 serves neighbours that share an operand: tiles are
    // numbered down bands of kBand rows, so that the 32 an XCD runs at a time
    // are about as many rows as columns.
    const int total = tiles_m * tiles_n * g.split, per = (total + 7) / 8;
    int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= total || (int)(blockIdx.x >> 3) >= per)
        return;
    const int slice = id % g.split;
    id /= g.split;
    const int band = id / (kBand * tiles_n), rest = id - band * (kBand * tiles_n);
    const int rows = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
    const int tm = band * kBand + rest % rows, tn = rest / rows;
    const int chunks = (g.K + C::KC - 1) / C::KC;
    C::template run<T, ANY>(g, tm * C::BM, tn * C::BN, slice * chunks / g.split,
                       (slice + 1) * chunks / g.split, id, slice, lds);
}

// f(a value of the output type).
template <class F>
hipError_t with_type(int out_dtype, F &&f)
{
    if (out_dtype == MOE_WNA16_BF16)
        return f(Bf16{});
    if (out_dtype == MOE_WNA16_FP16)
        return f(Fp16{});
    return f(0.f);
}

template <class C, bool ANY>
hipError_t launch_tile(const GemmArgs &g, int out_dtype, hipStream_t stream)
{
    const int tm = (g.T + C::BM - 1) / C::BM, tn = (g.N + C::BN - 1) / C::BN;
    const unsigned grid = (unsigned)((tm * tn * g.split + 7) / 8 * 8);
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_tile_kernel<C, decltype(zero), ANY>, dim3(grid), 64 * C::NW, stream, g,
                      tm, tn);
    });
}

template <int TC, int NW, int R, bool ANY>
hipError_t launch_stream(const GemmArgs &g, int out_dtype, hipStream_t stream)
{
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_stream_kernel<decltype(zero), TC, NW, R, ANY>,
                      dim3((unsigned)((g.N + 15) / 16)), 64 * NW, stream, g);
    });
}

bool aligned16(const GemmArgs &g)
{
    return (reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.w) |
            (uintptr_t)g.lda | (uintptr_t)g.ldw | (uintptr_t)g.K) % 16 == 0;
}

}  // namespace

namespace {

// The tiles, and what they cost in microseconds on an MI355X: launch, first
// copies and epilogue once; a chunk of 128 K with one workgroup a CU, when few
// CUs run one and when all do; a chunk for each of two workgroups a CU, where
// their LDS allows it; every further tile of a CU.  Fitted to N and T that fill
// the 256 CUs in part, once, twice and four times, at K from 2048 to 16384, with
// uniform codes: with those of activations most take less, up to a fifth (T = 2047,
// N = 2056, K = 4096: 25.2 us by the model, 21.8 to 22.7 measured).
// Large tiles do a chunk's products in less time (2.5 POP/s, where the clock
// falls for power; 64 x 64: 1.4), small ones cover few rows with more CUs.  128 x
// 192 serves sizes that 128 x 256 or 256 x 256 would leave in part idle; without
// it (K = 4096): T = 1280, N = 4096 24.8 -> 26.8 us; 2047, 2056 22.7 -> 25.9; 3000,
// 1536 23.7 -> 26.1; 3000, 3000 45.0 -> 53.8; 2048, 6144 58 -> 66; 3000, 6144 81 ->
// 103; and at K = 1024 768, 6144 11.5 -> 15.8; 1536, 3000 11.2 -> 16.4.
struct TileCost {
    int bm, bn;
    float once, few, all, two, more;
};
constexpr TileCost kTiles[] = {
    {256, 256, 10.6f, 1.30f, 1.73f, 0.f, 8.0f}, {128, 256, 9.5f, 0.42f, 0.76f, 0.f, 10.0f},
    {128, 192, 8.4f, 0.36f, 0.60f, 0.f, 8.0f},  {128, 128, 7.3f, 0.30f, 0.44f, 0.f, 5.5f},
    {128, 64, 5.5f, 0.255f, 0.30f, 0.542f, 1.3f}, {64, 64, 4.8f, 0.163f, 0.19f, 0.372f, 0.2f},
};
constexpr int kMaxSplit = 16;

// With K split over `split` workgroups a tile, the chunks are fewer, every
// workgroup writes its sums and the last one of a tile reads the others'.
// N = 512, T = 128, K = 16384 (64 x 64 tiles): 25.7 us whole, 12.7 us in eight;
// K = 4096: 10.1 us whole, 9.0 us in four, 10.6 us in eight.
float tile_cost(const TileCost &c, long long tiles, int chunks, int split)
{
    const long long groups = tiles * split;
    const float per_cu = (float)((groups + 255) / 256), each = (float)((chunks + split - 1) / split);
    const float pairs = c.two > 0.f ? (float)((groups + 255) / 256 / 2) : 0.f;
    const float one = c.few + (c.all - c.few) * (groups < 256 ? (float)groups / 256.f : 1.f);
    const float join =
        split > 1 ? 1.f + 0.35f * split + 0.006f / 4096.f * c.bm * c.bn * (float)groups : 0.f;
    return c.once + each * (pairs * c.two + (per_cu - 2.f * pairs) * one) + (per_cu - 1.f) * c.more +
           join;
}

}  // namespace

GemmPlan gemm_plan(int T, int N, int K)
{
    GemmPlan p{};
    p.split = 1;
    // Streaming against tiles (K split where the cost model splits it), us:
    //              N = 512, K = 4096  N = K = 4096  N = 16384, K = 4096  N = 512, K = 16384
    //   T = 4           3.8 / 7.8       5.5 / 9.1        14.6 / 19.2          6.6 / 11.5
    //   T = 16          4.0 / 7.9       5.6 / 9.2        16.7 / 19.5          8.0 / 11.6
    //   T = 32          4.9 / 7.9       6.7 / 9.2        21.1 / 19.9         10.6 / 11.7
    //   T = 64          6.7 / 8.0       8.4 / 9.4        26.6 / 20.6         15.5 / 11.8
    // Past 32 tokens the tiles are ahead where N or K is long (N = K = 16384, T = 64:
    // 88.2 / 64.3), and 1 to 3 us behind elsewhere.
    if (T <= 64) {
        p.variant = 0;
        p.bm = (T + 7) / 8 * 8;
        p.bn = 16;
        return p;
    }
    p.variant = 1;
    float best = 0.f;
    for (const TileCost &c : kTiles)
        for (int split = 1; split <= kMaxSplit; split *= 2) {
            const long long tiles = (long long)((T + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
            // at least two chunks a slice; the GPU is not filled twice to split
            if (split > 1 && (tiles * split > 512 || (K + 127) / 128 < 2 * split))
                break;
            const float t = tile_cost(c, tiles, (K + 127) / 128, split);
            if (p.bm == 0 || t < best) {
                best = t;
                p.bm = c.bm;
                p.bn = c.bn;
                p.split = split;
                p.workspace = split == 1 ? 0
                                         : kCounterBytes + (size_t)tiles * split * c.bm * c.bn * 4;
            }
        }
    return p;
}

namespace {

template <bool ANY>
hipError_t launch_planned(const GemmArgs &g, const GemmPlan &p, int out_dtype, hipStream_t stream)
{
    if (p.variant == 1) {
        // through registers, 256 x 256 would need more of them than there are:
        // two tiles of 128 x 256 (no more workspace than the planned tile)
        if constexpr (!ANY)
            if (p.bm == 256)
                return launch_tile<Tile8<256, 256, 2, 4, 2>, ANY>(g, out_dtype, stream);
        if (p.bn == 256)
            return launch_tile<Tile8<128, 256, 2, 4, ANY ? 2 : 3>, ANY>(g, out_dtype, stream);
        if (p.bn == 192)
            return launch_tile<Tile8<128, 192, 2, 4, ANY ? 2 : 3>, ANY>(g, out_dtype, stream);
        if (p.bn == 128)
            return launch_tile<Tile8<128, 128, 2, 4, ANY ? 2 : 4>, ANY>(g, out_dtype, stream);
        if (p.bm == 128)
            return launch_tile<Tile8<128, 64, 2, 2, ANY ? 2 : 3>, ANY>(g, out_dtype, stream);
        return launch_tile<Tile8<64, 64, 2, 2, ANY ? 2 : 4>, ANY>(g, out_dtype, stream);
    }
    // Up to 256 workgroups (one a CU): all of the LDS for one, so that most
    // of its K is in flight at once (N = 4096, K = 4096, T = 4: 5.5 us, with
    // half the waves 5.8 us).  More: two a CU, so that one starts while the
    // other joins (N = 8192: 7.9 us against 8.7 us, N = 16384: 14.8 against 16.8).
    const bool one = g.N <= 16 * 256;
    if (g.T <= 8)
        return one ? launch_stream<1, 16, 2, ANY>(g, out_dtype, stream)
                   : launch_stream<1, 8, 3, ANY>(g, out_dtype, stream);
    if (g.T <= 16)
        return one ? launch_stream<2, 16, 2, ANY>(g, out_dtype, stream)
                   : launch_stream<2, 8, 2, ANY>(g, out_dtype, stream);
    if (g.T <= 32)
        return launch_stream<4, 4, 3, ANY>(g, out_dtype, stream);
    return launch_stream<8, 4, 2, ANY>(g, out_dtype, stream);
}

}  // namespace

hipError_t launch_gemm_w8a8(const GemmArgs &g, const GemmPlan &p, int out_dtype,
                            hipStream_t stream)
{
    return aligned16(g) ? launch_planned<false>(g, p, out_dtype, stream)
                        : launch_planned<true>(g, p, out_dtype, stream);
}

}  // namespace wna16
