// Product in 8-bit floating point (e4m3) with a scale for each 128 elements of
// a token and each 128 x 128 block of the weight, plain and by expert:
//   out[t][n] = round( sum_b sa[t][b] sw[n / 128][b] sum_{k in b} a[t][k] w[n][k] + add[t][n] )
// One MFMA takes the 128 elements of a block at once (16 x 16 x 128), its sum in
// FP32.  The block's scale is the same for every channel of a wave's tile, so
// a result takes one product for the scale of its token and four FMAs for its
// four channels, which run beside the MFMAs.  Blocks are added in order, slices
// of K in order of the slices: results do not depend on timing.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "expert_ops.hpp"
#include "lds_copy.hpp"
#include "moe_wna16.h"
#include "wave.hpp"

namespace wna16 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// A lane's half of a 128-element row piece: 16 bytes of the first and of the
// second 64.  Which element sits where does not matter as long as both operands
// agree.
__device__ __forceinline__ v8i both(v4i lo, v4i hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ v4f mfma_block(v8i w, v8i a)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                            0, 0, 0);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Each active lane l's 4 bytes at p land at LDS address lds + l * 4.
__device__ __forceinline__ void copy4_to_lds(const void *p, uint32_t lds_in)
{
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_in);
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Which rows and weights a workgroup's tile has.
struct Where {
    int expert, row0, count;    // rows of the output
    int column;                 // tile column, -1: no such tile
};

// Grouped: an expert's rows, and how many tiles of bm rows they make.  Offsets are
// held inside [0, rows of the output].
__device__ __forceinline__ int tiles_of(const GemmFp8Args &g, int e, int bm, int &row0, int &rows)
{
    int lo = 0, hi = 0;
    if (e < g.experts) {
        lo = g.offsets[e];
        hi = g.offsets[e + 1];
    }
    lo = lo < 0 ? 0 : lo > g.T ? g.T : lo;
    hi = hi < lo ? lo : hi > g.T ? g.T : hi;
    row0 = lo;
    rows = hi - lo;
    return (rows + bm - 1) / bm;
}

// What four consecutive outputs of one token, from column n, need besides
// their sums: loaded while the operands are on their way.
template <class T>
struct Beside {
    Out4<T> add;

    __device__ __forceinline__ void load(const GemmFp8Args &g, int t, int n, int t_end)
    {
        add = Out4<T>{};
        if (t >= t_end || n >= g.N || !g.addend)
            return;
        const T *p = static_cast<const T *>(g.addend) + t * g.ld_add + n;
        if (n + 4 <= g.N) {
            add = *reinterpret_cast<const Out4<T> *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < g.N)
                    add.v[i] = p[i];
        }
    }
    __device__ __forceinline__ void emit(const GemmFp8Args &g, int t, int n, v4f acc, int t_end) const
    {
        if (t >= t_end || n >= g.N)
            return;
        T *o = static_cast<T *>(g.out) + t * g.ldo + n;
        Out4<T> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.v[i] = from_float<T>(g.addend ? acc[i] + to_float(add.v[i]) : acc[i]);
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

// ---------------------------------------------------------------------------
// Few tokens (decode): the weights are streamed once.  A workgroup owns 16
// channels and up to 8 * TC tokens; its waves take the blocks of K in turn,
// each through a ring of R stages of its own, and add their sums through LDS at
// the end.  A stage holds the block's 16 channels, the tokens, and their scales.
// ---------------------------------------------------------------------------
template <class T, int TC, int NW, int R>
__device__ __forceinline__ void stream_tile(const GemmFp8Args &g, const uint8_t *w,
                                            const float *w_scale, int n0, int t0, int count,
                                            char *lds)
{
    constexpr int MT = TC < 2 ? 1 : TC / 2, ROWS = 16 + 8 * TC;
    constexpr int STAGE = ROWS * 128 + 512, SCALES = ROWS * 128;   // 64 tokens', then the weight's
    constexpr int COPIES = ROWS / 8, ALL = COPIES + 2;
    static_assert(MT <= NW, "a wave for every 16 tokens");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char *ring = lds + wave * (R * STAGE);
    const uint32_t ring0 = lds_of(ring);
    const int crow = lane >> 3;
    uint32_t off[COPIES];
    const int cplace[2] = {place(crow, lane & 7) * 16, place(8 + crow, lane & 7) * 16};
    const uint8_t *wbase = w + (long long)n0 * g.ldw;
    const uint8_t *abase = g.rows ? g.a : g.a + (long long)t0 * g.lda;
    auto a_row = [&](int r) {               // of a, from abase: rows past the end repeat the last one
        r = r < count ? r : count - 1;
        if (!g.rows)
            return r;
        const int s = g.rows[t0 + r];
        return (unsigned)s < (unsigned)g.a_rows ? s : 0;
    };
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int row = i < 2 ? i * 8 + crow : (i - 2) * 8 + crow;
        const int last = g.N - 1 - n0;
        off[i] = i < 2 ? (uint32_t)(row < last ? row : last) * (uint32_t)g.ldw
                       : (uint32_t)a_row(row) * (uint32_t)g.lda;
        off[i] += (uint32_t)cplace[i & 1];
    }
    // lane l brings token l's scale (lanes past the tokens: none), lane 0 the weight's
    const float *sa = g.a_scale + (g.rows ? 0 : (long long)t0 * g.lda_s) +
                      (long long)a_row(lane < 8 * TC ? lane : 0) * g.lda_s;
    const float *sw = w_scale + (long long)(n0 >> 7) * g.ldw_s;
    const int chunks = (g.K + 127) / 128;
    auto copy = [&](int c, int stage) {
        const bool part = (c + 1) * 128 > g.K;
        const uint32_t st = ring0 + (uint32_t)(stage * STAGE);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            uint32_t o = off[i] + (uint32_t)(c * 128);
            // K past the end (a multiple of 16): the row's first piece is read
            // again, and the channels' registers are cleared below
            if (part && c * 128 + cplace[i & 1] >= g.K)
                o = off[i] - (uint32_t)cplace[i & 1];
            copy16_to_lds(i < 2 ? wbase : abase, o, st + i * 1024);
        }
        if (lane < 8 * TC)
            copy4_to_lds(sa + c, st + SCALES);
        if (lane < 1)
            copy4_to_lds(sw + c, st + SCALES + 256);
    };
    const int r = lane & 15, kq = lane >> 4;
    Beside<T> beside;
    const int t_end = t0 + count;
    if (wave < MT)
        beside.load(g, t0 + wave * 16 + r, n0 + kq * 4, t_end);
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        acc[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (wave + i * NW < chunks)
            copy(wave + i * NW, i);
    for (int c = wave, stage = 0; c < chunks; c += NW, stage = stage + 1 == R ? 0 : stage + 1) {
        // the copies behind this chunk's stay in flight
        if (c + (R - 1) * NW < chunks)
            wait_copies<(R - 1) * ALL>();
        else
            wait_copies<0>();
        const char *st = ring + stage * STAGE;
        v4i fw[2], fa[2][MT];
        float s[MT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fw[h] = *reinterpret_cast<const v4i *>(st + r * 128 + place(r, h * 4 + kq) * 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int row = TC == 1 ? 16 + (r & 7) : 16 + m * 16 + r;
                fa[h][m] = *reinterpret_cast<const v4i *>(st + row * 128 +
                                                          place(row, h * 4 + kq) * 16);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
            s[m] = *reinterpret_cast<const float *>(st + SCALES +
                                                    (TC == 1 ? r & 7 : m * 16 + r) * 4);
        const float ws = *reinterpret_cast<const float *>(st + SCALES + 256);
        if ((c + 1) * 128 > g.K) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (c * 128 + h * 64 + kq * 16 >= g.K)
                    fw[h] = v4i{0, 0, 0, 0};
        }
        if (c + R * NW < chunks) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read
            copy(c + R * NW, stage);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const v4f p = mfma_block(both(fw[0], fw[1]), both(fa[0][m], fa[1][m]));
            const float f = s[m] * ws;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[m][i] = __builtin_fmaf(p[i], f, acc[m][i]);
        }
    }
    __syncthreads();                                // every ring has been read
    // the waves' sums, in their order; wave m writes tokens [t0 + 16 m, +16)
    float *part = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        *reinterpret_cast<v4f *>(part + ((wave * MT + m) * 64 + lane) * 4) = acc[m];
    __syncthreads();
    if (wave < MT) {
        v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const v4f p = *reinterpret_cast<const v4f *>(part + ((i * MT + wave) * 64 + lane) * 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum[k] += p[k];
        }
        beside.emit(g, t0 + wave * 16 + (lane & 15), n0 + (lane >> 4) * 4, sum, t_end);
    }
}

template <int TC, int NW, int R>
constexpr int stream_lds()
{
    constexpr int ring = NW * R * ((16 + 8 * TC) * 128 + 512), part = NW * (TC < 2 ? 1 : TC / 2) * 1024;
    return ring > part ? ring : part;
}

template <class T, int TC, int NW, int R>
__global__ void __launch_bounds__(64 * NW) gemm_fp8_stream_kernel(GemmFp8Args g)
{
    __shared__ __attribute__((aligned(1024))) char lds[stream_lds<TC, NW, R>()];
    stream_tile<T, TC, NW, R>(g, g.w, g.w_scale, blockIdx.x * 16, 0, g.T, lds);
}

// A wave's search for tile `id`, where every expert in turn has its row tiles
// times `columns` tiles, rows first: 64 experts at a time.
__device__ __forceinline__ Where find_tile(const GemmFp8Args &g, int id, int bm, int columns)
{
    const int lane = threadIdx.x & 63;
    Where r{0, 0, 0, -1};
    int base = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
        int row0, rows;
        const int n = tiles_of(g, e0 + lane, bm, row0, rows);
        int incl = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d)
                incl += o;
        }
        const uint64_t past = __ballot((base + incl) * columns > id);
        if (past) {
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1);
            const int tiles = __builtin_amdgcn_readlane(n, l);
            const int rest = id - (base + __builtin_amdgcn_readlane(incl, l) - tiles) * columns;
            const int at = rest % tiles * bm, left = __builtin_amdgcn_readlane(rows, l) - at;
            r.expert = e0 + l;
            r.row0 = __builtin_amdgcn_readlane(row0, l) + at;
            r.count = left < bm ? left : bm;
            r.column = rest / tiles;
            break;
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    return r;
}

template <class T, int TC, int NW, int R>
__global__ void __launch_bounds__(64 * NW) gemm_fp8_grouped_stream_kernel(GemmFp8Args g)
{
    __shared__ __attribute__((aligned(1024))) char lds[stream_lds<TC, NW, R>()];
    const Where at = find_tile(g, blockIdx.y, 8 * TC, 1);
    if (at.column < 0)
        return;
    stream_tile<T, TC, NW, R>(g, g.w + at.expert * g.w_expert, g.w_scale + at.expert * g.ws_expert,
                              blockIdx.x * 16, at.row0, at.count, lds);
}

// ---------------------------------------------------------------------------
// Many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

// Tile of BM tokens x BN channels, WM x WN waves.  Operand rows of a block (128
// bytes) sit in LDS as 8 pieces of 16 bytes, swizzled by place(); a stage is one
// block of K, a ring has ST of them.  The scales of four blocks lie next to each
// other in memory; they are copied together, into one of two buffers.
//
// Pipeline: a wave holds the channels' operands of its block and up to four of
// the tokens', which it reads two steps of 16 tokens ahead.  Before the last step
// of block c comes the one barrier of a block: every wave holds all it needs of
// block c, and block c + 1 has arrived.  Behind it block c + ST is copied over
// block c, spread over a block's time, and block c + 1's operands are read while
// the last step of block c is multiplied.  A product's FMAs follow it three MFMAs
// later, so that none waits for the one before.
template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct TileF8 {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
    static constexpr int KC = 128, ST = ST_;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr int STAGE = (BM + BN) * KC;
    static constexpr int ACOPIES = BM / 8 / NW, COPIES = (BM + BN) / 8 / NW;   // 8 rows each
    static_assert((BM + BN) / 8 % NW == 0 && BM / 8 % NW == 0, "copies divide evenly");
    static constexpr int WCOLS = BN / WN;
    static_assert(128 % WCOLS == 0, "a wave's channels lie in one block");
    // scales: 16 bytes (four blocks) for each token and each 128 channels
    static constexpr int SROWS = BM + (BN + 127) / 128, SBUF = (SROWS * 16 + 63) / 64 * 64;
    static constexpr int SCOPIES = BM / 16;                 // of 16 tokens each
    static constexpr int SCALES = ST * STAGE, LDS = SCALES + 2 * SBUF;
    static constexpr int REGION = ST * STAGE / NW;          // a wave's, in the epilogue
    static constexpr int AR = MT < 4 ? 2 : 4;      // token operands held
    static constexpr int N = MT * NT, D = NT < 4 ? 2 : 3;   // FMAs D MFMAs behind
    static_assert(N % 4 == 0 && MT % AR == 0, "registers take turns");

    template <class T>
    static __device__ __forceinline__ void run(const GemmFp8Args &g, const uint8_t *w,
                                               const float *w_scale, int t0, int count, int n0,
                                               int c0, int c1, int tile, int slice, char *lds)
    {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds0 = lds_of(lds) + wave * 1024;
        const uint8_t *abase = g.rows ? g.a : g.a + (long long)t0 * g.lda;
        const uint8_t *wbase = w + (long long)n0 * g.ldw;
        auto a_row = [&](int r) {
            r = r < count ? r : count - 1;
            if (!g.rows)
                return r;
            const int s = g.rows[t0 + r];
            return (unsigned)s < (unsigned)g.a_rows ? s : 0;
        };
        // Copy i of this wave brings rows [8 * (i * NW + wave), +8).  Rows past
        // the end repeat the last row; their results are dropped.
        uint32_t off[COPIES];
        const int crow = lane >> 3;
        const int cplace = place(wave * 8 + crow, lane & 7) * 16;   // the same for every copy
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int row = ((i < ACOPIES ? i : i - ACOPIES) * NW + wave) * 8 + crow;
            const int last = g.N - 1 - n0;
            off[i] = i < ACOPIES ? (uint32_t)a_row(row) * (uint32_t)g.lda
                                 : (uint32_t)(row < last ? row : last) * (uint32_t)g.ldw;
            off[i] += (uint32_t)cplace;
        }
        // Scale copy i of this wave: tokens [16 * (i * NW + wave), +16), four blocks
        // each; one more of wave 0, the weight's.
        constexpr int SW = (SCOPIES + NW - 1) / NW;
        const int kb = (g.K + KC - 1) / KC;
        const float *sa[SW];
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            const int row = (i * NW + wave) * 16 + (lane >> 2);
            sa[i] = g.a_scale + (g.rows ? 0 : (long long)t0 * g.lda_s) +
                    (long long)a_row(row < BM ? row : BM - 1) * g.lda_s;
        }
        const int nblocks = (g.N + 127) / 128 - 1;
        int nb = n0 / 128 + (lane >> 2);
        nb = nb < nblocks ? nb : nblocks;
        const float *sw = w_scale + (long long)nb * g.ldw_s;
        const uint32_t scale0 = lds_of(lds) + SCALES;
        auto copy_scales = [&](int c) {                 // blocks [c, c + 4)
            const uint32_t buf = scale0 + ((c - c0) & 4 ? SBUF : 0);
            int b = c + (lane & 3);
            b = b < kb ? b : kb - 1;
#pragma unroll
            for (int i = 0; i < SW; ++i)
                if (i * NW + wave < SCOPIES)
                    copy4_to_lds(sa[i] + b, buf + (uint32_t)((i * NW + wave) * 256));
            if (wave == 0 && lane < 4 * (SROWS - BM))
                copy4_to_lds(sw + b, buf + BM * 16);
        };
        auto copy_part = [&](int c) {
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
        const int r = lane & 15, kq = lane >> 4;
        const int arow = wm * (MT * 16) + r, brow = BM + wn * (NT * 16) + r;
        // place() of the lane's rows is the same for every 16-row step
        const char *at[2] = {lds + arow * KC + place(arow, kq) * 16,
                             lds + arow * KC + place(arow, 4 + kq) * 16};
        const char *bt[2] = {lds + brow * KC + place(brow, kq) * 16,
                             lds + brow * KC + place(brow, 4 + kq) * 16};
        const char *sat = lds + SCALES + arow * 16;
        const char *swt = lds + SCALES + (BM + wn * WCOLS / 128) * 16;
        v8i fb[NT], fa[AR];
        float raw[AR], f[AR], ws = 0.f;
        v4f tmp[4], acc[NT][MT];
        auto read_b = [&](int n, int stage) {
            const int o = stage * STAGE + n * 16 * KC;
            fb[n] = both(*reinterpret_cast<const v4i *>(bt[0] + o),
                         *reinterpret_cast<const v4i *>(bt[1] + o));
        };
        auto read_a = [&](int m, int stage, int sbuf) {
            const int o = stage * STAGE + m * 16 * KC;
            fa[m % AR] = both(*reinterpret_cast<const v4i *>(at[0] + o),
                              *reinterpret_cast<const v4i *>(at[1] + o));
            raw[m % AR] = *reinterpret_cast<const float *>(sat + sbuf + m * 256);
        };
        auto add_up = [&](int j) {                      // the FMAs of product j
            const int m = j / NT, n = j % NT;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[n][m][i] = __builtin_fmaf(tmp[j % 4][i], f[m % AR], acc[n][m][i]);
        };
        auto product = [&](int j) {
            tmp[j % 4] = mfma_block(fb[j % NT], fa[j / NT % AR]);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[n][m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tmp[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < AR; ++i)
            f[i] = 0.f;
        const bool ragged = g.K % KC != 0;
        const int part = ragged ? kb - 1 : -1;          // the chunk of which K ends inside
        auto clear_past_k = [&](int c) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                v4i lo = __builtin_shufflevector(fb[n], fb[n], 0, 1, 2, 3);
                v4i hi = __builtin_shufflevector(fb[n], fb[n], 4, 5, 6, 7);
                if (c * KC + kq * 16 >= g.K)
                    lo = v4i{0, 0, 0, 0};
                if (c * KC + 64 + kq * 16 >= g.K)
                    hi = v4i{0, 0, 0, 0};
                fb[n] = both(lo, hi);
            }
        };
        // the first chunks
        copy_scales(c0);
#pragma unroll
        for (int i = 0; i < ST; ++i)
            if (c0 + i < c1) {
                if (c0 + i == part) {
                    copy_part(c0 + i);
                } else {
#pragma unroll
                    for (int k = 0; k < COPIES; ++k)
                        copy16_to_lds((k < ACOPIES ? abase : wbase) + (long long)(c0 + i) * KC,
                                      off[k], lds0 + i * STAGE + k * NW * 1024);
                }
            }
        if (c1 - c0 >= ST)
            wait_copies<(ST - 1) * COPIES>();
        else
            wait_copies<0>();
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
            read_b(n, 0);
        read_a(0, 0, 0);
        read_a(1, 0, 0);
        ws = *reinterpret_cast<const float *>(swt);
        if (c0 == part)
            clear_past_k(c0);
        // Steps 0 .. MT - 2 of a chunk, with act(j) behind product j.
        auto head = [&](int stage, int sbuf, auto &&act) {
#pragma unroll
            for (int j = 0; j < N - NT; ++j) {
                const int m = j / NT, n = j % NT;
                if (n == 0)
                    f[m % AR] = raw[m % AR] * ws;
                product(j);
                __builtin_amdgcn_sched_barrier(0);
                add_up(j >= D ? j - D : N - D + j);     // the first ones are the chunk before's
                if (n == (AR > 2 ? 1 : NT - 1) && m + 2 < MT)
                    read_a(m + 2, stage, sbuf);
                act(j);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // The last step, while block c + 1's first operands are read.
        auto last = [&](int next, int sbuf, auto &&act) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int j = N - NT + n;
                if (n == 0)
                    f[(MT - 1) % AR] = raw[(MT - 1) % AR] * ws;
                product(j);
                __builtin_amdgcn_sched_barrier(0);
                add_up(j - D);
                read_b(n, next);
                if (n == 0)
                    read_a(0, next, sbuf);
                if (n == (AR > 2 ? 1 : NT - 1))
                    read_a(1, next, sbuf);
                if (n == NT - 1)
                    ws = *reinterpret_cast<const float *>(swt + sbuf);
                act(n);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto scale_of = [&](int c) {                    // offset of the chunk's scales
            return ((c - c0) & 4 ? SBUF : 0) + ((c - c0) & 3) * 4;
        };
        head(0, 0, [](int) {});
        int stage = 0, c = c0;
        // One run of instructions without a branch: the compiler moves the FMAs out
        // of sight of their products otherwise, and runs out of registers.
        const int whole = part >= 0 && part < c1 ? c1 - 1 : c1;
        for (; c + ST < whole; ++c) {
            const int next = stage + 1 == ST ? 0 : stage + 1, cn = c + ST;
            // chunk c + 1 has arrived, and every wave holds the rest of chunk c
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            wait_copies<(ST - 2) * COPIES>();
            __syncthreads();
            if (((cn - c0) & 3) == 0)
                copy_scales(cn);
            const uint32_t st = lds0 + stage * STAGE;
            const uint8_t *an = abase + (long long)cn * KC, *wn_ = wbase + (long long)cn * KC;
            const int sbuf = scale_of(c + 1);
            // chunk cn over chunk c, the copies spread over the chunk's products
            auto spread = [&](int k) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    if (i * (N - NT) / COPIES == k)
                        copy16_to_lds(i < ACOPIES ? an : wn_, off[i], st + i * NW * 1024);
            };
            last(next, sbuf, spread);
            head(next, sbuf, [&](int j) { spread(j + NT); });
            stage = next;
        }
        for (;; ++c) {                                  // the last ones
            const int next = stage + 1 == ST ? 0 : stage + 1;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            wait_copies<0>();
            __syncthreads();
            if (c + ST < c1) {                          // the part of a chunk
                if (((c + ST - c0) & 3) == 0)
                    copy_scales(c + ST);
                copy_part(c + ST);
            }
            const int sbuf = scale_of(c + 1);
            last(next, sbuf, [](int) {});               // past the end: values that nobody uses
            if (c + 1 == c1)
                break;
            if (c + 1 == part)
                clear_past_k(c + 1);
            head(next, sbuf, [](int) {});
            stage = next;
        }
#pragma unroll
        for (int j = N - D; j < N; ++j)
            add_up(j);
        if (g.split == 1 || join(g, acc, tile, slice))
            epilogue<T>(g, t0 + wm * (MT * 16), t0 + count, n0 + wn * WCOLS, acc,
                        lds + wave * REGION);
    }

    // Split K: every workgroup of a tile leaves its sums in the workspace and
    // counts itself; the last one adds them up in the order of the slices and
    // writes the tile (true), so nobody waits and no order of arrival shows.  The
    // sums are written past the XCDs' caches (agent scope), and counted only
    // when every wave's have arrived.
    static __device__ __forceinline__ bool join(const GemmFp8Args &g, v4f (&acc)[NT][MT], int tile,
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
                    const uint64_t v = __float_as_uint(acc[n][m][2 * h]) |
                                       (uint64_t)__float_as_uint(acc[n][m][2 * h + 1]) << 32;
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
            const uint64_t *one = sums + (size_t)i * PER + at;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t v =
                            __hip_atomic_load(one + ((n * MT + m) * 2 + h) * 64, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
                        const float lo = __uint_as_float((uint32_t)v);
                        const float hi = __uint_as_float((uint32_t)(v >> 32));
                        acc[n][m][2 * h] = i ? acc[n][m][2 * h] + lo : lo;
                        acc[n][m][2 * h + 1] = i ? acc[n][m][2 * h + 1] + hi : hi;
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
    static __device__ __forceinline__ void epilogue(const GemmFp8Args &g, int t0, int t_end, int n0,
                                                    const v4f (&acc)[NT][MT], char *region)
    {
        constexpr int ROW = WCOLS * sizeof(T), PIECES = ROW / 16, EPP = 16 / sizeof(T);
        constexpr int MP = MT < 2 ? MT : 2;   // 16-row steps a pass
        static_assert(MT % MP == 0 && PIECES >= 4 && MP * 16 * ROW <= REGION, "passes fit");
        static_assert(MP * 16 * PIECES % 64 == 0, "whole stores");
        auto spread = [](int row) { return PIECES >= 8 ? (row >> 1) & 7 : (row >> 2) & 3; };
        const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
#pragma unroll
        for (int p = 0; p < MT / MP; ++p) {
            Out4<T> add[MP][NT];
            if (g.addend) {
#pragma unroll
                for (int mm = 0; mm < MP; ++mm)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        add[mm][n] = load_addend<T>(g, t0 + (p * MP + mm) * 16 + r, t_end,
                                                    n0 + n * 16 + kq * 4);
            }
#pragma unroll
            for (int mm = 0; mm < MP; ++mm) {
                const int m = p * MP + mm, row = mm * 16 + r;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int byte = (n * 16 + kq * 4) * (int)sizeof(T);
                    char *at = region + row * ROW + (((byte >> 4) ^ spread(row)) << 4) + (byte & 15);
                    Out4<T> v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float f = acc[n][m][i];
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
                const v4i v = *reinterpret_cast<const v4i *>(region + row * ROW +
                                                             ((c ^ spread(row)) << 4));
                store_piece<T>(g, t, t_end, n, v);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }

    template <class T>
    static __device__ __forceinline__ Out4<T> load_addend(const GemmFp8Args &g, int t, int t_end,
                                                          int n)
    {
        Out4<T> r{};
        if (t < t_end && n < g.N) {
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
    static __device__ __forceinline__ void store_piece(const GemmFp8Args &g, int t, int t_end, int n,
                                                       v4i v)
    {
        constexpr int EPP = 16 / sizeof(T);
        if (t >= t_end || n >= g.N)
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

template <class C, class T>
__global__ void __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_fp8_tile_kernel(GemmFp8Args g, int tiles_m, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
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
    const int chunks = (g.K + C::KC - 1) / C::KC, t0 = tm * C::BM;
    C::template run<T>(g, g.w, g.w_scale, t0, g.T - t0 < C::BM ? g.T - t0 : C::BM, tn * C::BN,
                       slice * chunks / g.split, (slice + 1) * chunks / g.split, id, slice, lds);
}

// By expert: the row tiles of all experts in order, each expert's columns of
// tiles one after another.  Each XCD takes a contiguous run of them.
template <class C, class T>
__global__ void __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_fp8_grouped_tile_kernel(GemmFp8Args g, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
    const int lane = threadIdx.x & 63;
    int tiles = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
        int row0, rows;
        int n = tiles_of(g, e0 + lane, C::BM, row0, rows);
        n += __shfl_xor(n, 32);
        n += __shfl_xor(n, 16);
        tiles += __builtin_amdgcn_readfirstlane(row_sum(n));
    }
    const int total = tiles * tiles_n, per = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total)
        return;
    const Where at = find_tile(g, id, C::BM, tiles_n);
    if (at.column < 0)
        return;
    C::template run<T>(g, g.w + at.expert * g.w_expert, g.w_scale + at.expert * g.ws_expert, at.row0,
                       at.count, at.column * C::BN, 0, (g.K + C::KC - 1) / C::KC, 0, 0, lds);
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

template <class C>
hipError_t launch_tile(const GemmFp8Args &g, int out_dtype, hipStream_t stream)
{
    const int tm = (g.T + C::BM - 1) / C::BM, tn = (g.N + C::BN - 1) / C::BN;
    const unsigned grid = (unsigned)((tm * tn * g.split + 7) / 8 * 8);
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_fp8_tile_kernel<C, decltype(zero)>, dim3(grid), 64 * C::NW, stream, g,
                      tm, tn);
    });
}

template <int TC, int NW, int R>
hipError_t launch_stream(const GemmFp8Args &g, int out_dtype, hipStream_t stream)
{
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_fp8_stream_kernel<decltype(zero), TC, NW, R>,
                      dim3((unsigned)((g.N + 15) / 16)), 64 * NW, stream, g);
    });
}

// Row tiles of bm rows that the experts can have at most: each expert ends with
// a part of one.
long long most_tiles(const GemmFp8Args &g, int bm)
{
    const int with_rows = g.experts < g.T ? g.experts : g.T;
    return (g.T + (long long)with_rows * (bm - 1)) / bm;
}

template <class C>
hipError_t launch_grouped_tile(const GemmFp8Args &g, int out_dtype, hipStream_t stream)
{
    const int tn = (g.N + C::BN - 1) / C::BN;
    const unsigned grid = (unsigned)((most_tiles(g, C::BM) * tn + 7) / 8 * 8);
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_fp8_grouped_tile_kernel<C, decltype(zero)>, dim3(grid), 64 * C::NW,
                      stream, g, tn);
    });
}

template <int TC, int NW, int R>
hipError_t launch_grouped_stream(const GemmFp8Args &g, int out_dtype, hipStream_t stream)
{
    return with_type(out_dtype, [&](auto zero) {
        return launch(gemm_fp8_grouped_stream_kernel<decltype(zero), TC, NW, R>,
                      dim3((unsigned)((g.N + 15) / 16), (unsigned)most_tiles(g, 8 * TC)), 64 * NW,
                      stream, g);
    });
}

// The tiles, and what they cost in microseconds on an MI355X: launch, first
// copies and epilogue once; a block of 128 K with one workgroup a CU, when few
// CUs run one and when all do; a block for each of two workgroups a CU, where
// their LDS allows it; every further tile of a CU.
struct TileCost {
    int bm, bn;
    float once, few, all, two, more;
};
constexpr TileCost kTiles[] = {
    {256, 256, 10.6f, 1.30f, 1.73f, 0.f, 8.0f}, {128, 256, 9.5f, 0.42f, 0.76f, 0.f, 10.0f},
    {128, 128, 7.3f, 0.30f, 0.44f, 0.f, 5.5f},  {128, 64, 5.5f, 0.255f, 0.30f, 0.542f, 1.3f},
    {64, 64, 4.8f, 0.163f, 0.19f, 0.372f, 0.2f},
};
constexpr int kMaxSplit = 16;
constexpr size_t kCounterBytes = MOE_WNA16_GEMM_SYNC_BYTES;

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

Fp8Plan gemm_fp8_plan(int T, int N, int K)
{
    Fp8Plan p{};
    p.split = 1;
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

hipError_t launch_gemm_fp8(const GemmFp8Args &g, const Fp8Plan &p, int out_dtype,
                           hipStream_t stream)
{
    if (p.variant == 1) {
        if (p.bm == 256)
            return launch_tile<TileF8<256, 256, 2, 4, 2>>(g, out_dtype, stream);
        if (p.bn == 256)
            return launch_tile<TileF8<128, 256, 2, 4, 3>>(g, out_dtype, stream);
        if (p.bn == 128)
            return launch_tile<TileF8<128, 128, 2, 4, 4>>(g, out_dtype, stream);
        if (p.bm == 128)
            return launch_tile<TileF8<128, 64, 2, 2, 3>>(g, out_dtype, stream);
        return launch_tile<TileF8<64, 64, 2, 2, 4>>(g, out_dtype, stream);
    }
    const bool one = g.N <= 16 * 256;
    if (g.T <= 8)
        return one ? launch_stream<1, 16, 2>(g, out_dtype, stream)
                   : launch_stream<1, 8, 3>(g, out_dtype, stream);
    if (g.T <= 16)
        return one ? launch_stream<2, 16, 2>(g, out_dtype, stream)
                   : launch_stream<2, 8, 2>(g, out_dtype, stream);
    if (g.T <= 32)
        return launch_stream<4, 4, 3>(g, out_dtype, stream);
    return launch_stream<8, 4, 2>(g, out_dtype, stream);
}

hipError_t launch_gemm_fp8_grouped(const GemmFp8Args &args, int out_dtype, hipStream_t stream)
{
    GemmFp8Args g = args;
    g.split = 1;
    const int with_rows = g.experts < g.T ? g.experts : g.T;
    const int rows = g.T / with_rows;           // of an expert, about
    if (rows <= 4)
        return launch_grouped_stream<1, 8, 3>(g, out_dtype, stream);
    if (rows <= 16)
        return launch_grouped_stream<2, 8, 2>(g, out_dtype, stream);
    if (rows <= 48)
        return launch_grouped_tile<TileF8<64, 128, 1, 4, 4>>(g, out_dtype, stream);
    if (rows <= 128)
        return launch_grouped_tile<TileF8<128, 128, 2, 4, 4>>(g, out_dtype, stream);
    return launch_grouped_tile<TileF8<256, 256, 2, 4, 2>>(g, out_dtype, stream);
}

}  // namespace wna16
