// Internal launchers of the operators for experts in 8-bit floating point (not
// part of the C ABI): e4m3 rows, their product plain and by expert, tokens
// sorted by expert and combined.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace wna16 {

struct QuantArgs {
    const void *x;                              // [T] rows of n; SwiGLU: of 2n, gate, then up
    long long x_stride, q_stride, s_stride;     // elements between rows
    int T, n;
    int blocks;                                 // a row's, set by the launch
    int shift;                                  // id / blocks for ids, set by the launch
    uint32_t magic;
    float alpha, beta, clamp;                   // SwiGLU; clamp = +inf: none
    uint8_t *q;
    float *scale;
};
constexpr int kMaxQuantRow = 1 << 17;
constexpr long long kMaxQuantBlocks = 1ll << 27;   // rows * blocks: below 2^32 threads
hipError_t launch_quant_fp8(const QuantArgs &a, bool swiglu, int dtype, hipStream_t stream);

// Tokens sorted by expert.
struct SortArgs {
    const int32_t *ids;                         // [T, topk]
    int T, topk, E;
    int per_group;                              // tokens a workgroup, set by the launch
    int chunk;                                  // tokens a counted chunk, set by the launch
    int32_t *tokens, *slots, *offsets;          // [T * topk], [T, topk], [E + 1]
    int32_t *counts;                            // workspace: [chunks][E] (many pairs)
    const char *x;                              // rows of row_bytes, or null
    long long x_stride, xs_stride;              // bytes
    int row_bytes;
    char *xs;
};
size_t sort_workspace(int T, int topk, int E);
hipError_t launch_sort_tokens(const SortArgs &a, hipStream_t stream);

struct CombineArgs {
    const void *y;                              // [R] rows of H
    const int32_t *slots;                       // [T, topk]
    const float *weights;                       // [T, topk], or null: ones
    const void *addend;                         // [T] rows of H, or null
    long long y_stride, add_stride, out_stride; // elements
    int T, topk, H, R;
    int threads;                                // a workgroup's, set by the launch
    void *out;
};
hipError_t launch_combine_tokens(const CombineArgs &a, int dtype, hipStream_t stream);

struct CombineGradArgs {
    const void *dout, *y;                       // [T], [R] rows of H; y null: no dw
    const int32_t *slots;
    const float *weights;                       // or null: ones
    const int32_t *used;                        // device: dy's rows from *used on get zeros; or null
    long long d_stride, y_stride, dy_stride;
    int T, topk, H, R;
    int threads;
    void *dy;                                   // or null
    float *dw;                                  // [T, topk], or null
};
hipError_t launch_combine_tokens_grad(const CombineGradArgs &a, int dtype, hipStream_t stream);

struct GemmFp8Args {
    const uint8_t *a, *w;                       // [T, K], [N, K] (grouped: [experts, N, K])
    const float *a_scale, *w_scale;             // rows of K / 128 blocks; w's for 128 channels
    const void *addend;                         // [T, N] of the output type, or null
    long long lda, ldw, lda_s, ldw_s, ld_add, ldo;   // elements between rows
    long long w_expert, ws_expert;              // elements between experts (grouped)
    int T, N, K;                                // T: rows of the output
    void *out;
    int split;                                  // K slices a tile, each its own workgroup
    int32_t *counters;                          // [tiles], zero between calls (split > 1)
    float *partial;                             // [tiles][split] sums (split > 1)
    const int32_t *offsets;                     // grouped: [experts + 1]
    const int32_t *rows;                        // grouped: a's row of each output row, or null
    int experts, a_rows;                        // grouped: a_rows of a that `rows` names
};
struct Fp8Plan {
    int tile;                                   // -1: few tokens, weights streamed
    int split;                                  // K slices a tile
    size_t workspace;
};
Fp8Plan gemm_fp8_plan(int T, int N, int K);
int gemm_fp8_grouped_tile(int experts, int R, int N, int K);
hipError_t launch_gemm_fp8(const GemmFp8Args &a, const Fp8Plan &p, int out_dtype,
                           hipStream_t stream);
hipError_t launch_gemm_fp8_grouped(const GemmFp8Args &a, int out_dtype, hipStream_t stream);

}  // namespace wna16
