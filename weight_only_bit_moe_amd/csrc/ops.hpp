// Internal launchers of the operators around the routed layer (not part of
// the C ABI): residual norm, expert routing, 8-bit product, 8-bit SwiGLU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace wna16 {

// OK when the current device is gfx950, else a moe_wna16_status (api.hip).
int check_device();

struct NormArgs {
    const void *x, *residual, *weight;          // residual may be null
    long long x_stride, r_stride, q_stride;     // elements between rows
    int T, H;
    int threads;                                // a row's, set by the launch
    float eps;
    void *residual_out, *y;                     // null: not written
    int8_t *q;                                  // null: no 8-bit output
    float *scale;
};
// dtype: moe_wna16_dtype of x, residual, weight, residual_out and y.
hipError_t launch_add_rmsnorm(const NormArgs &a, int dtype, hipStream_t stream);
constexpr int kMaxRow = 32768;                  // longest row of the row kernels
constexpr int kMaxRows = 1 << 21;               // a launch stays below 2^32 threads

struct SwigluArgs {
    const void *gu;                             // [T] rows of 2I: gate, then up
    long long gu_stride, q_stride;
    int T, I;
    int threads;                                // a row's, set by the launch
    float alpha, beta, clamp;                   // clamp = +inf: none
    int8_t *q;
    float *scale;
};
hipError_t launch_swiglu_quant(const SwigluArgs &a, int dtype, hipStream_t stream);

struct RouteArgs {
    const void *logits;                         // [T] rows of E
    const float *bias;                          // [E] or null
    long long stride;
    int T, E, topk, groups, topk_groups, renormalize;
    int per_group, span;                        // set by the launch
    float scale;
    int32_t *ids;                               // [T, topk]
    float *weights;                             // [T, topk]
};
hipError_t launch_route_topk(const RouteArgs &a, int dtype, int score, hipStream_t stream);

struct GemmArgs {
    const int8_t *a, *w;                        // [T, K], [N, K]
    const float *a_scale, *w_scale;             // [T], [N]
    const void *addend;                         // [T, N] of the output type, or null
    long long lda, ldw, ld_add, ldo;            // elements between rows
    int T, N, K;
    void *out;
    int split;                                  // K slices a tile, each its own workgroup
    int32_t *counters;                          // [tiles], zero between calls (split > 1)
    int32_t *partial;                           // [tiles][split] int32 sums (split > 1)
};
// Start of a product's workspace: the counters, at most one for each of the 512
// workgroups of a split product, then the partial sums.
constexpr size_t kCounterBytes = 4096;          // MOE_WNA16_GEMM_SYNC_BYTES
// Tiling of a product: a pure function of the sizes.
struct GemmPlan {
    int variant;                                // 0: few tokens, weights streamed, 1: tiles
    int bm, bn;                                 // output tile
    int split;                                  // K slices a tile
    size_t workspace;                           // bytes
};
GemmPlan gemm_plan(int T, int N, int K);
hipError_t launch_gemm_w8a8(const GemmArgs &a, const GemmPlan &p, int out_dtype,
                            hipStream_t stream);

}  // namespace wna16
