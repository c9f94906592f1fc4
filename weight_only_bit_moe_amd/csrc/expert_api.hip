// Host side of the operators for experts in 8-bit floating point
// (include/moe_wna16.h): argument checks and the launch on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>

#include "expert_ops.hpp"
#include "moe_wna16.h"
#include "ops.hpp"

namespace {

constexpr long long kMaxStride = 1ll << 23;     // products: 256 rows stay within 32-bit offsets
constexpr long long kMaxScaleStride = 1ll << 20;
constexpr int kMaxDim = 1 << 21;
constexpr int kMaxK = 1 << 17;
constexpr int kMaxPairs = 1 << 24;
constexpr int kMaxColumns = 1 << 20;
constexpr long long kMaxElements = 1ll << 62;   // strides in bytes stay within 64 bits

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_dtype(int d) { return d == MOE_WNA16_BF16 || d == MOE_WNA16_FP16 || d == MOE_WNA16_FP32; }

size_t size_of(int dtype) { return dtype == MOE_WNA16_FP32 ? 4 : 2; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_WNA16_OK : MOE_WNA16_EHIP; }

int blocks_of(int n) { return (n + 127) / 128; }

int quant(const void *x, bool swiglu, int T, int K, int64_t x_stride, int dtype, float alpha,
          float beta, float clamp, void *q_out, int64_t q_stride, float *scale_out,
          int64_t s_stride, hipStream_t stream)
{
    if (T < 0 || K <= 0 || !valid_dtype(dtype) || !std::isfinite(alpha) || !std::isfinite(beta) ||
        !(clamp > 0.f))
        return MOE_WNA16_EINVAL;
    if (K > wna16::kMaxQuantRow || T > wna16::kMaxRows ||
        (long long)T * blocks_of(K) > wna16::kMaxQuantBlocks)
        return MOE_WNA16_EUNSUPPORTED;
    if (x_stride < (swiglu ? 2ll : 1ll) * K || q_stride < K || s_stride < blocks_of(K))
        return MOE_WNA16_EINVAL;
    if (T == 0)
        return MOE_WNA16_OK;
    if (!x || !q_out || !scale_out)
        return MOE_WNA16_EINVAL;
    if (!aligned(x, size_of(dtype)) || !aligned(scale_out, 4))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::QuantArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.q_stride = q_stride;
    a.s_stride = s_stride;
    a.T = T;
    a.n = K;
    a.alpha = alpha;
    a.beta = beta;
    a.clamp = clamp;
    a.q = static_cast<uint8_t *>(q_out);
    a.scale = scale_out;
    return hip_status(wna16::launch_quant_fp8(a, swiglu, dtype, stream));
}

// Sizes and strides that both products check; T rows of output.
int check_product(int T, int N, int K, int64_t lda, int64_t lda_s, int64_t ldw, int64_t ldw_s,
                  int64_t ldo, int out_dtype)
{
    if (T < 0 || N < 0 || K <= 0 || !valid_dtype(out_dtype) || lda < K || ldw < K ||
        lda_s < blocks_of(K) || ldw_s < blocks_of(K) || ldo < N)
        return MOE_WNA16_EINVAL;
    if (T > kMaxDim || N > kMaxDim || K > kMaxK || K % 16 != 0 || lda >= kMaxStride ||
        ldw >= kMaxStride || ldo >= kMaxStride || lda_s >= kMaxScaleStride ||
        ldw_s >= kMaxScaleStride)
        return MOE_WNA16_EUNSUPPORTED;
    return MOE_WNA16_OK;
}

}  // namespace

extern "C" {

int moe_wna16_quant_fp8(const void *x, int T, int K, int64_t x_stride, int dtype, void *q_out,
                        int64_t q_stride, float *scale_out, int64_t s_stride, hipStream_t stream)
{
    return quant(x, false, T, K, x_stride, dtype, 1.f, 0.f, INFINITY, q_out, q_stride, scale_out,
                 s_stride, stream);
}

int moe_wna16_swiglu_quant_fp8(const void *gu, int T, int I, int64_t gu_stride, int dtype,
                               float alpha, float beta, float clamp, void *q_out, int64_t q_stride,
                               float *scale_out, int64_t s_stride, hipStream_t stream)
{
    return quant(gu, true, T, I, gu_stride, dtype, alpha, beta, clamp, q_out, q_stride, scale_out,
                 s_stride, stream);
}

int moe_wna16_gemm_fp8_workspace_size(int T, int N, int K, size_t *bytes_out)
{
    if (!bytes_out || T < 0 || N < 0 || K <= 0)
        return MOE_WNA16_EINVAL;
    if (T > kMaxDim || N > kMaxDim || K > kMaxK || K % 16 != 0)
        return MOE_WNA16_EUNSUPPORTED;
    *bytes_out = T == 0 || N == 0 ? 0 : wna16::gemm_fp8_plan(T, N, K).workspace;
    return MOE_WNA16_OK;
}

int moe_wna16_gemm_fp8(const void *a, const float *a_scale, const void *w, const float *w_scale,
                       const void *addend, int T, int N, int K, int64_t lda, int64_t lda_s,
                       int64_t ldw, int64_t ldw_s, int64_t ld_add, int64_t ldo, int out_dtype,
                       void *out, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    int st = check_product(T, N, K, lda, lda_s, ldw, ldw_s, ldo, out_dtype);
    if (st != MOE_WNA16_OK)
        return st;
    if (addend && ld_add < N)
        return MOE_WNA16_EINVAL;
    if (addend && ld_add >= kMaxStride)
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0 || N == 0)
        return MOE_WNA16_OK;
    if (!a || !a_scale || !w || !w_scale || !out)
        return MOE_WNA16_EINVAL;
    const size_t b = size_of(out_dtype);
    if (!aligned(a, 16) || !aligned(w, 16) || lda % 16 != 0 || ldw % 16 != 0 ||
        !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(addend, b) || !aligned(out, b) ||
        !aligned(workspace, 256))
        return MOE_WNA16_EALIGN;
    const wna16::Fp8Plan plan = wna16::gemm_fp8_plan(T, N, K);
    if (plan.workspace && !workspace)
        return MOE_WNA16_EINVAL;
    if (workspace_bytes < plan.workspace)
        return MOE_WNA16_EWORKSPACE;
    st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::GemmFp8Args g{};
    g.a = static_cast<const uint8_t *>(a);
    g.w = static_cast<const uint8_t *>(w);
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.addend = addend;
    g.lda = lda;
    g.ldw = ldw;
    g.lda_s = lda_s;
    g.ldw_s = ldw_s;
    g.ld_add = ld_add;
    g.ldo = ldo;
    g.T = T;
    g.N = N;
    g.K = K;
    g.out = out;
    g.split = plan.split;
    if (plan.split > 1) {
        g.counters = static_cast<int32_t *>(workspace);
        g.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                              MOE_WNA16_GEMM_SYNC_BYTES);
    }
    return hip_status(wna16::launch_gemm_fp8(g, plan, out_dtype, stream));
}

int moe_wna16_gemm_fp8_grouped(const void *a, const float *a_scale, const void *w,
                               const float *w_scale, const int32_t *offsets, const int32_t *rows,
                               int E, int a_rows, int R, int N, int K, int64_t lda, int64_t lda_s,
                               int64_t ldw, int64_t ldw_s, int64_t w_expert, int64_t ws_expert,
                               int64_t ldo, int out_dtype, void *out, hipStream_t stream)
{
    int st = check_product(R, N, K, lda, lda_s, ldw, ldw_s, ldo, out_dtype);
    if (st != MOE_WNA16_OK)
        return st;
    if (E <= 0 || a_rows < 0 || (R > 0 && a_rows == 0) || (!rows && a_rows < R) ||
        (E > 1 && N > 0 && (w_expert < (N - 1) * ldw + K ||
                            ws_expert < (blocks_of(N) - 1) * ldw_s + blocks_of(K))))
        return MOE_WNA16_EINVAL;
    if (E > 1024 || w_expert >= kMaxElements / 1024 || ws_expert >= kMaxElements / 4096 ||
        a_rows > kMaxDim || (rows && (a_rows * lda >= 1ll << 32 || a_rows * lda_s >= 1ll << 30)))
        return MOE_WNA16_EUNSUPPORTED;
    if (R == 0 || N == 0)
        return MOE_WNA16_OK;
    if (!a || !a_scale || !w || !w_scale || !offsets || !out)
        return MOE_WNA16_EINVAL;
    if (!aligned(a, 16) || !aligned(w, 16) || lda % 16 != 0 || ldw % 16 != 0 ||
        (E > 1 && w_expert % 16 != 0) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(out, size_of(out_dtype)))
        return MOE_WNA16_EALIGN;
    st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::GemmFp8Args g{};
    g.a = static_cast<const uint8_t *>(a);
    g.w = static_cast<const uint8_t *>(w);
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.lda = lda;
    g.ldw = ldw;
    g.lda_s = lda_s;
    g.ldw_s = ldw_s;
    g.ldo = ldo;
    g.w_expert = w_expert;
    g.ws_expert = ws_expert;
    g.T = R;
    g.N = N;
    g.K = K;
    g.out = out;
    g.split = 1;
    g.offsets = offsets;
    g.rows = rows;
    g.experts = E;
    g.a_rows = a_rows;
    return hip_status(wna16::launch_gemm_fp8_grouped(g, out_dtype, stream));
}

static int check_sort(int T, int topk, int E)
{
    if (T < 0 || topk <= 0 || E <= 0)
        return MOE_WNA16_EINVAL;
    return T > wna16::kMaxRows || topk > 64 || E > 1024 || (long long)T * topk > kMaxPairs
               ? MOE_WNA16_EUNSUPPORTED
               : MOE_WNA16_OK;
}

int moe_wna16_sort_tokens_workspace_size(int T, int topk, int E, size_t *bytes_out)
{
    if (!bytes_out)
        return MOE_WNA16_EINVAL;
    const int st = check_sort(T, topk, E);
    if (st != MOE_WNA16_OK)
        return st;
    *bytes_out = T == 0 ? 0 : wna16::sort_workspace(T, topk, E);
    return MOE_WNA16_OK;
}

int moe_wna16_sort_tokens(const int32_t *ids, int T, int topk, int E, const void *x, int H,
                          int64_t x_stride, int dtype, int32_t *tokens_out, int32_t *slots_out,
                          int32_t *offsets_out, void *xs_out, int64_t xs_stride, void *workspace,
                          size_t workspace_bytes, hipStream_t stream)
{
    int st = check_sort(T, topk, E);
    if (st != MOE_WNA16_OK)
        return st;
    if (x && (H <= 0 || !valid_dtype(dtype) || x_stride < H || xs_stride < H))
        return MOE_WNA16_EINVAL;
    if (x && (H > kMaxColumns || x_stride >= kMaxElements / 4 || xs_stride >= kMaxElements >> 26))
        return MOE_WNA16_EUNSUPPORTED;
    if (!offsets_out || (T > 0 && (!ids || !tokens_out || !slots_out || (x && !xs_out))))
        return MOE_WNA16_EINVAL;
    const size_t need = T == 0 ? 0 : wna16::sort_workspace(T, topk, E), b = size_of(dtype);
    if (!aligned(ids, 4) || !aligned(tokens_out, 4) || !aligned(slots_out, 4) ||
        !aligned(offsets_out, 4) || !aligned(workspace, 4) ||
        (x && (!aligned(x, b) || !aligned(xs_out, b))))
        return MOE_WNA16_EALIGN;
    if (need && !workspace)
        return MOE_WNA16_EINVAL;
    if (workspace_bytes < need)
        return MOE_WNA16_EWORKSPACE;
    st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::SortArgs a{};
    a.ids = ids;
    a.T = T;
    a.topk = topk;
    a.E = E;
    a.tokens = tokens_out;
    a.slots = slots_out;
    a.offsets = offsets_out;
    a.counts = static_cast<int32_t *>(workspace);
    if (x) {
        a.x = static_cast<const char *>(x);
        a.x_stride = x_stride * (int64_t)b;
        a.xs_stride = xs_stride * (int64_t)b;
        a.row_bytes = H * (int)b;
        a.xs = static_cast<char *>(xs_out);
    }
    return hip_status(wna16::launch_sort_tokens(a, stream));
}

int moe_wna16_combine_tokens(const void *y, const int32_t *slots, const float *weights,
                             const void *addend, int T, int topk, int H, int R, int64_t y_stride,
                             int64_t add_stride, int64_t out_stride, int dtype, void *out,
                             hipStream_t stream)
{
    if (T < 0 || topk <= 0 || H <= 0 || R < 0 || !valid_dtype(dtype) || y_stride < H ||
        (addend && add_stride < H) || out_stride < H)
        return MOE_WNA16_EINVAL;
    if (T > wna16::kMaxRows || topk > 64 || H > kMaxColumns || R > kMaxPairs)
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0)
        return MOE_WNA16_OK;
    if ((R > 0 && !y) || !slots || !out)
        return MOE_WNA16_EINVAL;
    const size_t b = size_of(dtype);
    if (!aligned(y, b) || !aligned(slots, 4) || !aligned(weights, 4) || !aligned(addend, b) ||
        !aligned(out, b))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::CombineArgs a{};
    a.y = y;
    a.slots = slots;
    a.weights = weights;
    a.addend = addend;
    a.y_stride = y_stride;
    a.add_stride = add_stride;
    a.out_stride = out_stride;
    a.T = T;
    a.topk = topk;
    a.H = H;
    a.R = R;
    a.out = out;
    return hip_status(wna16::launch_combine_tokens(a, dtype, stream));
}

int moe_wna16_combine_tokens_grad(const void *dout, const void *y, const int32_t *slots,
                                  const float *weights, const int32_t *used, int T, int topk, int H,
                                  int R, int64_t d_stride, int64_t y_stride, int64_t dy_stride,
                                  int dtype, void *dy, float *dw, hipStream_t stream)
{
    if (T < 0 || topk <= 0 || H <= 0 || R < 0 || !valid_dtype(dtype) || d_stride < H ||
        (dw && y_stride < H) || (dy && dy_stride < H) || (used && !dy && R > 0))
        return MOE_WNA16_EINVAL;
    if (T > wna16::kMaxRows || topk > 64 || H > (T > 0 ? wna16::kMaxRow : kMaxColumns) || R > kMaxPairs)
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0 && (!used || R == 0))
        return MOE_WNA16_OK;
    if ((T > 0 && (!dout || !slots)) || (!dy && !dw && R > 0) || (dw && R > 0 && !y))
        return MOE_WNA16_EINVAL;
    const size_t b = size_of(dtype);
    if (!aligned(dout, b) || !aligned(y, b) || !aligned(slots, 4) || !aligned(weights, 4) ||
        !aligned(used, 4) || !aligned(dy, b) || !aligned(dw, 4))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::CombineGradArgs a{};
    a.dout = dout;
    a.y = y;
    a.slots = slots;
    a.weights = weights;
    a.used = used;
    a.d_stride = d_stride;
    a.y_stride = y_stride;
    a.dy_stride = dy_stride;
    a.T = T;
    a.topk = topk;
    a.H = H;
    a.R = R;
    a.dy = dy;
    a.dw = dw;
    return hip_status(wna16::launch_combine_tokens_grad(a, dtype, stream));
}

}  // extern "C"
