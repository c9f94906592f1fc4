// Host side of the operators around the routed layer (include/moe_wna16.h):
// argument checks and the launch on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe_wna16.h"
#include "ops.hpp"

namespace {

constexpr long long kMaxStride = 1ll << 23;   // products: 256 rows stay within 32-bit offsets
constexpr int kMaxGemmDim = 1 << 21;
constexpr int kMaxGemmK = 131071;
static_assert(wna16::kCounterBytes == MOE_WNA16_GEMM_SYNC_BYTES, "the header states it");

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_dtype(int d) { return d == MOE_WNA16_BF16 || d == MOE_WNA16_FP16 || d == MOE_WNA16_FP32; }

size_t size_of(int dtype) { return dtype == MOE_WNA16_FP32 ? 4 : 2; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_WNA16_OK : MOE_WNA16_EHIP; }

}  // namespace

extern "C" {

int moe_wna16_add_rmsnorm(const void *x, const void *residual, const void *weight, int T, int H,
                          int64_t x_stride, int64_t r_stride, int dtype, float eps,
                          void *residual_out, void *y_out, int8_t *q_out, int64_t q_stride,
                          float *scale_out, hipStream_t stream)
{
    if (T < 0 || H <= 0 || !valid_dtype(dtype) || !std::isfinite(eps) || eps < 0.f)
        return MOE_WNA16_EINVAL;
    if (H > wna16::kMaxRow || T > wna16::kMaxRows)
        return MOE_WNA16_EUNSUPPORTED;
    if (x_stride < H || (residual && r_stride < H) || (q_out && q_stride < H))
        return MOE_WNA16_EINVAL;
    if (T == 0)
        return MOE_WNA16_OK;
    if (!x || !weight || (!y_out && !q_out) || (q_out && !scale_out))
        return MOE_WNA16_EINVAL;
    const size_t b = size_of(dtype);
    if (!aligned(x, b) || !aligned(residual, b) || !aligned(weight, b) ||
        !aligned(residual_out, b) || !aligned(y_out, b) || !aligned(scale_out, 4))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.x_stride = x_stride;
    a.r_stride = r_stride;
    a.q_stride = q_stride;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.residual_out = residual_out;
    a.y = y_out;
    a.q = q_out;
    a.scale = scale_out;
    return hip_status(wna16::launch_add_rmsnorm(a, dtype, stream));
}

int moe_wna16_route_topk(const void *logits, const float *bias, int T, int E, int64_t stride,
                         int dtype, int topk, int score, int groups, int topk_groups,
                         int renormalize, float scale, int32_t *ids_out, float *w_out,
                         hipStream_t stream)
{
    if (T < 0 || E <= 0 || topk <= 0 || topk > E || !valid_dtype(dtype) ||
        (score != MOE_WNA16_SOFTMAX && score != MOE_WNA16_SIGMOID) || groups <= 0 ||
        E % groups != 0 || topk_groups <= 0 || topk_groups > groups || stride < E ||
        !std::isfinite(scale))
        return MOE_WNA16_EINVAL;
    if (E > 1024 || topk > 64 || groups > 64 || T > wna16::kMaxRows)
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0)
        return MOE_WNA16_OK;
    if (!logits || !ids_out || !w_out)
        return MOE_WNA16_EINVAL;
    if (!aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(ids_out, 4) ||
        !aligned(w_out, 4))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.stride = stride;
    a.T = T;
    a.E = E;
    a.topk = topk;
    a.groups = groups;
    a.topk_groups = topk_groups;
    a.renormalize = renormalize;
    a.scale = scale;
    a.ids = ids_out;
    a.weights = w_out;
    return hip_status(wna16::launch_route_topk(a, dtype, score, stream));
}

static int check_gemm_sizes(int T, int N, int K)
{
    if (T < 0 || N < 0 || K <= 0)
        return MOE_WNA16_EINVAL;
    return T > kMaxGemmDim || N > kMaxGemmDim || K > kMaxGemmK ? MOE_WNA16_EUNSUPPORTED
                                                               : MOE_WNA16_OK;
}

int moe_wna16_gemm_w8a8_workspace_size(int T, int N, int K, size_t *bytes_out)
{
    if (!bytes_out)
        return MOE_WNA16_EINVAL;
    const int st = check_gemm_sizes(T, N, K);
    if (st != MOE_WNA16_OK)
        return st;
    *bytes_out = T == 0 || N == 0 ? 0 : wna16::gemm_plan(T, N, K).workspace;
    return MOE_WNA16_OK;
}

int moe_wna16_gemm_w8a8(const int8_t *a, const float *a_scale, const int8_t *w,
                        const float *w_scale, const void *addend, int T, int N, int K,
                        int64_t lda, int64_t ldw, int64_t ld_add, int64_t ldo, int out_dtype,
                        void *out, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    int st = check_gemm_sizes(T, N, K);
    if (st != MOE_WNA16_OK)
        return st;
    if (!valid_dtype(out_dtype) || lda < K || ldw < K || (addend && ld_add < N) || ldo < N)
        return MOE_WNA16_EINVAL;
    if (lda >= kMaxStride || ldw >= kMaxStride || ldo >= kMaxStride ||
        (addend && ld_add >= kMaxStride))
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0 || N == 0)
        return MOE_WNA16_OK;
    if (!a || !a_scale || !w || !w_scale || !out)
        return MOE_WNA16_EINVAL;
    const size_t b = size_of(out_dtype);
    if (!aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(addend, b) || !aligned(out, b) ||
        !aligned(workspace, 256))
        return MOE_WNA16_EALIGN;
    const wna16::GemmPlan plan = wna16::gemm_plan(T, N, K);
    if (plan.workspace && !workspace)
        return MOE_WNA16_EINVAL;
    if (workspace_bytes < plan.workspace)
        return MOE_WNA16_EWORKSPACE;
    st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::GemmArgs g{};
    g.a = a;
    g.w = w;
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.addend = addend;
    g.lda = lda;
    g.ldw = ldw;
    g.ld_add = ld_add;
    g.ldo = ldo;
    g.T = T;
    g.N = N;
    g.K = K;
    g.out = out;
    g.split = plan.split;
    if (plan.split > 1) {
        g.counters = static_cast<int32_t *>(workspace);
        g.partial = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) +
                                                wna16::kCounterBytes);
    }
    return hip_status(wna16::launch_gemm_w8a8(g, plan, out_dtype, stream));
}

int moe_wna16_swiglu_quant(const void *gu, int T, int I, int64_t gu_stride, int dtype, float alpha,
                           float beta, float clamp, int8_t *q_out, int64_t q_stride,
                           float *scale_out, hipStream_t stream)
{
    if (T < 0 || I <= 0 || !valid_dtype(dtype) || !std::isfinite(alpha) || !std::isfinite(beta) ||
        std::isnan(clamp) || !(clamp > 0.f) || gu_stride < 2ll * I || q_stride < I)
        return MOE_WNA16_EINVAL;
    if (I > wna16::kMaxRow || T > wna16::kMaxRows)
        return MOE_WNA16_EUNSUPPORTED;
    if (T == 0)
        return MOE_WNA16_OK;
    if (!gu || !q_out || !scale_out)
        return MOE_WNA16_EINVAL;
    if (!aligned(gu, size_of(dtype)) || !aligned(scale_out, 4))
        return MOE_WNA16_EALIGN;
    const int st = wna16::check_device();
    if (st != MOE_WNA16_OK)
        return st;
    wna16::SwigluArgs a{};
    a.gu = gu;
    a.gu_stride = gu_stride;
    a.q_stride = q_stride;
    a.T = T;
    a.I = I;
    a.alpha = alpha;
    a.beta = beta;
    a.clamp = clamp;
    a.q = q_out;
    a.scale = scale_out;
    return hip_status(wna16::launch_swiglu_quant(a, dtype, stream));
}

}  // extern "C"
