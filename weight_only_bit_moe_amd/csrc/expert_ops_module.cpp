// The operators for experts in 8-bit floating point in the Python module
// _block_ops: checks, allocation and the library call, as for the operators
// around the layer; and the graph nodes of sort and combine.  A node's gradient runs
// on torch's own thread without the interpreter: written in Python, small
// gradients waited for the interpreter's lock (forward and backward of 32 tokens: sort
// 86 -> 49 us, 54 since its graph's rows behind the last pair are cleared, combine 73 -> 52,
// where torch's product by two takes 43).
#include "torch_module.hpp"

#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>

namespace {

using namespace moe_module;

constexpr at::ScalarType kE4m3 = at::kFloat8_e4m3fn;

PyObject *n_x, *n_q, *n_scale, *n_gu, *n_alpha, *n_beta, *n_clamp, *n_a, *n_a_scale, *n_w,
    *n_w_scale, *n_addend, *n_out_dtype, *n_out, *n_workspace, *n_offsets, *n_rows, *n_ids,
    *n_experts, *n_tokens, *n_slots, *n_y, *n_weights;

constexpr int64_t kMaxGradientRow = 32768;          // moe_wna16_combine_tokens_grad's

int64_t blocks(int64_t n) { return (n + 127) / 128; }

at::ScalarType out_type(PyObject *o)
{
    if (!o)
        return at::kBFloat16;
    if (!THPDtype_Check(o))
        fail(PyExc_TypeError, "out_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

const void *optional_flat(PyObject *o, const char *name, c10::IntArrayRef shape,
                          at::ScalarType dtype, c10::Device dev)
{
    return o ? flat(tensor(o, name), name, shape, dtype, dev) : nullptr;
}

template <bool SWIGLU>
PyObject *quant(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *v[6] = {};                            // x, q, scale, alpha, beta, clamp
    const char *in = SWIGLU ? "gu" : "x";
    if constexpr (SWIGLU) {
        PyObject *const names[] = {n_gu, n_q, n_scale, n_alpha, n_beta, n_clamp};
        const Args<6> p("swiglu_quant_fp8", names, 1, 1, args, nargs, kw);
        std::copy(p.v, p.v + 6, v);
    } else {
        PyObject *const names[] = {n_x, n_q, n_scale};
        const Args<3> p("quant_fp8", names, 1, 1, args, nargs, kw);
        std::copy(p.v, p.v + 3, v);
    }
    const at::Tensor &x = matrix(v[0], in);
    if (SWIGLU && x.size(1) % 2)
        fail(PyExc_ValueError, "gu must hold gate and up halves of equal length");
    const int64_t T = x.size(0), K = SWIGLU ? x.size(1) / 2 : x.size(1);
    const c10::Device dev = x.device();
    const int code = dtype_code(x.scalar_type(), in);
    const int64_t xs = rows(x, in, x.sizes(), x.scalar_type(), dev);
    const float alpha = (float)number(v[3], 1.0), beta = (float)number(v[4], 0.0);
    const float clamp = (float)number(v[5], INFINITY);
    ensure_library();
    at::Tensor q = given_or_empty(v[1], "q", {T, K}, kE4m3, dev);
    at::Tensor scale = given_or_empty(v[2], "scale", {T, blocks(K)}, at::kFloat, dev);
    const int64_t qs = rows(q, "q", {T, K}, kE4m3, dev);
    const int64_t ss = rows(scale, "scale", {T, blocks(K)}, at::kFloat, dev);
    launch(SWIGLU ? "moe_wna16_swiglu_quant_fp8" : "moe_wna16_quant_fp8", dev, [&](hipStream_t s) {
        if constexpr (SWIGLU)
            return lib.swiglu_quant_fp8(x.data_ptr(), (int)T, (int)K, xs, code, alpha, beta, clamp,
                                        q.data_ptr(), qs, (float *)scale.data_ptr(), ss, s);
        else
            return lib.quant_fp8(x.data_ptr(), (int)T, (int)K, xs, code, q.data_ptr(), qs,
                                 (float *)scale.data_ptr(), ss, s);
    });
    return pair(q, scale);
}

PyObject *gemm_fp8(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_a,      n_a_scale,   n_w,   n_w_scale,
                               n_addend, n_out_dtype, n_out, n_workspace};
    const Args<8> p("gemm_fp8", names, 4, 4, args, nargs, kw);
    const at::Tensor &a = matrix(p.v[0], "a"), &w = matrix(p.v[2], "w");
    const int64_t T = a.size(0), K = a.size(1), N = w.size(0), kb = blocks(K);
    const c10::Device dev = a.device();
    const at::ScalarType dt = out_type(p.v[5]);
    const int code = dtype_code(dt, "out_dtype");
    const int64_t lda = rows(a, "a", {T, K}, kE4m3, dev);
    const int64_t ldw = rows(w, "w", {N, K}, kE4m3, dev);
    const at::Tensor &sa = tensor(p.v[1], "a_scale"), &sw = tensor(p.v[3], "w_scale");
    const int64_t lda_s = rows(sa, "a_scale", {T, kb}, at::kFloat, dev);
    const int64_t ldw_s = rows(sw, "w_scale", {blocks(N), kb}, at::kFloat, dev);
    const void *ap = nullptr;
    int64_t lad = N;
    if (p.v[4]) {
        const at::Tensor &add = tensor(p.v[4], "addend");
        lad = rows(add, "addend", {T, N}, dt, dev);
        ap = add.data_ptr();
    }
    ensure_library();
    at::Tensor out = given_or_empty(p.v[6], "out", {T, N}, dt, dev);
    const int64_t ldo = rows(out, "out", {T, N}, dt, dev);
    at::Tensor ws;
    if (p.v[7]) {
        ws = tensor(p.v[7], "workspace");
        flat(ws, "workspace", {ws.numel()}, at::kByte, dev);
    } else {
        size_t bytes = 0;
        if (lib.gemm_fp8_workspace_size((int)T, (int)N, (int)K, &bytes) == MOE_WNA16_OK && bytes)
            ws = fresh_workspace((int64_t)bytes, dev);
    }
    launch("moe_wna16_gemm_fp8", dev, [&](hipStream_t s) {
        return lib.gemm_fp8(a.data_ptr(), (const float *)sa.data_ptr(), w.data_ptr(),
                            (const float *)sw.data_ptr(), ap, (int)T, (int)N, (int)K, lda, lda_s,
                            ldw, ldw_s, lad, ldo, code, out.data_ptr(),
                            ws.defined() ? ws.data_ptr() : nullptr,
                            ws.defined() ? (size_t)ws.numel() : 0, s);
    });
    return THPVariable_Wrap(out);
}

// The strides of E matrices of contiguous rows: between rows, and between experts.
void expert_rows(const at::Tensor &t, const char *name, c10::IntArrayRef shape,
                 at::ScalarType dtype, c10::Device dev, int64_t &row, int64_t &expert)
{
    check(t, name, shape, dtype, dev);
    if (shape[2] > 1 && t.stride(2) != 1)
        fail(PyExc_ValueError, "%s must have contiguous rows", name);
    row = shape[1] <= 1 ? shape[2] : t.stride(1);
    expert = shape[0] <= 1 ? shape[1] * row : t.stride(0);
    if (row < shape[2] || (shape[0] > 1 && expert < (shape[1] - 1) * row + shape[2]))
        fail(PyExc_ValueError, "%s has overlapping rows", name);
}

PyObject *gemm_fp8_grouped(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_a, n_a_scale, n_w, n_w_scale, n_offsets, n_rows, n_out_dtype, n_out};
    const Args<8> p("gemm_fp8_grouped", names, 5, 5, args, nargs, kw);
    const at::Tensor &a = matrix(p.v[0], "a"), &w = tensor(p.v[2], "w");
    if (w.dim() != 3)
        fail(PyExc_ValueError, "w must be 3-D");
    const int64_t Ta = a.size(0), K = a.size(1), E = w.size(0), N = w.size(1), kb = blocks(K);
    if (E > INT32_MAX || N > INT32_MAX)
        fail(PyExc_ValueError, "w is too large");
    const c10::Device dev = a.device();
    const at::ScalarType dt = out_type(p.v[6]);
    const int code = dtype_code(dt, "out_dtype");
    const int64_t lda = rows(a, "a", {Ta, K}, kE4m3, dev);
    const at::Tensor &sa = tensor(p.v[1], "a_scale"), &sw = tensor(p.v[3], "w_scale");
    const int64_t lda_s = rows(sa, "a_scale", {Ta, kb}, at::kFloat, dev);
    int64_t ldw, we, ldw_s, se;
    expert_rows(w, "w", {E, N, K}, kE4m3, dev, ldw, we);
    expert_rows(sw, "w_scale", {E, blocks(N), kb}, at::kFloat, dev, ldw_s, se);
    const void *op = flat(tensor(p.v[4], "offsets"), "offsets", {E + 1}, at::kInt, dev);
    int64_t R = Ta;
    const void *rp = nullptr;
    if (p.v[5]) {
        const at::Tensor &r = tensor(p.v[5], "rows");
        R = r.numel();
        if (R > INT32_MAX)
            fail(PyExc_ValueError, "rows is too large");
        rp = flat(r, "rows", {R}, at::kInt, dev);
        if (!rp)                                    // no rows at all
            R = 0;
    }
    ensure_library();
    at::Tensor out = given_or_empty(p.v[7], "out", {R, N}, dt, dev);
    const int64_t ldo = rows(out, "out", {R, N}, dt, dev);
    launch("moe_wna16_gemm_fp8_grouped", dev, [&](hipStream_t s) {
        return lib.gemm_fp8_grouped(a.data_ptr(), (const float *)sa.data_ptr(), w.data_ptr(),
                                    (const float *)sw.data_ptr(), (const int32_t *)op,
                                    (const int32_t *)rp, (int)E, (int)Ta, (int)R, (int)N, (int)K,
                                    lda, lda_s, ldw, ldw_s, we, se, ldo, code, out.data_ptr(), s);
    });
    return THPVariable_Wrap(out);
}

const at::Tensor &expert_ids(PyObject *o, const char *name)
{
    const at::Tensor &t = matrix(o, name);
    flat(t, name, t.sizes(), at::kInt, t.device());
    return t;
}

// ---- gradients: without the interpreter's lock, on arguments checked before ------

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

int code_of(at::ScalarType t)
{
    return t == at::kBFloat16 ? MOE_WNA16_BF16 : t == at::kHalf ? MOE_WNA16_FP16 : MOE_WNA16_FP32;
}

template <class F>
void launch_plain(const char *name, c10::Device dev, F &&f)
{
    const c10::DeviceGuard guard(dev);
    const int st = f(c10::hip::getCurrentHIPStream(dev.index()).stream());
    TORCH_CHECK(st == MOE_WNA16_OK, name, ": status ", st);
}

// A gradient with rows that the kernels read (the graph also hands over expanded ones).
at::Tensor with_rows(const at::Tensor &d)
{
    return (d.size(1) <= 1 || d.stride(1) == 1) && (d.size(0) <= 1 || d.stride(0) >= d.size(1))
               ? d
               : d.contiguous();
}
int64_t row_stride(const at::Tensor &d) { return d.size(0) <= 1 ? d.size(1) : d.stride(0); }

// Results of a gradient carry no graph of their own: where one is asked for, they say so
// when it is used.
variable_list once(variable_list grads)
{
    if (!at::GradMode::is_enabled())
        return grads;
    for (at::Tensor &g : grads)
        if (g.defined()) {
            auto error = std::make_shared<torch::autograd::DelayedError>(
                "the gradients of sort_tokens and combine_tokens have no gradient", 1);
            g = (*error)({g.detach().set_requires_grad(true)})[0];
        }
    return grads;
}

struct Sorted {
    at::Tensor tokens, slots, offsets, x;       // x may be undefined
};

struct SortNode : torch::autograd::Function<SortNode> {
    // the values have been computed: what is left is their place in the graph
    static variable_list forward(AutogradContext *ctx, const at::Tensor &, const Sorted *r)
    {
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({r->slots});
        ctx->mark_non_differentiable({r->tokens, r->slots, r->offsets});
        return {r->tokens, r->slots, r->offsets, r->x};
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[3].defined())
            return {at::Tensor(), at::Tensor()};
        const at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor d = with_rows(grads[3]), slots = ctx->get_saved_variables()[0];
        const int64_t T = slots.size(0), H = d.size(1);
        at::Tensor dx = empty({T, H}, d.scalar_type(), d.device());
        launch_plain("moe_wna16_combine_tokens", d.device(), [&](hipStream_t s) {
            return lib.combine_tokens(d.data_ptr(), (const int32_t *)slots.data_ptr(), nullptr,
                                      nullptr, (int)T, (int)slots.size(1), (int)H, (int)d.size(0),
                                      row_stride(d), H, H, code_of(d.scalar_type()), dx.data_ptr(), s);
        });
        return once({dx, at::Tensor()});
    }
};

struct Combined {
    at::Tensor slots, offsets, out;             // offsets may be undefined
    bool y, weights, addend;                    // which require a gradient
};

struct CombineNode : torch::autograd::Function<CombineNode> {
    static variable_list forward(AutogradContext *ctx, const at::Tensor &y,
                                 const std::optional<at::Tensor> &weights,
                                 const std::optional<at::Tensor> &addend, const Combined *c)
    {
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({c->weights ? y : at::Tensor(), c->slots,
                                weights ? *weights : at::Tensor(), c->offsets});
        ctx->saved_data["rows"] = y.size(0);
        ctx->saved_data["wanted"] = (int64_t)(c->y + 2 * c->weights + 4 * c->addend);
        ctx->saved_data["given"] = (int64_t)(1 + 2 * weights.has_value() + 4 * addend.has_value());
        return {c->out};
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[0].defined())
            return {at::Tensor(), at::Tensor(), at::Tensor(), at::Tensor()};
        // which require a gradient, and of these (in order) which this call is asked for
        int64_t wanted = ctx->saved_data["wanted"].toInt();
        const int64_t R = ctx->saved_data["rows"].toInt();
        const int64_t given = ctx->saved_data["given"].toInt();
        for (int i = 0, edge = 0; i < 3; ++i)
            if (given >> i & 1 && !ctx->needs_input_grad(edge++))
                wanted &= ~(1ll << i);
        const variable_list saved = ctx->get_saved_variables();
        const at::Tensor &y = saved[0], &slots = saved[1], &weights = saved[2], &offsets = saved[3];
        at::Tensor dy, dw;
        if (wanted & 3) {
            const at::AutoDispatchBelowADInplaceOrView below;
            const at::Tensor d = with_rows(grads[0]);
            const int64_t T = slots.size(0), k = slots.size(1), H = d.size(1);
            const int32_t *used = nullptr;
            if (wanted & 1) {
                dy = empty({R, H}, d.scalar_type(), d.device());
                if (offsets.defined())
                    used = (const int32_t *)offsets.data_ptr() + offsets.numel() - 1;
                else
                    dy.zero_();                 // rows that no slot names
            }
            if (wanted & 2)
                dw = empty({T, k}, at::kFloat, d.device());
            launch_plain("moe_wna16_combine_tokens_grad", d.device(), [&](hipStream_t s) {
                return lib.combine_tokens_grad(
                    d.data_ptr(), dw.defined() ? y.data_ptr() : nullptr,
                    (const int32_t *)slots.data_ptr(),
                    weights.defined() ? (const float *)weights.data_ptr() : nullptr, used, (int)T,
                    (int)k, (int)H, (int)R, row_stride(d), dw.defined() ? row_stride(y) : H, H,
                    code_of(d.scalar_type()), dy.defined() ? dy.data_ptr() : nullptr,
                    dw.defined() ? (float *)dw.data_ptr() : nullptr, s);
            });
        }
        variable_list r = once({dy, dw});
        return {r[0], r[1], wanted & 4 ? grads[0] : at::Tensor(), at::Tensor()};
    }
};

// ---- sort and combine ------------------------------------------------------------

// They have reverse-mode gradients only: a tangent would be dropped without a word.
void no_tangent(const at::Tensor &t, const char *fn, const char *name)
{
    if (t._fw_grad(0).defined())
        fail(PyExc_NotImplementedError, "%s() has no forward-mode derivative, and %s has a tangent", fn,
             name);
}

// Values written into a tensor with a graph would leave it the gradient of the old ones.
void not_in_a_graph(PyObject *out)
{
    if (out && at::GradMode::is_enabled() && tensor(out, "out").requires_grad())
        fail(PyExc_ValueError, "out requires a gradient");
}

// GRAPH: the result is part of x's graph, and its rows behind the last sorted pair are
// cleared: a function of all rows between sort and combine has gradients of its
// parameters too, where their zeros meet those rows (0 * NaN is NaN).
template <bool GRAPH>
PyObject *sort_tokens(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_ids, n_experts, n_x, n_out};
    const Args<4> p("sort_tokens", names, 3, 2, args, nargs, kw);
    const at::Tensor &ids = expert_ids(p.v[0], "ids");
    const int E = integer(p.v[1], 0);
    const int64_t T = ids.size(0), k = ids.size(1), P = T * k;
    const c10::Device dev = ids.device();
    if (E < 1)
        fail(PyExc_ValueError, "experts must be at least 1");
    if (k < 1)
        fail(PyExc_ValueError, "ids must name at least one expert a token");
    ensure_library();
    Sorted r;
    at::Tensor &xs = r.x;
    const void *xp = nullptr;
    int64_t H = 0, xst = 0, xsst = 0;
    int code = MOE_WNA16_BF16;
    if (p.v[2]) {
        const at::Tensor &x = matrix(p.v[2], "x");
        no_tangent(x, "sort_tokens", "x");
        H = x.size(1);
        code = dtype_code(x.scalar_type(), "x");
        xst = rows(x, "x", {T, H}, x.scalar_type(), dev);
        xp = x.data_ptr();
        if (H < 1)
            fail(PyExc_ValueError, "x has no columns");
        not_in_a_graph(p.v[3]);
        xs = given_or_empty(p.v[3], "out", {P, H}, x.scalar_type(), dev);
        xsst = rows(xs, "out", {P, H}, x.scalar_type(), dev);
    } else if (p.v[3]) {
        fail(PyExc_ValueError, "out without x");
    }
    at::Tensor &tokens = r.tokens, &slots = r.slots, &offsets = r.offsets, ws;
    tokens = empty({P}, at::kInt, dev);
    slots = empty({T, k}, at::kInt, dev);
    offsets = empty({(int64_t)E + 1}, at::kInt, dev);
    size_t bytes = 0;
    if (lib.sort_tokens_workspace_size((int)T, (int)k, E, &bytes) == MOE_WNA16_OK && bytes)
        ws = empty({(int64_t)bytes}, at::kByte, dev);
    launch("moe_wna16_sort_tokens", dev, [&](hipStream_t s) {
        const int st = lib.sort_tokens(
            (const int32_t *)ids.data_ptr(), (int)T, (int)k, E, xp, (int)H, xst, code,
            (int32_t *)tokens.data_ptr(), (int32_t *)slots.data_ptr(), (int32_t *)offsets.data_ptr(),
            xp ? xs.data_ptr() : nullptr, xsst, bytes ? ws.data_ptr() : nullptr, bytes, s);
        if (!GRAPH || st != MOE_WNA16_OK)
            return st;
        return lib.combine_tokens_grad(nullptr, nullptr, nullptr, nullptr,
                                       (const int32_t *)offsets.data_ptr() + E, 0, (int)k, (int)H,
                                       (int)P, H, H, xsst, code, xs.data_ptr(), nullptr, s);
    });
    if constexpr (GRAPH) {
        const variable_list v = SortNode::apply(tensor(p.v[2], "x"), (const Sorted *)&r);
        r = Sorted{v[0], v[1], v[2], v[3]};
    }
    PyObject *d = PyDict_New();
    if (!d)
        throw Raised{};
    try {
        put(d, n_tokens, tokens);
        put(d, n_slots, slots);
        put(d, n_offsets, offsets);
        if (xs.defined())
            put(d, n_x, xs);
    } catch (...) {
        Py_DECREF(d);
        throw;
    }
    return d;
}

// GRAPH: the result is part of the graphs of y, weights and addend.
template <bool GRAPH>
PyObject *combine_tokens(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_y, n_slots, n_weights, n_addend, n_out, n_offsets};
    const Args<6> p("combine_tokens", names, 3, 2, args, nargs, kw);
    const at::Tensor &y = matrix(p.v[0], "y"), &slots = expert_ids(p.v[1], "slots");
    const int64_t R = y.size(0), H = y.size(1), T = slots.size(0), k = slots.size(1);
    const c10::Device dev = y.device();
    const at::ScalarType dt = y.scalar_type();
    const int code = dtype_code(dt, "y");
    if (H < 1 || k < 1)
        fail(PyExc_ValueError, "y has no columns, or slots names no rows");
    check(slots, "slots", {T, k}, at::kInt, dev);
    no_tangent(y, "combine_tokens", "y");
    const int64_t ys = rows(y, "y", {R, H}, dt, dev);
    const void *wp = optional_flat(p.v[2], "weights", {T, k}, at::kFloat, dev);
    if (p.v[2])
        no_tangent(tensor(p.v[2], "weights"), "combine_tokens", "weights");
    if (p.v[5]) {
        const at::Tensor &offsets = tensor(p.v[5], "offsets");
        flat(offsets, "offsets", {offsets.numel()}, at::kInt, dev);
        if (offsets.numel() < 1)
            fail(PyExc_ValueError, "offsets is empty");
    }
    const void *ap = nullptr;
    int64_t as = H;
    if (p.v[3]) {
        const at::Tensor &add = tensor(p.v[3], "addend");
        no_tangent(add, "combine_tokens", "addend");
        as = rows(add, "addend", {T, H}, dt, dev);
        ap = add.data_ptr();
    }
    if constexpr (GRAPH)            // here, not in the gradient
        if (H > kMaxGradientRow &&
            (y.requires_grad() || (p.v[2] && tensor(p.v[2], "weights").requires_grad())))
            fail(PyExc_ValueError, "y has rows of %lld elements, gradients are for up to %lld",
                 (long long)H, (long long)kMaxGradientRow);
    not_in_a_graph(p.v[4]);
    ensure_library();
    at::Tensor out = given_or_empty(p.v[4], "out", {T, H}, dt, dev);
    const int64_t os = rows(out, "out", {T, H}, dt, dev);
    launch("moe_wna16_combine_tokens", dev, [&](hipStream_t s) {
        return lib.combine_tokens(y.data_ptr(), (const int32_t *)slots.data_ptr(),
                                  (const float *)wp, ap, (int)T, (int)k, (int)H, (int)R, ys, as, os,
                                  code, out.data_ptr(), s);
    });
    if constexpr (GRAPH) {
        auto given = [&](int i) {
            return p.v[i] ? std::optional<at::Tensor>(THPVariable_Unpack(p.v[i])) : std::nullopt;
        };
        const std::optional<at::Tensor> w = given(2), add = given(3);
        Combined c{slots, {}, out, y.requires_grad(), w && w->requires_grad(),
                   add && add->requires_grad()};
        if (p.v[5])
            c.offsets = tensor(p.v[5], "offsets");
        out = CombineNode::apply(y, w, add, (const Combined *)&c)[0];
    }
    return THPVariable_Wrap(out);
}

const char k_quant_fp8[] = R"(quant_fp8(x, *, q=None, scale=None) -> (q, scale)

Rows x [T, K] (bf16, fp16 or fp32; rows may be strided) in 8-bit floating point:
codes float8_e4m3fn [T, K], and scale float32 [T, ceil(K / 128)], the smallest power
of two for each 128 elements under which the largest fits.  x is about q * scale,
with one rounding of each element to e4m3.  No gradient: outputs carry no graph.)";

const char k_swiglu_quant_fp8[] = R"(swiglu_quant_fp8(gu, *, alpha=1.0, beta=0.0, clamp=None, q=None, scale=None) -> (q, scale)

SwiGLU of rows gu = [gate (I), up (I)] [T, 2I] (bf16, fp16 or fp32; rows may be
strided) in 8-bit floating point, codes [T, I] and scales as quant_fp8's.  alpha,
beta, clamp as in forward().  No gradient: outputs carry no graph.)";

const char k_gemm_fp8[] = R"(gemm_fp8(a, a_scale, w, w_scale, *, addend=None, out_dtype=torch.bfloat16, out=None, workspace=None) -> out

The product of rows and a weight in 8-bit floating point, scaled by blocks of 128:
the sum over blocks b of a_scale[t, b] * w_scale[n // 128, b] * (a[t, b] . w[n, b]),
plus the addend, in FP32, rounded to out_dtype at the end.  (Of eight consecutive products
in k, bits below 2^-13 of the largest one's power of two are dropped by the matrix cores:
about 1.5e-5 of a result, which out_dtype float32 shows.)

a float8_e4m3fn [T, K], a_scale float32 [T, ceil(K / 128)], as quant_fp8 gives
them; w float8_e4m3fn [N, K], w_scale float32 [ceil(N / 128), ceil(K / 128)];
addend [T, N] of out_dtype (bf16, fp16, fp32).  Rows may be strided; K, the strides of
a and w and their addresses are multiples of 16.  out may be the addend.  workspace:
from gemm_fp8_workspace_for, kept by the caller and used by one call at a time;
allocated here when it is needed and not given.  No gradient: the output carries no
graph.)";

const char k_gemm_fp8_grouped[] = R"(gemm_fp8_grouped(a, a_scale, w, w_scale, offsets, *, rows=None, out_dtype=torch.bfloat16, out=None) -> out

gemm_fp8 for rows sorted by expert: row i of out, offsets[e] <= i < offsets[e + 1], is
the product of a's row rows[i] (row i without rows) with w[e].

a, a_scale as in gemm_fp8; w float8_e4m3fn [E, N, K], w_scale float32 [E, ceil(N / 128),
ceil(K / 128)]; offsets int32 [E + 1] and rows int32 [R] as sort_tokens returns them
("offsets", "tokens").  out [R, N]; its rows from offsets[E] on are not written.  No
gradient: the output carries no graph.)";

PyMethodDef methods[] = {
    {"quant_fp8", MOE_MODULE_FAST(quant<false>), METH_FASTCALL | METH_KEYWORDS, k_quant_fp8},
    {"swiglu_quant_fp8", MOE_MODULE_FAST(quant<true>), METH_FASTCALL | METH_KEYWORDS,
     k_swiglu_quant_fp8},
    {"gemm_fp8", MOE_MODULE_FAST(gemm_fp8), METH_FASTCALL | METH_KEYWORDS, k_gemm_fp8},
    {"gemm_fp8_grouped", MOE_MODULE_FAST(gemm_fp8_grouped), METH_FASTCALL | METH_KEYWORDS,
     k_gemm_fp8_grouped},
    {"sort_tokens", MOE_MODULE_FAST(sort_tokens<false>), METH_FASTCALL | METH_KEYWORDS, nullptr},
    {"sort_tokens_graph", MOE_MODULE_FAST(sort_tokens<true>), METH_FASTCALL | METH_KEYWORDS, nullptr},
    {"combine_tokens", MOE_MODULE_FAST(combine_tokens<false>), METH_FASTCALL | METH_KEYWORDS, nullptr},
    {"combine_tokens_graph", MOE_MODULE_FAST(combine_tokens<true>), METH_FASTCALL | METH_KEYWORDS,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

}  // namespace

bool moe_module::add_expert_ops(PyObject *module)
{
    struct { PyObject **at; const char *name; } const all[] = {
        {&n_x, "x"}, {&n_q, "q"}, {&n_scale, "scale"}, {&n_gu, "gu"}, {&n_alpha, "alpha"},
        {&n_beta, "beta"}, {&n_clamp, "clamp"}, {&n_a, "a"}, {&n_a_scale, "a_scale"}, {&n_w, "w"},
        {&n_w_scale, "w_scale"}, {&n_addend, "addend"}, {&n_out_dtype, "out_dtype"},
        {&n_out, "out"}, {&n_workspace, "workspace"}, {&n_offsets, "offsets"}, {&n_rows, "rows"},
        {&n_ids, "ids"}, {&n_experts, "experts"}, {&n_tokens, "tokens"}, {&n_slots, "slots"},
        {&n_y, "y"}, {&n_weights, "weights"}};
    for (const auto &n : all)
        if (!(*n.at = PyUnicode_InternFromString(n.name)))
            return false;
    return PyModule_AddFunctions(module, methods) == 0;
}
