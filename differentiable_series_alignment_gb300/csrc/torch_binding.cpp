// torch_binding.cpp -- the encoder operators as torch autograd functions: checks of arguments,
// torch's memory and streams, and calls of the C entry points of include/sdtw.h, nothing
// more. Compiled rather than written in Python because autograd runs a backward pass in a
// thread of its own, where every line of Python costs two or three times as much: the
// forward and backward of a layer norm of 16384 x 64 took some 300 us that way and 130 here.
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "../../include/sdtw.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using Maybe = std::optional<Tensor>;

int dtype_of(const Tensor& t, const char* name)
{
    switch (t.scalar_type()) {
        case at::kFloat: return SDTW_F32;
        case at::kBFloat16: return SDTW_BF16;
        case at::kHalf: return SDTW_F16;
        default: TORCH_CHECK_TYPE(false, name, " must be float32, bfloat16 or float16"); return 0;
    }
}
void check_cuda(const Tensor& t, const char* name)
{
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    dtype_of(t, name);
}
void check_sizes(const Tensor& t, const char* name)
{
    for (const int64_t n : t.sizes())
        TORCH_CHECK_VALUE(n <= std::numeric_limits<int>::max(), name, " has a dimension of ", n, ", more than 32 bits count");
}
// A status of a C entry point. It leaves a call as the package's SdtwError; autograd makes a RuntimeError of the same
// words of one from a backward pass.
struct StatusError : std::runtime_error {
    sdtw_status status;
    const char* where;
    StatusError(sdtw_status s, const char* w) : std::runtime_error(std::string(w) + ": " + sdtw_status_string(s)), status(s), where(w) {}
};
void check_status(sdtw_status s, const char* where)
{
    if (s != SDTW_OK) throw StatusError(s, where);
}
void once_only()
{
    TORCH_CHECK(!at::GradMode::is_enabled(), "the encoder operators are differentiable once");
}
void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
Tensor like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }   // contiguous
// Conversions that have nothing to do cost a call of the dispatcher each, a third of a small operator's time.
Tensor packed(const Tensor& t) { return t.is_contiguous() ? t : t.contiguous(); }
// Integers as the kernels take them. What lies outside 32 bits becomes the nearest end of their range, which is
// outside any table and beyond any length too.
Tensor as_int(Tensor t, const Tensor& beside)
{
    constexpr int64_t low = std::numeric_limits<int>::min(), high = std::numeric_limits<int>::max();
    if (t.scalar_type() == at::kUInt64) t = t.to(at::kDouble).clamp(0, static_cast<double>(high));
    if (t.scalar_type() == at::kLong || t.scalar_type() == at::kUInt32) t = t.to(at::kLong).clamp(low, high);
    return packed(t.scalar_type() == at::kInt && t.device() == beside.device() ? t : t.to(beside.device(), at::kInt));
}
Tensor workspace(size_t n, const Tensor& t)
{
    return n ? at::empty({static_cast<int64_t>(n)}, t.options().dtype(at::kByte)) : Tensor();
}
size_t bytes(const Tensor& ws) { return ws.defined() ? static_cast<size_t>(ws.numel()) : 0; }
Maybe given(const Tensor& t) { return t.defined() ? Maybe(t) : std::nullopt; }   // autograd takes no undefined inputs
Tensor value(const Maybe& t) { return t.has_value() ? *t : Tensor(); }
bool wants(const Tensor& t) { return t.defined() && t.requires_grad(); }
// Whether autograd records a call of these tensors. Tangents of forward mode would be lost: a tensor may carry one
// without requiring a gradient.
bool recording(std::initializer_list<Tensor> ts)
{
    const bool tangents = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    for (const Tensor& t : ts)
        TORCH_CHECK_NOT_IMPLEMENTED(!tangents || !t.defined() || !t._fw_grad(0).defined(), "the encoder operators have no forward-mode derivative");
    if (!at::GradMode::is_enabled()) return false;
    for (const Tensor& t : ts)
        if (wants(t)) return true;
    return false;
}

// ---- layer norm
Tensor norm_forward(const Tensor& x, const Tensor& w, const Tensor& b, double eps, const Tensor& stats)
{
    const c10::cuda::CUDAGuard guard(x.device());
    const int64_t C = x.size(-1), rows = x.numel() / C;
    Tensor y = like(x);
    if (rows == 0) return y;
    const Tensor& any = w.defined() ? w : b;
    float* mean = stats.defined() ? stats.data_ptr<float>() : nullptr;
    TORCH_CHECK_VALUE(C <= std::numeric_limits<int>::max(), "x's last dimension is too long");
    check_status(sdtw_layernorm_forward(ptr(x), ptr(w), ptr(b), rows, static_cast<int>(C), static_cast<float>(eps),
                                        dtype_of(x, "x"), any.defined() ? dtype_of(any, "weight") : SDTW_F32, ptr(y), mean,
                                        mean ? mean + rows : nullptr, stream()),
                 "sdtw_layernorm_forward");
    return y;
}

struct LayerNorm : torch::autograd::Function<LayerNorm> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Maybe& weight, const Maybe& bias, double eps)
    {
        const Tensor w = value(weight), b = value(bias);
        const Tensor stats = at::empty({2, x.numel() / x.size(-1)}, x.options().dtype(at::kFloat));
        Tensor y = norm_forward(x, w, b, eps, stats);
        ctx->save_for_backward({x, w, b, stats});
        ctx->saved_data["want"] = (wants(x) ? 1 : 0) | (wants(w) ? 2 : 0) | (wants(b) ? 4 : 0);
        return y;
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &w = saved[1], &b = saved[2], &stats = saved[3];
        const int64_t want = ctx->saved_data["want"].toInt();
        const c10::cuda::CUDAGuard guard(x.device());
        const int64_t C = x.size(-1), rows = x.numel() / C;
        Tensor dx, dw, db, ws;
        if (want & 1) dx = like(x);
        if (want & 2) dw = rows ? like(w) : at::zeros_like(w);
        if (want & 4) db = rows ? like(b) : at::zeros_like(b);
        if (rows) {
            if (want & 6) ws = workspace(sdtw_layernorm_workspace_bytes(rows, static_cast<int>(C)), x);
            const Tensor dy = packed(grads[0]);
            const Tensor& any = w.defined() ? w : b;
            float* mean = stats.data_ptr<float>();
            check_status(sdtw_layernorm_backward(ptr(dy), ptr(x), ptr(w), mean, mean + rows, rows, static_cast<int>(C),
                                                 dtype_of(x, "x"), any.defined() ? dtype_of(any, "weight") : SDTW_F32, ptr(dx),
                                                 ptr(dw), ptr(db), ptr(ws), bytes(ws), stream()),
                         "sdtw_layernorm_backward");
        }
        return {dx, dw, db, Tensor()};
    }
};

Tensor layer_norm(const Tensor& x_, const Maybe& weight, const Maybe& bias, double eps)
{
    check_cuda(x_, "x");
    TORCH_CHECK_VALUE(x_.dim() >= 1 && x_.size(-1) >= 1, "x must have a last dimension of at least 1");
    TORCH_CHECK_VALUE(eps >= 0 && std::isfinite(static_cast<float>(eps)), "eps must be >= 0 and finite in float32");
    Tensor w = value(weight), b = value(bias);
    for (int k = 0; k < 2; ++k) {
        const Tensor& t = k ? b : w;
        const char* name = k ? "bias" : "weight";
        if (!t.defined()) continue;
        check_cuda(t, name);
        TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == x_.size(-1), name, " must be (", x_.size(-1), ",)");
        TORCH_CHECK_TYPE(t.scalar_type() == x_.scalar_type() || t.scalar_type() == at::kFloat, name,
                         " must be float32 or of x's type");
        TORCH_CHECK_VALUE(t.device() == x_.device(), name, " must be on x's device");
    }
    TORCH_CHECK_TYPE(!w.defined() || !b.defined() || w.scalar_type() == b.scalar_type(), "weight and bias must be of one type");
    const Tensor x = packed(x_);
    if (w.defined()) w = packed(w);
    if (b.defined()) b = packed(b);
    if (recording({x, w, b})) return LayerNorm::apply(x, given(w), given(b), eps);
    return norm_forward(x, w, b, eps, Tensor());
}

// ---- rotary positions
Tensor with_features(const Tensor& t) { return t.stride(3) == 1 || t.size(3) == 1 ? t : t.contiguous(); }

variable_list rotate(const Tensor& q_, const Tensor& k_, const Tensor& table, const Tensor& positions, bool interleaved,
                     bool inverse)
{
    const c10::cuda::CUDAGuard guard(q_.device());
    const Tensor q = with_features(q_), k = k_.defined() ? with_features(k_) : Tensor();
    Tensor qo = like(q), ko = k.defined() ? like(k) : Tensor();
    // those that have something to turn; one of the two may have no heads
    const Tensor* in[2] = {nullptr, nullptr};
    void* out[2] = {nullptr, nullptr};
    long long stride[2][3] = {};
    int heads[2] = {0, 0}, count = 0;
    for (const auto& [t, o] : {std::pair(&q, &qo), std::pair(&k, &ko)}) {
        if (!t->defined() || t->numel() == 0) continue;
        for (int i = 0; i < 3; ++i) stride[count][i] = t->stride(i);
        in[count] = t, out[count] = ptr(*o), heads[count] = static_cast<int>(t->size(2)), ++count;
    }
    if (count) {
        const int N = static_cast<int>(q.size(1));
        // positions are 32 bits: what a longer table has beyond is out of their reach
        const int length = static_cast<int>(std::min<int64_t>(table.size(0), std::numeric_limits<int>::max()));
        check_status(sdtw_rotary(ptr(*in[0]), stride[0], count > 1 ? ptr(*in[1]) : nullptr, stride[1], static_cast<int>(q.size(0)), N,
                                 heads[0], heads[1], static_cast<int>(q.size(3)), static_cast<int>(2 * table.size(1)),
                                 table.data_ptr<float>(), length, positions.defined() ? positions.data_ptr<int>() : nullptr,
                                 positions.defined() && positions.dim() == 2 ? N : 0, interleaved, inverse, dtype_of(q, "q"), out[0],
                                 out[1], stream()),
                     "sdtw_rotary");
    }
    if (ko.defined()) return {qo, ko};
    return {qo};
}

struct Rotary : torch::autograd::Function<Rotary> {
    static variable_list forward(AutogradContext* ctx, const Tensor& q, const Maybe& k_, const Tensor& table,
                                 const Maybe& positions_, bool interleaved)
    {
        const Tensor k = value(k_), positions = value(positions_);
        ctx->save_for_backward({table, positions});
        ctx->saved_data["interleaved"] = interleaved;
        return rotate(q, k, table, positions, interleaved, false);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list saved = ctx->get_saved_variables();
        variable_list g = rotate(grads[0], grads.size() > 1 ? grads[1] : Tensor(), saved[0], saved[1],
                                 ctx->saved_data["interleaved"].toBool(), true);
        return {g[0], g.size() > 1 ? g[1] : Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

variable_list rotary(const Tensor& q, const Maybe& k_, const Tensor& table_, const Maybe& positions_, bool interleaved)
{
    check_cuda(q, "q");
    TORCH_CHECK_VALUE(q.dim() == 4, "q must be (B, N, H, D)");
    check_sizes(q, "q");
    const Tensor k = value(k_);
    if (k.defined()) {
        check_cuda(k, "k");
        TORCH_CHECK_TYPE(k.scalar_type() == q.scalar_type(), "k must be of q's type");
        TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == q.size(0) && k.size(1) == q.size(1) && k.size(3) == q.size(3) &&
                              k.device() == q.device(),
                          "k must be (B, N, H, D) with q's batch, positions and features, on q's device");
        check_sizes(k, "k");
    }
    TORCH_CHECK_VALUE(table_.dim() == 3 && table_.size(2) == 2 && table_.scalar_type() == at::kFloat && table_.device() == q.device(),
                      "table must be a (length, R / 2, 2) float32 tensor on q's device, as rotary_table gives");
    TORCH_CHECK_VALUE(table_.size(1) >= 1 && 2 * table_.size(1) <= q.size(3), "the table turns more features than a head has, or none");
    Tensor positions = value(positions_);
    if (positions.defined()) {
        TORCH_CHECK_VALUE(at::isIntegralType(positions.scalar_type(), false) &&
                              ((positions.dim() == 2 && positions.size(0) == q.size(0) && positions.size(1) == q.size(1)) ||
                               (positions.dim() == 1 && positions.size(0) == q.size(1))),
                          "positions must be (B, N) or (N,) integers");
        positions = as_int(positions, q);
    } else {
        TORCH_CHECK_VALUE(q.size(1) <= table_.size(0), "the table has fewer positions than q");
    }
    Tensor table = packed(table_.requires_grad() ? table_.detach() : table_);
    if (reinterpret_cast<uintptr_t>(table.data_ptr()) & 7) table = table.clone();   // a pair's cosine and sine are one load
    if (recording({q, k})) return Rotary::apply(q, given(k), table, given(positions), interleaved);
    return rotate(q, k, table, positions, interleaved, false);
}

// ---- attention
struct Masks {
    Tensor q_lengths, k_lengths;
    double scale;
    int64_t left, right;
};
sdtw_attention problem(const Tensor& q, const Tensor& k, const Tensor& v, const Masks& m)
{
    sdtw_attention a{};
    a.q = ptr(q), a.k = ptr(k), a.v = ptr(v);
    for (int i = 0; i < 3; ++i) a.q_stride[i] = q.stride(i), a.k_stride[i] = k.stride(i), a.v_stride[i] = v.stride(i);
    a.q_lengths = m.q_lengths.defined() ? m.q_lengths.data_ptr<int>() : nullptr;
    a.k_lengths = m.k_lengths.defined() ? m.k_lengths.data_ptr<int>() : nullptr;
    a.B = static_cast<int>(q.size(0)), a.N = static_cast<int>(q.size(1)), a.M = static_cast<int>(k.size(1));
    a.Hq = static_cast<int>(q.size(2)), a.Hkv = static_cast<int>(k.size(2)), a.D = static_cast<int>(q.size(3));
    a.dtype = dtype_of(q, "q");
    a.window_left = static_cast<int>(m.left), a.window_right = static_cast<int>(m.right);
    a.scale = static_cast<float>(m.scale);
    return a;
}

// out, what its rounding left (keep, 16-bit types) and lse (keep or want_lse)
std::array<Tensor, 3> attend(const Tensor& q, const Tensor& k, const Tensor& v, const Masks& m, bool keep, bool want_lse)
{
    const c10::cuda::CUDAGuard guard(q.device());
    Tensor out = like(q), rest, lse;
    if (keep && q.scalar_type() != at::kFloat) rest = like(q);
    if (keep || want_lse) lse = at::empty({q.size(0), q.size(2), q.size(1)}, q.options().dtype(at::kFloat));
    if (out.numel() == 0 || k.numel() == 0) {
        out.zero_();
        if (lse.defined()) lse.fill_(-std::numeric_limits<float>::infinity());
        return {out, rest, lse};
    }
    const sdtw_attention a = problem(q, k, v, m);
    const Tensor ws = workspace(sdtw_attention_workspace_bytes(&a, 0), q);
    check_status(sdtw_attention_forward(&a, ptr(out), ptr(rest), static_cast<float*>(ptr(lse)), ptr(ws), bytes(ws), stream()),
                 "sdtw_attention_forward");
    return {out, rest, lse};
}

struct Attention : torch::autograd::Function<Attention> {
    static variable_list forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v, const Maybe& ql,
                                 const Maybe& kl, double scale, int64_t left, int64_t right)
    {
        const Tensor q_lengths = value(ql), k_lengths = value(kl);
        const auto got = attend(q, k, v, {q_lengths, k_lengths, scale, left, right}, true, true);
        ctx->save_for_backward({q, k, v, got[0], got[1], got[2], q_lengths, k_lengths});
        ctx->saved_data["scale"] = scale;
        ctx->saved_data["left"] = left;
        ctx->saved_data["right"] = right;
        ctx->saved_data["want"] = (wants(q) ? 1 : 0) | (wants(k) ? 2 : 0) | (wants(v) ? 4 : 0);
        ctx->mark_non_differentiable({got[2]});
        return {got[0], got[2]};
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list s = ctx->get_saved_variables();
        const Tensor &q = s[0], &k = s[1], &v = s[2], &out = s[3], &rest = s[4], &lse = s[5];
        const Masks m{s[6], s[7], ctx->saved_data["scale"].toDouble(), ctx->saved_data["left"].toInt(), ctx->saved_data["right"].toInt()};
        const int64_t want = ctx->saved_data["want"].toInt();
        const c10::cuda::CUDAGuard guard(q.device());
        Tensor dq, dk, dv;
        if (want & 1) dq = like(q);
        if (want & 6) dk = like(k), dv = like(v);
        if (q.numel() == 0 || k.numel() == 0) {
            for (Tensor* t : {&dq, &dk, &dv})
                if (t->defined()) t->zero_();
        } else if (want) {
            const sdtw_attention a = problem(q, k, v, m);
            const Tensor ws = workspace(sdtw_attention_workspace_bytes(&a, 1), q);
            const Tensor dout = packed(grads[0]);
            check_status(sdtw_attention_backward(&a, ptr(out), ptr(rest), static_cast<float*>(ptr(lse)), ptr(dout), ptr(dq), ptr(dk),
                                                 ptr(dv), ptr(ws), bytes(ws), stream()),
                         "sdtw_attention_backward");
        }
        return {dq, want & 2 ? dk : Tensor(), want & 4 ? dv : Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

Tensor lengths_of(const Maybe& t, const Tensor& q, const char* name)
{
    if (!t.has_value() || !t->defined()) return Tensor();
    TORCH_CHECK_VALUE(at::isIntegralType(t->scalar_type(), false) && t->dim() == 1 && t->size(0) == q.size(0), name,
                      " must be a (B,) integer tensor");
    return as_int(*t, q);
}

// (out,) or (out, lse)
variable_list attention(const Tensor& q_, const Tensor& k_, const Tensor& v_, bool causal, std::optional<int64_t> window,
                        const Maybe& q_lengths, const Maybe& k_lengths, std::optional<double> scale_, bool return_lse)
{
    const Tensor* in[3] = {&q_, &k_, &v_};
    const char* names[3] = {"q", "k", "v"};
    for (int i = 0; i < 3; ++i) {
        check_cuda(*in[i], names[i]);
        TORCH_CHECK_TYPE(in[i]->scalar_type() == q_.scalar_type(), names[i], " must be of q's type");
        TORCH_CHECK_VALUE(in[i]->dim() == 4 && in[i]->device() == q_.device(), names[i], " must be (B, L, H, D), on q's device");
        check_sizes(*in[i], names[i]);
    }
    TORCH_CHECK_VALUE(k_.sizes() == v_.sizes() && k_.size(0) == q_.size(0) && k_.size(3) == q_.size(3),
                      "k and v must both be (B, M, Hkv, D) with q's batch and features");
    const int64_t D = q_.size(3), Hq = q_.size(2), Hkv = k_.size(2);
    TORCH_CHECK_VALUE(D >= 1 && D <= 128, "the head size must be 1 to 128");
    TORCH_CHECK_VALUE(Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0, "the query heads must be a multiple of the key heads");
    TORCH_CHECK_VALUE(!window || *window >= 1, "window must be >= 1");
    const double scale = scale_ ? *scale_ : 1.0 / std::sqrt(static_cast<double>(D));
    TORCH_CHECK_VALUE(static_cast<float>(scale) > 0 && std::isfinite(static_cast<float>(scale)), "scale must be > 0 and finite in float32");
    const int64_t left = window ? std::min<int64_t>(*window - 1, std::numeric_limits<int>::max() - 1) : -1;
    const int64_t right = causal ? 0 : left;
    const Tensor ql = lengths_of(q_lengths, q_, "q_lengths"), kl = lengths_of(k_lengths, q_, "k_lengths");
    const Tensor q = with_features(q_), k = with_features(k_), v = with_features(v_);
    if (recording({q, k, v})) {
        variable_list r = Attention::apply(q, k, v, given(ql), given(kl), scale, left, right);
        if (!return_lse) r.resize(1);
        return r;
    }
    const auto got = attend(q, k, v, {ql, kl, scale, left, right}, false, return_lse);
    if (return_lse) return {got[0], got[2]};
    return {got[0]};
}

// ---- group norm
Tensor group_forward(const Tensor& x, const Tensor& w, const Tensor& b, const Tensor& lengths, int64_t groups, double eps, int64_t activation,
                     const Tensor& stats)
{
    const c10::cuda::CUDAGuard guard(x.device());
    Tensor y = like(x);
    if (x.numel() == 0) return y;
    const int B = static_cast<int>(x.size(0)), C = static_cast<int>(x.size(-1)), S = static_cast<int>(x.numel() / x.size(0) / C);
    const Tensor& any = w.defined() ? w : b;
    float* mean = stats.defined() ? stats.data_ptr<float>() : nullptr;
    const Tensor ws = workspace(sdtw_groupnorm_workspace_bytes(B, S, static_cast<int>(groups), C, dtype_of(x, "x"), 0), x);
    check_status(sdtw_groupnorm_forward(ptr(x), ptr(w), ptr(b), static_cast<int*>(ptr(lengths)), B, S, static_cast<int>(groups), C,
                                        static_cast<float>(eps), static_cast<int>(activation), dtype_of(x, "x"),
                                        any.defined() ? dtype_of(any, "weight") : SDTW_F32, ptr(y), mean,
                                        mean ? mean + B * groups : nullptr, ptr(ws), bytes(ws), stream()),
                 "sdtw_groupnorm_forward");
    return y;
}

struct GroupNorm : torch::autograd::Function<GroupNorm> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Maybe& weight, const Maybe& bias, const Maybe& lengths_,
                          int64_t groups, double eps, int64_t activation)
    {
        const Tensor w = value(weight), b = value(bias), lengths = value(lengths_);
        const Tensor stats = at::empty({2, x.size(0), groups}, x.options().dtype(at::kFloat));
        Tensor y = group_forward(x, w, b, lengths, groups, eps, activation, stats);
        ctx->save_for_backward({x, w, b, lengths, stats});
        ctx->saved_data["groups"] = groups;
        ctx->saved_data["activation"] = activation;
        ctx->saved_data["want"] = (wants(x) ? 1 : 0) | (wants(w) ? 2 : 0) | (wants(b) ? 4 : 0);
        return y;
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &w = saved[1], &b = saved[2], &lengths = saved[3], &stats = saved[4];
        const int groups = static_cast<int>(ctx->saved_data["groups"].toInt());
        const int64_t want = ctx->saved_data["want"].toInt();
        const c10::cuda::CUDAGuard guard(x.device());
        const bool some = x.numel() != 0;
        Tensor dx, dw, db;
        if (want & 1) dx = like(x);
        if (want & 2) dw = some ? like(w) : at::zeros_like(w);
        if (want & 4) db = some ? like(b) : at::zeros_like(b);
        if (some) {
            const int B = static_cast<int>(x.size(0)), C = static_cast<int>(x.size(-1)), S = static_cast<int>(x.numel() / x.size(0) / C);
            const Tensor ws = workspace(sdtw_groupnorm_workspace_bytes(B, S, groups, C, dtype_of(x, "x"), 1), x);
            const Tensor dy = packed(grads[0]);
            const Tensor& any = w.defined() ? w : b;
            float* mean = stats.data_ptr<float>();
            check_status(sdtw_groupnorm_backward(ptr(dy), ptr(x), ptr(w), ptr(b), static_cast<int*>(ptr(lengths)), mean,
                                                 mean + static_cast<int64_t>(B) * groups, B, S, groups, C,
                                                 static_cast<int>(ctx->saved_data["activation"].toInt()), dtype_of(x, "x"),
                                                 any.defined() ? dtype_of(any, "weight") : SDTW_F32, ptr(dx), ptr(dw), ptr(db),
                                                 ptr(ws), bytes(ws), stream()),
                         "sdtw_groupnorm_backward");
        }
        return {dx, dw, db, Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

Tensor group_norm(const Tensor& x_, int64_t groups, const Maybe& weight, const Maybe& bias, double eps, int64_t activation,
                  const Maybe& lengths_)
{
    check_cuda(x_, "x");
    TORCH_CHECK_VALUE(x_.dim() >= 2 && x_.size(-1) >= 1, "x must be (B, ..., C) with at least one channel");
    check_sizes(x_, "x");
    TORCH_CHECK_VALUE(groups >= 1 && x_.size(-1) % groups == 0, "groups must divide the channels, ", x_.size(-1));
    TORCH_CHECK_VALUE(eps >= 0 && std::isfinite(static_cast<float>(eps)), "eps must be >= 0 and finite in float32");
    TORCH_CHECK_VALUE(x_.numel() == 0 || x_.numel() / x_.size(0) / x_.size(-1) <= std::numeric_limits<int>::max(),
                      "x has more positions than 32 bits count");
    Tensor w = value(weight), b = value(bias);
    for (int k = 0; k < 2; ++k) {
        const Tensor& t = k ? b : w;
        const char* name = k ? "bias" : "weight";
        if (!t.defined()) continue;
        check_cuda(t, name);
        TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == x_.size(-1), name, " must be (", x_.size(-1), ",)");
        TORCH_CHECK_TYPE(t.scalar_type() == x_.scalar_type() || t.scalar_type() == at::kFloat, name,
                         " must be float32 or of x's type");
        TORCH_CHECK_VALUE(t.device() == x_.device(), name, " must be on x's device");
    }
    TORCH_CHECK_TYPE(!w.defined() || !b.defined() || w.scalar_type() == b.scalar_type(), "weight and bias must be of one type");
    const Tensor lengths = lengths_of(lengths_, x_, "lengths");
    TORCH_CHECK_VALUE(!lengths.defined() || x_.dim() == 3, "lengths needs x of (B, N, C)");
    const Tensor x = packed(x_);
    if (w.defined()) w = packed(w);
    if (b.defined()) b = packed(b);
    if (recording({x, w, b})) return GroupNorm::apply(x, given(w), given(b), given(lengths), groups, eps, activation);
    return group_forward(x, w, b, lengths, groups, eps, activation, Tensor());
}

// ---- gated recurrence
// channels side by side, and rows of a stride that the kernels take
Tensor with_channels(const Tensor& t) { return (t.stride(2) == 1 || t.size(2) == 1) && t.stride(1) > 0 && t.stride(1) <= 1 << 23 ? t : t.contiguous(); }

sdtw_recurrence recurrence(const Tensor& x, const Tensor& gate, const Tensor& state, const Tensor& lengths, bool reverse, bool tied)
{
    sdtw_recurrence a{};
    a.x = ptr(x), a.gate = ptr(gate), a.state = static_cast<float*>(ptr(state)), a.lengths = static_cast<int*>(ptr(lengths));
    for (int i = 0; i < 2; ++i) a.x_stride[i] = x.stride(i), a.gate_stride[i] = gate.stride(i);
    a.B = static_cast<int>(x.size(0)), a.N = static_cast<int>(x.size(1)), a.C = static_cast<int>(x.size(2));
    a.dtype = dtype_of(x, "x"), a.reverse = reverse, a.tied = tied;
    return a;
}

// h, last (want_last) and the states for the backward pass (keep)
std::array<Tensor, 3> recur(const Tensor& x, const Tensor& gate, const Tensor& state, const Tensor& lengths, bool reverse, bool tied,
                            bool want_last, bool keep)
{
    const c10::cuda::CUDAGuard guard(x.device());
    const auto f32 = x.options().dtype(at::kFloat);
    Tensor h = like(x), last, kept;
    if (want_last) last = at::empty({x.size(0), x.size(2)}, f32);
    if (x.numel() == 0) {
        if (want_last) state.defined() ? last.copy_(state) : last.zero_();
        return {h, last, kept};
    }
    if (keep) kept = at::empty({x.size(0), (x.size(1) + SDTW_RECURRENCE_STEP - 1) / SDTW_RECURRENCE_STEP, x.size(2)}, f32);
    const sdtw_recurrence a = recurrence(x, gate, state, lengths, reverse, tied);
    check_status(sdtw_recurrence_forward(&a, ptr(h), static_cast<float*>(ptr(last)), static_cast<float*>(ptr(kept)), stream()),
                 "sdtw_recurrence_forward");
    return {h, last, kept};
}

struct Recurrence : torch::autograd::Function<Recurrence> {
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& gate, const Maybe& state_, const Maybe& lengths_,
                                 bool reverse, bool tied)
    {
        const Tensor state = value(state_), lengths = value(lengths_);
        const auto got = recur(x, gate, state, lengths, reverse, tied, true, true);
        ctx->save_for_backward({x, gate, state, lengths, got[2]});
        ctx->saved_data["reverse"] = reverse;
        ctx->saved_data["tied"] = tied;
        ctx->saved_data["want"] = (wants(x) ? 1 : 0) | (wants(gate) ? 2 : 0) | (wants(state) ? 4 : 0);
        ctx->set_materialize_grads(false);   // an output that the loss does not use costs nothing
        return {got[0], got[1]};
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list s = ctx->get_saved_variables();
        const Tensor &x = s[0], &gate = s[1], &state = s[2], &lengths = s[3], &kept = s[4];
        const int64_t want = ctx->saved_data["want"].toInt();
        if (!grads[0].defined() && !grads[1].defined()) return variable_list(6);
        const c10::cuda::CUDAGuard guard(x.device());
        Tensor dx = like(x), dgate = like(x), dstate;
        if (want & 4) dstate = like(state);
        if (x.numel() == 0) {
            if (want & 4) grads[1].defined() ? dstate.copy_(grads[1]) : dstate.zero_();
        } else {
            const sdtw_recurrence a = recurrence(x, gate, state, lengths, ctx->saved_data["reverse"].toBool(), ctx->saved_data["tied"].toBool());
            const Tensor dh = grads[0].defined() ? packed(grads[0]) : Tensor(), dlast = grads[1].defined() ? packed(grads[1]) : Tensor();
            check_status(sdtw_recurrence_backward(&a, kept.data_ptr<float>(), ptr(dh), static_cast<float*>(ptr(dlast)), ptr(dx), ptr(dgate),
                                                  static_cast<float*>(ptr(dstate)), stream()),
                         "sdtw_recurrence_backward");
        }
        return {want & 1 ? dx : Tensor(), want & 2 ? dgate : Tensor(), dstate, Tensor(), Tensor(), Tensor()};
    }
};

// (h,) or (h, last)
variable_list gated_recurrence(const Tensor& x_, const Tensor& gate_, const Maybe& state_, const Maybe& lengths_, bool reverse, bool tied,
                               bool return_state)
{
    check_cuda(x_, "x");
    check_cuda(gate_, "gate");
    TORCH_CHECK_VALUE(x_.dim() == 3, "x must be (B, N, C)");
    check_sizes(x_, "x");
    TORCH_CHECK_TYPE(gate_.scalar_type() == x_.scalar_type(), "gate must be of x's type");
    TORCH_CHECK_VALUE(gate_.sizes() == x_.sizes() && gate_.device() == x_.device(), "gate must have x's shape, on x's device");
    Tensor state = value(state_);
    if (state.defined()) {
        TORCH_CHECK_TYPE(state.scalar_type() == at::kFloat, "state must be float32");
        TORCH_CHECK_VALUE(state.dim() == 2 && state.size(0) == x_.size(0) && state.size(1) == x_.size(2) && state.device() == x_.device(),
                          "state must be (B, C), on x's device");
        state = packed(state);
    }
    const Tensor lengths = lengths_of(lengths_, x_, "lengths");
    const Tensor x = with_channels(x_), gate = with_channels(gate_);
    if (recording({x, gate, state})) {
        variable_list r = Recurrence::apply(x, gate, given(state), given(lengths), reverse, tied);
        if (!return_state) r.resize(1);
        return r;
    }
    const auto got = recur(x, gate, state, lengths, reverse, tied, return_state, false);
    if (return_state) return {got[0], got[1]};
    return {got[0]};
}

// ---- gated linear units
sdtw_gated gated(const Tensor& x, const Tensor& wg, const Tensor& wu, const Tensor& bg, const Tensor& bu, int64_t activation)
{
    sdtw_gated a{};
    a.x = ptr(x), a.gate_weight = ptr(wg), a.up_weight = ptr(wu), a.gate_bias = ptr(bg), a.up_bias = ptr(bu);
    a.x_stride = x.stride(0), a.gate_stride = wg.stride(0), a.up_stride = wu.stride(0);
    a.R = x.size(0), a.K = static_cast<int>(x.size(1)), a.F = static_cast<int>(wg.size(0));
    a.dtype = dtype_of(x, "x"), a.activation = static_cast<int>(activation);
    return a;
}

Tensor gate_forward(const Tensor& x, const Tensor& wg, const Tensor& wu, const Tensor& bg, const Tensor& bu, int64_t activation)
{
    const c10::cuda::CUDAGuard guard(x.device());
    Tensor h = at::empty({x.size(0), wg.size(0)}, x.options());
    if (x.size(0) == 0) return h;
    const sdtw_gated a = gated(x, wg, wu, bg, bu, activation);
    const Tensor ws = workspace(sdtw_gated_workspace_bytes(&a, 0), x);
    check_status(sdtw_gated_forward(&a, ptr(h), ptr(ws), bytes(ws), stream()), "sdtw_gated_forward");
    return h;
}

struct GatedLinear : torch::autograd::Function<GatedLinear> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& wg, const Tensor& wu, const Maybe& bg_, const Maybe& bu_,
                          int64_t activation)
    {
        const Tensor bg = value(bg_), bu = value(bu_);
        ctx->save_for_backward({x, wg, wu, bg, bu});
        ctx->saved_data["activation"] = activation;
        ctx->saved_data["want"] = (wants(x) ? 1 : 0) | (wants(wg) ? 2 : 0) | (wants(wu) ? 4 : 0) | (wants(bg) ? 8 : 0) | (wants(bu) ? 16 : 0);
        return gate_forward(x, wg, wu, bg, bu, activation);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        once_only();
        const variable_list s = ctx->get_saved_variables();
        const Tensor& x = s[0];
        const int64_t want = ctx->saved_data["want"].toInt();
        const c10::cuda::CUDAGuard guard(x.device());
        variable_list d(6);
        const bool some = x.size(0) != 0;
        for (int i = 0; i < 5; ++i)
            if (want >> i & 1) d[i] = some ? like(s[i]) : at::zeros(s[i].sizes(), s[i].options());
        if (some && want) {
            const sdtw_gated a = gated(x, s[1], s[2], s[3], s[4], ctx->saved_data["activation"].toInt());
            const Tensor ws = workspace(sdtw_gated_workspace_bytes(&a, 1), x);
            const Tensor dh = packed(grads[0]);
            check_status(sdtw_gated_backward(&a, ptr(dh), ptr(d[0]), ptr(d[1]), ptr(d[2]), ptr(d[3]), ptr(d[4]), ptr(ws), bytes(ws), stream()),
                         "sdtw_gated_backward");
        }
        return d;
    }
};

Tensor gated_linear(const Tensor& x_, const Tensor& wg_, const Tensor& wu_, const Maybe& bg_, const Maybe& bu_, int64_t activation)
{
    check_cuda(x_, "x");
    TORCH_CHECK_VALUE(x_.dim() >= 1 && x_.size(-1) >= 1, "x must have a last dimension of at least 1");
    const int64_t K = x_.size(-1);
    const Tensor* weights[2] = {&wg_, &wu_};
    const char* names[4] = {"gate_weight", "up_weight", "gate_bias", "up_bias"};
    for (int i = 0; i < 2; ++i) {
        check_cuda(*weights[i], names[i]);
        TORCH_CHECK_TYPE(weights[i]->scalar_type() == x_.scalar_type(), names[i], " must be of x's type");
        TORCH_CHECK_VALUE(weights[i]->dim() == 2 && weights[i]->size(1) == K && weights[i]->size(0) == wg_.size(0) && wg_.size(0) >= 1 &&
                              weights[i]->device() == x_.device(),
                          names[i], " must be (F, ", K, ") as the other weight, with F >= 1, on x's device");
        check_sizes(*weights[i], names[i]);
    }
    Tensor bg = value(bg_), bu = value(bu_);
    for (int i = 0; i < 2; ++i) {
        const Tensor& t = i ? bu : bg;
        if (!t.defined()) continue;
        check_cuda(t, names[2 + i]);
        TORCH_CHECK_TYPE(t.scalar_type() == x_.scalar_type(), names[2 + i], " must be of x's type");
        TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == wg_.size(0) && t.device() == x_.device(), names[2 + i], " must be (F,), on x's device");
    }
    // rows of any stride where features are contiguous; what does not flatten to that is copied
    auto rows = [](const Tensor& t) { return t.stride(1) == 1 || t.size(1) == 1 ? t : t.contiguous(); };
    const Tensor x = rows(x_.dim() == 2 ? x_ : x_.reshape({x_.numel() / K, K})), wg = rows(wg_), wu = rows(wu_);
    if (bg.defined()) bg = packed(bg);
    if (bu.defined()) bu = packed(bu);
    const Tensor h = recording({x, wg, wu, bg, bu}) ? GatedLinear::apply(x, wg, wu, given(bg), given(bu), activation)
                                                    : gate_forward(x, wg, wu, bg, bu, activation);
    if (x_.dim() == 2) return h;
    std::vector<int64_t> shape(x_.sizes().begin(), x_.sizes().end());
    shape.back() = wg.size(0);
    return h.view(shape);
}

}  // namespace

PYBIND11_MODULE(_binding, m)
{
    py::register_local_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError& e) {
            const py::object error = py::module_::import("differentiable_series_alignment_gb300._lib").attr("SdtwError");
            PyErr_SetObject(error.ptr(), error(static_cast<int>(e.status), e.where).ptr());
        }
    });
    m.def("layer_norm", &layer_norm);
    m.def("rotary", &rotary);
    m.def("attention", &attention);
    m.def("group_norm", &group_norm);
    m.def("gated_recurrence", &gated_recurrence);
    m.def("gated_linear", &gated_linear);
}
