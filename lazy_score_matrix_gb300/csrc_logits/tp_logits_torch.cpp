// PyTorch binding of include/tp_logits.h: argument checks, outputs from PyTorch's allocator, the current stream, the
// autograd functions and the libtp call. Nothing here computes on the data.
//
// In C++, unlike the ctypes binding of tp.h: these calls sit in decoding loops and training steps where a kernel
// takes 10 us. A call through ctypes and torch's Python API cost 20 us of the caller's time on a Grace core and
// a Python autograd function 110 us more than a native one, most of it for moving the interpreter's data to autograd's
// thread and back.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <array>
#include <optional>
#include <string>
#include <tuple>
#include <vector>

#include "tp_logits.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
using torch::autograd::variable_list;

constexpr int64_t kStats = 8;  // floats per row that a forward leaves for its backward
constexpr int64_t kMaxList = 128;

// A failed call: the package's TPError, with libtp's message.
void check(tp_status s, const char* where) {
    if (s == TP_OK) return;
    pybind11::gil_scoped_acquire gil;
    pybind11::module_::import("lazy_score_matrix_gb300._lib").attr("check")((int)s, where);
}

// (group, row stride, group stride) of the rows t[..., :], or none when two strides do not describe them.
std::optional<std::array<int64_t, 3>> row_strides(const Tensor& t) {
    const int64_t last = t.dim() - 1, M = t.size(last);
    if (M > 1 && t.stride(last) != 1) return std::nullopt;
    std::vector<std::array<int64_t, 2>> dims;  // leading sizes and strides, adjacent ones joined where they can be
    for (int64_t i = 0; i < last; ++i) {
        const int64_t n = t.size(i), st = t.stride(i);
        if (n == 1) continue;
        if (!dims.empty() && dims.back()[1] == st * n) dims.back() = {dims.back()[0] * n, st};
        else dims.push_back({n, st});
    }
    if (dims.size() > 2) return std::nullopt;
    if (dims.size() == 2) return std::array<int64_t, 3>{dims[1][0], dims[1][1], dims[0][1]};
    if (dims.size() == 1) return std::array<int64_t, 3>{dims[0][0], dims[0][1], 0};
    return std::array<int64_t, 3>{1, M, 0};
}

struct Rows {
    tp_rows r;
    Tensor t;  // what r points into: a contiguous copy where the strides need one
};

Rows rows_of(const Tensor& t, const char* name, bool copy = true) {
    tp_rows r{};
    switch (t.scalar_type()) {
        case at::kFloat: r.dtype = TP_ROWS_F32; break;
        case at::kHalf: r.dtype = TP_ROWS_F16; break;
        case at::kBFloat16: r.dtype = TP_ROWS_BF16; break;
        default: TORCH_CHECK_TYPE(false, name, " must be a float32, float16 or bfloat16 tensor, got ", t.scalar_type());
    }
    TORCH_CHECK_VALUE(t.dim() >= 1 && t.size(-1) >= 1, name, " must have shape [..., M] with M >= 1, got ", t.sizes());
    TORCH_CHECK_VALUE(t.is_cuda(), "libtp runs on CUDA tensors only (no CPU fallback)");
    r.M = t.size(-1);
    r.N = t.numel() / r.M;
    Tensor kept = t;
    auto s = row_strides(t);
    if (!s) {
        TORCH_CHECK_VALUE(copy, name, ": its rows must be contiguous and lie at one stride, or at two");
        kept = t.contiguous();
        s = std::array<int64_t, 3>{r.N, r.M, 0};
    }
    r.group = (*s)[0], r.row_stride = (*s)[1], r.group_stride = (*s)[2];
    r.data = kept.data_ptr();
    return Rows{r, std::move(kept)};
}

tp_rows dense(const tp_rows& like, const Tensor& t) {
    tp_rows r = like;
    r.group = r.N, r.row_stride = r.M, r.group_stride = 0;
    r.data = t.data_ptr();
    return r;
}

// A dense per-row array of the call: dtype checked or converted, contiguous, on the logits' device.
Tensor side(const OptTensor& o, at::ScalarType type, const char* name, at::IntArrayRef shape, const Tensor& like) {
    if (!o || !o->defined()) return Tensor();
    const Tensor& t = *o;
    const bool whole = at::isIntegralType(t.scalar_type(), /*includeBool=*/false);
    TORCH_CHECK_TYPE(type == at::kLong ? whole : at::isFloatingType(t.scalar_type()), name, " must be ",
                     type == at::kLong ? "an integer" : "a floating-point", " tensor, got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
    TORCH_CHECK_VALUE(t.device() == like.device(), "all tensors must be on the same device");
    return t.to(type).contiguous();
}

template <class T>
T* ptr(const Tensor& t) {
    return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

at::IntArrayRef lead_of(const Tensor& t) { return t.sizes().slice(0, t.dim() - 1); }
std::vector<int64_t> with(at::IntArrayRef lead, int64_t n) {
    std::vector<int64_t> s(lead.begin(), lead.end());
    s.push_back(n);
    return s;
}

// A gradient of a backward that has none of its own: under create_graph it raises where it is differentiated.
Tensor once(Tensor g) {
    if (!at::GradMode::is_enabled()) return g;
    auto e = std::make_shared<torch::autograd::DelayedError>("libtp's backwards cannot be differentiated again", 1);
    return (*e)({g.detach().set_requires_grad(true)})[0];
}

Tensor dense_grad(const Tensor& g) { return g.defined() ? g.contiguous() : g; }

// --- token_logprobs ---------------------------------------------------------------------------------------------

struct Logprobs {
    Tensor logprobs, entropy, top_logprobs, top_ids, stats;
};

Logprobs logprobs_forward(const Rows& x, const Tensor& tokens, double temperature, int64_t top, bool stats) {
    const auto f32 = x.t.options().dtype(at::kFloat);
    const auto lead = lead_of(x.t);
    Logprobs o;
    if (tokens.defined()) o.logprobs = at::empty(lead, f32);
    o.entropy = at::empty(lead, f32);
    if (top) {
        const auto shape = with(lead, top);
        o.top_logprobs = at::empty(shape, f32);
        o.top_ids = at::empty(shape, f32.dtype(at::kLong));
    }
    if (stats) o.stats = at::empty({x.r.N, kStats}, f32);
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_token_logprobs(&x.r, ptr<const int64_t>(tokens), temperature, (int)top, ptr<float>(o.logprobs),
                                ptr<float>(o.entropy), ptr<float>(o.stats), ptr<float>(o.top_logprobs),
                                ptr<int64_t>(o.top_ids), stream_of(x.t)),
              "tp_token_logprobs");
    }
    return o;
}

struct LogprobsFn : torch::autograd::Function<LogprobsFn> {
    // outputs: entropy, then log probabilities (with tokens), then alternatives (with top)
    static variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& logits, const Tensor& tokens,
                                 double temperature, int64_t top) {
        const Rows x = rows_of(logits, "logits");
        const Logprobs o = logprobs_forward(x, tokens, temperature, top, true);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({x.t, tokens, o.stats});
        ctx->saved_data["T"] = temperature;
        variable_list out{o.entropy};
        if (tokens.defined()) out.push_back(o.logprobs);
        if (top) {
            ctx->mark_non_differentiable({o.top_logprobs, o.top_ids});
            out.push_back(o.top_logprobs);
            out.push_back(o.top_ids);
        }
        return out;
    }
    static variable_list backward(torch::autograd::AutogradContext* ctx, const variable_list& grads) {
        const auto saved = ctx->get_saved_variables();
        const Tensor &tokens = saved[1], &stats = saved[2];
        const Tensor g_h = dense_grad(grads[0]), g_lp = tokens.defined() ? dense_grad(grads[1]) : Tensor();
        if (!g_h.defined() && !g_lp.defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
        const Rows x = rows_of(saved[0], "logits");  // a saved tensor may come back at another address
        Tensor grad = at::empty(x.t.sizes(), x.t.options());
        if (x.r.N) {
            const c10::cuda::CUDAGuard guard(x.t.device());
            const tp_rows g = dense(x.r, grad);
            check(tp_token_logprobs_backward(&x.r, ptr<const int64_t>(tokens), ctx->saved_data["T"].toDouble(),
                                             ptr<const float>(stats), ptr<const float>(g_lp), ptr<const float>(g_h), &g,
                                             stream_of(x.t)),
                  "tp_token_logprobs_backward");
        }
        return {once(grad), Tensor(), Tensor(), Tensor()};
    }
};

using Four = std::tuple<OptTensor, Tensor, OptTensor, OptTensor>;

OptTensor maybe(const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; }

Four token_logprobs(const Tensor& logits, const OptTensor& tokens_, double temperature, int64_t top) {
    Rows x = rows_of(logits, "logits");
    TORCH_CHECK_VALUE(top >= 0 && top <= kMaxList && top <= x.r.M, "top must be in [0, min(M, 128)], got ", top);
    const Tensor tokens = side(tokens_, at::kLong, "tokens", lead_of(logits), logits);
    if (!(at::GradMode::is_enabled() && logits.requires_grad())) {
        const Logprobs o = logprobs_forward(x, tokens, temperature, top, false);
        return {maybe(o.logprobs), o.entropy, maybe(o.top_logprobs), maybe(o.top_ids)};
    }
    const auto out = LogprobsFn::apply(logits, tokens, temperature, top);
    const size_t at = tokens.defined() ? 2 : 1;
    return {tokens.defined() ? OptTensor(out[1]) : std::nullopt, out[0], top ? OptTensor(out[at]) : std::nullopt,
            top ? OptTensor(out[at + 1]) : std::nullopt};
}

// --- topk_distillation ------------------------------------------------------------------------------------------

struct Teacher {
    Tensor ids, values;
    int K;
};

Teacher teacher_of(const Tensor& ids, const Tensor& values, const Tensor& logits) {
    TORCH_CHECK_VALUE(ids.dim() >= 1 && ids.size(-1) >= 1 && ids.size(-1) <= kMaxList,
                      "a teacher's list has 1 to 128 columns a row, got ", ids.sizes());
    const auto shape = with(lead_of(logits), ids.size(-1));
    return Teacher{side(ids, at::kLong, "teacher_ids", shape, logits), side(values, at::kFloat, "teacher_values", shape, logits),
                   (int)ids.size(-1)};
}

std::pair<Tensor, Tensor> distillation_forward(const Rows& x, const Teacher& y, double temperature, bool rest, bool want_stats) {
    const auto f32 = x.t.options().dtype(at::kFloat);
    Tensor loss = at::empty(lead_of(x.t), f32), stats = want_stats ? at::empty({x.r.N, kStats}, f32) : Tensor();
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_topk_distillation(&x.r, y.K, ptr<const int64_t>(y.ids), ptr<const float>(y.values), temperature, rest,
                                   ptr<float>(loss), ptr<float>(stats), stream_of(x.t)),
              "tp_topk_distillation");
    }
    return {loss, stats};
}

struct DistillationFn : torch::autograd::Function<DistillationFn> {
    static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& logits, const Tensor& ids, const Tensor& values,
                          double temperature, bool rest) {
        const Rows x = rows_of(logits, "logits");
        const auto [loss, stats] = distillation_forward(x, Teacher{ids, values, (int)ids.size(-1)}, temperature, rest, true);
        ctx->save_for_backward({x.t, ids, values, stats});
        ctx->saved_data["T"] = temperature;
        ctx->saved_data["rest"] = rest;
        return loss;
    }
    static variable_list backward(torch::autograd::AutogradContext* ctx, const variable_list& grads) {
        const auto saved = ctx->get_saved_variables();
        const Rows x = rows_of(saved[0], "logits");
        const Tensor g_loss = dense_grad(grads[0]);
        Tensor grad = at::empty(x.t.sizes(), x.t.options());
        if (x.r.N) {
            const c10::cuda::CUDAGuard guard(x.t.device());
            const tp_rows g = dense(x.r, grad);
            check(tp_topk_distillation_backward(&x.r, (int)saved[1].size(-1), ptr<const int64_t>(saved[1]),
                                                ptr<const float>(saved[2]), ctx->saved_data["T"].toDouble(),
                                                ctx->saved_data["rest"].toBool(), ptr<const float>(saved[3]),
                                                ptr<const float>(g_loss), &g, stream_of(x.t)),
                  "tp_topk_distillation_backward");
        }
        return {once(grad), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

Tensor topk_distillation(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest) {
    const Rows x = rows_of(logits, "logits");
    const bool grad = at::GradMode::is_enabled();
    TORCH_CHECK_VALUE(!(grad && values.requires_grad()),
                      "topk_distillation: the teacher's list is a constant; pass teacher_values.detach()");
    const Teacher y = teacher_of(ids, values, logits);
    if (grad && logits.requires_grad()) return DistillationFn::apply(logits, y.ids, y.values, temperature, rest);
    return distillation_forward(x, y, temperature, rest, false).first;
}

std::tuple<Tensor, Tensor> topk_distillation_grad(const Tensor& logits, const Tensor& ids, const Tensor& values,
                                                  const OptTensor& weights, double temperature, bool rest,
                                                  const OptTensor& out) {
    const at::NoGradGuard no_grad;
    const Rows x = rows_of(logits, "logits");
    const Teacher y = teacher_of(ids, values, logits);
    const Tensor w = side(weights, at::kFloat, "weights", lead_of(logits), logits);
    const auto f32 = x.t.options().dtype(at::kFloat);
    Tensor grad;
    tp_rows g;
    if (out) {
        grad = *out;
        TORCH_CHECK_VALUE(grad.sizes() == logits.sizes() && grad.scalar_type() == logits.scalar_type() &&
                              grad.device() == logits.device(),
                          "out must have the logits' shape, dtype and device");
        g = rows_of(grad, "out", /*copy=*/false).r;
    } else {
        grad = at::empty(x.t.sizes(), x.t.options());
        g = dense(x.r, grad);
    }
    Tensor loss = at::empty(lead_of(x.t), f32), stats = at::empty({x.r.N, kStats}, f32);
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_topk_distillation_grad(&x.r, y.K, ptr<const int64_t>(y.ids), ptr<const float>(y.values), ptr<const float>(w),
                                        temperature, rest, ptr<float>(loss), ptr<float>(stats), &g, stream_of(x.t)),
              "tp_topk_distillation_grad");
    }
    if (out) torch::autograd::impl::bump_version(grad);  // a graph that saved it must not use it any more
    return {loss, grad};
}

}  // namespace

PYBIND11_MODULE(_tp_logits, m) {
    m.def("token_logprobs", &token_logprobs);
    m.def("topk_distillation", &topk_distillation);
    m.def("topk_distillation_grad", &topk_distillation_grad);
    m.def("row_strides", &row_strides);
}
