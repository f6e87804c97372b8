// PyTorch binding of include/tp_logits.h: argument checks, outputs from PyTorch's allocator, the current stream, the
// autograd functions and the libtp call, as operators of PyTorch's dispatcher. Nothing here computes on the data.
//
// In C++, unlike the ctypes binding of tp.h: these calls sit in decoding loops and training steps where a kernel
// takes 10 us. A call through ctypes and torch's Python API cost 20 us of the caller's time on a Grace core and
// a Python autograd function 110 us more than a native one, most of it for moving the interpreter's data to autograd's
// thread and back.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>
#include <torch/library.h>

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

void check_device(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda() || t.is_meta(), "libtp runs on CUDA tensors only (no CPU fallback)"); }

tp_rows_dtype check_rows_type(const Tensor& t, const char* name) {
    const auto type = t.scalar_type();
    TORCH_CHECK_TYPE(type == at::kFloat || type == at::kHalf || type == at::kBFloat16, name,
                     " must be a float32, float16 or bfloat16 tensor, got ", type);
    TORCH_CHECK_VALUE(t.dim() >= 1 && t.size(-1) >= 1, name, " must have shape [..., M] with M >= 1, got ", t.sizes());
    return type == at::kFloat ? TP_ROWS_F32 : type == at::kHalf ? TP_ROWS_F16 : TP_ROWS_BF16;
}

Rows rows_of(const Tensor& t, const char* name, bool copy = true) {
    tp_rows r{};
    r.dtype = check_rows_type(t, name);
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

// the logits as a backward keeps them: a copy where rows_of would make one, once for both directions
Tensor readable(const Tensor& t) { return row_strides(t) ? t : t.contiguous(); }

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

OptTensor maybe(const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; }

// --- operators ---------------------------------------------------------------------------------------------------
//
// Calls go through PyTorch's dispatcher as operators with a schema, so that whatever records calls (jit.trace, make_fx)
// records them, runs them again on replay and finds their gradients there, and fake tensors get shapes. Outside the
// dispatcher a trace would hold nothing of a call but the allocation of its outputs.
//
//   CUDA      allocates the outputs and calls libtp
//   Meta      the outputs' shapes and types
//   Autograd  the autograd function where a gradient may be asked for; else straight on

template <class F>
auto op_of(const char* name) {
    const std::string full = std::string("lazy_score_matrix_gb300::") + name;
    return c10::Dispatcher::singleton().findSchemaOrThrow(full.c_str(), "").template typed<F>();
}

// No forward-mode derivatives, as the lazy consumers have none: a tangent is refused, not dropped.
bool tangent(const Tensor& t) { return t.defined() && t._fw_grad(/*level=*/0).defined(); }
bool tangent(const OptTensor& t) { return t && tangent(*t); }
template <class... T>
void refuse_tangents(const char* where, const T&... tensors) {
    TORCH_CHECK_NOT_IMPLEMENTED(!(tangent(tensors) || ...), where, ": no forward-mode derivative; libtp has reverse mode only");
}

using below_autograd = at::AutoDispatchBelowADInplaceOrView;

// Whether a call on these tensors is the CUDA function's alone: no subclass, mode, trace or transform, no tangent, no
// profiler that wants to see operators. (Undefined tensors do not count.) It then runs that function directly: the
// dispatcher's two passes add 0.3 us to the 2.1 that a call takes on a Grace core without its launch, and with the launch
// behind them 1 to 2, a third of a short row's kernel; to a call and its gradient by autograd, 8 us.
template <class... T>
bool plain(const T&... tensors) {
    constexpr auto ordinary =
        c10::DispatchKeySet({c10::DispatchKey::Dense, c10::DispatchKey::BackendSelect, c10::DispatchKey::ADInplaceOrView}) |
        c10::autograd_dispatch_keyset | c10::autocast_dispatch_keyset;
    auto keys = c10::impl::tls_local_dispatch_key_set().included_;
    const auto add = [&](const Tensor& t) {
        if (!t.defined()) return true;
        keys = keys | t.key_set();
        return t.is_cuda() && !tangent(t);
    };
    const bool cuda = (add(tensors) && ...);
    return cuda && !(keys.raw_repr() & ~ordinary.raw_repr() & ~c10::full_backend_mask) &&
           !at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION);
}
bool wants_grad(const Tensor& t) { return at::GradMode::is_enabled() && t.requires_grad(); }

// --- token_logprobs ---------------------------------------------------------------------------------------------

struct Logprobs {
    Tensor entropy, logprobs, top_logprobs, top_ids, stats;
    // as the operator returns them: those that there are
    std::vector<Tensor> list() const {
        std::vector<Tensor> o;
        o.reserve(5);
        for (const Tensor* t : {&entropy, &logprobs, &top_logprobs, &top_ids, &stats})
            if (t->defined()) o.push_back(*t);
        return o;
    }
};

Logprobs logprobs_outputs(const Tensor& logits, bool tokens, int64_t top, bool stats) {
    check_rows_type(logits, "logits");
    TORCH_CHECK_VALUE(top >= 0 && top <= kMaxList && top <= logits.size(-1), "top must be in [0, min(M, 128)], got ", top);
    const auto f32 = logits.options().dtype(at::kFloat);
    const auto lead = lead_of(logits);
    Logprobs o;
    if (tokens) o.logprobs = at::empty(lead, f32);
    o.entropy = at::empty(lead, f32);
    if (top) {
        const auto shape = with(lead, top);
        o.top_logprobs = at::empty(shape, f32);
        o.top_ids = at::empty(shape, f32.dtype(at::kLong));
    }
    if (stats) o.stats = at::empty({logits.numel() / logits.size(-1), kStats}, f32);
    return o;
}

Logprobs logprobs_forward(const Tensor& logits, const OptTensor& tokens_, double temperature, int64_t top, bool stats) {
    const Rows x = rows_of(logits, "logits");
    const Tensor tokens = side(tokens_, at::kLong, "tokens", lead_of(logits), logits);
    const Logprobs o = logprobs_outputs(logits, tokens.defined(), top, stats);
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_token_logprobs(&x.r, ptr<const int64_t>(tokens), temperature, (int)top, ptr<float>(o.logprobs), ptr<float>(o.entropy),
                                ptr<float>(o.stats), ptr<float>(o.top_logprobs), ptr<int64_t>(o.top_ids), stream_of(x.t)),
              "tp_token_logprobs");
    }
    return o;
}

std::vector<Tensor> logprobs_cuda(const Tensor& logits, const OptTensor& tokens, double temperature, int64_t top, bool stats) {
    return logprobs_forward(logits, tokens, temperature, top, stats).list();
}
std::vector<Tensor> logprobs_meta(const Tensor& logits, const OptTensor& tokens, double, int64_t top, bool stats) {
    return logprobs_outputs(logits, side(tokens, at::kLong, "tokens", lead_of(logits), logits).defined(), top, stats).list();
}
std::vector<Tensor> logprobs_op(const Tensor& logits, const OptTensor& tokens, double temperature, int64_t top, bool stats) {
    static const auto op = op_of<decltype(logprobs_op)>("token_logprobs");
    return op.call(logits, tokens, temperature, top, stats);
}

Tensor logprobs_backward_meta(const Tensor& logits, const OptTensor&, double, const Tensor&, const OptTensor&, const OptTensor&) {
    return at::empty(logits.sizes(), logits.options());
}

Tensor logprobs_backward_cuda(const Tensor& logits, const OptTensor& tokens_, double temperature, const Tensor& stats_,
                              const OptTensor& g_logprobs, const OptTensor& g_entropy) {
    const Rows x = rows_of(logits, "logits");
    const auto lead = lead_of(logits);
    const Tensor tokens = side(tokens_, at::kLong, "tokens", lead, logits), stats = side(stats_, at::kFloat, "stats", {x.r.N, kStats}, logits);
    const Tensor g_lp = side(g_logprobs, at::kFloat, "grad_logprobs", lead, logits), g_h = side(g_entropy, at::kFloat, "grad_entropy", lead, logits);
    Tensor grad = at::empty(logits.sizes(), logits.options());
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        const tp_rows g = dense(x.r, grad);
        check(tp_token_logprobs_backward(&x.r, ptr<const int64_t>(tokens), temperature, ptr<const float>(stats), ptr<const float>(g_lp),
                                         ptr<const float>(g_h), &g, stream_of(x.t)),
              "tp_token_logprobs_backward");
    }
    return grad;
}

Tensor logprobs_backward_op(const Tensor& logits, const OptTensor& tokens, double temperature, const Tensor& stats,
                            const OptTensor& g_logprobs, const OptTensor& g_entropy) {
    static const auto op = op_of<decltype(logprobs_backward_op)>("token_logprobs_backward");
    return op.call(logits, tokens, temperature, stats, g_logprobs, g_entropy);
}

struct LogprobsFn : torch::autograd::Function<LogprobsFn> {
    // tokens as an optional: autograd takes a Tensor argument for one that is defined
    static variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& logits, const OptTensor& tokens,
                                 double temperature, int64_t top) {
        const below_autograd guard;
        const Tensor x = readable(logits), t = tokens ? *tokens : Tensor();
        auto out = plain(x, t) ? logprobs_cuda(x, tokens, temperature, top, true) : logprobs_op(x, tokens, temperature, top, true);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({x, t, out.back()});
        out.pop_back();
        ctx->saved_data["T"] = temperature;
        if (top) ctx->mark_non_differentiable({out.end() - 2, out.end()});
        return out;
    }
    static variable_list backward(torch::autograd::AutogradContext* ctx, const variable_list& grads) {
        const auto saved = ctx->get_saved_variables();
        const Tensor &tokens = saved[1], &g_h = grads[0], g_lp = tokens.defined() ? grads[1] : Tensor();
        refuse_tangents("token_logprobs", g_h, g_lp);
        if (!g_h.defined() && !g_lp.defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
        const auto grad = [&] {
            const below_autograd guard;
            const auto call = plain(saved[0], tokens, saved[2], g_lp, g_h) ? logprobs_backward_cuda : logprobs_backward_op;
            return call(saved[0], maybe(tokens), ctx->saved_data["T"].toDouble(), saved[2], maybe(g_lp), maybe(g_h));
        };
        return {once(grad()), Tensor(), Tensor(), Tensor()};
    }
};

std::vector<Tensor> logprobs_autograd(const Tensor& logits, const OptTensor& tokens_, double temperature, int64_t top, bool stats) {
    refuse_tangents("token_logprobs", logits);
    if (wants_grad(logits)) {
        check_rows_type(logits, "logits");
        TORCH_CHECK(!stats, "token_logprobs: the statistics are for the backward, which autograd calls here");
        return LogprobsFn::apply(logits, maybe(side(tokens_, at::kLong, "tokens", lead_of(logits), logits)), temperature, top);
    }
    const below_autograd guard;
    return logprobs_op(logits, tokens_, temperature, top, stats);
}

using Four = std::tuple<OptTensor, Tensor, OptTensor, OptTensor>;

Four token_logprobs(const Tensor& logits, const OptTensor& tokens, double temperature, int64_t top) {
    check_device(logits);
    const bool direct = tokens ? plain(logits, *tokens) : plain(logits);
    if (direct && !wants_grad(logits)) {
        const Logprobs o = logprobs_forward(logits, tokens, temperature, top, false);
        return {maybe(o.logprobs), o.entropy, maybe(o.top_logprobs), maybe(o.top_ids)};
    }
    const auto out = (direct ? logprobs_autograd : logprobs_op)(logits, tokens, temperature, top, false);
    const size_t at = tokens ? 2 : 1;
    return {tokens ? OptTensor(out[1]) : std::nullopt, out[0], top ? OptTensor(out[at]) : std::nullopt,
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

struct Distillation {
    Tensor loss, stats;
    std::vector<Tensor> list() const { return stats.defined() ? std::vector<Tensor>{loss, stats} : std::vector<Tensor>{loss}; }
};

Distillation distillation_outputs(const Tensor& logits, bool stats) {
    check_rows_type(logits, "logits");
    const auto f32 = logits.options().dtype(at::kFloat);
    return {at::empty(lead_of(logits), f32), stats ? at::empty({logits.numel() / logits.size(-1), kStats}, f32) : Tensor()};
}

Distillation distillation_forward(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest, bool stats) {
    const Rows x = rows_of(logits, "logits");
    const Teacher y = teacher_of(ids, values, logits);
    const Distillation o = distillation_outputs(logits, stats);
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_topk_distillation(&x.r, y.K, ptr<const int64_t>(y.ids), ptr<const float>(y.values), temperature, rest,
                                   ptr<float>(o.loss), ptr<float>(o.stats), stream_of(x.t)),
              "tp_topk_distillation");
    }
    return o;
}

std::vector<Tensor> distillation_cuda(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest,
                                      bool stats) {
    return distillation_forward(logits, ids, values, temperature, rest, stats).list();
}
std::vector<Tensor> distillation_meta(const Tensor& logits, const Tensor& ids, const Tensor& values, double, bool, bool stats) {
    const Distillation o = distillation_outputs(logits, stats);
    teacher_of(ids, values, logits);
    return o.list();
}
std::vector<Tensor> distillation_op(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest,
                                    bool stats) {
    static const auto op = op_of<decltype(distillation_op)>("topk_distillation");
    return op.call(logits, ids, values, temperature, rest, stats);
}

Tensor distillation_backward_meta(const Tensor& logits, const Tensor&, const Tensor&, double, bool, const Tensor&, const Tensor&) {
    return at::empty(logits.sizes(), logits.options());
}

Tensor distillation_backward_cuda(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest,
                                  const Tensor& stats_, const Tensor& g_loss) {
    const Rows x = rows_of(logits, "logits");
    const Teacher y = teacher_of(ids, values, logits);
    const Tensor stats = side(stats_, at::kFloat, "stats", {x.r.N, kStats}, logits), g = side(g_loss, at::kFloat, "grad_loss", lead_of(logits), logits);
    Tensor grad = at::empty(logits.sizes(), logits.options());
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        const tp_rows rows = dense(x.r, grad);
        check(tp_topk_distillation_backward(&x.r, y.K, ptr<const int64_t>(y.ids), ptr<const float>(y.values), temperature, rest,
                                            ptr<const float>(stats), ptr<const float>(g), &rows, stream_of(x.t)),
              "tp_topk_distillation_backward");
    }
    return grad;
}

Tensor distillation_backward_op(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest,
                                const Tensor& stats, const Tensor& g_loss) {
    static const auto op = op_of<decltype(distillation_backward_op)>("topk_distillation_backward");
    return op.call(logits, ids, values, temperature, rest, stats, g_loss);
}

struct DistillationFn : torch::autograd::Function<DistillationFn> {
    static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& logits, const Tensor& ids, const Tensor& values,
                          double temperature, bool rest) {
        const below_autograd guard;
        const Tensor x = readable(logits);
        const auto out = (plain(x, ids, values) ? distillation_cuda : distillation_op)(x, ids, values, temperature, rest, true);
        ctx->save_for_backward({x, ids, values, out[1]});
        ctx->saved_data["T"] = temperature;
        ctx->saved_data["rest"] = rest;
        return out[0];
    }
    static variable_list backward(torch::autograd::AutogradContext* ctx, const variable_list& grads) {
        const auto saved = ctx->get_saved_variables();
        refuse_tangents("topk_distillation", grads[0]);
        const auto grad = [&] {
            const below_autograd guard;
            const auto call = plain(saved[0], saved[1], saved[2], saved[3], grads[0]) ? distillation_backward_cuda : distillation_backward_op;
            return call(saved[0], saved[1], saved[2], ctx->saved_data["T"].toDouble(), ctx->saved_data["rest"].toBool(), saved[3], grads[0]);
        };
        return {once(grad()), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

std::vector<Tensor> distillation_autograd(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest,
                                          bool stats) {
    refuse_tangents("topk_distillation", logits, values);
    TORCH_CHECK_VALUE(!wants_grad(values), "topk_distillation: the teacher's list is a constant; pass teacher_values.detach()");
    if (wants_grad(logits)) {
        check_rows_type(logits, "logits");
        const Teacher y = teacher_of(ids, values, logits);
        TORCH_CHECK(!stats, "topk_distillation: the statistics are for the backward, which autograd calls here");
        return {DistillationFn::apply(logits, y.ids, y.values, temperature, rest)};
    }
    const below_autograd guard;
    return distillation_op(logits, ids, values, temperature, rest, stats);
}

Tensor topk_distillation(const Tensor& logits, const Tensor& ids, const Tensor& values, double temperature, bool rest) {
    check_device(logits);
    const bool direct = plain(logits, ids, values);
    if (direct && !wants_grad(logits) && !wants_grad(values)) return distillation_forward(logits, ids, values, temperature, rest, false).loss;
    return (direct ? distillation_autograd : distillation_op)(logits, ids, values, temperature, rest, false)[0];
}

// The loss, and its gradient into `grad` (rows g).
Tensor distillation_grad_into(const Rows& x, const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                              double temperature, bool rest, const tp_rows& g) {
    const Teacher y = teacher_of(ids, values, logits);
    const Tensor w = side(weights, at::kFloat, "weights", lead_of(logits), logits);
    const Distillation o = distillation_outputs(logits, true);
    if (x.r.N) {
        const c10::cuda::CUDAGuard guard(x.t.device());
        check(tp_topk_distillation_grad(&x.r, y.K, ptr<const int64_t>(y.ids), ptr<const float>(y.values), ptr<const float>(w),
                                        temperature, rest, ptr<float>(o.loss), ptr<float>(o.stats), &g, stream_of(x.t)),
              "tp_topk_distillation_grad");
    }
    return o.loss;
}

std::tuple<Tensor, Tensor> distillation_grad_meta(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                                  double, bool) {
    const Tensor loss = distillation_outputs(logits, false).loss;
    teacher_of(ids, values, logits);
    side(weights, at::kFloat, "weights", lead_of(logits), logits);
    return {loss, at::empty(logits.sizes(), logits.options())};
}
std::tuple<Tensor, Tensor> distillation_grad_cuda(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                                  double temperature, bool rest) {
    const Rows x = rows_of(logits, "logits");
    const Tensor grad = at::empty(logits.sizes(), logits.options());
    return {distillation_grad_into(x, logits, ids, values, weights, temperature, rest, dense(x.r, grad)), grad};
}
std::tuple<Tensor, Tensor> distillation_grad_op(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                                double temperature, bool rest) {
    static const auto op = op_of<decltype(distillation_grad_op)>("topk_distillation_grad");
    return op.call(logits, ids, values, weights, temperature, rest);
}
std::tuple<Tensor, Tensor> distillation_grad_autograd(const Tensor& logits, const Tensor& ids, const Tensor& values,
                                                      const OptTensor& weights, double temperature, bool rest) {
    refuse_tangents("topk_distillation_grad", logits, values, weights);
    const below_autograd guard;
    return distillation_grad_op(logits, ids, values, weights, temperature, rest);
}

void check_out(const Tensor& logits, const Tensor& out) {
    TORCH_CHECK_VALUE(out.sizes() == logits.sizes() && out.scalar_type() == logits.scalar_type() && out.device() == logits.device(),
                      "out must have the logits' shape, dtype and device");
    // bump_version would say so too, but behind the write
    TORCH_CHECK(!out.is_inference() || c10::InferenceMode::is_enabled(),
                "out was made under inference mode and cannot be written outside of it");
}
Tensor distillation_grad_out_meta(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights, double,
                                  bool, Tensor& out) {
    check_out(logits, out);
    return std::get<0>(distillation_grad_meta(logits, ids, values, weights, 1.0, false));
}
Tensor distillation_grad_out_cuda(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                  double temperature, bool rest, Tensor& out) {
    const Rows x = rows_of(logits, "logits");
    check_out(logits, out);
    const Tensor loss = distillation_grad_into(x, logits, ids, values, weights, temperature, rest, rows_of(out, "out", /*copy=*/false).r);
    torch::autograd::impl::bump_version(out);  // a graph that saved it must not use it any more
    return loss;
}
Tensor distillation_grad_out_op(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                double temperature, bool rest, Tensor& out) {
    static const auto op = op_of<decltype(distillation_grad_out_op)>("topk_distillation_grad_out");
    return op.call(logits, ids, values, weights, temperature, rest, out);
}
Tensor distillation_grad_out_autograd(const Tensor& logits, const Tensor& ids, const Tensor& values, const OptTensor& weights,
                                      double temperature, bool rest, Tensor& out) {
    refuse_tangents("topk_distillation_grad", logits, values, weights, out);
    const below_autograd guard;
    return distillation_grad_out_op(logits, ids, values, weights, temperature, rest, out);
}

std::tuple<Tensor, Tensor> topk_distillation_grad(const Tensor& logits, const Tensor& ids, const Tensor& values,
                                                  const OptTensor& weights, double temperature, bool rest,
                                                  const OptTensor& out) {
    check_device(logits);
    const at::NoGradGuard no_grad;
    const bool direct = weights ? plain(logits, ids, values, *weights) : plain(logits, ids, values);
    if (!out) {
        if (direct) return distillation_grad_cuda(logits, ids, values, weights, temperature, rest);
        return distillation_grad_op(logits, ids, values, weights, temperature, rest);
    }
    Tensor grad = *out;
    const Tensor loss = direct && plain(grad) ? distillation_grad_out_cuda(logits, ids, values, weights, temperature, rest, grad)
                                              : distillation_grad_out_op(logits, ids, values, weights, temperature, rest, grad);
    return {loss, grad};
}

}  // namespace

TORCH_LIBRARY(lazy_score_matrix_gb300, m) {
    m.def("token_logprobs(Tensor logits, Tensor? tokens, float temperature, int top, bool stats) -> Tensor[]");
    m.def("token_logprobs_backward(Tensor logits, Tensor? tokens, float temperature, Tensor stats, Tensor? grad_logprobs, "
          "Tensor? grad_entropy) -> Tensor");
    m.def("topk_distillation(Tensor logits, Tensor ids, Tensor values, float temperature, bool rest, bool stats) -> Tensor[]");
    m.def("topk_distillation_backward(Tensor logits, Tensor ids, Tensor values, float temperature, bool rest, Tensor stats, "
          "Tensor grad_loss) -> Tensor");
    m.def("topk_distillation_grad(Tensor logits, Tensor ids, Tensor values, Tensor? weights, float temperature, bool rest) -> "
          "(Tensor, Tensor)");
    m.def("topk_distillation_grad_out(Tensor logits, Tensor ids, Tensor values, Tensor? weights, float temperature, bool rest, "
          "Tensor(a!) out) -> Tensor");
}
TORCH_LIBRARY_IMPL(lazy_score_matrix_gb300, CUDA, m) {
    m.impl("token_logprobs", &logprobs_cuda);
    m.impl("token_logprobs_backward", &logprobs_backward_cuda);
    m.impl("topk_distillation", &distillation_cuda);
    m.impl("topk_distillation_backward", &distillation_backward_cuda);
    m.impl("topk_distillation_grad", &distillation_grad_cuda);
    m.impl("topk_distillation_grad_out", &distillation_grad_out_cuda);
}
TORCH_LIBRARY_IMPL(lazy_score_matrix_gb300, Meta, m) {
    m.impl("token_logprobs", &logprobs_meta);
    m.impl("token_logprobs_backward", &logprobs_backward_meta);
    m.impl("topk_distillation", &distillation_meta);
    m.impl("topk_distillation_backward", &distillation_backward_meta);
    m.impl("topk_distillation_grad", &distillation_grad_meta);
    m.impl("topk_distillation_grad_out", &distillation_grad_out_meta);
}
TORCH_LIBRARY_IMPL(lazy_score_matrix_gb300, Autograd, m) {
    m.impl("token_logprobs", &logprobs_autograd);
    m.impl("topk_distillation", &distillation_autograd);
    m.impl("topk_distillation_grad", &distillation_grad_autograd);
    m.impl("topk_distillation_grad_out", &distillation_grad_out_autograd);
}

PYBIND11_MODULE(_tp_logits, m) {
    m.def("token_logprobs", &token_logprobs);
    m.def("topk_distillation", &topk_distillation);
    m.def("topk_distillation_grad", &topk_distillation_grad);
    m.def("row_strides", &row_strides);
}
