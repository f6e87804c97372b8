// The C entries of the stored-row consumers (declared in include/tp_logits.h): argument validation and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "tp_launch.h"
#include "tp_logits.h"
#include "tp_logits_args.h"

namespace tp {
void set_last_error(const std::string& msg);  // tp_api.cu
tp_status launched(int n);                    // tp_api.cu: counts launches, checks the launch error
tp_status injected_fault(const char* entry);  // tp_status.cu: TP_FAULT_INJECT
}  // namespace tp

using namespace tp;
using namespace tp::rows;

namespace {

#define TP_CHECK(expr)                          \
    do {                                        \
        const tp_status tp_check_s = (expr);    \
        if (tp_check_s != TP_OK) return tp_check_s; \
    } while (0)

tp_status invalid(const std::string& msg) {
    set_last_error(msg);
    return TP_ERR_INVALID_ARG;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t rows_esize(const tp_rows* r) { return r->dtype == TP_ROWS_F32 ? 4 : 2; }

// bytes from data to the end of the last row
int64_t rows_extent(const tp_rows* r) {
    const int64_t groups = r->N / r->group;
    return ((groups > 1 ? (groups - 1) * r->group_stride : 0) + (r->group - 1) * r->row_stride + r->M) * (int64_t)rows_esize(r);
}

tp_status check_rows(const tp_rows* r, const char* name, bool written) {
    const std::string n(name);
    if (!r) return invalid(n + " is NULL");
    if (r->dtype != TP_ROWS_F32 && r->dtype != TP_ROWS_F16 && r->dtype != TP_ROWS_BF16)
        return invalid(n + ": dtype must be TP_ROWS_F32, TP_ROWS_F16 or TP_ROWS_BF16");
    constexpr int64_t lim = int64_t(1) << 31;
    if (r->N < 1 || r->M < 1 || r->N >= lim || r->M > lim / 2) return invalid(n + ": N must be in [1, 2^31) and M in [1, 2^30]");
    if (r->group < 1 || r->group > r->N || r->N % r->group) return invalid(n + ": N must be a multiple of group >= 1");
    const int64_t groups = r->N / r->group;
    const int64_t gs = groups > 1 ? r->group_stride : 0, rs = r->group > 1 ? r->row_stride : 0;
    constexpr int64_t most = int64_t(1) << 61;  // of any offset, so that no sum of two leaves 64 bits
    if (rs < 0 || gs < 0 || rs > most / r->N || gs > most / r->N) return invalid(n + ": strides must be >= 0 and span less than 2^61 elements");
    if (!r->data) return invalid(n + ": data is NULL");
    if (!aligned(r->data, rows_esize(r))) return invalid(n + ": data not aligned to the element size");
    if (written) {
        const bool rows_inside = (r->group == 1 || rs >= r->M) && (groups == 1 || gs >= (r->group - 1) * rs + r->M);
        const bool groups_inside = (groups == 1 || gs >= r->M) && (r->group == 1 || rs >= (groups - 1) * gs + r->M);
        if (!rows_inside && !groups_inside) return invalid(n + ": rows that are written overlap one another");
    }
    return TP_OK;
}

struct Span {
    const void* p;
    int64_t bytes;
    const char* name;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// Every pointer aligned to its element, no output on an input or another output.
tp_status check_spans(std::initializer_list<Span> in, std::initializer_list<Span> out) {
    for (const Span* o = out.begin(); o != out.end(); ++o) {
        for (const Span& i : in)
            if (overlap(*o, i)) return invalid(std::string(o->name) + " overlaps input " + i.name);
        for (const Span* p = o + 1; p != out.end(); ++p)
            if (overlap(*o, *p)) return invalid(std::string(o->name) + " overlaps output " + p->name);
    }
    return TP_OK;
}

tp_status check_ptr(const void* p, const char* name, size_t es, bool required = true) {
    if (!p) return required ? invalid(std::string(name) + " is NULL") : TP_OK;
    if (!aligned(p, es)) return invalid(std::string(name) + " not aligned to the element size");
    return TP_OK;
}

tp_status check_temperature(double t) {
    if (!(t >= 1e-3 && t <= 1e3)) return invalid("temperature must be in [1e-3, 1e3]");
    return TP_OK;
}

// Whether an offset at + k step, |k| < n, comes closer to 0 than `near` by way of f(at + k step); only the two k about
// -at / step can, where step >= near.
template <class F>
bool near_zero(int64_t at, int64_t step, int64_t n, F f) {
    if (n == 1) return f(at);
    const int64_t k0 = -at / step - (-at % step < 0);
    for (int64_t k = k0; k <= k0 + 1; ++k)
        if (k > -n && k < n && f(at + k * step)) return true;
    return false;
}

// Whether rows at the same strides, which do not overlap among themselves, share an element: a row of one then lies less
// than M from a row of the other. The smaller stride's rows fill less than one step of the larger.
bool share_elements(const tp_rows* x, const tp_rows* g) {
    const int64_t at = (static_cast<const char*>(g->data) - static_cast<const char*>(x->data)) / (int64_t)rows_esize(x);
    const int64_t groups = x->N / x->group;
    const bool swap = x->group > 1 && groups > 1 && x->row_stride > x->group_stride;
    const int64_t outer = swap ? x->row_stride : x->group_stride, inner = swap ? x->group_stride : x->row_stride;
    return near_zero(at, outer, swap ? x->group : groups, [&](int64_t a) {
        return near_zero(a, inner, swap ? groups : x->group, [&](int64_t b) { return b > -x->M && b < x->M; });
    });
}

// grad: rows of the logits' type and shape; either the logits themselves or apart from them
tp_status check_grad(const tp_rows* x, const tp_rows* g) {
    TP_CHECK(check_rows(g, "grad", true));
    if (g->dtype != x->dtype || g->N != x->N || g->M != x->M) return invalid("grad must have the logits' dtype, N and M");
    const bool alike = g->group == x->group && (g->group == 1 || g->row_stride == x->row_stride) &&
                       (g->group == g->N || g->group_stride == x->group_stride);
    if (alike && g->data == x->data) return TP_OK;
    if (overlap({x->data, rows_extent(x), ""}, {g->data, rows_extent(g), ""}) && (!alike || share_elements(x, g)))
        return invalid("grad overlaps the logits without being the same rows");
    return TP_OK;
}

View view(const tp_rows* r) {
    View v;
    v.data = r->data;
    v.row_stride = r->row_stride;
    v.group_stride = r->group < r->N ? r->group_stride : 0;
    v.M = (int)r->M;
    v.group = (int)r->group;
    v.grouped = r->group < r->N;
    return v;
}

Scale scale_of(double t) {
    Scale s;
    const double inv = 1.0 / t;
    s.inv = (float)inv;
    s.inv_lo = (float)(inv - (double)s.inv);
    const double c = 1.4426950408889634074 / t;
    s.c = (float)c;
    s.c_hi = std::nextafterf((float)c, 0.f);  // below c whichever way it rounded
    s.c_lo = (float)(c - (double)s.c_hi);
    s.delta = (float)(inv - (double)s.c * 0.69314718055994530942);
    return s;
}

// one body for every entry: no exception leaves the library
template <class F>
tp_status entry(F&& body) noexcept {
    try {
        return body();
    } catch (...) {
        return TP_ERR_INVALID_ARG;  // out of host memory while a message was formed
    }
}

tp_status logprob_common(const tp_rows* x, const int64_t* tokens, double t) {
    TP_CHECK(check_rows(x, "logits", false));
    TP_CHECK(check_ptr(tokens, "tokens", 8, false));
    return check_temperature(t);
}

tp_status distill_common(const tp_rows* x, int K, const int64_t* ids, const float* values, double t, int rest) {
    TP_CHECK(check_rows(x, "logits", false));
    if (K < 1 || K > kMaxList) return invalid("K must be in [1, 128]");
    TP_CHECK(check_ptr(ids, "ids", 8));
    TP_CHECK(check_ptr(values, "values", 4));
    if (rest != 0 && rest != 1) return invalid("rest must be 0 or 1");
    return check_temperature(t);
}

DistillArgs distill_args(const tp_rows* x, int K, const int64_t* ids, const float* values, double t, int rest) {
    DistillArgs a{};
    a.x = view(x);
    a.N = x->N;
    a.ids = ids;
    a.values = values;
    a.K = K;
    a.rest = rest;
    a.sc = scale_of(t);
    return a;
}

}  // namespace

extern "C" {

tp_status tp_token_logprobs(const tp_rows* x, const int64_t* tokens, double temperature, int top, float* logprobs,
                            float* entropy, float* stats, float* top_logprobs, int64_t* top_ids, void* stream) {
    return entry([&]() -> tp_status {
        TP_CHECK(logprob_common(x, tokens, temperature));
        if (top < 0 || top > kMaxList || top > x->M) return invalid("top must be in [0, min(M, 128)]");
        TP_CHECK(check_ptr(logprobs, "logprobs", 4, tokens != nullptr));
        if (!tokens && logprobs) return invalid("logprobs given without tokens");
        TP_CHECK(check_ptr(entropy, "entropy", 4));
        TP_CHECK(check_ptr(stats, "stats", 4, false));
        TP_CHECK(check_ptr(top_logprobs, "top_logprobs", 4, top > 0));
        TP_CHECK(check_ptr(top_ids, "top_ids", 8, top > 0));
        if (top == 0 && (top_logprobs || top_ids)) return invalid("top_logprobs or top_ids given with top = 0");
        const int64_t N = x->N;
        TP_CHECK(check_spans({{x->data, rows_extent(x), "logits"}, {tokens, N * 8, "tokens"}},
                             {{logprobs, N * 4, "logprobs"},
                              {entropy, N * 4, "entropy"},
                              {stats, N * kStats * 4, "stats"},
                              {top_logprobs, N * top * 4, "top_logprobs"},
                              {top_ids, N * top * 8, "top_ids"}}));
        TP_CHECK(injected_fault("token_logprobs"));
        LogprobArgs a{};
        a.x = view(x);
        a.N = N;
        a.tokens = tokens;
        a.sc = scale_of(temperature);
        a.top = top;
        a.logprobs = logprobs;
        a.entropy = entropy;
        a.stats = stats;
        a.top_logprobs = top_logprobs;
        a.top_ids = top_ids;
        launch_logprobs(x->dtype, a, static_cast<cudaStream_t>(stream));
        return launched(1);
    });
}

tp_status tp_token_logprobs_backward(const tp_rows* x, const int64_t* tokens, double temperature, const float* stats,
                                     const float* grad_logprobs, const float* grad_entropy, const tp_rows* grad,
                                     void* stream) {
    return entry([&]() -> tp_status {
        TP_CHECK(logprob_common(x, tokens, temperature));
        TP_CHECK(check_ptr(stats, "stats", 4));
        TP_CHECK(check_ptr(grad_logprobs, "grad_logprobs", 4, false));
        TP_CHECK(check_ptr(grad_entropy, "grad_entropy", 4, false));
        if (!grad_logprobs && !grad_entropy) return invalid("grad_logprobs and grad_entropy are both NULL");
        if (grad_logprobs && !tokens) return invalid("grad_logprobs given without tokens");
        TP_CHECK(check_grad(x, grad));
        const int64_t N = x->N;
        TP_CHECK(check_spans({{tokens, N * 8, "tokens"},
                              {stats, N * kStats * 4, "stats"},
                              {grad_logprobs, N * 4, "grad_logprobs"},
                              {grad_entropy, N * 4, "grad_entropy"}},
                             {{grad->data, rows_extent(grad), "grad"}}));
        TP_CHECK(injected_fault("token_logprobs_backward"));
        LogprobArgs a{};
        a.x = view(x);
        a.N = N;
        a.tokens = tokens;
        a.sc = scale_of(temperature);
        a.stats = const_cast<float*>(stats);
        a.g_logprob = grad_logprobs;
        a.g_entropy = grad_entropy;
        a.g = view(grad);
        launch_logprobs_backward(x->dtype, a, static_cast<cudaStream_t>(stream));
        return launched(1);
    });
}

tp_status tp_topk_distillation(const tp_rows* x, int K, const int64_t* ids, const float* values, double temperature,
                               int rest, float* loss, float* stats, void* stream) {
    return entry([&]() -> tp_status {
        TP_CHECK(distill_common(x, K, ids, values, temperature, rest));
        TP_CHECK(check_ptr(loss, "loss", 4));
        TP_CHECK(check_ptr(stats, "stats", 4, false));
        const int64_t N = x->N;
        TP_CHECK(check_spans({{x->data, rows_extent(x), "logits"}, {ids, N * K * 8, "ids"}, {values, N * K * 4, "values"}},
                             {{loss, N * 4, "loss"}, {stats, N * kStats * 4, "stats"}}));
        TP_CHECK(injected_fault("topk_distillation"));
        DistillArgs a = distill_args(x, K, ids, values, temperature, rest);
        a.loss = loss;
        a.stats = stats;
        launch_distill(x->dtype, a, static_cast<cudaStream_t>(stream));
        return launched(1);
    });
}

tp_status tp_topk_distillation_backward(const tp_rows* x, int K, const int64_t* ids, const float* values,
                                        double temperature, int rest, const float* stats, const float* grad_loss,
                                        const tp_rows* grad, void* stream) {
    return entry([&]() -> tp_status {
        TP_CHECK(distill_common(x, K, ids, values, temperature, rest));
        TP_CHECK(check_ptr(stats, "stats", 4));
        TP_CHECK(check_ptr(grad_loss, "grad_loss", 4));
        TP_CHECK(check_grad(x, grad));
        const int64_t N = x->N;
        TP_CHECK(check_spans({{ids, N * K * 8, "ids"},
                              {values, N * K * 4, "values"},
                              {stats, N * kStats * 4, "stats"},
                              {grad_loss, N * 4, "grad_loss"}},
                             {{grad->data, rows_extent(grad), "grad"}}));
        TP_CHECK(injected_fault("topk_distillation_backward"));
        DistillArgs a = distill_args(x, K, ids, values, temperature, rest);
        a.stats = const_cast<float*>(stats);
        a.weights = grad_loss;
        a.g = view(grad);
        launch_distill_backward(x->dtype, a, static_cast<cudaStream_t>(stream));
        return launched(1);
    });
}

tp_status tp_topk_distillation_grad(const tp_rows* x, int K, const int64_t* ids, const float* values,
                                    const float* weights, double temperature, int rest, float* loss, float* stats,
                                    const tp_rows* grad, void* stream) {
    return entry([&]() -> tp_status {
        TP_CHECK(distill_common(x, K, ids, values, temperature, rest));
        TP_CHECK(check_ptr(weights, "weights", 4, false));
        TP_CHECK(check_ptr(loss, "loss", 4));
        TP_CHECK(check_ptr(stats, "stats", 4));
        TP_CHECK(check_grad(x, grad));
        const int64_t N = x->N;
        TP_CHECK(check_spans({{ids, N * K * 8, "ids"}, {values, N * K * 4, "values"}, {weights, N * 4, "weights"}},
                             {{loss, N * 4, "loss"}, {stats, N * kStats * 4, "stats"}, {grad->data, rows_extent(grad), "grad"}}));
        TP_CHECK(check_spans({{x->data, rows_extent(x), "logits"}}, {{loss, N * 4, "loss"}, {stats, N * kStats * 4, "stats"}}));
        TP_CHECK(injected_fault("topk_distillation_grad"));
        DistillArgs a = distill_args(x, K, ids, values, temperature, rest);
        a.loss = loss;
        a.stats = stats;
        a.weights = weights;
        a.g = view(grad);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        launch_distill_grad(x->dtype, a, s);
        return launched(1);
    });
}

}  // extern "C"
