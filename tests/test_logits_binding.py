"""What PyTorch's machinery around a call does with the stored-row consumers: tracing, forward-mode derivatives, function
transforms, saved tensors that come back otherwise, inference mode."""
import pytest
import torch
import torch.utils.checkpoint
from torch.autograd import forward_ad
from torch.fx.experimental.proxy_tensor import make_fx

import lazy_score_matrix_gb300 as tp
from tests.test_logits import check_logprobs, scores

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(seed, n=6, m=901, k=7, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(n, m, device=DEV, generator=g) * 3).to(dtype)
    tokens = torch.randint(0, m, (n,), device=DEV, generator=g)
    y = torch.log_softmax(x.float() + torch.randn(n, m, device=DEV, generator=g), 1)
    values, ids = y.topk(k, 1)
    return x, tokens, ids, values, torch.rand(n, device=DEV, generator=g) + 0.5


def no_grad_calls(x, tokens, ids, values, w):
    r = tp.token_logprobs(x, tokens, temperature=0.8, top=5)
    only = tp.token_logprobs(x)
    loss, grad = tp.topk_distillation_grad(x, ids, values, w, rest=True)
    return (r.logprobs, r.entropy, r.top_logprobs, r.top_ids, only.entropy, tp.topk_distillation(x, ids, values), loss, grad)


def in_place(x, tokens, ids, values, w):
    y = x * 1.0
    loss, grad = tp.topk_distillation_grad(y, ids, values, w, out=y)
    return loss, grad, y


def differentiable(x, tokens, ids, values, w):
    r = tp.token_logprobs(x, tokens)
    return (r.logprobs * w).sum() + 0.1 * r.entropy.sum() + (tp.topk_distillation(x, ids, values, rest=True) * w).sum()


def traced_by_jit(f, args):
    return torch.jit.trace(f, args, check_trace=False)


def traced_by_fx(f, args):
    return make_fx(f)(*args)


TRACERS = {"jit": traced_by_jit, "fx": traced_by_fx}


@pytest.mark.parametrize("tracer", TRACERS)
@pytest.mark.parametrize("calls", [no_grad_calls, in_place])
def test_traced_calls_run_again(tracer, calls):
    traced = TRACERS[tracer](calls, inputs(1))
    for seed in (1, 2, 3):
        want = calls(*inputs(seed))
        keep = [torch.randn(6, 901, device=DEV) for _ in range(4)]  # other values in the freed blocks
        got = traced(*inputs(seed))
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del keep


def test_gradients_of_a_traced_call():
    x, *rest = inputs(1)
    traced = traced_by_jit(differentiable, (x.requires_grad_(True), *rest))
    for seed in (1, 2):
        y, *rest = inputs(seed)
        leaves = [y.clone().requires_grad_(True) for _ in range(2)]
        got, want = traced(leaves[0], *rest), differentiable(leaves[1], *rest)
        assert torch.equal(got, want)
        got.backward()
        want.backward()
        assert torch.equal(leaves[0].grad, leaves[1].grad)


def test_a_traced_gradient():
    # the whole step, its backward included, as a graph of operators
    def step(x, *rest):
        y = x.detach().requires_grad_(True)
        return torch.autograd.grad(differentiable(y, *rest), y)[0]

    traced = make_fx(step)(*inputs(1))
    for seed in (1, 2):
        assert torch.equal(traced(*inputs(seed)), step(*inputs(seed)))


def test_traced_under_inference_mode_and_reduced_types():
    with torch.inference_mode():
        traced = traced_by_jit(no_grad_calls, inputs(1, dtype=torch.bfloat16))
        args = inputs(2, dtype=torch.bfloat16)
        assert all(torch.equal(a, b) for a, b in zip(traced(*args), no_grad_calls(*args)))


def test_shapes_without_data():
    # fake tensors: shapes and types of every result, nothing launched
    from torch._subclasses.fake_tensor import FakeTensorMode
    args = inputs(1, dtype=torch.float16)
    want = no_grad_calls(*args)
    with FakeTensorMode() as mode:
        got = no_grad_calls(*(mode.from_tensor(t) for t in args))
    assert [(t.shape, t.dtype, t.device.type) for t in got] == [(t.shape, t.dtype, "cuda") for t in want]


def test_forward_mode_is_refused():
    x, tokens, ids, values, w = inputs(1)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        dual_values, dual_w = forward_ad.make_dual(values, torch.ones_like(values)), forward_ad.make_dual(w, torch.ones_like(w))
        calls = [lambda: tp.token_logprobs(dual, tokens), lambda: tp.token_logprobs(dual, top=3), lambda: tp.topk_distillation(dual, ids, values),
                 lambda: tp.topk_distillation(x, ids, dual_values), lambda: tp.topk_distillation_grad(dual, ids, values, w),
                 lambda: tp.topk_distillation_grad(x, ids, dual_values, w), lambda: tp.topk_distillation_grad(x, ids, values, dual_w),
                 lambda: tp.topk_distillation_grad(x, ids, values, w, out=dual)]
        for i, call in enumerate(calls):
            with pytest.raises(NotImplementedError):
                call()
                pytest.fail(f"call {i} was accepted")
            with pytest.raises(NotImplementedError), torch.no_grad():
                call()
                pytest.fail(f"call {i} was accepted under no_grad")
        # a tangent of an upstream gradient, on the way back
        leaf = x.detach().requires_grad_(True)
        for out in (tp.token_logprobs(leaf, tokens).logprobs, tp.token_logprobs(leaf).entropy, tp.topk_distillation(leaf, ids, values)):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(out, leaf, dual_w)
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda t: tp.token_logprobs(t, tokens).logprobs, (x,), (torch.ones_like(x),))
    assert torch.isfinite(tp.token_logprobs(x, tokens).logprobs).all()


def test_function_transforms_are_right_or_refused():
    x, tokens, ids, values, w = inputs(1)
    calls = [(lambda: torch.vmap(lambda a, t: tp.token_logprobs(a, t).logprobs)(x, tokens), lambda: tp.token_logprobs(x, tokens).logprobs),
             (lambda: torch.vmap(lambda a, i, v: tp.topk_distillation(a, i, v))(x, ids, values), lambda: tp.topk_distillation(x, ids, values)),
             (lambda: torch.func.grad(lambda a: tp.token_logprobs(a, tokens).entropy.sum())(x),
              lambda: torch.autograd.grad(tp.token_logprobs(y, tokens).entropy.sum(), y)[0])]
    y = x.detach().requires_grad_(True)
    for transform, plain in calls:
        try:
            got = transform()
        except (NotImplementedError, RuntimeError):
            continue
        assert (got - plain()).abs().max() < 1e-5


def test_saved_tensors_in_another_layout():
    # hooks that bring a saved tensor back with other strides
    x, tokens, ids, values, w = inputs(1, n=12)
    x, tokens, ids, values, w = x.view(3, 4, -1), tokens.view(3, 4), ids.view(3, 4, -1), values.view(3, 4, -1), w.view(3, 4)

    def grad():
        leaf = x.detach().requires_grad_(True)
        return torch.autograd.grad(differentiable(leaf, tokens, ids, values, w), leaf)[0]

    want = grad()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.transpose(0, -1).contiguous().transpose(0, -1)):
        got = grad()
    assert torch.equal(got, want)


def test_negated_views():
    # a view that PyTorch negates when it is read
    x, tokens, ids, values, w = inputs(1, n=1)
    neg = torch.complex(torch.zeros_like(w), -w).conj().imag
    assert neg.is_neg() and torch.equal(neg, w)
    assert torch.equal(tp.topk_distillation_grad(x, ids, values, neg)[1], tp.topk_distillation_grad(x, ids, values, w)[1])


def test_output_made_under_inference_mode():
    x, tokens, ids, values, w = inputs(1)
    want = tp.topk_distillation_grad(x, ids, values, w)[1]
    with torch.inference_mode():
        out = torch.full_like(x, 7.0)
        assert torch.equal(tp.topk_distillation_grad(x, ids, values, w, out=out)[1], want)
        out.fill_(7.0)
    with pytest.raises(RuntimeError):  # as any write to it outside
        tp.topk_distillation_grad(x, ids, values, w, out=out)
    assert (out == 7.0).all()  # and nothing was written


@pytest.mark.parametrize("n,m", [(3, 2), (5, 261), (4, 20011), (1300, 700)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("top", [0, 2])
def test_entropy_and_its_gradient_without_tokens(n, m, dtype, top):
    x = scores(min(n, 6), m, dtype, m).repeat((n + 5) // 6, 1)[:n]
    check_logprobs(x[:6], None, 0.9, top)
    leaves = [x.to(DEV).requires_grad_(True) for _ in range(2)]
    # the same alternatives on both sides: with and without them a row's sums are split over other threads
    r = tp.token_logprobs(leaves[0], temperature=0.9, top=top)
    w = tp.token_logprobs(leaves[1], torch.zeros(n, dtype=torch.int64, device=DEV), temperature=0.9, top=top)
    assert r.logprobs is None and torch.equal(r.entropy, w.entropy)
    grads = [torch.autograd.grad(o.entropy.sum(), leaf)[0] for o, leaf in zip((r, w), leaves)]
    assert torch.equal(*grads)


def whole_step(x, *rest):
    leaf = x.detach().requires_grad_(True)
    loss = differentiable(leaf, *rest) - 0.2 * tp.token_logprobs(leaf).entropy.mean()
    loss.backward()
    return [loss.detach(), leaf.grad, *no_grad_calls(x, *rest)]


def under_profiler(args):
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
        got = whole_step(*args)
    assert {"lazy_score_matrix_gb300::token_logprobs", "lazy_score_matrix_gb300::topk_distillation_grad"} <= {e.name for e in p.events()}
    return got


def under_checkpoint(args):
    x, *rest = args
    leaf = x.detach().requires_grad_(True)
    loss = torch.utils.checkpoint.checkpoint(lambda t: differentiable(t, *rest) - 0.2 * tp.token_logprobs(t).entropy.mean(), leaf, use_reentrant=False)
    loss.backward()
    return [loss.detach(), leaf.grad, *no_grad_calls(*args)]


def under(manager):
    def run(args):
        with manager():
            return whole_step(*args)
    return run


def on_another_thread(args):
    import threading
    got = []
    t = threading.Thread(target=lambda: got.extend(whole_step(*args)))
    t.start()
    t.join()
    return got


TOOLS = {"profiler": under_profiler, "checkpoint": under_checkpoint, "anomaly mode": under(lambda: torch.autograd.set_detect_anomaly(True)),
         "autocast": under(lambda: torch.autocast("cuda", dtype=torch.bfloat16)), "saved on the CPU": under(torch.autograd.graph.save_on_cpu),
         "another thread": on_another_thread}


@pytest.mark.parametrize("tool", TOOLS)
def test_the_same_results_under_pytorch_tools(tool):
    args = inputs(4, dtype=torch.bfloat16)
    want, got = whole_step(*args), TOOLS[tool](args)
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_gradient_traced_without_data():
    def step(x, *rest):
        y = x.detach().requires_grad_(True)
        return torch.autograd.grad(differentiable(y, *rest), y)[0]

    traced = make_fx(step, tracing_mode="fake")(*inputs(1))
    assert torch.equal(traced(*inputs(2)), step(*inputs(2)))
