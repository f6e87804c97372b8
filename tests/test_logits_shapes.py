"""Stored score rows, for each way in which a kernel's threads share rows (a warp, a CTA, several CTAs or a cluster a row): the
C entries' outputs stay inside their buffers, gradients over the scores and in groups of rows, ties over more columns than
any buffer of candidates holds."""
import pytest
import torch

import lazy_score_matrix_gb300 as tp
from lazy_score_matrix_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = {torch.float32: _lib.TP_ROWS_F32, torch.float16: _lib.TP_ROWS_F16, torch.bfloat16: _lib.TP_ROWS_BF16}
SHAPES = [(9, 1003, torch.bfloat16), (1302, 261, torch.float32), (1302, 4099, torch.bfloat16), (651, 9001, torch.float32), (6, 150001, torch.bfloat16),
          (42, 70001, torch.float16), (162, 100003, torch.float32)]


def stream():
    return torch.cuda.current_stream().cuda_stream


def rows(t, n, m, group=None, gs=0):
    return _lib.tp_rows(CODE[t.dtype], n, m, group or n, m, gs, t.data_ptr())


def problem(n, m, dtype, k=48):
    """Scores, tokens (some left out), lists spread over the whole row with columns named twice, weights."""
    g = torch.Generator(device=DEV).manual_seed(n + m)
    x = (torch.randn(n, m, device=DEV, generator=g) * 3).to(dtype)
    tok = torch.randint(0, m, (n,), device=DEV, generator=g)
    tok[2::7] = -1
    ids = (torch.arange(k, device=DEV) * (m - 1) // (k - 1)).repeat(n, 1)
    ids[:, 5], ids[:, 40] = ids[:, 4], ids[:, 20]
    ids[3::8] = -1
    values = torch.randn(n, k, device=DEV, generator=g) - 6.0
    return x, tok, ids, values, torch.randn(n, device=DEV, generator=g), torch.randn(n, device=DEV, generator=g)


class Calls:
    """The five C entries on one problem."""

    def __init__(self, n, m, dtype, top=0):
        self.n, self.m, self.lib = n, m, _lib.load()
        self.x, self.tok, self.ids, self.values, self.g1, self.g2 = problem(n, m, dtype)
        self.k, self.top = self.ids.shape[1], top

    def logprobs(self, lp, h, stats, tv=None, ti=None):
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        _lib.check(self.lib.tp_token_logprobs(rows(self.x, self.n, self.m), self.tok.data_ptr(), 0.9, self.top, lp.data_ptr(), h.data_ptr(),
                                              stats.data_ptr(), p(tv), p(ti), stream()), "token_logprobs")

    def logprobs_backward(self, x, stats, grad):
        _lib.check(self.lib.tp_token_logprobs_backward(rows(x, self.n, self.m), self.tok.data_ptr(), 0.9, stats.data_ptr(), self.g1.data_ptr(),
                                                       self.g2.data_ptr(), grad, stream()), "token_logprobs_backward")

    def distill(self, rest, loss, stats):
        _lib.check(self.lib.tp_topk_distillation(rows(self.x, self.n, self.m), self.k, self.ids.data_ptr(), self.values.data_ptr(), 1.2, rest,
                                                 loss.data_ptr(), stats.data_ptr(), stream()), "topk_distillation")

    def distill_backward(self, rest, x, stats, grad):
        _lib.check(self.lib.tp_topk_distillation_backward(rows(x, self.n, self.m), self.k, self.ids.data_ptr(), self.values.data_ptr(), 1.2, rest,
                                                          stats.data_ptr(), self.g1.data_ptr(), grad, stream()), "topk_distillation_backward")

    def distill_grad(self, rest, x, loss, stats, grad):
        _lib.check(self.lib.tp_topk_distillation_grad(rows(x, self.n, self.m), self.k, self.ids.data_ptr(), self.values.data_ptr(),
                                                      self.g1.data_ptr(), 1.2, rest, loss.data_ptr(), stats.data_ptr(), grad, stream()),
                   "topk_distillation_grad")


class Guarded:
    """An array with guard elements on both sides; it starts at an odd element."""

    def __init__(self, count, dtype):
        self.whole = torch.full((count + 200,), -77, dtype=dtype, device=DEV)
        self.inner = self.whole[61:61 + count]

    def data_ptr(self):
        return self.inner.data_ptr()

    def check(self, what):
        assert (self.whole[:61] == -77).all() and (self.whole[61 + self.inner.numel():] == -77).all(), what
        assert not (self.inner == -77).any(), what


@pytest.mark.parametrize("n,m,dtype", SHAPES)
@pytest.mark.parametrize("top", [1, 32, 128])
def test_outputs_stay_inside_their_buffers(n, m, dtype, top):
    c = Calls(n, m, dtype, top)
    f, i = torch.float32, torch.int64
    a = {"logprobs": Guarded(n, f), "entropy": Guarded(n, f), "stats": Guarded(n * 8, f), "top_logprobs": Guarded(n * top, f),
         "top_ids": Guarded(n * top, i), "loss": Guarded(n, f), "distillation stats": Guarded(n * 8, f), "loss at once": Guarded(n, f),
         "stats at once": Guarded(n * 8, f)}
    grads = {name: Guarded(n * m, dtype) for name in ("grad", "distillation grad", "grad at once")}
    grad = lambda name: _lib.tp_rows(CODE[dtype], n, m, n, m, 0, grads[name].data_ptr())  # noqa: E731
    for rest in (0, 1):
        c.logprobs(a["logprobs"], a["entropy"], a["stats"], a["top_logprobs"], a["top_ids"])
        c.logprobs_backward(c.x, a["stats"], grad("grad"))
        c.distill(rest, a["loss"], a["distillation stats"])
        c.distill_backward(rest, c.x, a["distillation stats"], grad("distillation grad"))
        c.distill_grad(rest, c.x, a["loss at once"], a["stats at once"], grad("grad at once"))
        torch.cuda.synchronize()
        for name, buf in {**a, **grads}.items():
            buf.check(name)


@pytest.mark.parametrize("n,m,dtype", SHAPES)
@pytest.mark.parametrize("rest", [0, 1])
def test_gradients_over_the_scores_and_in_groups(n, m, dtype, rest):
    # each backward into its own scores, and into rows with one behind every third left alone: the bits of a plain one
    c = Calls(n, m, dtype)
    new = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    lp, h, loss, st, dst = new(n), new(n), new(n), new(n, 8), new(n, 8)
    c.logprobs(lp, h, st)
    c.distill(rest, loss, dst)
    entries = {"token_logprobs": lambda x, g: c.logprobs_backward(x, st, g), "topk_distillation": lambda x, g: c.distill_backward(rest, x, dst, g),
               "at once": lambda x, g: c.distill_grad(rest, x, new(n), new(n, 8), g)}
    for name, call in entries.items():
        plain = torch.empty_like(c.x)
        call(c.x, rows(plain, n, m))
        over = c.x.clone()
        call(over, rows(over, n, m))
        assert torch.equal(over, plain), name
        apart = torch.full((n // 3, 4, m), 7.0, dtype=dtype, device=DEV)
        call(c.x, rows(apart, n, m, 3, 4 * m))
        assert torch.equal(apart[:, :3].reshape(n, m), plain), name
        assert (apart[:, 3] == 7).all(), name


@pytest.mark.parametrize("n,m,dtype", SHAPES)
def test_output_in_groups_from_python(n, m, dtype):
    c = Calls(n, m, dtype)
    x, ids, values, w = (t.view(3, n // 3, *t.shape[1:]) for t in (c.x, c.ids, c.values, c.g1))
    want = tp.topk_distillation_grad(x, ids, values, w, rest=True)
    out = torch.full((3, n // 3 + 1, m), 7.0, dtype=dtype, device=DEV)
    loss, grad = tp.topk_distillation_grad(x, ids, values, w, rest=True, out=out[:, 1:])
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1]) and (out[:, 0] == 7).all()


TIES = [(1, 300007, 128), (2, 131072, 128), (60, 131072, 128), (650, 9001, 100), (650, 20011, 128), (1300, 4099, 32), (1300, 700, 20), (1300, 512, 32),
        (300, 9001, 128), (620, 300007, 33)]


@pytest.mark.parametrize("n,m,top", TIES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["equal", "two values", "equal but the last"])
def test_ties_over_whole_rows(n, m, top, dtype, kind):
    i = torch.arange(m, device=DEV)
    row = {"equal": torch.full((m,), 2.0, device=DEV), "two values": (i % 5 == 3).float(), "equal but the last": (i == m - 1).float()}[kind].to(dtype)
    r = tp.token_logprobs(row.expand(n, m).contiguous(), top=top)
    order = torch.sort(row.float(), descending=True, stable=True).indices[:top]
    assert torch.equal(r.top_ids, order.expand(n, top))
    want = torch.log_softmax(row.double(), 0)[order]
    # u (13 + 2 a + 3 l) for the log of the sum, doubled, and the result's rounding: a below 1, l and |want| below 13
    assert (r.top_logprobs - want).abs().max() < 2.0 ** -24 * (2 * (13 + 2 + 39 + 3 + 13) + 13)
