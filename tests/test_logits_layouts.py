"""Stored score rows: gradients written between the scores of one buffer, without sharing an element of them."""
import random

import pytest
import torch

import lazy_score_matrix_gb300 as tp
from lazy_score_matrix_gb300 import _lib
from lazy_score_matrix_gb300 import build as tpbuild
from tests.test_logits import scores, teacher_list

DEV = "cuda"
FAKE = 0x7F0000000000  # never dereferenced
IDS, VALUES, LOSS, STATS = (FAKE + (i << 36) for i in range(1, 5))


def elements(at, n, m, group, rs, gs):
    return [set(range(at + i // group * gs + i % group * rs, at + i // group * gs + i % group * rs + m)) for i in range(n)]


def test_rows_between_rows_are_told_from_rows_on_rows(monkeypatch):
    # every accepted pair shares no element or all of them, every refused one shares some; against sets of elements
    tpbuild.build()
    lib = _lib.load()
    monkeypatch.setenv("TP_FAULT_INJECT", "topk_distillation_grad")  # what is accepted ends in the injected fault
    rng = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        m, group, groups = rng.randint(1, 5), rng.randint(1, 4), rng.randint(1, 4)
        n, inner, outer = group * groups, rng.randint(m, 3 * m), 0
        swap = rng.random() < 0.5  # groups inside rows
        counts = (groups, group) if swap else (group, groups)
        outer = (counts[0] - 1) * inner + m + rng.randint(0, 2 * m + 3)
        rs, gs = (outer, inner) if swap else (inner, outer)
        delta = rng.randint(-3 * outer, 3 * outer)
        x = _lib.tp_rows(0, n, m, group, rs, gs, FAKE)
        g = _lib.tp_rows(0, n, m, group, rs, gs, FAKE + 4 * delta)
        a, b = elements(0, n, m, group, rs, gs), elements(delta, n, m, group, rs, gs)
        free = a == b or not set().union(*a) & set().union(*b)
        status = lib.tp_topk_distillation_grad(x, 2, IDS, VALUES, None, 1.0, 0, LOSS, STATS, g, None)
        assert status == (_lib.TP_ERR_CUDA if free else _lib.TP_ERR_INVALID_ARG), (n, m, group, rs, gs, delta)
        seen[free] += 1
    assert min(seen.values()) > 1500
    # rows at other strides: whole spans count
    for x, g in (((6, 10, 6, 40, 0), (6, 10, 6, 20, 0)), ((6, 10, 3, 20, 200), (6, 10, 6, 20, 0))):
        call = lambda at: lib.tp_topk_distillation_grad(_lib.tp_rows(0, *x, FAKE), 2, IDS, VALUES, None, 1.0, 0, LOSS, STATS,  # noqa: E731
                                                        _lib.tp_rows(0, *g, at), None)
        assert call(FAKE + 4 * 12) == _lib.TP_ERR_INVALID_ARG and call(FAKE + 4 * 100000) == _lib.TP_ERR_CUDA


BETWEEN = {
    "halves of a row": lambda b, n, m: (b.view(n, 2 * m)[:, :m], b.view(n, 2 * m)[:, m:]),
    "second half first": lambda b, n, m: (b.view(n, 2 * m)[:, m:], b.view(n, 2 * m)[:, :m]),
    "every other row": lambda b, n, m: (b.view(2 * n, m)[::2], b.view(2 * n, m)[1::2]),
    "groups": lambda b, n, m: (b.view(3, 2, n // 3, m)[:, 0], b.view(3, 2, n // 3, m)[:, 1]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("layout", BETWEEN)
@pytest.mark.parametrize("n,m,dtype", [(6, 701, torch.bfloat16), (12, 40001, torch.float32), (1500, 333, torch.float16), (660, 9001, torch.bfloat16)])
def test_gradient_between_the_scores(layout, n, m, dtype):
    buf = torch.full((2 * n * m,), 7.0, dtype=dtype, device=DEV)
    x, out = BETWEEN[layout](buf, n, m)
    src = scores(n, m, dtype, m)
    x.copy_(src.to(DEV).view(x.shape))
    ids, values = (t.to(DEV).view(*x.shape[:-1], -1) for t in teacher_list(src, 9, 1.0, True, 2))
    want = tp.topk_distillation_grad(x, ids, values, rest=True)  # the same rows: at another alignment sums may round otherwise
    loss, grad = tp.topk_distillation_grad(x, ids, values, rest=True, out=out)
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
    assert grad.data_ptr() == out.data_ptr() and torch.equal(x.cpu().view(n, m), src)
