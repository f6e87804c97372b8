"""Stored score rows on the GPU: token_logprobs and topk_distillation, forward and backward, against plain 64-bit
forms at the sizes, masks, strides and lists where they can go wrong (bounds derived in _rows_ref.py)."""
import pytest
import torch

import lazy_score_matrix_gb300 as tp
from lazy_score_matrix_gb300 import _lib
from tests import _rows_ref as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]
NEG = float("-inf")
DEV = "cuda"


def scores(n, m, dtype, seed, spread=3.0):
    """[n, m]: a background, and a few tall columns a row."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, m, generator=g) * spread
    x.scatter_(1, torch.randint(0, m, (n, 3), generator=g), torch.randn(n, 3, generator=g) + 9)
    return x.to(dtype)


def check_logprobs(x, tokens, T=1.0, top=0, grads=True, run=None):
    """x [n, m] on the CPU in its dtype, tokens a list or None."""
    n, m = x.shape
    g = torch.Generator().manual_seed(n + m)
    g1, g2 = torch.randn(n, generator=g), torch.randn(n, generator=g) * 0.3
    xg = (run or (lambda t: t.to(DEV)))(x)
    assert torch.equal(torch.nan_to_num(xg.cpu().float()), torch.nan_to_num(x.float()))
    leaf = xg.detach().requires_grad_(grads)
    tok = None if tokens is None else torch.tensor(tokens, device=DEV)
    r = tp.token_logprobs(leaf, tok, temperature=T, top=top)
    grad = None
    if grads:
        if tok is None:
            grad, = torch.autograd.grad(r.entropy, leaf, g2.to(DEV))
        else:
            grad, = torch.autograd.grad((r.logprobs, r.entropy), leaf, (g1.to(DEV), g2.to(DEV)))
        assert grad.dtype == x.dtype and grad.shape == x.shape
    assert r.entropy.dtype == torch.float32
    for i in range(n):
        w = ref.logprobs(x[i].double(), None if tok is None else tokens[i], T, top, 0.0 if tok is None else float(g1[i]), float(g2[i]))
        if tok is not None:
            ref.close(r.logprobs[i], w["lp"], w["lp_tol"], what=f"logprob of row {i}")
        ref.close(r.entropy[i], w["h"], w["h_tol"], what=f"entropy of row {i}")
        if top:
            assert r.top_ids[i].tolist() == w["top_ids"], f"alternatives of row {i}"
            ref.close(r.top_logprobs[i], w["top_lp"], w["top_tol"], what=f"alternatives of row {i}")
        if grads:
            ref.close(grad[i], w["grad"], w["grad_tol"], x.dtype, what=f"gradient of row {i}")
    return r


def teacher_list(x, k, T, rest, seed):
    """A teacher near the student: ids, values [n, k] on the CPU."""
    g = torch.Generator().manual_seed(seed)
    y = x.float() + 0.7 * T * torch.randn(x.shape, generator=g)
    y = torch.where(y > NEG, y, torch.full_like(y, -30.0))
    if rest:
        y = torch.log_softmax(y / T, 1)
    values, ids = y.topk(k, 1)
    return ids, values


def check_distill(x, ids, values, T=1.0, rest=False, run=None, weights=True):
    n, m = x.shape
    w = torch.rand(n, generator=torch.Generator().manual_seed(n * m)) + 0.5 if weights else torch.ones(n)
    xg = (run or (lambda t: t.to(DEV)))(x)
    leaf = xg.detach().requires_grad_(True)
    a = (ids.to(DEV), values.to(DEV))
    loss = tp.topk_distillation(leaf, *a, temperature=T, rest=rest)
    grad, = torch.autograd.grad(loss, leaf, w.to(DEV))
    alone = tp.topk_distillation(xg, *a, temperature=T, rest=rest)
    loss2, grad2 = tp.topk_distillation_grad(xg, *a, w.to(DEV) if weights else None, temperature=T, rest=rest)
    assert torch.equal(alone, loss.detach())
    for i in range(n):
        e = ref.distill(x[i].double(), ids[i].tolist(), values[i].tolist(), T, rest, float(w[i]))
        for name, l, gr in (("autograd", loss, grad), ("at once", loss2, grad2)):
            ref.close(l[i].detach(), e["loss"], e["loss_tol"], what=f"loss of row {i} ({name})")
            ref.close(gr[i], e["grad"], e["grad_tol"], x.dtype, what=f"gradient of row {i} ({name})")
    return loss


# --- sizes and types ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m", [(1, 1), (3, 2), (5, 7), (4, 8), (2, 9), (9, 33), (17, 129), (3, 260), (2, 1000), (2, 4097), (1, 8192),
                                 (2, 16391), (1, 70001)])
def test_logprobs_sizes(n, m, dtype):
    x = scores(n, m, dtype, n * 1000 + m)
    check_logprobs(x, [(i * 37) % m for i in range(n)], 0.8, min(m, 20))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m,k", [(1, 1, 1), (3, 2, 2), (4, 9, 5), (5, 129, 128), (3, 1000, 33), (2, 4097, 100), (2, 16391, 64), (1, 70001, 128)])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_sizes(n, m, k, rest, dtype):
    x = scores(n, m, dtype, n * 1000 + m + 1)
    check_distill(x, *teacher_list(x, k, 1.3, rest, m), 1.3, rest)


@pytest.mark.parametrize("n", [1, 2, 151, 153, 700])
def test_row_counts(n):
    x = scores(n, 600, torch.bfloat16, n)
    check_logprobs(x, [(i * 7) % 600 if i % 5 else -1 for i in range(n)], top=3)
    check_distill(x[:40], *teacher_list(x[:40], 8, 1.0, True, 3), 1.0, True)


@pytest.mark.parametrize("top", [1, 2, 5, 31, 32, 33, 64, 127, 128])
@pytest.mark.parametrize("m", [128, 1537, 20011])
def test_top_counts(top, m):
    check_logprobs(scores(2, m, torch.bfloat16, top), [0, m - 1], top=top, grads=False)


@pytest.mark.parametrize("T", [1e-3, 0.05, 0.7, 1.0, 3.0, 1e3])
def test_temperatures(T):
    x = scores(3, 1500, torch.float32, 5)
    check_logprobs(x, [1, 2, 3], T, 9)
    check_distill(x, *teacher_list(x, 12, min(T, 3.0), False, 9), T, False)
    if T >= 0.5:
        check_distill(x, *teacher_list(x, 12, T, True, 9), T, True)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_rows_and_many_elements(dtype):
    # rows of an ordinary vocabulary, checked whole against fp64 torch (the row-by-row form is slow here)
    n, m, T = 24, 131075, 1.0
    x = scores(n, m, dtype, 77).to(DEV)
    tok = torch.arange(n, device=DEV) * 5003
    leaf = x.detach().requires_grad_(True)
    r = tp.token_logprobs(leaf, tok, top=50)
    g1 = torch.linspace(-1, 1, n, device=DEV)
    grad, = torch.autograd.grad(r.logprobs, leaf, g1)
    logp = torch.log_softmax(x.double(), 1)
    p = logp.exp()
    assert (r.logprobs - logp[torch.arange(n), tok]).abs().max() < 64 * ref.U * 12  # u (13 + 2 a + 3 l), a and l below 12
    assert (r.entropy + (p * logp).sum(1)).abs().max() < 2 * ref.U * (13 + 5 * 12 + 16 * 12 + 2 * 144)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :50]
    assert torch.equal(r.top_ids, order)
    want = -p * g1.double()[:, None]
    want[torch.arange(n), tok] += g1.double()
    tol = 2 * ref.U * 120 * p * g1.abs()[:, None] + ref.STEP[dtype] * 1.001 * want.abs() + ref.TINY[dtype] + 8 * ref.U * g1.abs()[:, None] * (want > 0)
    assert ((grad.double() - want).abs() <= tol).all()


# The kernels' shapes: a warp a row, a CTA a row, a cluster a row, one CTA alone on an SM; every one with rows at odd
# addresses, some left out, masked columns, and lists that lie across the parts of a long row. Checked whole against
# fp64 torch, with _rows_ref.py's bounds formed for all rows at once.
SHAPES = [(1300, 261, torch.float32), (1300, 4099, torch.bfloat16), (1216, 8001, torch.float32), (650, 9001, torch.float32),
          (610, 100003, torch.bfloat16), (300, 32003, torch.float32), (40, 70001, torch.float16), (5, 150001, torch.bfloat16),
          (2, 300007, torch.bfloat16), (160, 100003, torch.float32), (620, 300007, torch.float16)]


def _bounds(x, T):
    """fp64 rows: d = (x - max)/T, p, log p, l, a, E d^2, and the bound of l."""
    d = (x - x.amax(1, keepdim=True)) / T
    l = d.exp().sum(1, keepdim=True).log()
    p = (d - l).exp()
    dd = torch.where(p > 0, d, 0.0)
    a, a2 = -(p * dd).sum(1, keepdim=True), (p * dd * dd).sum(1, keepdim=True)
    return d, p, d - l, l, a, a2, ref.U * (13 + 2 * a + 3 * l)


def _device_scores(n, m, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, m, device=DEV, generator=g) * 3
    x.scatter_(1, torch.randint(0, m, (n, 3), device=DEV, generator=g), torch.randn(n, 3, device=DEV, generator=g) + 9)
    x[:, torch.rand(m, device=DEV, generator=g) < 0.1] = NEG
    return x.to(dtype)


@pytest.mark.parametrize("n,m,dtype", SHAPES)
def test_logprobs_shapes(n, m, dtype):
    T, U = 0.9, ref.U
    x = _device_scores(n, m, dtype, n + m)
    i = torch.arange(n, device=DEV)
    tok = (i * 7919) % m
    tok[3::11] = -1
    kept = tok >= 0
    g1, g2 = torch.linspace(-1, 1, n, device=DEV), torch.linspace(0.2, -0.3, n, device=DEV)
    for top in (20, 100):
        leaf = x.detach().requires_grad_(top == 20)
        r = tp.token_logprobs(leaf, tok, temperature=T, top=top)
        x64 = x.double()
        d, p, logp, l, a, a2, l_tol = _bounds(x64, T)
        t = tok.clamp(min=0)[:, None]
        lp, dt = logp.gather(1, t)[:, 0], d.gather(1, t)[:, 0]
        fin = kept & (lp > NEG)
        assert (r.logprobs[~kept] == 0).all() and (r.logprobs[kept & (lp == NEG)] == NEG).all()
        tol = 2 * (l_tol[:, 0] + U * (3 * dt.abs() + lp.abs())) + U * lp.abs()
        assert ((r.logprobs.double() - lp).abs() <= tol)[fin].all()
        h = -torch.where(p > 0, p * logp, 0.0).sum(1, keepdim=True)
        h_tol = 2 * (l_tol + U * (16 * a + 2 * a2 + h)) + U * h
        assert ((r.entropy.double() - h[:, 0]).abs() <= h_tol[:, 0])[kept].all() and (r.entropy[~kept] == 0).all()
        order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(r.top_ids[kept], order[kept]) and (r.top_ids[~kept] == -1).all()
        v, dv = logp.gather(1, order), d.gather(1, order)
        assert ((r.top_logprobs.double() - v).abs() <= 2 * (l_tol + U * (3 * dv.abs() + v.abs())) + U * v.abs())[kept].all()
        if top == 20:
            grad, = torch.autograd.grad((r.logprobs, r.entropy), leaf, (g1, g2))
            w1, w2 = (torch.where(kept, w, 0.0).double()[:, None] for w in (g1, g2))
            lf = torch.where(p > 0, logp, 0.0)
            want = -p * (w1 + w2 * (lf + h))
            want[i, t[:, 0]] += w1[:, 0]
            want /= T
            dc = d.clamp(min=-200.0).abs()
            mag = w1.abs() + w2.abs() * (lf.abs() + h)
            tol = 2 * ((p + ref.FLUSH) * mag * (l_tol + U * (4 * (dc + l) + 10)) + p * w2.abs() * (h_tol + l_tol + 4 * U * (dc + l)) + 4 * U * w1.abs()) / T
            assert ((grad.double() - want).abs() <= tol + ref.STEP[dtype] * 1.001 * want.abs() + ref.TINY[dtype]).all()
            del grad, want, mag, tol, lf, dc
        del x64, d, p, logp, order


# Many rows of few columns: one score a register of a warp, at every count of registers and about its ends; ties that let
# every column through, masked columns, rows left out, rows at odd addresses.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 289, 384, 385, 511, 512, 513])
def test_many_short_rows(m, dtype):
    n, top = 1217, min(m, 32)
    i = torch.arange(n)
    x = scores(n, m, dtype, m)
    x[0::5] = 2.0  # all equal
    x[1::5] = (torch.arange(m) % 3 * 0.5).to(dtype)
    x[2::5, ::3] = NEG
    x[7::50] = NEG
    x[12::50, 1:] = NEG
    tok = i * 7 % m
    tok[4::13] = -100
    buf = torch.full((n, m + 3), float("nan"), dtype=dtype, device=DEV)
    buf[:, 1:1 + m] = x.to(DEV)
    leaf = buf[:, 1:1 + m].detach().requires_grad_(True)
    r = tp.token_logprobs(leaf, tok.to(DEV), temperature=0.8, top=top)
    none = tp.token_logprobs(buf[:, 1:1 + m], tok.to(DEV), temperature=0.8)
    assert torch.equal(none.logprobs, r.logprobs) and torch.equal(none.entropy, r.entropy)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top]
    order = torch.where((x.float().gather(1, order) > NEG) & (tok >= 0)[:, None], order, -1)
    assert torch.equal(r.top_ids.cpu(), order)
    g1, g2 = torch.linspace(-1, 1, n), torch.linspace(0.2, -0.3, n)
    grad, = torch.autograd.grad((r.logprobs, r.entropy), leaf, (g1.to(DEV), g2.to(DEV)))
    for k in list(range(26)) + list(range(26, n, 83)) + [n - 1]:
        w = ref.logprobs(x[k].double(), int(tok[k]), 0.8, top, float(g1[k]), float(g2[k]))
        ref.close(r.logprobs[k].detach(), w["lp"], w["lp_tol"], what=f"logprob of row {k}")
        ref.close(r.entropy[k].detach(), w["h"], w["h_tol"], what=f"entropy of row {k}")
        ref.close(r.top_logprobs[k], w["top_lp"], w["top_tol"], what=f"alternatives of row {k}")
        ref.close(grad[k], w["grad"], w["grad_tol"], dtype, what=f"gradient of row {k}")


@pytest.mark.parametrize("n,m,dtype", SHAPES)
@pytest.mark.parametrize("rest", [False, True])
def test_distill_shapes(n, m, dtype, rest):
    T, K, U = 1.2, 50, ref.U
    x = _device_scores(n, m, dtype, n * 3 + m)
    g = torch.Generator(device=DEV).manual_seed(7)
    y = torch.where(x > NEG, x.float(), -40.0) + 0.7 * T * torch.randn(n, m, device=DEV, generator=g)
    if rest:
        y = torch.log_softmax(y.double() / T, 1).float()
    values, ids = y.topk(K, 1)
    if rest:
        values = values - 0.3  # a share for the others everywhere
    del y
    ids[2::9, K // 2:] = -1
    ids[5::13] = -1
    values[7::10, 3] = NEG
    w = torch.rand(n, device=DEV, generator=g) + 0.5
    leaf = x.detach().requires_grad_(True)
    loss = tp.topk_distillation(leaf, ids, values, temperature=T, rest=rest)
    grad, = torch.autograd.grad(loss, leaf, w)
    loss2, grad2 = tp.topk_distillation_grad(x, ids, values, w, temperature=T, rest=rest)
    inplace = x.clone()
    loss3, _ = tp.topk_distillation_grad(inplace, ids, values, w, temperature=T, rest=rest, out=inplace)
    assert torch.equal(loss2, loss3) and torch.equal(grad2, inplace)
    del inplace
    d, p, logp, l, a, _, l_tol = _bounds(x.double(), T)
    ok = (ids >= 0) & (values > NEG)
    kept = ok.any(1, keepdim=True)
    at = ids.clamp(min=0)
    logq = torch.where(ok, values.double() if rest else values.double() / T, NEG)
    if not rest:
        logq = logq - torch.logsumexp(logq, 1, keepdim=True).clamp(min=-1e300)
    q = torch.where(ok, logq.exp(), 0.0)
    want = (torch.where(q > 0, q * (logq - logp.gather(1, at)), 0.0)).sum(1, keepdim=True)
    Z = q.sum(1, keepdim=True)
    listed = torch.zeros(n, m + 1, dtype=torch.bool, device=DEV).scatter_(1, torch.where(ok, at, m), True)[:, :m]
    share = torch.zeros(n, m, dtype=torch.float64, device=DEV).scatter_add_(1, at, q)
    dc = d.clamp(min=-200.0).abs()
    if rest:
        other = torch.where(listed, NEG, x.double())
        dr, r, _, lr, ar, _, lr_tol = _bounds(other, T)
        gap = ((other.amax(1, keepdim=True) - x.double().amax(1, keepdim=True)) / T)
        log_pr = gap + lr - l
        q_r = torch.where(kept & (1 - Z >= 2.0 ** -20), 1 - Z, 0.0)
        want = want + torch.where(q_r > 0, q_r * (q_r.clamp(min=1e-300).log() - log_pr), 0.0)
        Z = Z + q_r
        p_r = log_pr.exp()
        gen = torch.where(listed, p * Z, (Z * p_r - q_r) * r)
        coef_tol = Z * p_r * (l_tol + lr_tol + U * (4 * gap.abs() + 4 * l + 4 * lr + 8)) + 8 * U * (K ** 0.5 + 1)
        gen_tol = torch.where(listed, p * Z * (l_tol + U * (4 * (dc + l) + 8)),
                              r * (coef_tol + (Z * p_r - q_r).abs() * (lr_tol + U * (4 * (dr.clamp(min=-200.0).abs() + lr) + 8))))
        loss_tol = 2 * (Z * (l_tol + lr_tol) + U * want.abs() + 1e-13) + U * want.abs()
        del other, dr, r
    else:
        gen, gen_tol = p * Z, p * Z * (l_tol + U * (4 * (dc + l) + 8))
        loss_tol = 2 * (Z * l_tol + U * want.abs() + 1e-13) + U * want.abs()
    want = torch.where(kept, want, 0.0)[:, 0]
    spread = torch.where(q > 0, logq.abs(), 0.0).amax(1, keepdim=True).clamp(max=200.0)
    wg = torch.where(kept[:, 0], w, 0.0).double()[:, None]
    gw = wg * (gen - share) / T
    tol = 2 * (wg / T) * (ref.FLUSH + gen_tol + share * U * (12 + 6 * spread)) + 2 * U * gw.abs() + ref.STEP[dtype] * 1.001 * gw.abs() + ref.TINY[dtype]
    for name, lo, gr in (("autograd", loss.detach(), grad), ("at once", loss2, grad2)):
        assert ((lo.double() - want).abs() <= loss_tol[:, 0])[kept[:, 0]].all() and (lo[~kept[:, 0]] == 0).all(), name
        assert ((gr.double() - gw).abs() <= tol).all(), name


# --- masks, ties, orders ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_columns_and_rows(dtype):
    m = 2500
    x = scores(6, m, dtype, 2)
    low = torch.finfo(dtype).min
    x[0, ::2] = NEG                  # half the columns
    x[1, :] = NEG                    # the whole row
    x[2, :] = NEG                    # all but three
    x[2, [5, 1200, 2499]] = torch.tensor([1.0, 3.0, 3.0], dtype=dtype)
    x[3, :] = low                    # masked by the type's lowest value, all but three
    x[3, [7, 1201, 2000]] = torch.tensor([1.0, 3.0, 3.0], dtype=dtype)
    x[4, :] = low                    # that value throughout: uniform
    x[5, 1:] = NEG                   # one column
    check_logprobs(x, [1, 4, 1200, 9, 3, 0], top=10)
    check_logprobs(x, [2, 4, 6, 7, 3, 5], 2.5, 10)
    for rest in (False, True):
        ids, values = teacher_list(x, 9, 1.0, rest, 5)
        ids[2], ids[5] = torch.tensor([5, 1200, 2499] * 3), torch.zeros(9, dtype=torch.int64)
        values = values - 3.0  # some share for the rest
        keep = [0, 1, 2, 4, 5]
        check_distill(x[keep], ids[keep], values[keep], 1.0, rest)


def test_lowest_value_outside_the_list():
    # every unlisted column masked by the lowest value: their class has no probability, the listed ones all of it
    x = torch.full((1, 900), torch.finfo(torch.float32).min)
    ids = torch.tensor([[3, 500, 899, -1]])
    x[0, ids[0, :3]] = torch.tensor([1.0, 2.0, 0.5])
    values = torch.tensor([[0.25, 0.5, 0.25, 0.0]]).log()
    loss, grad = tp.topk_distillation_grad(x.to(DEV), ids.to(DEV), values.to(DEV), rest=True)
    e = ref.distill(x[0].double(), ids[0].tolist(), values[0].tolist(), 1.0, False)  # q as a softmax of its logarithms
    ref.close(loss, e["loss"], e["loss_tol"])
    ref.close(grad, e["grad"], e["grad_tol"] + 1e-6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "steps", "zeros"])
def test_ties_and_orders(kind, dtype):
    m = 9001
    i = torch.arange(m)
    x = {"equal": torch.full((m,), 2.0), "ascending": i * (4.0 / m), "descending": i.flip(0) * (4.0 / m), "steps": (i % 7).float(),
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0)}[kind]
    check_logprobs(x.to(dtype)[None].repeat(2, 1), [0, m - 1], top=128, grads=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_magnitudes(dtype):
    x = scores(3, 700, dtype, 8).float()
    x = (x + torch.tensor([[3.0e4], [-3.0e4], [0.0]])).to(dtype)
    check_logprobs(x, [0, 5, 699], top=4)
    if dtype == torch.float32:
        big = torch.randn(2, 700, generator=torch.Generator().manual_seed(1)) * 1e37
        check_logprobs(big, [3, 4], top=4)


def test_left_out_rows_are_not_read():
    x = scores(8, 1000, torch.bfloat16, 3)
    x[[1, 4]] = float("nan")
    tokens = [3, -100, 7, 8, 1000, 9, -1, 2**40]
    check_logprobs(x, tokens, top=5)
    ids, values = teacher_list(x.nan_to_num(), 6, 1.0, True, 3)
    ids[1], values[4] = -1, NEG
    ids[6] = torch.tensor([-1, 1000, 2**40, -(2**40), -7, 1001])
    check_distill(x, ids, values, 1.0, True)
    check_distill(x, ids, values, 1.0, False)


def test_nan_and_inf_reach_the_results():
    x = scores(3, 5000, torch.float32, 3).to(DEV)
    x[0, 4321] = float("nan")
    x[1, 17] = float("inf")
    leaf = x.detach().requires_grad_(True)
    r = tp.token_logprobs(leaf, torch.tensor([5, 6, 7], device=DEV))
    assert r.logprobs.isnan().tolist() == [True, True, False] and r.entropy.isnan().tolist() == [True, True, False]
    for rest in (False, True):
        loss = tp.topk_distillation(x, torch.tensor([[1, 2]] * 3, device=DEV), torch.full((3, 2), -1.0, device=DEV), rest=rest)
        assert loss.isnan().tolist() == [True, True, False]


@pytest.mark.parametrize("rest", [False, True])
def test_nan_in_a_teacher_list_shows(rest):
    x = scores(3, 300, torch.float32, 3).to(DEV)
    values = torch.full((3, 5), -2.0, device=DEV)
    values[1, 2] = float("nan")
    loss = tp.topk_distillation(x, torch.arange(5, device=DEV).repeat(3, 1), values, rest=rest)
    assert loss.isnan().tolist() == [False, True, False]


@pytest.mark.parametrize("rest", [False, True])
def test_lists_with_repeats_gaps_and_any_order(rest):
    x = scores(4, 777, torch.float32, 6)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, 777, (4, 40), generator=g)
    ids[:, 10:20] = ids[:, :10]      # columns listed twice, some three times
    ids[:, 30:33] = ids[:, :3]
    ids[1, ::3] = -1
    values = torch.randn(4, 40, generator=g) - 5.0
    values[2, 5:9] = NEG
    ids[3], values[3, 1:] = 776, NEG  # one entry, the last column
    check_distill(x, ids, values, 0.9, rest)


def test_rest_without_room():
    # every column listed: no class is left; shares that sum to more than one leave it nothing
    x = scores(2, 40, torch.float32, 6)
    ids = torch.arange(40)[None].repeat(2, 1)
    values = torch.log_softmax(x + torch.randn(2, 40, generator=torch.Generator().manual_seed(2)), 1)
    check_distill(x, ids, values, 1.0, True)
    check_distill(x, ids[:, :30], values[:, :30] + 1.0, 1.0, True)


def test_listed_column_that_the_student_forbids():
    x = scores(1, 100, torch.float32, 6)
    x[0, 7] = NEG
    loss, grad = tp.topk_distillation_grad(x.to(DEV), torch.tensor([[3, 7]], device=DEV), torch.zeros(1, 2, device=DEV))
    assert loss.item() == float("inf") and torch.isfinite(grad).all() and abs(grad[0, 7].item() + 0.5) < 1e-6


# --- layouts ------------------------------------------------------------------------------------------------------


LAYOUTS = {
    "padded vocabulary": lambda x: torch.cat([x, torch.full((x.shape[0], 13), 60.0, dtype=x.dtype)], 1).to(DEV)[:, :x.shape[1]],
    "odd offset": lambda x: torch.cat([torch.zeros(3, dtype=x.dtype), x.reshape(-1)]).to(DEV)[3:].view(x.shape),
    "every other row": lambda x: torch.stack([x, -x], 1).to(DEV)[:, 0],
    "transposed": lambda x: x.t().contiguous().to(DEV).t(),
    "every other column": lambda x: torch.stack([x, -x], 2).to(DEV)[..., 0],
}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [515, 16391])
def test_layouts(layout, dtype, m):
    x = scores(5, m, dtype, 12)
    check_logprobs(x, [0, 1, -1, m - 1, 77], top=6, run=LAYOUTS[layout])
    for rest in (False, True):
        check_distill(x, *teacher_list(x, 20, 1.0, rest, 1), 1.0, rest, run=LAYOUTS[layout])


def test_batches_and_shifted_views():
    b, s, m = 3, 5, 701
    x = scores(b * s, m, torch.bfloat16, 4).to(DEV).view(b, s, m)
    tok = torch.randint(0, m, (b, s), device=DEV)
    whole = tp.token_logprobs(x.reshape(-1, m), tok.reshape(-1), top=4)
    for view, t in ((x[:, :-1], tok[:, :-1]), (x[:, 1:], tok[:, 1:]), (x.transpose(0, 1), tok.t()), (x[:, ::2], tok[:, ::2])):
        r = tp.token_logprobs(view, t, top=4)
        same = lambda a, k: torch.equal(a, k)  # noqa: E731
        index = torch.arange(b * s, device=DEV).view(b, s)
        at = (index[:, :-1], index[:, 1:], index.t(), index[:, ::2])[[v.shape == view.shape and v.stride() == view.stride() and
                                                                      v.data_ptr() == view.data_ptr() for v in
                                                                      (x[:, :-1], x[:, 1:], x.transpose(0, 1), x[:, ::2])].index(True)]
        for f in ("logprobs", "entropy", "top_logprobs", "top_ids"):
            assert same(getattr(r, f), getattr(whole, f)[at]), f
        assert _lib.logits_binding().row_strides(view) is not None  # read where it lies
    leaf = x.detach().requires_grad_(True)
    tp.token_logprobs(leaf[:, :-1], tok[:, :-1]).logprobs.sum().backward()
    flat = x.reshape(-1, m).detach().requires_grad_(True)
    lp = tp.token_logprobs(flat, tok.reshape(-1)).logprobs.view(b, s)
    lp[:, :-1].sum().backward()
    assert torch.equal(leaf.grad.view(-1, m), flat.grad)
    one = tp.token_logprobs(x[1, 2], tok[1, 2], top=4)  # no leading dimension
    assert one.logprobs.shape == () and torch.equal(one.top_ids, whole.top_ids[1 * s + 2])
    shared = x[:1, 0].expand(6, m)  # one row seen six times
    r = tp.token_logprobs(shared, tok[0, :1].expand(6))
    assert torch.equal(r.logprobs, whole.logprobs[:1].expand(6))


def test_empty_batches():
    x = torch.empty(0, 4, 33, device=DEV, dtype=torch.bfloat16).requires_grad_(True)
    r = tp.token_logprobs(x, torch.empty(0, 4, dtype=torch.int64, device=DEV), top=3)
    assert r.logprobs.shape == (0, 4) and r.top_ids.shape == (0, 4, 3)
    r.logprobs.sum().backward()
    assert x.grad.shape == x.shape
    loss, grad = tp.topk_distillation_grad(x.detach(), torch.empty(0, 4, 2, dtype=torch.int64, device=DEV), torch.empty(0, 4, 2, device=DEV))
    assert loss.shape == (0, 4) and grad.shape == (0, 4, 33)


def test_offsets_beyond_32_bits():
    # 2^31 elements lie before the last rows; only those rows are looked at
    m, n = 131071, 16600
    big = torch.zeros(n, m, dtype=torch.bfloat16, device=DEV)
    assert n * m > 2**31 and (n - 3) * m > 2**31
    x = scores(3, m, torch.bfloat16, 1)
    big[-3:] = x.to(DEV)
    tok = torch.full((n,), -1, device=DEV)
    tok[-3:] = torch.tensor([5, 6, m - 1], device=DEV)
    r = tp.token_logprobs(big, tok, top=5)
    ids, values = teacher_list(x, 7, 1.0, True, 2)
    ids_all = torch.full((n, 7), -1, device=DEV)
    ids_all[-3:] = ids.to(DEV)
    values_all = torch.zeros(n, 7, device=DEV)
    values_all[-3:] = values.to(DEV)
    loss, grad = tp.topk_distillation_grad(big, ids_all, values_all, rest=True, out=big)
    assert grad is big
    # against 64 bits, not against a call on these rows alone: that one splits a row over more threads and may
    # round its sums another way
    for i, t in enumerate([5, 6, m - 1]):
        w, e = ref.logprobs(x[i].double(), t, 1.0, 5), ref.distill(x[i].double(), ids[i].tolist(), values[i].tolist(), 1.0, True)
        ref.close(r.logprobs[n - 3 + i], w["lp"], w["lp_tol"])
        ref.close(r.entropy[n - 3 + i], w["h"], w["h_tol"])
        assert r.top_ids[n - 3 + i].tolist() == w["top_ids"]
        ref.close(loss[n - 3 + i], e["loss"], e["loss_tol"])
        ref.close(grad[n - 3 + i], e["grad"], e["grad_tol"], torch.bfloat16)
    assert (loss[:-3] == 0).all() and int(torch.count_nonzero(grad[-200:-3])) == 0


# --- gradients against differences --------------------------------------------------------------------------------


def test_gradients_against_differences():
    n, m, T = 3, 300, 1.2
    x = scores(n, m, torch.float32, 9)
    v = torch.randn(n, m, generator=torch.Generator().manual_seed(3))
    tokens, g1, g2 = [4, 299, 7], [0.7, -1.1, 0.4], [0.3, 0.2, -0.6]
    leaf = x.to(DEV).requires_grad_(True)
    r = tp.token_logprobs(leaf, torch.tensor(tokens, device=DEV), temperature=T)
    got, = torch.autograd.grad((r.logprobs, r.entropy), leaf, (torch.tensor(g1, device=DEV), torch.tensor(g2, device=DEV)))
    h = 1e-4

    def both(f):
        return (f(x.double() + h * v.double()) - f(x.double() - h * v.double())) / (2 * h)

    def of_lp(y):
        rows = [ref.logprobs(y[i], tokens[i], T, 0) for i in range(n)]
        return sum(a * w["lp"] + b * w["h"] for a, b, w in zip(g1, g2, rows))

    assert abs(float((got.cpu().double() * v).sum()) - both(of_lp)) < 2e-6  # h^2 third derivatives, fp32 gradient
    for rest in (False, True):
        ids, values = teacher_list(x, 11, T, rest, 8)
        _, grad = tp.topk_distillation_grad(x.to(DEV), ids.to(DEV), values.to(DEV), torch.tensor(g1, device=DEV), temperature=T, rest=rest)
        diff = both(lambda y: sum(a * ref.distill(y[i], ids[i].tolist(), values[i].tolist(), T, rest)["loss"] for i, a in enumerate(g1)))
        assert abs(float((grad.cpu().double() * v).sum()) - diff) < 2e-6


# --- use ----------------------------------------------------------------------------------------------------------


def test_teacher_to_student_together():
    # the teacher's list, the student's loss and gradient, one step down the gradient lowers every row's loss
    teacher, student = scores(20, 3001, torch.bfloat16, 1).to(DEV), scores(20, 3001, torch.float32, 2).to(DEV)
    for T in (1.0, 2.0):
        t = tp.token_logprobs(teacher, top=64, temperature=T)
        loss, grad = tp.topk_distillation_grad(student, t.top_ids, t.top_logprobs, temperature=T, rest=True)
        after = tp.topk_distillation(student - 0.05 * grad, t.top_ids, t.top_logprobs, temperature=T, rest=True)
        assert (loss > 0).all() and (after < loss).all()
        same = tp.topk_distillation(teacher, t.top_ids, t.top_logprobs, temperature=T, rest=True)
        assert same.abs().max() < 2e-6  # the student is the teacher: the values' rounding is left, 64 u |log q| q
    leaf = student.requires_grad_(True)
    lp = tp.token_logprobs(leaf, t.top_ids[:, 0])
    (tp.topk_distillation(leaf, t.top_ids, t.top_logprobs, rest=True).mean() - 0.1 * lp.logprobs.mean() - 0.01 * lp.entropy.mean()).backward()
    assert torch.isfinite(leaf.grad).all() and leaf.grad.abs().sum() > 0


def test_only_one_upstream_gradient():
    x, tok = scores(4, 900, torch.float32, 3).to(DEV), torch.tensor([1, -1, 3, 899], device=DEV)
    parts = []
    for names in (("logprobs",), ("entropy",), ("logprobs", "entropy")):
        leaf = x.detach().requires_grad_(True)
        r = tp.token_logprobs(leaf, tok, top=2)
        assert not r.top_logprobs.requires_grad and not r.top_ids.requires_grad
        sum(getattr(r, f).sum() for f in names).backward()
        parts.append(leaf.grad)
    assert (parts[0] + parts[1] - parts[2]).abs().max() < 1e-6


def test_in_place_and_given_output():
    x = scores(6, 2000, torch.bfloat16, 3).to(DEV)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 12, 1.0, True, 3))
    loss, grad = tp.topk_distillation_grad(x, ids, values, rest=True)
    pad = torch.full((6, 2003), 7.0, dtype=torch.bfloat16, device=DEV)
    _, g = tp.topk_distillation_grad(x, ids, values, rest=True, out=pad[:, 1:2001])
    assert torch.equal(g, grad) and (pad[:, 0] == 7).all() and (pad[:, 2001:] == 7).all()
    y = x.clone()
    l2, g2 = tp.topk_distillation_grad(y, ids, values, rest=True, out=y)
    assert g2 is y and torch.equal(y, grad) and torch.equal(loss, l2)
    leaf = x.clone().requires_grad_(True)
    hold = tp.token_logprobs(leaf * 1.0, ids[:, 0])
    z = leaf * 1.0
    kept = tp.token_logprobs(z, ids[:, 0])
    tp.topk_distillation_grad(z, ids, values, out=z)
    with pytest.raises(RuntimeError):  # the graph of `kept` needs the overwritten scores
        kept.logprobs.sum().backward()
    hold.logprobs.sum().backward()


def test_saved_tensors_that_move():
    # hooks that bring saved tensors back at another address
    x = scores(4, 700, torch.float32, 3).to(DEV)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 6, 1.0, False, 3))

    def grads(view):
        leaf = x.detach().requires_grad_(True)
        y = view(leaf)
        r = tp.token_logprobs(y, ids[:, 0])
        return torch.autograd.grad(r.logprobs.sum() + r.entropy.sum() + tp.topk_distillation(y, ids, values).sum(), leaf)[0]

    for view in (lambda t: t, lambda t: torch.cat([t, t], 1)[:, :700], lambda t: t.t().contiguous().t()):
        want = grads(view)
        with torch.autograd.graph.save_on_cpu():
            got = grads(view)
        assert torch.equal(got, want)


def test_leading_shapes_that_need_a_copy():
    x = scores(2 * 3 * 4, 90, torch.bfloat16, 4).to(DEV).view(2, 3, 4, 90)[:, :2, :3]
    r, want = tp.token_logprobs(x, top=3), tp.token_logprobs(x.reshape(-1, 90), top=3)
    assert r.top_ids.shape == (2, 2, 3, 3) and torch.equal(r.top_ids.reshape(-1, 3), want.top_ids)
    assert torch.equal(r.entropy.reshape(-1), want.entropy)


def test_integer_types_and_teacher_types():
    x = scores(4, 500, torch.float32, 3).to(DEV)
    tok = torch.tensor([1, 2, -1, 4], device=DEV)
    a = tp.token_logprobs(x, tok)
    assert torch.equal(a.logprobs, tp.token_logprobs(x, tok.int()).logprobs)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 5, 1.0, False, 3))
    values = values.half().float()
    assert torch.equal(tp.topk_distillation(x, ids, values), tp.topk_distillation(x, ids.int(), values.half()))


def test_same_bits_every_time():
    x = scores(300, 5003, torch.bfloat16, 3).to(DEV)
    tok = torch.arange(300, device=DEV)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 64, 1.0, True, 3))
    first = tp.token_logprobs(x, tok, top=40)[:] + tp.topk_distillation_grad(x, ids, values, rest=True)
    for _ in range(3):
        again = tp.token_logprobs(x, tok, top=40)[:] + tp.topk_distillation_grad(x, ids, values, rest=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams_and_overlapping_calls():
    x = [scores(64, 20000, torch.bfloat16, i).to(DEV) for i in range(3)]
    ids, values = zip(*[[t.to(DEV) for t in teacher_list(y.cpu(), 32, 1.0, True, 3)] for y in x])
    want = [tp.topk_distillation_grad(*a, rest=True) + tp.token_logprobs(a[0], a[1][:, 0], top=32)[:] for a in zip(x, ids, values)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s, a in zip(streams, zip(x, ids, values)):
        with torch.cuda.stream(s):
            got.append(tp.topk_distillation_grad(*a, rest=True) + tp.token_logprobs(a[0], a[1][:, 0], top=32)[:])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for w, g in zip(want, got) for p, q in zip(w, g))


def test_captured_and_replayed():
    x = scores(16, 9000, torch.bfloat16, 5).to(DEV)
    tok = torch.arange(16, device=DEV) * 3
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 20, 1.0, True, 3))

    def step(x, leaf):
        r = tp.token_logprobs(x, tok, top=10)
        loss, grad = tp.topk_distillation_grad(x, ids, values, rest=True)
        q = tp.token_logprobs(leaf, tok)
        g, = torch.autograd.grad(q.logprobs.sum() + q.entropy.sum(), leaf)
        return [r.logprobs, r.entropy, r.top_logprobs, r.top_ids, loss, grad, g]

    static = torch.zeros_like(x)
    leaf = static.detach().requires_grad_(True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(static, leaf)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(static, leaf)
    for seed in (5, 6):
        y = scores(16, 9000, torch.bfloat16, seed).to(DEV)
        static.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = step(y, y.detach().requires_grad_(True))
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_outputs_stay_inside_their_buffers():
    # guard elements around every output of the C entries come back untouched, every output element is written
    n, m, k, top = 9, 1003, 7, 11
    x = scores(n, m, torch.bfloat16, 3).to(DEV)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), k, 1.0, True, 3))
    tok = torch.arange(n, device=DEV)
    lib = _lib.load()
    rows = _lib.tp_rows(_lib.TP_ROWS_BF16, n, m, n, m, 0, x.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream

    def buf(count, dtype):
        t = torch.full((count + 128,), -77, dtype=dtype, device=DEV)
        return t, t[64:64 + count]

    f, i = torch.float32, torch.int64
    bufs = {"lp": buf(n, f), "h": buf(n, f), "stats": buf(n * 8, f), "tv": buf(n * top, f), "ti": buf(n * top, i), "loss": buf(n, f),
            "dstats": buf(n * 8, f), "grad": buf(n * m, x.dtype), "grad2": buf(n * m, x.dtype)}
    p = {a: b[1].data_ptr() for a, b in bufs.items()}
    grad = lambda a: _lib.tp_rows(rows.dtype, n, m, n, m, 0, p[a])  # noqa: E731
    g1 = torch.ones(n, device=DEV)
    _lib.launch_count(reset=True)
    _lib.check(lib.tp_token_logprobs(rows, tok.data_ptr(), 1.0, top, p["lp"], p["h"], p["stats"], p["tv"], p["ti"], stream), "fwd")
    _lib.check(lib.tp_token_logprobs_backward(rows, tok.data_ptr(), 1.0, p["stats"], g1.data_ptr(), None, grad("grad"), stream), "bwd")
    _lib.check(lib.tp_topk_distillation_grad(rows, k, ids.data_ptr(), values.data_ptr(), None, 1.0, 1, p["loss"], p["dstats"], grad("grad2"),
                                             stream), "grad")
    assert _lib.launch_count() >= 3
    torch.cuda.synchronize()
    for name, (whole, inner) in bufs.items():
        assert (whole[:64] == -77).all() and (whole[-64:] == -77).all(), name
        assert not (inner == -77).any(), name


@pytest.mark.parametrize("entry", ["token_logprobs", "token_logprobs_backward", "topk_distillation", "topk_distillation_backward",
                                   "topk_distillation_grad"])
def test_a_failed_call_raises_and_leaves_the_process_usable(entry, monkeypatch):
    x = scores(4, 300, torch.float32, 3).to(DEV)
    ids, values = (t.to(DEV) for t in teacher_list(x.cpu(), 4, 1.0, False, 3))

    def step():
        leaf = x.detach().requires_grad_(True)
        (tp.token_logprobs(leaf, ids[:, 0]).logprobs.sum() + tp.topk_distillation(leaf, ids, values).sum()).backward()
        return leaf.grad, tp.topk_distillation_grad(x, ids, values)[1]

    want = step()
    monkeypatch.setenv("TP_FAULT_INJECT", entry)
    with pytest.raises(_lib.TPError) as e:
        step()
    assert e.value.status == _lib.TP_ERR_CUDA and entry in str(e.value)
    monkeypatch.delenv("TP_FAULT_INJECT")
    assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_refusals():
    x = torch.zeros(4, 50, device=DEV)
    tok, ids, val = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 3, dtype=torch.int64, device=DEV), torch.zeros(4, 3, device=DEV)
    bad = [
        (TypeError, lambda: tp.token_logprobs(x.double())),
        (TypeError, lambda: tp.token_logprobs(x.long())),
        (ValueError, lambda: tp.token_logprobs(x.cpu())),
        (ValueError, lambda: tp.token_logprobs(x[:, :0])),
        (ValueError, lambda: tp.token_logprobs(x, tok[:3])),
        (TypeError, lambda: tp.token_logprobs(x, tok.float())),
        (TypeError, lambda: tp.token_logprobs(x, tok.bool())),
        (ValueError, lambda: tp.token_logprobs(x, tok.cpu())),
        (ValueError, lambda: tp.token_logprobs(x, tok, top=51)),
        (ValueError, lambda: tp.token_logprobs(torch.zeros(1, 500, device=DEV), top=129)),
        (ValueError, lambda: tp.token_logprobs(x, tok, top=-1)),
        (_lib.TPError, lambda: tp.token_logprobs(x, tok, temperature=0.0)),
        (_lib.TPError, lambda: tp.token_logprobs(x, tok, temperature=float("nan"))),
        (_lib.TPError, lambda: tp.token_logprobs(x, tok, temperature=2e3)),
        (ValueError, lambda: tp.topk_distillation(x, ids[:, :0], val[:, :0])),
        (ValueError, lambda: tp.topk_distillation(x, ids, val[:, :2])),
        (ValueError, lambda: tp.topk_distillation(x, ids[:2], val[:2])),
        (TypeError, lambda: tp.topk_distillation(x, ids.float(), val)),
        (TypeError, lambda: tp.topk_distillation(x, ids, ids)),
        (ValueError, lambda: tp.topk_distillation(x, ids.cpu(), val)),
        (ValueError, lambda: tp.topk_distillation(x, ids, val.clone().requires_grad_(True))),
        (ValueError, lambda: tp.topk_distillation(torch.zeros(1, 500, device=DEV), torch.zeros(1, 129, dtype=torch.int64, device=DEV),
                                                  torch.zeros(1, 129, device=DEV))),
        (ValueError, lambda: tp.topk_distillation_grad(x, ids, val, torch.ones(3, device=DEV))),
        (ValueError, lambda: tp.topk_distillation_grad(x, ids, val, out=torch.zeros(4, 49, device=DEV))),
        (ValueError, lambda: tp.topk_distillation_grad(x, ids, val, out=torch.zeros(4, 50, device=DEV, dtype=torch.float16))),
        (ValueError, lambda: tp.topk_distillation_grad(x, ids, val, out=torch.zeros(50, 4, device=DEV).t())),
        (_lib.TPError, lambda: tp.topk_distillation_grad(x, ids, val, out=x[:1].expand(4, 50))),
        (_lib.TPError, lambda: tp.topk_distillation_grad(x[:3], ids[:3], val[:3], out=x[1:])),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was accepted")
    leaf = x.clone().requires_grad_(True)
    g, = torch.autograd.grad(tp.token_logprobs(leaf, tok).logprobs.sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
