"""Plain 64-bit forms of the stored-row consumers, row by row from their definitions, with error bounds of the
fp32 kernels derived from the formulas.

u = 2^-24 is the largest relative rounding of an fp32 operation. What the kernels evaluate per column, with
d = x - m (m the row's maximum): e = ex2(d c), c = log2(e)/T. ex2 is off by at most 2^-22, the product and the
difference by u each, so e is off by 4u + 2u |d|/T relatively. A sum of e is off by the mean of that, 4u + 2u a
with a = E_p |d|/T, and by the additions' own rounding: at most eight that are not compensated, 8u. ln of it:
one fp32 logarithm, 2u |ln s|, and its result's rounding. Hence for l = ln s

    |delta l| <= u (13 + 2 a + 3 l)

which every bound below starts from; each is then doubled, once for all, for second-order terms. ex2 gives 0 below
2^-126 (FLUSH): a probability is off by that much besides, before its factors."""
import math

import torch

U = 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}  # half the smallest step; below fp32's normal range
FLUSH = 2.0 ** -126
NEG = float("-inf")


def row_state(x, T):
    """x: one row, float64. (d/T, p, log p, l, a, E d^2/T^2), the masked columns with p = 0."""
    m = x.max()
    d = (x - m) / T
    e = d.exp()
    s = e.sum()
    p = e / s
    dd = torch.where(p > 0, d, torch.zeros_like(d))
    return d, p, d - s.log(), float(s.log()), float((p * -dd).sum()), float((p * dd * dd).sum())


def logprobs(x, token, T, top, g_lp=0.0, g_h=0.0):
    """One row x [M] (float64). dict of lp, h, top_lp, top_ids, grad and the bounds lp_tol, h_tol, top_tol, grad_tol."""
    M = x.shape[0]
    zero = torch.zeros(M, dtype=torch.float64)
    if token is not None and not 0 <= token < M:
        return {"lp": 0.0, "h": 0.0, "top_lp": [NEG] * top, "top_ids": [-1] * top, "grad": zero, "lp_tol": 0.0, "h_tol": 0.0,
                "top_tol": [0.0] * top, "grad_tol": zero}
    if (x == NEG).all():
        return {"lp": NEG, "h": 0.0, "top_lp": [NEG] * top, "top_ids": [-1] * top, "grad": zero, "lp_tol": 0.0, "h_tol": 0.0,
                "top_tol": [0.0] * top, "grad_tol": zero}
    d, p, logp, l, a, a2 = row_state(x, T)
    l_tol = U * (13 + 2 * a + 3 * l)
    # entropy l - h/(s T): the mean of d under weights off by 4u + 2u|d| each, its sum's rounding 8u, the division
    h = -float(torch.where(p > 0, p * logp, zero).sum())
    out = {"h": h, "h_tol": 2 * (l_tol + U * (16 * a + 2 * a2 + h))}
    order = sorted(range(M), key=lambda v: (-float(x[v]), v))[:top]
    order = [v for v in order if x[v] > NEG]
    out["top_ids"] = order + [-1] * (top - len(order))
    # d/T: a difference, a rounded 1/T and a product, then one subtraction
    one = lambda v: 2 * (l_tol + U * (3 * abs(float(d[v])) + abs(float(logp[v]))))  # noqa: E731
    out["top_lp"] = [float(logp[v]) for v in order] + [NEG] * (top - len(order))
    out["top_tol"] = [one(v) for v in order] + [0.0] * (top - len(order))
    grad, tol = zero.clone(), zero.clone()
    if token is not None:
        out["lp"], out["lp_tol"] = float(logp[token]), one(token) if x[token] > NEG else 0.0
        grad[token] += g_lp
        tol[token] += 4 * U * abs(g_lp)
    fin = torch.where(p > 0, logp, zero)
    inner = -g_lp - g_h * (fin + h)
    grad = (grad + p * inner) / T
    # p from log2 p = (x - m) c - l log2(e): off by l_tol and 4u (|d| + l) and ex2's 4u; the bracket by its terms' roundings
    p_rel = l_tol + U * (4 * (d.clamp(min=-200.0).abs() + l) + 4)
    mag = abs(g_lp) + abs(g_h) * (fin.abs() + abs(h))
    tol = 2 * (tol + FLUSH * mag + p * mag * (p_rel + 6 * U) + p * abs(g_h) * (out["h_tol"] + l_tol + 4 * U * (d.clamp(min=-200.0).abs() + l))) / T
    return {**out, "grad": grad, "grad_tol": tol}


def distill(x, ids, values, T, rest, w=1.0):
    """One row. ids, values: lists of K. dict of loss, grad, loss_tol, grad_tol."""
    M = x.shape[0]
    zero = torch.zeros(M, dtype=torch.float64)
    entries = [(v, float(y)) for v, y in zip(ids, values) if 0 <= v < M and float(y) > NEG]
    if not entries:
        return {"loss": 0.0, "grad": zero, "loss_tol": 0.0, "grad_tol": zero}
    if rest:
        logq = [y for _, y in entries]
    else:
        top = max(y for _, y in entries) / T
        s = sum(math.exp(y / T - top) for _, y in entries)
        logq = [y / T - top - math.log(s) for _, y in entries]
    q = [math.exp(v) for v in logq]
    if (x == NEG).all():
        return {"loss": math.inf if any(v > 0 for v in q) else 0.0, "grad": zero, "loss_tol": 0.0, "grad_tol": zero}
    d, p, logp, l, a, _ = row_state(x, T)
    l_tol = U * (13 + 2 * a + 3 * l)
    loss = sum(qk * (lq - float(logp[v])) for qk, lq, (v, _) in zip(q, logq, entries) if qk > 0)
    Z = sum(q)
    share = zero.clone()
    for qk, (v, _) in zip(q, entries):
        share[v] += qk
    listed = torch.zeros(M, dtype=torch.bool)
    listed[[v for v, _ in entries]] = True
    # the list's own arithmetic is in 64 bits; the row's sum gives l_tol, and the last rounding
    scale = sum(qk for qk in q)
    q_r, r, p_r, lr_tol, lr = 0.0, zero, 0.0, 0.0, 0.0
    if rest:
        other = torch.where(listed, torch.full_like(x, NEG), x)
        if (other > NEG).any():
            q_r = 1.0 - Z if 1.0 - Z >= 2.0 ** -20 else 0.0
            dr, r, _, lr, ar, _ = row_state(other, T)
            lr_tol = U * (13 + 2 * ar + 3 * lr)
            log_pr = float((other.max() - x.max()) / T) + lr - l
            p_r = math.exp(log_pr)
            if q_r > 0:
                loss += q_r * (math.log(q_r) - log_pr)
            scale += q_r
            Z += q_r
    loss_tol = 2 * (scale * (l_tol + lr_tol) + U * abs(loss) + 1e-13)
    gen = p * Z
    gen_tol = p * Z * (l_tol + U * (4 * (d.clamp(min=-200.0).abs() + l) + 8))
    if rest and (r > 0).any():
        dc = dr.clamp(min=-200.0).abs()
        gap = abs(float((other.max() - x.max()) / T))
        # Z p_r - q_r: p_r from exp of (gap + lr - l), q_r = Z - sum q in fp32
        coef_tol = Z * p_r * (l_tol + lr_tol + U * (4 * min(gap, 200.0) + 4 * l + 4 * lr + 8)) + 8 * U * (len(q) ** 0.5 + 1)
        gen = torch.where(listed, gen, (Z * p_r - q_r) * r)
        gen_tol = torch.where(listed, gen_tol, r * (coef_tol + abs(Z * p_r - q_r) * (lr_tol + U * (4 * (dc + lr) + 8))))
    spread = max((abs(v) for qk, v in zip(q, logq) if qk > 0), default=0.0)
    grad = w * (gen - share) / T
    tol = 2 * abs(w) * (FLUSH + gen_tol + share * U * (12 + 6 * min(spread, 200.0)) + U * grad.abs() * T / max(abs(w), 1e-30)) / T
    return {"loss": loss, "grad": grad, "loss_tol": loss_tol, "grad_tol": tol}


def close(got, want, tol, dtype=torch.float32, what=""):
    """Elementwise |got - want| <= tol + the rounding of `dtype`; infinities equal."""
    got, want, tol = (torch.as_tensor(t.detach() if isinstance(t, torch.Tensor) else t, dtype=torch.float64).reshape(-1).cpu() for t in (got, want, tol))
    inf = torch.isinf(want)
    assert (got[inf] == want[inf]).all(), f"{what}: infinite entries differ"
    g, w, t = got[~inf], want[~inf], tol[~inf]
    assert torch.isfinite(g).all(), f"{what}: not finite"
    over = (g - w).abs() - (t + STEP[dtype] * w.abs() * 1.001 + TINY[dtype])
    assert g.numel() == 0 or float(over.max()) <= 0, f"{what}: off by {float((g - w).abs().max()):.3g}, {float(over.max()):.3g} over its bound"
