"""Operators on stored score rows (a model's logits [N, M]): cases, inputs, plain forms and 64-bit values.

Two operators, each forward and backward:

``token_logprobs``      log probability of one given token a row, the row's entropy and its top alternatives
                        (values and ids, ties to the lower id); backward of log probability and entropy.
``topk_distillation``   KL divergence of a student's row from a teacher's list of top values, over the list alone or
                        with the unlisted columns as one more class ("rest"); loss alone, loss then backward, and
                        loss and gradient in one call for row weights known beforehand.

The plain forms below state what each computes:
  x = logits / T, p = softmax(x), lse = log sum exp x
  logprob = x_t - lse;  H = -sum p log p;  a token outside [0, M) leaves its row out (zeros, (-inf, -1), not read)
  d/dx_v = g_lp ([v = t] - p_v) - g_H p_v (log p_v + H)
  list entries count where the id is in [0, M) and the value is above -inf; a row without one is left out
  plain: q = softmax of the listed values / T;  rest: q = exp(values), q_r = 1 - sum q, 0 where that is below 2^-20
  (what the rounding of fp32 log probabilities can leave of a full list)
  loss = sum q_k (log q_k - log p_k) [+ q_r (log q_r - log p_r), p_r the mass of the unlisted columns]
"""
import numpy as np
import torch

own = False

LEAST_REST = 2.0 ** -20

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # serving: one sequence decodes one token and reports its log probability and 20 alternatives
        {"name": "decode one", "op": "logprobs", "rows": 1, "vocab": 131072, "pad": 0, "dtype": "bf16", "top": 20, "temperature": 0.7,
         "masked": False, "padded": False},
        # serving: a batch of sequences under a grammar that forbids part of an odd-sized vocabulary
        {"name": "decode batch", "op": "logprobs", "rows": 64, "vocab": 100003, "pad": 0, "dtype": "fp16", "top": 5, "temperature": 1.0,
         "masked": True, "padded": False},
        # evaluation: the log probabilities and entropies of a long prompt's own tokens
        {"name": "score prompt", "op": "logprobs", "rows": 4096, "vocab": 131072, "pad": 0, "dtype": "bf16", "top": 0, "temperature": 1.0,
         "masked": False, "padded": True},
        # distillation's teacher side: the list that the student is trained on
        {"name": "teacher list", "op": "logprobs", "rows": 2048, "vocab": 65536, "pad": 0, "dtype": "bf16", "top": 64, "temperature": 2.0,
         "masked": False, "padded": True},
        # a byte-level model: few columns, many rows
        {"name": "bytes", "op": "logprobs", "rows": 32768, "vocab": 261, "pad": 0, "dtype": "fp32", "top": 8, "temperature": 1.0,
         "masked": False, "padded": True},
        # policy gradient with an entropy bonus: a small fp32 model, and a large bf16 one
        {"name": "policy small", "op": "logprobs_train", "rows": 300, "vocab": 32003, "pad": 0, "dtype": "fp32", "temperature": 0.8, "padded": True},
        {"name": "policy large", "op": "logprobs_train", "rows": 4096, "vocab": 131072, "pad": 0, "dtype": "bf16", "temperature": 1.0,
         "padded": True},
        # distillation: a micro-batch; an evaluation pass; training through autograd on logits whose vocabulary is padded
        {"name": "distil micro", "op": "distil_grad", "rows": 8, "vocab": 32000, "pad": 0, "dtype": "fp16", "k": 16, "temperature": 1.0,
         "rest": False, "padded": False},
        {"name": "distil eval", "op": "distil", "rows": 2048, "vocab": 100352, "pad": 0, "dtype": "bf16", "k": 32, "temperature": 2.0,
         "rest": True, "padded": True},
        {"name": "distil autograd", "op": "distil_train", "rows": 1021, "vocab": 50001, "pad": 47, "dtype": "fp32", "k": 50, "temperature": 1.5,
         "rest": True, "padded": True},
        # distillation at scale, loss and gradient at once: over the list alone, and with the rest as a class
        {"name": "distil large", "op": "distil_grad", "rows": 8192, "vocab": 131072, "pad": 0, "dtype": "bf16", "k": 64, "temperature": 2.0,
         "rest": False, "padded": True},
        {"name": "distil rest", "op": "distil_grad", "rows": 3000, "vocab": 150016, "pad": 0, "dtype": "bf16", "k": 128, "temperature": 1.0,
         "rest": True, "padded": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_train", "distil", "distil_train", "distil_grad"])
    vocab = _log_uniform(rng, 200, 160000)
    if rng.random() < 0.5:
        vocab -= vocab % 64
    top = rng.choice([0, 1, 5, 20, 64, 128]) if op == "logprobs" else 0
    most = 1 << (27 if top else 29)  # elements of one case
    rows = _log_uniform(rng, 1, max(1, min(16384, most // vocab)))
    case = {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 0, 1, 24, 61]), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "temperature": rng.choice([0.6, 1.0, 1.0, 1.7, 3.0]), "padded": rows > 1 and rng.random() < 0.6}
    if op == "logprobs":
        case |= {"top": top, "masked": rng.random() < 0.3}
    if op.startswith("distil"):
        case |= {"k": rng.choice([1, 8, 20, 33, 64, 100, 128]), "rest": rng.random() < 0.5}
    return case


def _left_out(case):
    """Rows that a batch's padding leaves out: every twentieth."""
    return (case["rows"] + 12) // 20 if case["padded"] else 0


def work(case):
    n, m, es = case["rows"], case["vocab"], TYPES[case["dtype"]].itemsize
    kept = n - _left_out(case)
    op = case["op"]
    grad = op in ("logprobs_train", "distil_train", "distil_grad")
    side = n * (8 + 8 + 12 * case.get("top", 0)) if op.startswith("logprobs") else n * (4 + 12 * case["k"])
    if grad:
        side += 8 * n
    return {"bytes": kept * m * es + (n * m * es if grad else 0) + side, "flops": kept * m * (6 + (4 if grad else 0))}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, m, t = case["rows"], case["vocab"], TYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    # a flat background, columns that are likelier than others throughout, and a few tall columns in each row
    x = rnd(n, m + case["pad"]).mul_(2.0).add_(rnd(m + case["pad"]).mul_(1.5))
    tall = torch.randint(0, m, (n, 8), device="cuda", generator=g)
    x.scatter_(1, tall, rnd(n, 8).add_(10.0))
    if case.get("masked"):
        x[:, torch.rand(m + case["pad"], device="cuda", generator=g) < 0.3] = -float("inf")
    left = (torch.arange(n, device="cuda") % 20 == 7) if case["padded"] else torch.zeros(n, dtype=torch.bool, device="cuda")
    state = {"case": case, "logits": x.to(t, copy=True)[:, :m]}
    scale = 8.0 if t == torch.float16 else 1.0 / n  # a mean over rows; in fp16 under a loss scale that keeps it in range
    if case["op"].startswith("logprobs"):
        tokens = torch.where(torch.rand(n, device="cuda", generator=g) < 0.8, tall[:, 0], torch.randint(0, m, (n,), device="cuda", generator=g))
        state["tokens"] = torch.where(left, -100, tokens)
        state["g_logprob"], state["g_entropy"] = rnd(n) * scale, torch.full((n,), 0.01 * scale, device="cuda")
        return state
    # the teacher agrees with the student but for noise; a tenth of the lists is shorter than the others
    k, T = min(case["k"], m), case["temperature"]
    y = x[:, :m].add_(rnd(n, m).mul_(0.7 * T))
    if case["rest"]:
        y = y.div_(T)
        y -= y.amax(1, keepdim=True)
        y -= y.exp().sum(1, keepdim=True).log()
    values, ids = y.topk(k, dim=1)
    short = torch.where(torch.rand(n, device="cuda", generator=g) < 0.1, max(1, k // 3), k)
    gone = (torch.arange(k, device="cuda")[None] >= short[:, None]) | left[:, None]
    state["ids"] = torch.where(gone, -1, ids)
    state["values"] = torch.where(gone, -float("inf"), values)
    state["weights"] = torch.rand(n, device="cuda", generator=g).add_(0.5).mul_(scale)
    return state


# ---------------------------------------------------------------------------------------------------------------
# plain forms: the passes over [N, M] in fp32, what is left for [N, K] in 64 bits, and the row sums of a distillation
# too (a student near its teacher leaves differences below fp32's step)
# ---------------------------------------------------------------------------------------------------------------


def _softmax_state(logits, T, sums):
    """The row's maximum (0 for a row of -inf alone), d = (x - max)/T, exp(d), their sum in the type `sums`."""
    x = logits.float()
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -float("inf"), torch.zeros_like(m), m)
    d = (x - m) / T
    e = d.exp()
    return m, d, e, e.sum(1, keepdim=True, dtype=sums).double()


def _at(logits, m, T, ids):
    """(x - max)/T at some columns of each row."""
    return (logits.gather(1, ids).double() - m.double()) / T


def _top(logits, k):
    """Ids of the k largest of each row: unique integer keys, the value's order above, the lower id first below."""
    x = logits.float() + 0.0
    b = x.view(torch.int32)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    key = key.topk(k, dim=1).values
    return x.shape[1] - 1 - (key & 0xFFFFFFFF)


def _plain_logprobs(s):
    c, logits, tokens, T = s["case"], s["logits"], s["tokens"], s["case"]["temperature"]
    ok = (tokens >= 0) & (tokens < c["vocab"])
    t = torch.where(ok, tokens, 0)[:, None]
    m, d, e, z = _softmax_state(logits, T, torch.float32)
    ls = z.log()
    lp = torch.where(z > 0, _at(logits, m, T, t) - ls, -float("inf"))
    h = torch.where(z > 0, ls - (e * torch.where(e > 0, d, 0.0)).sum(1, keepdim=True) / z, 0.0)
    out = {"logprobs": torch.where(ok, lp[:, 0], 0.0).float(), "entropy": torch.where(ok, h[:, 0], 0.0).float()}
    if c["op"] == "logprobs_train":
        p = e / torch.where(z > 0, z, 1.0).float()
        g1, g2 = (torch.where(ok, s[n], 0.0)[:, None] for n in ("g_logprob", "g_entropy"))
        inner = -g1 - g2 * (torch.where(e > 0, d - ls.float(), 0.0) + h.float())
        out["grad"] = (p * inner).scatter_add_(1, t, g1).div_(T).to(logits.dtype)
        return out
    if c["top"]:
        ids = _top(logits, min(c["top"], c["vocab"]))
        dk = _at(logits, m, T, ids)
        keep = ok[:, None] & (dk > -float("inf"))
        out["top_logprobs"], out["top_ids"] = torch.where(keep, dk - ls, -float("inf")).float(), torch.where(keep, ids, -1)
    return out


def _plain_distil(s):
    c, logits, T = s["case"], s["logits"], s["case"]["temperature"]
    valid = (s["ids"] >= 0) & (s["ids"] < c["vocab"]) & (s["values"] > -float("inf"))
    ids, kept = torch.where(valid, s["ids"], 0), valid.any(1, keepdim=True)
    values = torch.where(valid, s["values"].double(), -float("inf"))
    m, d, e, z = _softmax_state(logits, T, torch.float64)
    ls = z.log()
    if c["rest"]:
        q = values.exp()
        # unlisted columns: marked by their ids, what does not count in a column behind the last
        free = torch.ones(d.shape[0], d.shape[1] + 1, dtype=torch.bool, device=d.device)
        free = free.scatter_(1, torch.where(valid, ids, c["vocab"]), False)[:, :-1]
        dr = torch.where(free, d, -float("inf"))
        mr = dr.amax(1, keepdim=True)
        some = mr > -float("inf")
        mr = torch.where(some, mr, 0.0)
        er = (dr - mr).exp()
        zr = er.sum(1, keepdim=True, dtype=torch.float64)
        logp_r = torch.where(some, zr.log() + mr.double() - ls, 0.0)
        q_r = 1.0 - q.sum(1, keepdim=True)
        q_r = torch.where(some & kept & (q_r >= LEAST_REST), q_r, 0.0)
        logq = torch.where(valid, values, 0.0)
    else:
        y = values / T
        y = y - torch.where(kept, y.amax(1, keepdim=True), 0.0)
        zq = torch.where(kept, y.exp().sum(1, keepdim=True), 1.0)
        q, logq = y.exp() / zq, torch.where(valid, y - zq.log(), 0.0)
        q_r = torch.zeros_like(zq)
    loss = (q * torch.where(q > 0, logq - (_at(logits, m, T, ids) - ls), 0.0)).sum(1, keepdim=True)
    if c["rest"]:
        loss += q_r * (torch.where(q_r > 0, q_r.log(), 0.0) - logp_r)
    out = {"loss": loss[:, 0].float()}
    if c["op"] == "distil":
        return out
    Z = torch.where(kept, q.sum(1, keepdim=True) + q_r, 0.0)
    grad = e * (Z / z).float()
    if c["rest"]:
        grad = torch.where(free, ((Z * logp_r.exp() - q_r) / torch.where(zr > 0, zr, 1.0)).float() * er, grad)
    grad = grad.scatter_add_(1, ids, -q.float()).mul_(s["weights"][:, None] / T)
    out["grad"] = grad.to(logits.dtype)
    return out


# ---------------------------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------------------------


def _own_run(s):
    import lazy_score_matrix_gb300 as tp

    c, T, logits = s["case"], s["case"]["temperature"], s["logits"]
    if c["op"] == "logprobs":
        r = tp.token_logprobs(logits, s["tokens"], temperature=T, top=min(c["top"], c["vocab"]))
        out = {"logprobs": r.logprobs, "entropy": r.entropy}
        if c["top"]:
            out |= {"top_logprobs": r.top_logprobs, "top_ids": r.top_ids}
        return out
    if c["op"] == "logprobs_train":
        x = logits.detach().requires_grad_(True)
        r = tp.token_logprobs(x, s["tokens"], temperature=T)
        grad, = torch.autograd.grad((r.logprobs, r.entropy), x, (s["g_logprob"], s["g_entropy"]))
        return {"logprobs": r.logprobs.detach(), "entropy": r.entropy.detach(), "grad": grad}
    if c["op"] == "distil":
        return {"loss": tp.topk_distillation(logits, s["ids"], s["values"], temperature=T, rest=c["rest"])}
    if c["op"] == "distil_train":
        x = logits.detach().requires_grad_(True)
        loss = tp.topk_distillation(x, s["ids"], s["values"], temperature=T, rest=c["rest"])
        grad, = torch.autograd.grad(loss, x, s["weights"])
        return {"loss": loss.detach(), "grad": grad}
    loss, grad = tp.topk_distillation_grad(logits, s["ids"], s["values"], s["weights"], temperature=T, rest=c["rest"])
    return {"loss": loss, "grad": grad}


def run(state):
    if own:
        return _own_run(state)
    if state["case"]["op"].startswith("logprobs"):
        return _plain_logprobs(state)
    return _plain_distil(state)


# ---------------------------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    T, m, n = case["temperature"], case["vocab"], case["rows"]
    x = s["logits"].double().div_(T)
    lse = torch.logsumexp(x, 1)
    rows = torch.arange(n, device="cuda")
    if case["op"].startswith("logprobs"):
        tok = s["tokens"]
        ok = (tok >= 0) & (tok < m)
        logp = x.sub_(lse[:, None])
        lp = logp[rows, tok.clamp(0, m - 1)]
        plogp = torch.special.xlogy(logp.exp(), logp.exp()) if case.get("masked") else logp.exp().mul_(logp)
        h = -plogp.sum(1)
        out = {"logprobs": torch.where(ok, lp, 0.0), "entropy": torch.where(ok, h, 0.0)}
        if case["op"] == "logprobs_train":
            p = logp.exp()
            g1, g2 = s["g_logprob"].double() * ok, s["g_entropy"].double() * ok
            grad = -(plogp + p * h[:, None]) * g2[:, None] - p * g1[:, None]
            grad[rows[ok], tok[ok]] += g1[ok]
            out["grad"] = grad / T
        elif case["top"]:
            k = min(case["top"], m)
            order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k]
            v = torch.gather(logp, 1, order)
            keep = ok[:, None] & torch.isfinite(v)
            out["top_logprobs"] = torch.where(keep, v, -np.inf)
            out["top_ids"] = torch.where(keep, order, -1)
        return out
    valid = (s["ids"] >= 0) & (s["ids"] < m) & torch.isfinite(s["values"])
    y = s["values"].double()
    r, k = valid.nonzero(as_tuple=True)  # the entries that count, one by one
    v = s["ids"][r, k]
    kept = valid.any(1)
    if case["rest"]:
        logq = y[r, k]
    else:
        logq = (y / T)[r, k] - torch.logsumexp(torch.where(valid, y / T, -np.inf), 1)[r]
    q = logq.exp()
    total = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, r, q)
    loss = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, r, q * (logq - (x[r, v] - lse[r])))
    grad = case["op"] != "distil"
    w = s["weights"].double()
    if not case["rest"]:
        if not grad:
            return {"loss": loss}
        p = x.sub_(lse[:, None]).exp_().mul_(total[:, None])
        p.index_put_((r, v), -q, accumulate=True)
        return {"loss": loss, "grad": p.mul_((w / T)[:, None])}
    q_r = torch.where(kept & (1 - total >= LEAST_REST), 1 - total, 0.0)
    at_list = x[r, v]
    x[r, v] = -np.inf
    R = torch.logsumexp(x, 1)
    q_r = torch.where(torch.isfinite(R), q_r, 0.0)
    p_r = (R - lse).exp()
    loss += torch.where(q_r > 0, q_r * (q_r.clamp(min=1e-300).log() - (R - lse)), 0.0)
    if not grad:
        return {"loss": loss}
    Z = (total + q_r) * kept
    out = (x - torch.where(torch.isfinite(R), R, 0.0)[:, None]).exp_().mul_((Z * p_r - q_r)[:, None])
    out[r, v] = Z[r] * (at_list - lse[r]).exp()
    out.index_put_((r, v), -q, accumulate=True)
    return {"loss": loss, "grad": out.mul_((w / T)[:, None])}
