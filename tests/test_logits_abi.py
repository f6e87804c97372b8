"""The C entries of include/tp_logits.h on the CPU: exported, and every invalid call refused before anything is
launched (the fake device addresses are never touched); the 64-bit forms the GPU tests compare with, pinned to
torch's own log_softmax and autograd."""
import ctypes
import subprocess

import pytest
import torch

from lazy_score_matrix_gb300 import _lib
from lazy_score_matrix_gb300 import build as tpbuild
from tests import _rows_ref as ref

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced
TOK, OUT, ENT, STATS, TOPV, TOPI, GRAD = (FAKE + (i << 32) for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    tpbuild.build()
    return _lib.load()


def rows(N=6, M=100, dtype=0, group=None, rs=None, gs=0, data=FAKE):
    return _lib.tp_rows(dtype, N, M, N if group is None else group, M if rs is None else rs, gs, data)


def test_exports_every_logits_symbol(lib):
    declared = _lib.header_symbols(_lib.LOGITS_HEADER)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(declared) == set(_lib.LOGITS_SIGNATURES) and set(declared) <= exported


def logprobs(lib, x=None, tok=TOK, T=1.0, top=0, lp=OUT, h=ENT, st=None, tv=None, ti=None):
    return lib.tp_token_logprobs(x if x is not None else rows(), tok, T, top, lp, h, st, tv, ti, None)


def logprobs_bwd(lib, x=None, tok=TOK, T=1.0, st=STATS, g1=OUT, g2=ENT, g=None):
    return lib.tp_token_logprobs_backward(x if x is not None else rows(), tok, T, st, g1, g2, g if g is not None else rows(data=GRAD), None)


def distill(lib, x=None, K=4, ids=TOK, val=TOPV, T=1.0, rest=0, loss=OUT, st=None):
    return lib.tp_topk_distillation(x if x is not None else rows(), K, ids, val, T, rest, loss, st, None)


def distill_grad(lib, x=None, K=4, ids=TOK, val=TOPV, w=None, T=1.0, rest=0, loss=OUT, st=STATS, g=None):
    return lib.tp_topk_distillation_grad(x if x is not None else rows(), K, ids, val, w, T, rest, loss, st,
                                         g if g is not None else rows(data=GRAD), None)


BAD = {
    "rows NULL data": lambda l: logprobs(l, rows(data=None)),
    "rows dtype": lambda l: logprobs(l, rows(dtype=3)),
    "rows N 0": lambda l: logprobs(l, rows(N=0, group=1)),
    "rows M 0": lambda l: logprobs(l, rows(M=0)),
    "rows N too large": lambda l: logprobs(l, rows(N=1 << 31)),
    "rows M too large": lambda l: logprobs(l, rows(M=1 << 31)),
    "rows group 0": lambda l: logprobs(l, rows(group=0)),
    "rows group not a divisor": lambda l: logprobs(l, rows(N=6, group=4)),
    "rows negative stride": lambda l: logprobs(l, rows(rs=-1)),
    "rows negative group stride": lambda l: logprobs(l, rows(group=3, gs=-5)),
    "rows stride beyond 64 bits": lambda l: logprobs(l, rows(rs=1 << 60)),
    "rows unaligned": lambda l: logprobs(l, rows(data=FAKE + 2)),
    "rows unaligned half": lambda l: logprobs(l, rows(dtype=1, data=FAKE + 1)),
    "tokens unaligned": lambda l: logprobs(l, tok=TOK + 4),
    "logprobs missing": lambda l: logprobs(l, lp=None),
    "logprobs without tokens": lambda l: logprobs(l, tok=None),
    "entropy missing": lambda l: logprobs(l, h=None),
    "temperature 0": lambda l: logprobs(l, T=0.0),
    "temperature negative": lambda l: logprobs(l, T=-1.0),
    "temperature NaN": lambda l: logprobs(l, T=float("nan")),
    "temperature too large": lambda l: logprobs(l, T=1e4),
    "top negative": lambda l: logprobs(l, top=-1, tv=TOPV, ti=TOPI),
    "top above 128": lambda l: logprobs(l, rows(M=1000), top=129, tv=TOPV, ti=TOPI),
    "top above M": lambda l: logprobs(l, top=101, tv=TOPV, ti=TOPI),
    "top ids missing": lambda l: logprobs(l, top=3, tv=TOPV),
    "top values missing": lambda l: logprobs(l, top=3, ti=TOPI),
    "top arrays without top": lambda l: logprobs(l, tv=TOPV, ti=TOPI),
    "output on the logits": lambda l: logprobs(l, lp=FAKE + 8),
    "outputs on each other": lambda l: logprobs(l, lp=OUT, h=OUT + 4),
    "output on the tokens": lambda l: logprobs(l, h=TOK + 8),
    "stats on the entropy": lambda l: logprobs(l, st=ENT + 20),
    "backward stats missing": lambda l: logprobs_bwd(l, st=None),
    "backward no upstream": lambda l: logprobs_bwd(l, g1=None, g2=None),
    "backward upstream without tokens": lambda l: logprobs_bwd(l, tok=None),
    "backward grad dtype": lambda l: logprobs_bwd(l, g=rows(dtype=2, data=GRAD)),
    "backward grad N": lambda l: logprobs_bwd(l, g=rows(N=5, data=GRAD)),
    "backward grad M": lambda l: logprobs_bwd(l, g=rows(M=99, data=GRAD)),
    "backward grad rows overlap": lambda l: logprobs_bwd(l, g=rows(rs=99, data=GRAD)),
    "backward grad rows expanded": lambda l: logprobs_bwd(l, g=rows(rs=0, data=GRAD)),
    "backward grad groups overlap": lambda l: logprobs_bwd(l, g=rows(group=3, gs=250, data=GRAD)),
    "backward grad shifted on the logits": lambda l: logprobs_bwd(l, g=rows(data=FAKE + 400)),
    "backward grad on the stats": lambda l: logprobs_bwd(l, g=rows(data=STATS)),
    "distillation K 0": lambda l: distill(l, K=0),
    "distillation K 129": lambda l: distill(l, K=129),
    "distillation ids missing": lambda l: distill(l, ids=None),
    "distillation values missing": lambda l: distill(l, val=None),
    "distillation rest": lambda l: distill(l, rest=2),
    "distillation loss missing": lambda l: distill(l, loss=None),
    "distillation temperature": lambda l: distill(l, T=float("inf")),
    "distillation loss on the values": lambda l: distill(l, loss=TOPV),
    "at once stats missing": lambda l: distill_grad(l, st=None),
    "at once loss on the grad": lambda l: distill_grad(l, loss=GRAD + 16),
    "at once loss on the logits": lambda l: distill_grad(l, loss=FAKE + 16),
    "at once grad on the weights": lambda l: distill_grad(l, w=GRAD + 64),
    "at once grad partly on the logits": lambda l: distill_grad(l, g=rows(data=FAKE + 1200)),
    "at once logits, other stride": lambda l: distill_grad(l, rows(rs=120), g=rows()),
}


@pytest.mark.parametrize("case", BAD)
def test_invalid_calls_are_refused(lib, case):
    _lib.launch_count(reset=True)
    assert BAD[case](lib) == _lib.TP_ERR_INVALID_ARG
    assert lib.tp_last_error() and _lib.launch_count() == 0


def test_fault_injection(lib, monkeypatch):
    calls = {"token_logprobs": lambda: logprobs(lib), "token_logprobs_backward": lambda: logprobs_bwd(lib), "topk_distillation": lambda: distill(lib),
             "topk_distillation_backward": lambda: lib.tp_topk_distillation_backward(rows(), 4, TOK, TOPV, 1.0, 0, STATS, OUT, rows(data=GRAD), None),
             "topk_distillation_grad": lambda: distill_grad(lib)}
    _lib.launch_count(reset=True)
    for name, call in calls.items():
        monkeypatch.setenv("TP_FAULT_INJECT", name)
        assert call() == _lib.TP_ERR_CUDA, name
        assert b"fault injected" in lib.tp_last_error()
    # valid forms of the layouts: in place, interleaved groups, one row, a group stride that is not read
    monkeypatch.setenv("TP_FAULT_INJECT", "topk_distillation_grad")
    for x, g in ((rows(), rows()), (rows(group=2, rs=300, gs=100), rows(group=2, rs=300, gs=100, data=GRAD)), (rows(N=1, rs=0), rows(N=1, rs=0, data=GRAD)),
                 (rows(gs=5), rows(gs=7)), (rows(rs=0), rows(data=GRAD))):
        assert distill_grad(lib, x, g=g) == _lib.TP_ERR_CUDA
    assert _lib.launch_count() == 0


def test_row_strides(lib):
    x = torch.empty(4, 6, 10)
    for view, want in ((x, (24, 10, 0)), (x[:, :-1], (5, 10, 60)), (x.transpose(0, 1), (4, 60, 10)), (x[:, :, :7], (24, 10, 0)),
                       (x[0, 0], (1, 10, 0)), (x[:1, 2:3], (1, 10, 0)), (x[..., ::2], None), (torch.empty(2, 3, 4, 5)[:, :2, :3], None),
                       (torch.empty(3, 1).t().expand(7, 3), (7, 0, 0))):
        got = _lib.logits_binding().row_strides(view)
        assert (tuple(got) if got else None) == want, (tuple(view.shape), view.stride())
        if want:  # every row where the strides say
            flat = view.reshape(-1, view.shape[-1])
            off = torch.arange(view.untyped_storage().size() // 4).as_strided(view.shape, view.stride(), view.storage_offset()).reshape(flat.shape)
            for i in range(flat.shape[0]):
                assert off[i, 0] - view.storage_offset() == (i // want[0]) * want[2] + (i % want[0]) * want[1]


@pytest.mark.parametrize("seed", range(6))
def test_plain_forms_agree_with_autograd(seed):
    g = torch.Generator().manual_seed(seed)
    m, T = 30 + seed, 0.6 + 0.3 * seed
    x = (torch.randn(m, generator=g, dtype=torch.float64) * 2).requires_grad_(True)
    logp = torch.log_softmax(x / T, 0)
    H = -(logp.exp() * logp).sum()
    want, = torch.autograd.grad(0.7 * logp[3] - 1.3 * H, x)
    w = ref.logprobs(x.detach(), 3, T, 4, 0.7, -1.3)
    assert abs(w["lp"] - float(logp[3].detach())) < 1e-12 and abs(w["h"] - float(H.detach())) < 1e-12
    assert (w["grad"] - want).abs().max() < 1e-12
    assert w["top_ids"] == torch.topk(x.detach(), 4).indices.tolist()
    ids = torch.tensor([5, 1, 9, 5])
    y = torch.randn(4, generator=g, dtype=torch.float64) - 3.0
    logp = torch.log_softmax(x / T, 0)
    q = torch.softmax(y / T, 0)
    loss = (q * (q.log() - logp[ids])).sum()
    want, = torch.autograd.grad(2.0 * loss, x)
    d = ref.distill(x.detach(), ids.tolist(), y.tolist(), T, False, 2.0)
    assert abs(d["loss"] - float(loss.detach())) < 1e-12 and (d["grad"] - want).abs().max() < 1e-12
    logp = torch.log_softmax(x / T, 0)
    others = torch.ones(m, dtype=torch.bool)
    others[ids] = False
    q, q_r = y.exp(), 1 - y.exp().sum()
    loss = (q * (y - logp[ids])).sum() + q_r * (q_r.log() - torch.logsumexp(logp[others], 0))
    want, = torch.autograd.grad(loss, x)
    d = ref.distill(x.detach(), ids.tolist(), y.tolist(), T, True)
    assert abs(d["loss"] - float(loss.detach())) < 1e-12 and (d["grad"] - want).abs().max() < 1e-12


def test_two_word_tables_are_right():
    """The tables of csrc_logits/tp_logits_two.cuh, recomputed in 60-digit decimal arithmetic: 2^(j/32) and -ln c as
    the nearest float and the nearest float to what is left, c the multiple of 2^-9 nearest to 1/(1 + (i + 1/2)/32);
    the words of ln 2 and ln2/32 sum to them."""
    import os
    import re
    import struct
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    src = open(os.path.join(_lib.PKG, "csrc_logits", "tp_logits_two.cuh")).read()
    number = r"-?0x[0-9a-f.]+p[+-]\d+|0\.f|0x0\.0p[+-]\d+"

    def table(name):
        body = src[src.index(name):]
        body = body[body.index("= {") + 3:body.index("};")]
        return [[float.fromhex(v.rstrip("f")) if "x" in v else 0.0 for v in re.findall(number, row)] for row in re.findall(r"\{([^{}]*)\}", body)]

    f32 = lambda v: struct.unpack("f", struct.pack("f", float(v)))[0]  # noqa: E731
    ln2 = Decimal(2).ln()
    exps, lns = table("kExpTab[32]"), table("kLnTab[32]")
    assert len(exps) == len(lns) == 32
    for j, (h, lo) in enumerate(exps):
        want = Decimal(2) ** (Decimal(j) / 32)
        assert h == f32(want) and lo == f32(want - Decimal(h)), j
    for i, (c, h, lo) in enumerate(r[:3] for r in lns):
        mid = 1 + (Decimal(i) + Decimal("0.5")) / 32
        assert Decimal(c) * 512 == (512 / mid).to_integral_value() and abs(Decimal(c) * mid - 1) < Decimal(1) / 500, i
        want = -Decimal(c).ln()
        assert h == f32(want) and lo == f32(want - Decimal(h)), i
    words = lambda names: [Decimal(float.fromhex(re.search(n + r" = (" + number + ")", src).group(1).rstrip("f"))) for n in names]  # noqa: E731
    l1, l2, l3 = words(["kL1", "kL2", "kL3"])
    assert abs(l1 + l2 + l3 - ln2 / 32) < Decimal(2) ** -52 and l1 * 2 ** 17 % 1 == 0 and l2 * 2 ** 28 % 1 == 0
    hi, lo = words(["kLn2Hi", "kLn2Lo"])
    assert abs(hi + lo - ln2) < Decimal(2) ** -38 and hi * 2 ** 14 % 1 == 0
