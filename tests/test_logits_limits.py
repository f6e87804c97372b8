"""Stored score rows at the ends of fp32's range: columns masked by the type's lowest value at any temperature, and
upstream gradients far above one. Against the 64-bit forms of _rows_ref.py."""
import math

import pytest
import torch

import lazy_score_matrix_gb300 as tp
from tests import _rows_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEG = float("-inf")


def check_list(row, ids, shares, T, rest, n, w=0.75):
    """One row of scores, n times over, against shares of some of its columns: the loss and both forms' gradients."""
    ids, values = torch.tensor(ids), torch.tensor(shares, dtype=torch.float64).log().mul(1.0 if rest else T).float()
    e = ref.distill(row.double(), ids.tolist(), values.tolist(), T, rest, w)
    big = 2.0 ** 128 * (1 - 2.0 ** -25)  # rounds to infinity in fp32
    want = e["loss"] if e["loss"] < big else math.inf
    # A distance beyond 1e30 is 12u off: its product with the share 1, a lane's four terms 3, the lanes 5, the shares' scale 2, the
    # last product 1.
    tol = e["loss_tol"] + (12 * ref.U * want if math.isfinite(want) and want > 1e30 else 0.0)
    x = row.to(DEV).expand(n, -1).contiguous()
    a = (ids.to(DEV).expand(n, -1), values.to(DEV).expand(n, -1))
    leaf = x.detach().requires_grad_(True)
    loss = tp.topk_distillation(leaf, *a, temperature=T, rest=rest)
    grad, = torch.autograd.grad(loss, leaf, torch.full((n,), w, device=DEV))
    loss2, grad2 = tp.topk_distillation_grad(x, *a, torch.full((n,), w, device=DEV), temperature=T, rest=rest)
    for name, lo, gr in (("autograd", loss.detach(), grad), ("at once", loss2, grad2)):
        assert torch.equal(lo, lo[:1].expand(n)) and torch.equal(gr, gr[:1].expand(n, -1)), name
        ref.close(lo[0], want, tol, what=f"loss ({name})")
        ref.close(gr[0], e["grad"], e["grad_tol"], row.dtype, what=f"gradient ({name})")


SHAPES = [(2, 900), (2, 40000), (1300, 300)]  # a CTA, a cluster and a warp a row
TEMPERATURES = [0.1, 0.5, 0.7, 0.9, 1.0, 2.0]


@pytest.mark.parametrize("n,m", SHAPES)
@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("left", [0.0, 2.0 ** -6, 2.0 ** -4])
def test_unlisted_columns_at_the_lowest_value(n, m, T, dtype, left):
    # the unlisted class has probability 0; with a share it costs that share of the distance
    row = torch.full((m,), torch.finfo(dtype).min, dtype=dtype)
    ids = [3, m // 2, m - 1, -1]
    row[ids[:3]] = torch.tensor([1.0, 2.0, 0.5], dtype=dtype)
    check_list(row, ids, [0.25, 0.5 - left, 0.25, 0.3], T, True, n)
    check_list(row, ids, [0.25, 0.5, 0.25, 0.3], T, False, n)
    row[7] = NEG
    check_list(row, ids, [0.25, 0.5 - left, 0.25, 0.3], T, True, n)


@pytest.mark.parametrize("n,m", SHAPES)
@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_listed_columns_at_the_lowest_value(n, m, T, dtype):
    row = (torch.randn(m, generator=torch.Generator().manual_seed(m)) * 2).to(dtype)
    ids = [5, m // 3, m - 2, m - 1]
    row[ids[:3]] = torch.finfo(dtype).min
    row[ids[3]] = 1.5
    check_list(row, ids[:3], [0.01, 0.02, 0.005], T, True, n)      # all of the list
    check_list(row, ids, [0.01, 0.02, 0.005, 0.7], T, True, n)     # but one
    check_list(row, ids, [0.01, 0.02, 0.005, 0.965], T, False, n)
    if T != 1.0:  # at T = 1 the sum of the shares' roundings decides between the largest value and infinity
        check_list(row, ids[:3], [0.25, 0.5, 0.25], T, False, n)
    row[ids[1]] = NEG
    check_list(row, ids, [0.01, 0.02, 0.005, 0.7], T, True, n)
    row[:] = torch.finfo(dtype).min  # the lowest value throughout: uniform
    check_list(row, ids, [0.1, 0.2, 0.05, 0.5], T, True, n)
    check_list(row, ids, [0.1, 0.2, 0.2, 0.5], T, False, n)


@pytest.mark.parametrize("T", [0.5, 0.9, 1.0, 3.0])
def test_a_distance_beyond_the_range(T):
    # the difference of two scores leaves fp32's range itself: shares small enough bring the loss back into it
    m = 700
    row = torch.full((m,), -3e38)
    row[9] = 3e38
    check_list(row, [9, 20], [0.9, 0.01], T, True, 2)
    check_list(row, [20, 9], [0.01, 0.99], T, False, 2)


@pytest.mark.parametrize("n,m", SHAPES)
@pytest.mark.parametrize("T", [0.5, 0.9, 1.0, 3.0])
def test_log_probabilities_beyond_the_range_of_a_difference(n, m, T):
    row = torch.full((m,), -3e38)
    row[9], row[20], row[21] = 3e38, -1e38, NEG
    tokens = torch.tensor([9, 20, 5, 21], device=DEV).repeat(n)[:n]
    r = tp.token_logprobs(row.to(DEV).expand(n, m).contiguous(), tokens, temperature=T, top=7)
    big = 2.0 ** 128 * (1 - 2.0 ** -25)
    for i in range(min(n, 4)):
        w = ref.logprobs(row.double(), int(tokens[i]), T, 7)
        out = lambda v: NEG if v <= -big else v  # noqa: E731
        ref.close(r.logprobs[i], out(w["lp"]), w["lp_tol"])
        ref.close(r.top_logprobs[i], [out(v) for v in w["top_lp"]], w["top_tol"])
        assert r.top_ids[i].tolist() == w["top_ids"] and r.entropy[i] == 0


@pytest.mark.parametrize("rest", [False, True])
def test_infinite_and_nan_scores_still_show(rest):
    x = torch.full((4, 600), torch.finfo(torch.float32).min, device=DEV)
    x[:, :3] = 1.0
    x[0, 300] = float("inf")
    x[1, 1] = float("inf")
    x[2, 300] = float("nan")
    ids = torch.tensor([[0, 1, 2]], device=DEV).expand(4, 3)
    values = torch.tensor([[0.3, 0.3, 0.3]], device=DEV).log().expand(4, 3)
    for loss in (tp.topk_distillation(x, ids, values, temperature=0.7, rest=rest),
                 tp.topk_distillation_grad(x, ids, values, temperature=0.7, rest=rest)[0]):
        assert loss.isnan().tolist() == [True, True, True, False]


@pytest.mark.parametrize("n,m", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,g_h", [(1e-3, 5e5), (1.0, 1e9), (0.5, -1e20), (2.0, 3e30)])
def test_masked_columns_under_a_large_entropy_gradient(n, m, dtype, T, g_h):
    g = torch.Generator().manual_seed(m)
    row = (torch.randn(m, generator=g) * 2 * T).to(dtype)
    row[::3] = NEG
    row[1::3] = torch.finfo(dtype).min
    token = 2
    leaf = row.to(DEV).expand(n, -1).contiguous().requires_grad_(True)
    r = tp.token_logprobs(leaf, torch.full((n,), token, device=DEV), temperature=T)
    grad, = torch.autograd.grad((r.logprobs, r.entropy), leaf, (torch.full((n,), 1.5, device=DEV), torch.full((n,), g_h, device=DEV)))
    w = ref.logprobs(row.double(), token, T, 0, 1.5, g_h)
    if float(w["grad"].abs().max()) < torch.finfo(dtype).max:
        ref.close(grad[0], w["grad"], w["grad_tol"], dtype)
    assert torch.equal(grad, grad[:1].expand(n, -1))
    masked = torch.ones(m, dtype=torch.bool)
    masked[2::3] = False
    assert int(torch.count_nonzero(grad[0].cpu()[masked])) == 0
