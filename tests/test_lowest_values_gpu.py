"""Logits masked with their type's lowest value at temperatures below 1, where their distance from the row's largest
logit passes fp32: their log-probabilities are -inf as token_logp's, never NaN. Against 64-bit formulas, rounded to
fp32 (so that what passes fp32 is -inf there too); tolerances as in test_top_gpu.py and test_distill_gpu.py."""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_distill_gpu import UNIT, close, data, reference, weights

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(T, V, dtype, live):
    """A few ordinary logits to a row, at places of their own, among the lowest value; the last row has nothing else."""
    x = torch.full((T, V), torch.finfo(dtype).min, device=DEV, dtype=dtype)
    at = torch.stack([torch.randperm(V, device=DEV, generator=gen(i))[:live] for i in range(T)])
    x.scatter_(1, at, (torch.randn((T, live), device=DEV, generator=gen(77)) * 3 + 5).to(dtype))
    if T > 1:
        x[-1] = torch.finfo(dtype).min
    return x


@pytest.mark.parametrize("temperature", [0.5, 0.7, 2.0 ** -20, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,live,k", [(3, 50257, 5, 64), (2, 50257, 70, 64), (1300, 3001, 3, 30), (9, 300, 20, 100), (3, 20011, 10, 400),
                                        (2, 700, 1, 1)])
def test_lists(T, V, live, k, dtype, temperature):
    x = rows(T, V, TYPES[dtype], live)
    got = zg.top_logits(x, k, temperature=temperature)
    z = x.double() / temperature
    v, at = torch.sort(z, dim=1, descending=True, stable=True)
    total = torch.log(torch.exp(v - v[:, :1]).sum(1, keepdim=True))
    logp = (v[:, :k] - v[:, :1]) - total
    rest = (v[:, k:k + 1] - v[:, :1])[:, 0] + torch.log(torch.exp(v[:, k:] - v[:, k:k + 1]).sum(1)) - total[:, 0]
    R = torch.clamp(z.amax(1) - z.amin(1), max=28.0) + math.log(V)
    E = 2.0 ** -22 * (8 + R) + 2.0 ** -24 * V / 128
    assert torch.equal(got.index, at[:, :k])
    for what, a, b, tol in (("logp", got.logp, logp, E[:, None]), ("lse", got.lse, (v[:, :1] + total)[:, 0], E), ("rest", got.rest, rest, E)):
        b = b.float().double()
        close(a, b, tol * (1 + b.abs().nan_to_num(posinf=0)), what)
    # what token_logp says of the same places
    for i in (0, k // 2, k - 1):
        want = zg.token_logp(x, got.index[:, i].contiguous(), temperature=temperature).logp
        close(got.logp[:, i], want.double(), E * (1 + want.double().abs().nan_to_num(posinf=0)), "token_logp")


@pytest.mark.parametrize("temperature", [0.5, 0.7])
@pytest.mark.parametrize("V,T,dtype", [(3000, 6, "bf16"), (50257, 6, "fp32"), (50257, 320, "bf16"), (150000, 6, "bf16"), (3000, 1300, "fp16")])
def test_distillation(V, T, dtype, temperature):
    x, y, index, lp, rest = data(T, V, 12, dtype, 3, masked=0.0, short=False)
    low = torch.finfo(x.dtype).min
    x[0, V - V // 50:] = low       # a padded vocabulary; its target is a masked place
    y[0] = V - 1
    x[1].scatter_(0, index[1, 3:5], low)  # in the list, the target among them
    y[1] = index[1, 3]
    only = torch.full((V,), low, device=DEV, dtype=x.dtype)
    only[index[2]] = x[2, index[2]]  # all of the rest
    x[2], y[2] = only, index[2, 1]
    for kind in ("reverse", "js"):
        for ce_coef in (0.0, 0.25):
            w = weights(y, None, "sum")
            D, logp, grad, dtol, ltol, gtol = reference(x, y, index, lp, rest, w, kind, "rest", 0.5, 1.0, ce_coef, temperature)
            r = zg.distill_loss(x, y, index, lp, rest, kind=kind, ce_coef=ce_coef, reduce="sum", temperature=temperature)
            lf = logp.float().double()
            close(r.logp, lf, ltol.nan_to_num(posinf=0), "logp")
            close(r.token_kl, D, dtol, "token_kl")
            close(r.dlogits, grad, gtol + UNIT[dtype] * grad.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0), "dlogits")
            want = (w * (D - (ce_coef * lf if ce_coef else 0.0))).sum()
            assert not r.loss.isnan() and (r.loss == want if not want.isfinite() else
                                           abs(r.loss.double() - want) <= (w * (dtol + ce_coef * ltol)).sum() + 2.0 ** -22 * (D + lf.abs()).sum())


def test_a_list_of_masked_places_reaches_the_loss():
    """A teacher's list longer than its unmasked places, handed on as it is: its masked entries are not there."""
    V, k = 5000, 30
    teacher = rows(4, V, torch.bfloat16, 7)[:3]
    top = zg.top_logits(teacher, k, temperature=0.5)
    assert bool((top.logp[:, 7:] == -math.inf).all()) and bool(top.logp[:, :7].isfinite().all()) and bool((top.rest == -math.inf).all())
    x = torch.randn((3, V), device=DEV, generator=gen(3))
    y = top.index[:, 0].contiguous()
    r = zg.distill_loss(x, y, top.index, top.logp, top.rest, temperature=0.5)
    w = weights(y, None, "token")
    D, _, grad, dtol, _, gtol = reference(x, y, top.index, top.logp, top.rest, w, "forward", "rest", 0.5, 1.0, 0.0, 0.5)
    close(r.token_kl, D, dtol, "token_kl")
    close(r.dlogits, grad, gtol + UNIT["fp32"] * grad.abs(), "dlogits")
