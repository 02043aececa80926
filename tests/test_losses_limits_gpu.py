"""Limits of the losses on every way that their kernels take a row: a warp each, one CTA with a small
and with a large slice, a cluster for few rows, a cluster for long rows, and two passes for rows that
no cluster holds. Against the 64-bit formulas and bounds of test_losses_gpu.py.
"""
import ctypes
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_losses_gpu import (DEV, TYPES, UNIT, bound, check, gen, make_logits, make_targets, reference, reference_grad)

pytestmark = pytest.mark.gpu

WAYS = {  # T, V, dtype
    "warp": (1300, 600, "bf16"), "warp fp32": (1300, 517, "fp32"), "small CTA": (160, 20011, "bf16"), "CTA": (160, 50257, "fp16"),
    "cluster of few rows": (14, 50257, "bf16"), "cluster fp32": (14, 50304, "fp32"), "cluster of long rows": (310, 60001, "bf16"),
    "two passes": (310, 131073, "bf16"), "two passes, few rows": (14, 300001, "fp32"),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def policy_with_entropy(x, y, adv, old, coef):
    """zero_policy_loss through the C ABI with an entropy buffer whatever the coefficient."""
    from zero_gradient_reduce_scatter_gb300.losses import KL, REDUCE, Logits, Policy
    from zero_gradient_reduce_scatter_gb300.losses import TYPES as CODES
    T, V = x.shape
    f = lambda *s: torch.full(s, math.nan, device=DEV)  # noqa: E731
    r = dict(loss=f(1), clip=f(1), kl=f(1), logp=f(T), entropy=f(T), dlogits=torch.empty_like(x))
    a = Logits(x.data_ptr(), y.data_ptr(), T, V, x.stride(0), CODES[x.dtype], 1.0)
    p = Policy(adv.data_ptr(), None if old is None else old.data_ptr(), None, None, 0, 0.2, 0.2, 0.0, 0.0, coef, KL["k3"], REDUCE["sum"], 0,
               r["loss"].data_ptr(), r["clip"].data_ptr(), r["kl"].data_ptr(), r["logp"].data_ptr(), r["entropy"].data_ptr(),
               r["dlogits"].data_ptr(), r["dlogits"].stride(0))
    size = zg._lib().zero_policy_workspace(T)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    zg._check(zg._lib().zero_policy_loss(ctypes.byref(a), ctypes.byref(p), ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream),
              "zero_policy_loss")
    return r


@pytest.mark.parametrize("way", WAYS)
def test_entropy_without_a_coefficient(way):
    """An entropy buffer beside entropy_coef = 0 receives the entropies, whichever kernel runs, and
    changes nothing else beyond the bounds."""
    T, V, dtype = WAYS[way]
    x, _ = make_logits(T, V, dtype, 31)
    y = make_targets(T, V, 32)
    adv = torch.randn(T, device=DEV, generator=gen(33))
    logq, lp, _, ent = reference(x, y)
    E = bound(x)
    old = (lp - 0.05).float()
    r = policy_with_entropy(x, y, adv, old, 0.0)
    check(r["entropy"], ent, E * (1 + ent), "entropy")
    check(r["logp"], lp, E, "logp")
    q = zg.policy_loss(x, y, adv, old, reduce="sum")
    # 2 E per unit of the coefficient r A (r below 1.06 here), in the loss and in every gradient entry, of either call
    size = 1.06 * adv.double().abs() * (1 + lp.abs()) * E
    assert abs(float(r["loss"]) - float(q.loss)) <= 4 * float(size.sum()) + 2.0 ** -20 * float(adv.abs().sum())
    g = torch.where(y >= 0, -torch.exp(lp - old.double()) * adv.double(), torch.zeros_like(lp))
    want = reference_grad(logq, y, g, None, ent, 1.0)
    hot = torch.zeros_like(logq).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    tol = (4 * size + 2.0 ** -21 * g.abs())[:, None] * (torch.exp(logq) + hot) + UNIT[dtype] * want.abs() + 2.0 ** -100
    if dtype == "fp16":
        tol = tol + 2.0 ** -25
    for d in (r["dlogits"], q.dlogits):
        assert bool(((d.double() - want).abs() <= tol).all())
