"""distill_loss on lists at the edge of what the call allows: renormalised lists whose probabilities, or whose sum, pass fp32; mixtures of nearly one side.
Against test_distill_gpu's reference; its tolerances, in which a renormalised log-probability lp - log sum exp is off by
its own rounding and that of lp at its distance from the list's largest, which count as |log p| does."""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_distill_gpu import UNIT, close, data, reference, weights

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("T,V,k,dtype", [(12, 3000, 20, "fp32"), (1300, 3000, 64, "bf16"), (12, 50257, 300, "bf16"), (320, 20011, 64, "fp16"),
                                         (8, 150001, 512, "bf16")])
@pytest.mark.parametrize("offset", [-500.0, -104.0, -90.0, -64.0, -30.0, 0.0, 60.0, 64.0, 95.0, 600.0])
def test_renormalised_lists_of_any_size(T, V, k, dtype, offset):
    """Lists of a distribution's far tail, and of a teacher's unnormalised logits: a constant leaves them as they are."""
    x, y, index, lp, _ = data(T, V, k, dtype, 3)
    lp = (lp + offset).contiguous()
    index[0] = -1  # a list of nothing
    w = weights(y, None, "sum")
    D, logp, grad, dtol, ltol, gtol = reference(x, y, index[:], lp, None, w, "forward", "renormalise", 0.5, 1.0, 0.2, 1.0)
    D[0], grad[0] = 0.0, 0.0
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise", ce_coef=0.2, reduce="sum")
    close(r.token_kl[1:], D[1:], dtol[1:], "token_kl")
    close(r.logp, logp, ltol, "logp")
    close(r.dlogits[1:], grad[1:], (gtol + UNIT[dtype] * grad.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0))[1:], "dlogits")
    assert r.token_kl[0] == 0 and bool(r.dlogits[0].isfinite().all())


def test_renormalised_lists_of_unequal_parts():
    """Entries that lie hundreds apart, in any order and in every warp's part of a list."""
    T, V, k = 40, 9001, 200
    x, y, index, _, _ = data(T, V, k, "fp32", 5, short=False)
    g = torch.Generator(device=DEV).manual_seed(4)
    lp = (torch.rand((T, k), device=DEV, generator=g) * 800 - 400).contiguous()
    lp[1] -= 400
    lp[2] += 500
    lp[3, :100] = -1000.0
    w = weights(y, None, "token")
    far = lp.double() - lp.double().amax(1, keepdim=True)  # the reference's exponentials end at e^709
    D, _, grad, dtol, _, gtol = reference(x, y, index, far, None, w, "forward", "renormalise", 0.5, 1.0, 0.0, 1.0)
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise")
    close(r.token_kl, D, dtol, "token_kl")
    close(r.dlogits, grad, gtol + UNIT["fp32"] * grad.abs(), "dlogits")
    lp[4, 7] = float("inf")
    lp[5, 7] = float("nan")
    y[4] = y[5] = 3
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise")
    assert bool(r.dlogits[4:6].isnan().all()) and bool(r.token_kl[4:6].isnan().all()) and bool(r.dlogits[6:].isfinite().all())


@pytest.mark.parametrize("T,V,k,dtype", [(12, 3000, 20, "fp32"), (12, 50257, 64, "bf16"), (320, 20011, 300, "fp32")])
@pytest.mark.parametrize("mix", [0.2, 0.999, 1 - 1e-5, 1 - 1e-7, 1 - 1e-9, 1 - 2.0 ** -53])
def test_mixtures_of_little_student(mix, T, V, k, dtype):
    """The gradient is of the size of 1 - mix and right relative to that: an entry's c = (1 - mix) q log(q / m) is off by r's own error,
    by 2^-20 of the logarithm and by its q's. A teacher that is sure of its list has log(q / m) = -log(1 - mix) for the rest."""
    x, y, index, lp, rest = data(T, V, k, dtype, 9, short=False)
    rest[0] = -math.inf
    other = 1.0 - mix
    logq = torch.log_softmax(x.double(), 1)
    member = torch.zeros((T, V), dtype=torch.bool, device=DEV).scatter_(1, index, True)
    lqr = torch.logsumexp(logq.masked_fill(member, -math.inf), 1, keepdim=True)
    lq, P = torch.cat([logq.gather(1, index), lqr], 1), torch.cat([lp, rest[:, None]], 1).double()
    p, q, r = P.exp(), lq.exp(), P - lq
    qm = torch.where(r > 0, -(r + torch.log1p(other * torch.expm1(-r))), -torch.log(other + mix * torch.exp(r)))
    qm = torch.where(r.abs() < 0.1, -torch.log1p(mix * torch.expm1(r)), qm)  # so that nothing cancels
    c = other * q * qm
    C = c.sum(1, keepdim=True)
    entry = torch.full((T, V), k, dtype=torch.int64, device=DEV).scatter_(1, index, torch.arange(k, device=DEV).expand(T, k))
    cond, prob = torch.where(member, 1.0, torch.exp(logq - lqr)), logq.exp()
    E = 2.0 ** -22 * (36 + math.log(V)) + 2.0 ** -24 * V / 256
    l = E * (2 + torch.where(P.isfinite(), P, 0.0).abs() + lq.abs())
    ctol = other * q * (l + 2.0 ** -20 * (qm.abs() + 1)) * (1 + qm.abs()) + 2 * E * c.abs()
    w = weights(y, None, "sum")
    got = zg.distill_loss(x, y, index, lp, rest, kind="js", mix=mix, reduce="sum")
    grad = (c.gather(1, entry) * cond - C * prob) * w[:, None]
    gtol = ctol.gather(1, entry) * cond + (ctol.sum(1, keepdim=True) + 2 * E * C.abs()) * prob
    close(got.dlogits, grad, gtol + UNIT[dtype] * grad.abs() + 2.0 ** -110, "dlogits")


@pytest.mark.parametrize("mix", [1e-300, 1e-50, 1e-30, 1e-9, 1e-4, 1 - 1e-4, 1 - 1e-9, 1 - 2.0 ** -53])
def test_mixtures_of_any_size(mix):
    """Also where one side has no probability in an entry: a teacher sure of its list, a student without the rest, a logit of -inf."""
    T, V, k = 12, 3000, 20
    x, y, index, lp, rest = data(T, V, k, "fp32", 9, short=False)
    rest[0] = -math.inf
    only = torch.full((V,), -math.inf, device=DEV)
    only[index[1]] = x[1, index[1]]
    x[1], y[1] = only, index[1, 0]
    x[2, index[2, 3]], y[2] = -math.inf, index[2, 4]
    w = weights(y, None, "sum")
    D, logp, grad, dtol, ltol, gtol = reference(x, y, index, lp, rest, w, "js", "rest", mix, 1.0, 0.0, 1.0)
    r = zg.distill_loss(x, y, index, lp, rest, kind="js", mix=mix, reduce="sum")
    close(r.token_kl, D, dtol, "token_kl")
    close(r.dlogits, grad, gtol + UNIT["fp32"] * grad.abs(), "dlogits")


@pytest.mark.parametrize("mix", [0.1, 0.2, 0.8])
@pytest.mark.parametrize("T,V", [(6, 5000), (6, 50257), (320, 20001)])
def test_mixtures_by_differences(mix, T, V):
    """The gradient of unequal mixtures against central differences of D itself, written here from m = mix p + (1 - mix) q alone."""
    x, y, index, lp, rest = data(T, V, 16, "fp32", 5, short=False)
    w = weights(y, None, "token")
    member = torch.zeros((T, V), dtype=torch.bool, device=DEV).scatter_(1, index, True)
    P = torch.cat([lp, rest[:, None]], 1).double()

    def loss(z):
        logq = torch.log_softmax(z, 1)
        lq = torch.cat([logq.gather(1, index), torch.logsumexp(logq.masked_fill(member, -math.inf), 1, keepdim=True)], 1)
        p, q = P.exp(), lq.exp()
        lm = torch.log(mix * p + (1 - mix) * q)
        return float((w * (mix * p * (P - lm) + (1 - mix) * q * (lq - lm)).sum(1)).sum())

    r = zg.distill_loss(x, y, index, lp, rest, kind="js", mix=mix)
    assert abs(r.loss.item() - loss(x.double())) <= 2.0 ** -18 * (1 + loss(x.double()))
    g = torch.Generator(device=DEV).manual_seed(9)
    d = torch.randn((T, V), device=DEV, generator=g, dtype=torch.float64).scatter_(1, index, 3.0)
    slope = (loss(x.double() + 1e-4 * d) - loss(x.double() - 1e-4 * d)) / 2e-4
    # third derivatives times 1e-8, and gradients off by 2^-18 of themselves
    assert abs(slope - float((r.dlogits.double() * d).sum())) <= 1e-5 * float((r.dlogits.double() * d).abs().sum()) + 1e-7
