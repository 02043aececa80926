"""distill_loss without a teacher's rest: p_rest = max(1 - sum p, 2^-24) of lists that hold nearly all of the teacher,
against a student that has most of its probability elsewhere.

Tolerances: test_distill_gpu's with p_rest given in 64 bits, and p_rest's own error beside them. The sum is formed in whole
numbers of 2^-48 from exponentials off by at most 2^-39 of themselves (together at most 1) and a unit each (513 of them,
2^-39): 2^-38 in all, divided by p_rest relative to it, rho. An entry with
p (1 + rho) moves D by at most (p + q) rho (1 + |r|), its own derivative c by the same, and so the sum C of all."""
import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_distill_gpu import TYPES, UNIT, close, reference, weights

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def lists(T, V, k, rests, seed):
    """Places, and log-probabilities in fp32 that leave about rests[t]."""
    index = torch.stack([torch.randperm(V, device=DEV, generator=gen(seed + i))[:k] for i in range(min(T, 40))])
    index = index.repeat((T + len(index) - 1) // len(index), 1)[:T].contiguous()
    z = torch.randn((T, k), device=DEV, generator=gen(seed), dtype=torch.float64) * 2
    lp = torch.log_softmax(z, 1) + torch.log1p(-rests)[:, None]
    return index, lp.float().contiguous()


@pytest.mark.parametrize("T,V,k,dtype", [(12, 3000, 64, "fp32"), (1300, 3000, 64, "bf16"), (12, 50257, 300, "bf16"), (400, 20011, 64, "fp16"),
                                         (320, 50257, 5, "bf16"), (12, 150001, 512, "bf16"), (40, 40, 32, "fp32"), (340, 9001, 512, "fp32")])
@pytest.mark.parametrize("kind", ["forward", "reverse", "js"])
def test_rests_of_little_probability(T, V, k, dtype, kind):
    rests = torch.tensor([1e-2, 1e-3, 1e-4, 1e-5, 3e-6, 1e-6, 7e-7, 5e-7, 3e-7, 2e-7, 1e-7, 0.0], dtype=torch.float64, device=DEV)
    rests = rests.repeat(T // 12 + 1)[:T]
    index, lp = lists(T, V, k, rests, 3)
    x = torch.randn((T, V), device=DEV, generator=gen(5)).to(TYPES[dtype])
    y = index[:, 0].contiguous()
    left = 1.0 - torch.exp(lp.double()).sum(1)
    pr = torch.log(left.clamp(min=2.0 ** -24))
    assert T < 12 or bool((left < 2.0 ** -24).any()) and bool((left > 2.0 ** -24).any())
    w = weights(y, None, "sum")
    for ce_coef, temperature in ((0.0, 1.0), (0.3, 2.0)):
        D, logp, grad, dtol, ltol, gtol = reference(x, y, index, lp, pr, w, kind, "rest", 0.5, 1.0, ce_coef, temperature)
        r = zg.distill_loss(x, y, index, lp, None, kind=kind, ce_coef=ce_coef, reduce="sum", temperature=temperature)
        logq = torch.log_softmax(x.double() / temperature, 1)
        member = torch.zeros_like(logq, dtype=torch.bool).scatter_(1, index, True)
        lqr = torch.logsumexp(logq.masked_fill(member, -torch.inf), 1)
        p, q, ratio = pr.exp(), lqr.exp(), (pr - lqr).abs()
        moved = (p + q) * 2.0 ** -38 / p * (1 + ratio)
        close(r.token_kl, D, dtol + moved, "token_kl")
        close(r.logp, logp, ltol, "logp")
        cond = torch.where(member, 0.0, torch.exp(logq - lqr[:, None]))
        gtol = gtol + moved[:, None] * (cond + logq.exp()) / temperature
        close(r.dlogits, grad, gtol + UNIT[dtype] * grad.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0), "dlogits")
