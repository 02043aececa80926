"""The README's distillation snippet, run as written (its placeholders filled in), against autograd through the
same loss written in torch."""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


class Net:
    def __init__(self, w):
        self.w = w

    def states(self, rows):
        return torch.tanh(rows @ self.w)


def test_readme_distillation():
    """Everything in fp32: what autograd adds up in another order agrees to 2^-16 of the gradients' norms (a
    few hundred additions and products, each off by 2^-24)."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, V, D = 60, 803, 32
    wte = (torch.randn((V, D), device=DEV, generator=g) / 8).requires_grad_()
    wte.grad = torch.zeros_like(wte)
    model = Net((torch.randn((D, D), device=DEV, generator=g) / 16).requires_grad_())
    teacher_logits = torch.randn((T, V), device=DEV, generator=g) * 2
    tokens = torch.randint(0, V, (T,), device=DEV, generator=g)
    tokens[7:12] = tokens[0]
    targets = tokens.roll(-1).clone()
    targets[::6] = -1
    offsets = torch.tensor([0, 10, 30, 60], device=DEV)

    with torch.no_grad():
        top = zg.top_logits(teacher_logits, 64, targets, temperature=2.0)  # lists; masked rows are not read
    rows = zg.embedding(wte.detach(), tokens, scale=wte.shape[1] ** 0.5).requires_grad_()
    logits = model.states(rows) @ wte.T
    r = zg.distill_loss(logits.detach(), targets, top.index, top.logp, top.rest, offsets=offsets,
                        kind="forward", ce_coef=0.1, reduce="sequence", temperature=2.0)
    logits.backward(r.dlogits)                                         # wte.grad: the output product's part
    zg.embedding_backward(tokens, rows.grad, wte.shape[0], scale=wte.shape[1] ** 0.5,
                          out=wte.grad, accumulate=True)               # and the embedding's

    live = targets >= 0
    w = torch.zeros(T, device=DEV)
    for a, b in ((0, 10), (10, 30), (30, 60)):
        w[a:b] = live[a:b] / live[a:b].sum() / 3
    logq = torch.log_softmax(model.states(wte[tokens] * D ** 0.5) @ wte.T / 2.0, 1)
    logp = torch.log_softmax(teacher_logits / 2.0, 1)
    at = torch.topk(teacher_logits, 64, dim=1).indices
    mask = torch.zeros_like(logq, dtype=torch.bool).scatter_(1, at, True)
    p, q = logp.gather(1, at), logq.gather(1, at)
    pr, qr = (torch.logsumexp(v.masked_fill(mask, -math.inf), 1) for v in (logp, logq))
    kl = (p.exp() * (p - q)).sum(1) + pr.exp() * (pr - qr)
    loss = (w * (kl - 0.1 * logq.gather(1, targets.clamp(min=0)[:, None])[:, 0])).sum()
    want = torch.autograd.grad(loss, [wte, model.w])
    assert abs(loss.item() - r.loss.item()) <= 1e-5 * loss.item()
    for a, b in zip((wte.grad, model.w.grad), want):
        assert float((a - b).norm()) <= 2.0 ** -16 * float(b.norm())
