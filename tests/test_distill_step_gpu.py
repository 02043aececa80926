"""A teacher's lists, the student's loss, the embedding's gradient on the tied matrix, clipping and the ZeRO step
together: the distillation of the post-training example, and its gradients against autograd through the same
loss written in torch."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def test_distillation_runs():
    import post_training_step as ex
    log = ex.train("distill", 8)
    assert len(log) == 8 and all(math.isfinite(a) and math.isfinite(b) and b > 0 for a, b, _ in log)


def test_gradients_reach_the_parameters():
    """Every parameter's gradient against autograd through the divergence in torch, from the same bf16 logits.
    Both round dlogits (2^-8 of each entry), the products behind it are the same kernels, and the tied matrix'
    gradient is a sum of two numbers, rounded once here and three times by autograd: 2^-6 of the norm."""
    import post_training_step as ex
    import zero_gradient_reduce_scatter_gb300 as zg
    g = torch.Generator(device="cuda").manual_seed(3)
    model, teacher = ex.Model(g), ex.Model(g)
    for p in model.params:
        p.grad = torch.zeros_like(p)
    tokens, targets, offsets = ex.batch(g)
    r = ex.distill(model, teacher, tokens, targets, offsets, ce_coef=0.3)

    logits = (model.hidden(tokens) @ model.params[0].T).float()
    with torch.no_grad():
        top = zg.top_logits(teacher.hidden(tokens) @ teacher.params[0].T, 16)
    live = targets >= 0
    logq = torch.log_softmax(logits, 1)
    lq = logq.gather(1, top.index)
    p = top.logp.exp()
    outside = torch.zeros_like(logits).scatter(1, top.index, 1.0)
    rest = torch.logsumexp(logq.masked_fill(outside > 0, -math.inf), 1)
    kl = (p * (top.logp - lq)).sum(1) + top.rest.exp() * (top.rest - rest)
    loss = ((kl - 0.3 * logq.gather(1, targets.clamp(min=0)[:, None])[:, 0]) * live).sum() / live.sum()
    want = torch.autograd.grad(loss, model.params)
    assert abs(loss.item() - r.loss.item()) <= 1e-5 * loss.item()
    for a, b in zip(model.params, want):
        assert float((a.grad - b).float().norm()) <= 2.0 ** -6 * float(b.float().norm())


def test_one_stream_of_calls_in_a_graph():
    """The calls of a step captured together and replayed with new contents, against the same calls one by one."""
    import zero_gradient_reduce_scatter_gb300 as zg
    g = torch.Generator(device="cuda").manual_seed(4)
    T, V, D, k = 300, 5003, 48, 32
    tokens = torch.randint(0, V, (T,), device="cuda", generator=g)
    wte = torch.randn((V, D), device="cuda", generator=g).bfloat16()
    z = torch.randn((T, V), device="cuda", generator=g)

    def step():
        top = zg.top_logits(z, k)
        rows = zg.embedding(wte, tokens, scale=2.0)
        logits = rows @ wte.T
        r = zg.distill_loss(logits, tokens, top.index, top.logp, top.rest, kind="js")
        grad = zg.embedding_backward(tokens, r.dlogits @ wte, V, scale=2.0)
        flat = torch.empty_like(grad)
        return r.loss, grad, zg.GradClip([grad], [flat]), flat

    loss, grad, plan, flat = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        top = zg.top_logits(z, k)
        rows = zg.embedding(wte, tokens, scale=2.0)
        r = zg.distill_loss(rows @ wte.T, tokens, top.index, top.logp, top.rest, kind="js")
        zg.embedding_backward(tokens, r.dlogits @ wte, V, scale=2.0, out=grad)
        norm = plan.clip(1e-3)
    for seed in (5, 6):
        h = torch.Generator(device="cuda").manual_seed(seed)
        z.copy_(torch.randn((T, V), device="cuda", generator=h))
        tokens.copy_(torch.randint(0, V, (T,), device="cuda", generator=h))
        graph.replay()
        held = [x.clone() for x in (r.loss, grad, norm.norm, flat)]
        loss2, grad2, plan2, flat2 = step()
        c = plan2.clip(1e-3)
        for a, b in zip(held, (loss2, grad2, c.norm, flat2)):
            assert torch.equal(a, b)
