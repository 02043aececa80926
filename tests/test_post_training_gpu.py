"""The post-training example: reference log-probabilities, loss, gradients, clipping and the ZeRO
step together, and its gradient against autograd through the same loss written in torch."""
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


def test_preference_training_separates_the_pairs():
    import post_training_step as ex
    log = ex.train("preference", 25)
    # at the start model and reference are one: every margin is 0 up to bf16 logits' rounding
    # (about 2^-9 of a logit of 10, over 23 tokens, times beta 0.2: below 0.15)
    assert abs(log[0][0] - math.log(2)) < 0.15
    assert all(math.isfinite(a) and math.isfinite(b) and b > 0 for a, b, _ in log)
    assert sum(a for a, _, _ in log[-5:]) / 5 < 0.5 * log[0][0]
    assert log[-1][2] > log[0][2]


def test_policy_training_raises_the_rewarded_answers():
    import post_training_step as ex
    log = ex.train("policy", 25)
    assert all(math.isfinite(a) and math.isfinite(b) and b > 0 for a, b, _ in log)
    assert sum(gap for _, _, gap in log[-5:]) / 5 > sum(gap for _, _, gap in log[:5]) / 5


def test_gradients_reach_the_parameters():
    """d loss / d parameters through dlogits against autograd through the loss in torch, both from
    the same bf16 logits. dlogits is rounded to bf16 (2^-8 of each entry) in both, and the products
    behind it are the same kernels: 2^-6 of each gradient's norm covers two roundings."""
    import post_training_step as ex
    import zero_gradient_reduce_scatter_gb300 as zg
    g = torch.Generator(device="cuda").manual_seed(3)
    model = ex.Model(g)
    tokens, targets, offsets = ex.batch(g)
    ref = torch.randn(tokens.numel(), device="cuda", generator=g) - 7
    logits = model.hidden(tokens) @ model.params[0].T
    r = zg.preference_loss(logits.detach(), targets, offsets, ref, beta=0.2, label_smoothing=0.1)
    got = torch.autograd.grad(logits, model.params, r.dlogits, retain_graph=True)
    live = targets >= 0
    logp = torch.log_softmax(logits.float(), 1).gather(1, targets.clamp(min=0)[:, None])[:, 0]
    ratio = torch.where(live, logp - ref, torch.zeros_like(logp)).view(2 * ex.PAIRS, -1).sum(1)
    s = 0.2 * (ratio[0::2] - ratio[1::2])
    loss = -(0.9 * torch.nn.functional.logsigmoid(s) + 0.1 * torch.nn.functional.logsigmoid(-s)).mean()
    want = torch.autograd.grad(loss, model.params)
    assert abs(loss.item() - r.loss.item()) <= 1e-5 * loss.item()
    for a, b in zip(got, want):
        assert float((a - b).float().norm()) <= 2.0 ** -6 * float(b.float().norm())
