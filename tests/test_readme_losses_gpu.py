"""The README's snippets around the losses and the clipping, run as written (its placeholders filled in),
against autograd through the same loss and against the step on gradients packed by hand."""
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


def test_readme_step_behind_a_policy_loss():
    """Two steps; the parameters after each against a step on gradients that autograd gives the loss written
    in torch, clipped by torch. Both gradients come from bf16 logits' gradients and agree to 2^-7 of their
    norm; AdamW's first step is lr in every lane whatever the gradient's size, so what is compared is the
    packed gradient itself."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, V, D = 36, 257, 32
    hidden = torch.randn((T, D), device=DEV, generator=g).bfloat16()
    frozen_hidden, frozen_wte = hidden, (torch.randn((V, D), device=DEV, generator=g) / 4).bfloat16()
    params = [frozen_wte.clone().requires_grad_(), (torch.randn((D, D), device=DEV, generator=g) / 6).bfloat16().requires_grad_()]
    targets = torch.randint(0, V, (T,), device=DEV, generator=g)
    targets[::6] = -1
    offsets = torch.tensor([0, 10, 22, 36], device=DEV)
    advantages = torch.randn(3, device=DEV, generator=g)
    live = targets >= 0
    numel = [p.numel() for p in params]
    opt = zg.ZeroOptimizer(numel, M=1, stage=2, master_init=torch.cat([p.detach().float().reshape(-1) for p in params]))
    grads = opt.new_grad_buffers()
    clip = None
    old_logp = None
    for step in range(2):
        logits = (hidden + hidden @ params[1]) @ params[0].T
        if old_logp is None:
            old_logp = zg.token_logp(logits.detach(), targets).logp - 0.03

        ref = zg.linear_logp(frozen_hidden, frozen_wte, targets).logp      # reference, no logits in memory
        r = zg.policy_loss(logits.detach(), targets, advantages, old_logp, ref, offsets=offsets,
                           kl_coef=0.02, entropy_coef=0.001, reduce="sequence")

        logq = torch.log_softmax(logits.float(), 1)
        lp = torch.where(live, logq.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
        seq = torch.searchsorted(offsets[1:], torch.arange(T, device=DEV), right=True)
        A, ratio, d = advantages[seq], torch.exp(lp - old_logp), ref - lp
        per = torch.maximum(-ratio * A, -ratio.clamp(0.8, 1.2) * A) + 0.02 * (torch.exp(d) - d - 1) + 0.001 * (logq.exp() * logq).sum(1)
        count = torch.zeros(3, device=DEV).index_add_(0, seq, live.float())
        loss = torch.where(live, per / count[seq] / 3, 0.0).sum()
        want = torch.cat([x.float().reshape(-1) for x in torch.autograd.grad(loss, params, retain_graph=True)])

        logits.backward(r.dlogits)                                         # autograd from here on
        if clip is None:                                                   # a plan over these tensors: made once
            clip = zg.GradClip.into(opt, [p.grad for p in params], grads[0])
        c = clip.clip(max_norm=1.0, grads=[p.grad for p in params])        # norm, clipped, into the flat buffer

        assert abs(loss.item() - r.loss.item()) <= 1e-5 * (1 + abs(loss.item()))
        norm = float(want.norm())
        assert abs(float(c.norm) - norm) <= 2.0 ** -7 * norm
        got = torch.cat([opt.tensor_view(grads[0], i) for i in range(2)]).float()
        assert float((got - want * min(1.0, 1.0 / norm)).norm()) <= 2.0 ** -6 * min(norm, 1.0)

        opt.step(grads, zg.Hyper(lr=1e-5))
        for p in params:
            p.grad.zero_()                                                 # kept, not set to None: the plan holds them
        with torch.no_grad():
            for p, x in zip(params, opt.params().split(numel)):
                p.copy_(x.view_as(p))
    # what the snippet avoids: gradients set to None and made anew are not the plan's
    before = clip.grads[0].clone()
    params[0].grad = None
    ((hidden @ params[0].T).sum() * 1e-3).backward()
    with pytest.raises(ValueError):
        clip.clip(max_norm=1.0, grads=[p.grad for p in params])
    assert torch.equal(clip.grads[0], before)


def test_readme_clipping_by_the_averaged_gradient():
    """Packed without clipping and clipped in the step: the same bits as a step on buffers filled by hand."""
    numel = [1000, 3, 4099]
    w0 = torch.randn(sum(numel), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 0.02
    opt, hand = (zg.ZeroOptimizer(numel, M=2, stage=2, master_init=w0) for _ in range(2))
    grads, want = opt.new_grad_buffers(), hand.new_grad_buffers()
    g = torch.Generator(device=DEV).manual_seed(2)
    own = [[torch.randn(n, device=DEV, generator=g) for n in numel] for _ in range(2)]
    packs = [zg.GradClip.into(opt, own[rank], grads[rank]) for rank in range(2)]

    for rank in range(len(grads)):                                     # a plan per rank
        packs[rank].clip(max_norm=math.inf)                            # into the flat buffer as they are
    opt.step(grads, zg.Hyper(lr=1e-5, clip=True, max_grad_norm=1.0))

    for rank in range(2):
        for i, x in enumerate(own[rank]):
            hand.tensor_view(want[rank], i).copy_(x.bfloat16())
    hand.step(want, zg.Hyper(lr=1e-5, clip=True, max_grad_norm=1.0))
    assert opt.last_norm()[0] > 1.0 and all(torch.equal(a, b) for a, b in zip(grads, want))
    assert torch.equal(opt.params(), hand.params()) and torch.equal(opt.master, hand.master)
