"""Preference, policy or distillation training of a tiny language model, end to end on one GPU.

    python examples/post_training_step.py [preference|policy|distill] [steps]

Each step is what a post-training loop does around the optimizer: the frozen reference model's
log-probabilities without its logits (``linear_logp``), the trained model's loss with its gradient
on the logits (``preference_loss`` or ``policy_loss``), autograd for the parameters' gradients,
their global norm and clipping straight into the flat gradient buffer (``GradClip.into``), and one
ZeRO step, whose bf16 parameters go back to the model.

Distillation has a teacher of its own in place of the reference: its most likely tokens
(``top_logits``), the student's divergence from them with its gradient (``distill_loss``), and the
embedding's rows and their gradient by the library too (``embedding``, ``embedding_backward``), added to
the gradient that the output product leaves on the same matrix.

The model predicts the next token from the last two (embeddings, one hidden layer, the embedding
again as the vocabulary matrix). The task is synthetic: answers made of even tokens are preferred.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_gradient_reduce_scatter_gb300 as zg  # noqa: E402

VOCAB, DIM, PROMPT, ANSWER, PAIRS = 1021, 64, 5, 23, 12


class Model:
    """Parameters as separate tensors, in the order the optimizer holds them."""

    def __init__(self, generator):
        shapes = [(VOCAB, DIM), (2 * DIM, 4 * DIM), (4 * DIM, DIM)]
        std = [0.5, (2 * DIM) ** -0.5, (4 * DIM) ** -0.5]
        self.params = [torch.randn(s, device="cuda", generator=generator).mul_(k).to(torch.bfloat16).requires_grad_()
                       for s, k in zip(shapes, std)]

    def hidden(self, tokens):
        """[T, DIM] states that predict the token after each of `tokens`."""
        wte = self.params[0]
        return self.states(torch.cat([wte[tokens], wte[tokens.roll(1)]], 1))

    def states(self, pair):
        """The same from the rows of each token and of the one before it, [T, 2 DIM]."""
        _, w1, w2 = self.params
        return torch.nn.functional.gelu(pair @ w1) @ w2

    def load(self, flat):
        """Take the optimizer's parameters (bf16, in tensor order)."""
        with torch.no_grad():
            for p, x in zip(self.params, flat.split([p.numel() for p in self.params])):
                p.copy_(x.view_as(p))


def batch(generator):
    """Packed prompts with a good (even) and a bad (any) answer each: tokens, the target after each
    token (-1 in prompts and at the ends), and sequence offsets."""
    tokens, targets = [], []
    for i in range(2 * PAIRS):
        prompt = torch.randint(0, VOCAB, (PROMPT,), device="cuda", generator=generator)
        answer = torch.randint(0, VOCAB // 2, (ANSWER,), device="cuda", generator=generator)
        answer = 2 * answer if i % 2 == 0 else 2 * answer + 1
        seq = torch.cat([prompt, answer])
        after = torch.cat([seq[1:], seq.new_full((1,), -1)])
        after[:PROMPT - 1] = -1
        tokens.append(seq)
        targets.append(after)
    n = PROMPT + ANSWER
    offsets = torch.arange(0, (2 * PAIRS + 1) * n, n, device="cuda")
    return torch.cat(tokens), torch.cat(targets), offsets


def both(tokens):
    """Each token, and behind them the token before each."""
    return torch.cat([tokens, tokens.roll(1)])


def distill(model, teacher, tokens, targets, offsets, **kw):
    """The distillation loss of a batch; its gradients are added to the parameters' own."""
    wte = model.params[0]
    with torch.no_grad():
        top = zg.top_logits(teacher.hidden(tokens) @ teacher.params[0].T, 16, targets)
    rows = zg.embedding(wte.detach(), both(tokens)).requires_grad_()
    logits = model.states(rows.view(2, -1, DIM).transpose(0, 1).reshape(-1, 2 * DIM)) @ wte.T
    r = zg.distill_loss(logits.detach(), targets, top.index, top.logp, top.rest, offsets=offsets, **kw)
    logits.backward(r.dlogits)  # the output product's part of wte's gradient
    zg.embedding_backward(both(tokens), rows.grad, VOCAB, out=wte.grad, accumulate=True)  # and the embedding's
    return r


def prefer(kind, model, reference, tokens, targets, offsets):
    """The preference or policy loss of a batch; its gradients are added to the parameters' own."""
    wte = model.params[0]
    with torch.no_grad():
        ref = zg.linear_logp(reference.hidden(tokens), reference.params[0], targets).logp
        old = zg.linear_logp(model.hidden(tokens), wte.detach(), targets).logp if kind == "policy" else None
    logits = model.hidden(tokens) @ wte.T
    if kind == "preference":
        r = zg.preference_loss(logits.detach(), targets, offsets, ref, beta=0.2)
    else:
        advantages = torch.tensor([1.0, -1.0] * PAIRS, device="cuda")
        r = zg.policy_loss(logits.detach(), targets, advantages, old, ref, offsets=offsets, clip_high=0.28, kl_coef=0.02,
                           entropy_coef=0.001, reduce="sequence")
    logits.backward(r.dlogits)
    return r


def train(kind="preference", steps=20, seed=0):
    """Returns each step's (loss, gradient norm before clipping, log-probability of the good answers
    above the bad ones', mean over pairs)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(g)
    frozen = [p.detach().clone() for p in model.params]  # the reference: the model at the start
    numel = [p.numel() for p in model.params]
    w0 = torch.cat([p.detach().float().reshape(-1) for p in model.params])
    opt = zg.ZeroOptimizer(numel, M=1, stage=2, master_init=w0)
    flat = opt.new_grad_buffers()[0]
    for p in model.params:
        p.grad = torch.zeros_like(p)  # kept, so that one clipping plan serves every step
    clip = zg.GradClip.into(opt, [p.grad for p in model.params], flat)
    reference = Model.__new__(Model)
    reference.params = frozen
    teacher = Model(torch.Generator(device="cuda").manual_seed(seed + 1)) if kind == "distill" else None
    log = []
    for _ in range(steps):
        tokens, targets, offsets = batch(g)
        for p in model.params:
            p.grad.zero_()
        if kind == "distill":
            r = distill(model, teacher, tokens, targets, offsets, reduce="sequence", ce_coef=0.1)
        else:
            r = prefer(kind, model, reference, tokens, targets, offsets)
        c = clip.clip(1.0)
        opt.step([flat], zg.Hyper(lr=2e-3, weight_decay=0.0))
        model.load(opt.params())
        answers = r.logp.view(PAIRS, 2, -1).sum(2)
        log.append((r.loss, c.norm, (answers[:, 0] - answers[:, 1]).mean()))
    assert opt.sync_status() == 0
    return [tuple(float(v) for v in row) for row in log]


if __name__ == "__main__":
    kind = sys.argv[1] if len(sys.argv) > 1 else "preference"
    for i, (loss, norm, gap) in enumerate(train(kind, int(sys.argv[2]) if len(sys.argv) > 2 else 20)):
        print(f"step {i:3d}  loss {loss:9.5f}  gradient norm {norm:8.4f}  good above bad {gap:8.3f}")
