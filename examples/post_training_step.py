"""Preference or policy training of a tiny language model, end to end on one GPU.

    python examples/post_training_step.py [preference|policy] [steps]

Each step is what a post-training loop does around the optimizer: the frozen reference model's
log-probabilities without its logits (``linear_logp``), the trained model's loss with its gradient
on the logits (``preference_loss`` or ``policy_loss``), autograd for the parameters' gradients,
their global norm and clipping straight into the flat gradient buffer (``GradClip.into``), and one
ZeRO step, whose bf16 parameters go back to the model.

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
        wte, w1, w2 = self.params
        pair = torch.cat([wte[tokens], wte[tokens.roll(1)]], 1)
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
    log = []
    for _ in range(steps):
        tokens, targets, offsets = batch(g)
        with torch.no_grad():
            ref = zg.linear_logp(reference.hidden(tokens), frozen[0], targets).logp
            old = zg.linear_logp(model.hidden(tokens), model.params[0].detach(), targets).logp if kind == "policy" else None
        logits = model.hidden(tokens) @ model.params[0].T
        if kind == "preference":
            r = zg.preference_loss(logits.detach(), targets, offsets, ref, beta=0.2)
        else:
            advantages = torch.tensor([1.0, -1.0] * PAIRS, device="cuda")
            r = zg.policy_loss(logits.detach(), targets, advantages, old, ref, offsets=offsets, clip_high=0.28, kl_coef=0.02,
                               entropy_coef=0.001, reduce="sequence")
        for p in model.params:
            p.grad.zero_()
        logits.backward(r.dlogits)
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
