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


def extremes(way, seed):
    """Logits whose rows 1, 3, 5 ... hold masks: -inf or the type's lowest value over parts, over all
    but one token, over the target itself, in the middle of the vocabulary."""
    T, V, dtype = WAYS[way]
    low = torch.finfo(TYPES[dtype]).min
    x, _ = make_logits(T, V, dtype, seed)
    y = torch.randint(0, V // 2, (T,), device=DEV, generator=gen(seed + 1))
    x[1, V // 2:] = -math.inf
    x[3, V // 2:] = low
    x[5, V // 3:V // 3 + V // 7] = -math.inf     # in the middle
    y[5] = 1
    x[7, :] = low                                # nothing allowed, by the lowest value: uniform
    x[9, :] = -math.inf                          # one token allowed, and it is the target
    x[9, V - 1] = 2.0
    y[9] = V - 1
    x[11, V // 2:] = low                         # the target is masked by the lowest value
    y[11] = V - 2
    x[13, V // 2:] = -math.inf                   # the target is masked by -inf
    y[13] = V - 2
    return x, y


@pytest.mark.parametrize("entropy_coef", [0.0, 0.02])
@pytest.mark.parametrize("way", WAYS)
def test_policy_loss_of_masked_rows(way, entropy_coef):
    T, V, dtype = WAYS[way]
    x, y = extremes(way, 41)
    adv = torch.randn(T, device=DEV, generator=gen(43)) + 0.3
    logq, lp, _, ent = reference(x, y)
    gone = lp < -1e4                             # a ratio of exactly 0, in fp32 as in 64 bits
    assert gone.tolist()[:14] == [False] * 11 + [True, False, True]
    old = torch.where(gone, torch.full_like(lp, -5.0), lp - 0.05).float()
    q = zg.policy_loss(x, y, adv, old, reduce="sum", entropy_coef=entropy_coef)
    A, near = adv.double(), torch.where(gone, torch.zeros_like(lp), lp)
    r = torch.exp(lp - old.double())
    live = torch.where(gone & (A < 0), torch.zeros_like(A), torch.ones_like(A))   # below the clip: no gradient, a constant loss
    surrogate = torch.where(gone & (A < 0), -0.8 * A, -r * A)
    E = bound(x) * (1 + near.abs())
    size = r * A.abs() + entropy_coef * (1 + ent)
    check(q.logp[~gone], lp[~gone], bound(x)[~gone], "logp")
    assert bool((q.logp[gone] < -1e4).all())
    assert abs(float(q.loss) - float((surrogate - entropy_coef * ent).sum())) <= float((2 * E * size + 2.0 ** -20 * (surrogate.abs() + entropy_coef * ent)).sum())
    g = -r * A * live
    h = torch.full_like(g, -entropy_coef) if entropy_coef else None
    want = reference_grad(logq, y, g, h, ent, 1.0)
    p = torch.exp(logq)
    hot = torch.zeros_like(p).scatter_(1, y[:, None], 1.0)
    plogp = torch.where(p > 0, p * logq.abs(), torch.zeros_like(p))
    tol = ((4 * E * size + 2.0 ** -21 * size)[:, None] * (p + hot) + (2 * E * entropy_coef)[:, None] * plogp)
    tol = tol + UNIT[dtype] * want.abs() + 2.0 ** -100 + (2.0 ** -25 if dtype == "fp16" else 0.0)
    err = (q.dlogits.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), q.dlogits[bad][:3].tolist(), want[bad][:3].tolist())
    inplace = zg.policy_loss(x, y, adv, old, reduce="sum", entropy_coef=entropy_coef, out=x)
    assert torch.equal(x, q.dlogits) and torch.equal(inplace.loss, q.loss)


@pytest.mark.parametrize("entropy_coef", [0.0, 0.02])
@pytest.mark.parametrize("way", WAYS)
def test_policy_loss_of_rows_without_a_value(way, entropy_coef):
    """NaN, +inf, a target past the vocabulary: NaN for that token and in the loss, and every other row's
    gradient bit for bit what it is without them; a row of -inf alone: gradient 0."""
    T, V, dtype = WAYS[way]
    x, _ = make_logits(T, V, dtype, 51)
    y = torch.randint(0, V, (T,), device=DEV, generator=gen(52))
    adv = torch.randn(T, device=DEV, generator=gen(53))
    old = (reference(x, y)[1] - 0.05).float()
    kw = dict(reduce="sum", entropy_coef=entropy_coef)
    bad = [2, 4, 6, 8]
    x[2, V // 3] = math.nan
    x[4, V // 3] = math.inf
    y[6] = V + 3
    x[8, y[8]] = math.nan
    x[10, :] = -math.inf
    masked = y.clone()
    masked[bad] = -1
    want = zg.policy_loss(x, masked, adv, old, **kw)
    assert bool(want.loss.isfinite()) and want.logp[10] == -math.inf and bool((want.dlogits[10] == 0).all())
    assert bool((want.dlogits[bad] == 0).all()) and bool(want.dlogits.isfinite().all())
    q = zg.policy_loss(x, y, adv, old, **kw)
    assert bool(q.loss.isnan()) and bool(q.logp[bad].isnan().all()) and bool(q.dlogits[bad].isnan().all())
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[bad] = False
    assert torch.equal(q.dlogits[rest], want.dlogits[rest]) and torch.equal(q.logp[rest], want.logp[rest])


@pytest.mark.parametrize("way", WAYS)
def test_preference_loss_of_extreme_rows(way):
    """Masked rows in two pairs; in a third a target that cannot be scored: NaN in that pair and the mean,
    nothing in the others."""
    T, V, dtype = WAYS[way]
    x, y = extremes(way, 61)
    y[11], y[13] = 3, 4                          # targets among the allowed tokens
    x[0, V // 3] = math.nan
    off = torch.tensor([0, 1, 2, 8, T - 2, T - 2, T], device=DEV)
    logq, lp, _, ent = reference(x, y)
    E = bound(x) * (1 + lp.abs())
    ref = (torch.where(lp.isfinite(), lp, torch.zeros_like(lp)) - 0.01).float()
    r = zg.preference_loss(x, y, off, ref, beta=0.1)
    assert bool(r.loss.isnan()) and bool(r.pair_loss[0].isnan()) and bool(r.dlogits[:2].isnan().all())
    check(r.logp[1:], lp[1:], bound(x)[1:], "logp")
    for i, (a, b, c) in ((1, (2, 8, T - 2)), (2, (T - 2, T - 2, T))):
        d = (lp - ref.double())
        m, err = float(d[a:b].sum() - d[b:c].sum()), float(E[a:c].sum())
        loss = math.log1p(math.exp(-0.1 * m))
        assert abs(float(r.pair_loss[i]) - loss) <= 0.1 * err + 2.0 ** -22
        dm = -0.1 / (1 + math.exp(0.1 * m)) / 3
        for lo, hi, s in ((a, b, dm), (b, c, -dm)):
            if lo == hi:
                continue
            g = torch.full((hi - lo,), s, device=DEV, dtype=torch.float64)
            want = reference_grad(logq[lo:hi], y[lo:hi], g, None, ent[lo:hi], 1.0)
            p = torch.exp(logq[lo:hi])
            hot = torch.zeros_like(p).scatter_(1, y[lo:hi, None], 1.0)
            # the coefficient follows the margin with a slope below beta times itself
            tol = abs(s) * (2 * E[lo:hi, None] + 0.1 * err + 2.0 ** -22) * (p + hot) + UNIT[dtype] * want.abs() + 2.0 ** -100
            if dtype == "fp16":
                tol = tol + 2.0 ** -25
            assert bool(((r.dlogits[lo:hi].double() - want).abs() <= tol).all()), (i, lo)


@pytest.mark.parametrize("way", WAYS)
def test_masked_target_under_the_current_policy(way):
    """Without old_logp the ratio is 1, also where the target's probability is 0; NaN stays NaN."""
    T, V, dtype = WAYS[way]
    x, _ = make_logits(T, V, dtype, 71)
    y = torch.randint(0, V // 2, (T,), device=DEV, generator=gen(72))
    x[1, V // 2:] = -math.inf
    y[1] = V - 1
    adv = torch.full((T,), 0.5, device=DEV)
    q = zg.policy_loss(x, y, adv, reduce="sum")
    assert q.logp[1] == -math.inf and abs(float(q.loss) + 0.5 * T) <= 2.0 ** -22 * T
    logq, _, _, ent = reference(x, y)
    want = reference_grad(logq, y, -adv.double(), None, ent, 1.0)[1]
    p = torch.exp(logq[1])
    tol = 0.5 * (2 * bound(x)[1] + 2.0 ** -21) * p + UNIT[dtype] * want.abs() + 2.0 ** -100 + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert bool(((q.dlogits[1].double() - want).abs() <= tol).all())
    x[2, 5] = math.nan
    assert bool(zg.policy_loss(x, y, adv, reduce="sum").loss.isnan())


def test_kl_of_a_masked_target_is_infinite():
    """exp(d) - d - 1 at d = inf, the third estimator where the policy gives a target no probability."""
    x, _ = make_logits(20, 300, "bf16", 81)
    y = torch.randint(0, 150, (20,), device=DEV, generator=gen(82))
    x[4, 150:] = -math.inf
    y[4] = 200
    zero = torch.zeros(20, device=DEV)
    for kl in ("k2", "k3"):
        assert float(zg.policy_loss(x, y, zero, zero - 5, zero - 5, kl=kl).kl) == math.inf
    x[5, 3] = math.nan
    assert bool(zg.policy_loss(x, y, zero, zero - 5, zero - 5).kl.isnan())


@pytest.mark.parametrize("way", WAYS)
def test_no_advantage_beside_a_ratio_past_fp32(way):
    """Advantage 0, as in a group whose rewards are all equal: no surrogate whatever the ratio, of which
    exp(logp - old_logp) may be no fp32 number."""
    T, V, dtype = WAYS[way]
    x, _ = make_logits(T, V, dtype, 91)
    y = torch.randint(0, V, (T,), device=DEV, generator=gen(92))
    adv = torch.zeros(T, device=DEV)
    old = torch.full((T,), -5.0, device=DEV)
    old[1] = -200.0
    q = zg.policy_loss(x, y, adv, old, reduce="sum")
    assert float(q.loss) == 0 and float(q.clip_fraction) == 0 and bool((q.dlogits == 0).all())


def test_pairs_of_no_tokens_in_a_graph():
    """A batch of no rows is captured like any other."""
    x, y = torch.empty((0, 40), device=DEV, dtype=torch.bfloat16), torch.empty(0, dtype=torch.int64, device=DEV)
    off = torch.zeros(2 * 700 + 1, dtype=torch.int64, device=DEV)
    want = zg.preference_loss(x, y, off)
    import gc
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = zg.preference_loss(x, y, off)
    for _ in range(2):
        r.loss.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.loss, want.loss) and abs(float(r.loss) - math.log(2)) <= 2.0 ** -23


@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("T,V", [(60000, 67), (1000, 1031)])
def test_entropy_beside_an_unlikely_target(T, V, temperature):
    """One token takes nearly all of the probability and the target is up to e^50 times less likely: the
    entropy, small, keeps the bound that the roundings of log p have."""
    x = torch.randn((T, V), device=DEV, generator=gen(1))
    y = torch.randint(1, V, (T,), device=DEV, generator=gen(2))
    x[:, 0] = x[:, 1:].amax(1) + 3 * torch.rand(T, device=DEV, generator=gen(4)) + 1
    gap = torch.linspace(0.0, 50.0, T, device=DEV) * temperature
    x.scatter_(1, y[:, None], (x[:, 0] - gap)[:, None])
    f = zg.token_logp(x, y, entropy=True, temperature=temperature)
    _, lp, lse, ent = reference(x, y, temperature)
    E = bound(x, temperature)
    check(f.entropy, ent, E * (1 + ent), "entropy")
    check(f.lse, lse, E, "lse")
    check(f.logp, lp, E, "logp")
    q = zg.policy_loss(x, y, torch.ones(T, device=DEV), entropy_coef=0.02, temperature=temperature)
    check(q.entropy, ent, E * (1 + ent), "entropy")


@pytest.mark.parametrize("sign", [1, -1])
def test_gradients_at_large_margins(sign):
    """A sigmoid loss far on either side: its slope sigmoid(-s) is formed without cancellation, down to
    where fp32 ends. The margin is a sum of 2 n log-probabilities, each within E (1 + |log p|), and the
    slope's relative error is at most that of s, beta times it and one rounding of s, and 2^-21 beside."""
    n, V, beta = 8, 257, 1.0
    x, _ = make_logits(12 * n, V, "fp32", 5)
    y = make_targets(12 * n, V, 6, masked=0.0)
    off = torch.arange(0, 12 * n + 1, n, device=DEV)
    logq, lp, _, ent = reference(x, y)
    ref = lp.float()
    for i, s in enumerate((20.0, 37.0, 45.0, 60.0, 80.0, 200.0)):   # of the pair's margin
        ref[2 * i * n] -= sign * s
    r = zg.preference_loss(x, y, off, ref, beta=beta)
    d = lp - ref.double()
    E = bound(x) * (1 + lp.abs())
    for i in range(6):
        a, b, c = 2 * i * n, (2 * i + 1) * n, (2 * i + 2) * n
        m = float(d[a:b].sum() - d[b:c].sum())
        t = math.exp(-abs(m))
        slope = -beta * (t if m > 0 else 1.0) / (1 + t) / 6
        err = float(E[a:c].sum()) + 2.0 ** -23 * abs(m) + 2.0 ** -21
        for lo, hi, g in ((a, b, slope), (b, c, -slope)):
            want = reference_grad(logq[lo:hi], y[lo:hi], torch.full((n,), g, device=DEV, dtype=torch.float64), None, ent[lo:hi], 1.0)
            p = torch.exp(logq[lo:hi])
            hot = torch.zeros_like(p).scatter_(1, y[lo:hi, None], 1.0)
            tol = abs(g) * (2 * E[lo:hi, None] + err) * (p + hot) + 2.0 ** -24 * want.abs() + 2.0 ** -126
            assert bool(((r.dlogits[lo:hi].double() - want).abs() <= tol).all()), (i, m)
