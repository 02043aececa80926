"""Token log-probabilities, the preference and policy losses and their gradients, against
64-bit formulas written here with elementary operations.

Tolerances. u = 2^-24 is fp32's rounding. A term's exponent d = (x - m) c carries three roundings
of a number of at most R = max |z - max z| that matters (terms below 2^-40 of the largest are
lost in the sum anyway, so R is cut at 28) plus log V, the exponential 2^-22, and a sum of n/256
terms in a row at most n/256 roundings. So log p and the entropy are within
    E = 2^-22 (8 + R) + 2^-24 n / 256,
times 1 + |value| for the final roundings. A gradient entry p (g + h (log p + H)) / temperature takes
the relative error of p, E, and in the bracket the absolute ones of log p and H, E (1 + |log p|) and
E (1 + H): in all 2 E p (|g| + |h| (1 + |log p| + H)) / temperature. It is then rounded once to its type (half its spacing: 2^-8, 2^-11, 2^-24), with half the
smallest fp16 number, 2^-25, where that type underflows. Losses are sums of such terms: their
bound is the sum of the terms' bounds.
"""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {k: torch.finfo(t).eps / 2 for k, t in TYPES.items()}  # 2^-8, 2^-11, 2^-24
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_logits(T, V, dtype, seed, stride=None, offset=0, spread=3.0):
    """[T, V] logits inside a larger allocation: row stride `stride`, first element at `offset`;
    what lies between rows is NaN, which no call may read."""
    stride = stride or V
    flat = torch.full((offset + max(T, 1) * stride + 16,), float("nan"), device=DEV, dtype=TYPES[dtype])
    x = flat[offset:].as_strided((T, V), (stride, 1))
    x.copy_(torch.randn((T, V), device=DEV, generator=gen(seed)) * spread)
    return x, flat


def make_targets(T, V, seed, masked=0.25):
    y = torch.randint(0, V, (T,), device=DEV, generator=gen(seed + 1))
    if masked:
        y = torch.where(torch.rand(T, device=DEV, generator=gen(seed + 2)) < masked, torch.full_like(y, -1), y)
    return y


def reference(x, y, temperature=1.0):
    """(log q over the vocabulary, logp, lse, entropy) in 64 bits; rows without a target 0."""
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s = torch.exp(z - m).sum(1, keepdim=True)
    lse = m + torch.log(s)
    # not z - lse: where |m| is large, log s is below its rounding even in 64 bits
    logq = torch.where(z == -math.inf, torch.full_like(z, -math.inf), (z - m) - torch.log(s))
    q = torch.exp(logq)
    ent = -torch.where(q > 0, q * logq, torch.zeros_like(q)).sum(1)
    live = y >= 0
    lp = logq.gather(1, y.clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(lp)
    return logq, torch.where(live, lp, zero), torch.where(live, lse[:, 0], zero), torch.where(live, ent, zero)


def bound(x, temperature=1.0):
    z = x.double() / temperature
    V = x.shape[1]
    m = torch.where(z.isfinite(), z, torch.full_like(z, -math.inf)).amax(1)
    m = torch.where(m.isfinite(), m, torch.zeros_like(m))
    low = torch.where(z.isfinite(), z, m[:, None]).amin(1)
    R = torch.clamp(m - low, max=28.0) + math.log(V)
    return 2.0 ** -22 * (8 + R) + 2.0 ** -24 * V / 256


def reference_grad(logq, y, g, h, ent, temperature):
    q = torch.exp(logq)
    hot = torch.zeros_like(q).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    d = g[:, None] * (hot - q)
    if h is not None:
        d = d - h[:, None] * torch.where(q > 0, q * (logq + ent[:, None]), torch.zeros_like(q))
    return torch.where((y >= 0)[:, None], d / temperature, torch.zeros_like(d))


def check_grad(got, want, logq, y, g, h, ent, E, dtype, temperature):
    q = torch.exp(logq)
    size = g.abs()[:, None].expand_as(q)
    if h is not None:
        size = size + h.abs()[:, None] * (1 + torch.where(q > 0, logq.abs(), torch.zeros_like(q)) + ent[:, None])
    # the target's entry g (1 - p) cancels: its error is that of p and of g
    hot = torch.zeros_like(q).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    tol = (2 * E[:, None] * q * size + hot * g.abs()[:, None] * 2.0 ** -22) / temperature + UNIT[dtype] * want.abs() + 2.0 ** -100
    if dtype == "fp16":
        tol = tol + 2.0 ** -25
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), (got.double() - want).abs().max().item(), bad.nonzero()[:3].tolist())


def check(got, want, E, what):
    tol = E * (1 + want.abs())
    err = (got.double() - want).abs()
    assert got.dtype == torch.float32 and bool((err <= tol).all()), (what, err.max().item(), (err - tol).max().item())


SHAPES = [  # T, V, stride, offset
    (1, 1, None, 0), (1, 50257, None, 0), (3, 7, None, 1), (5, 8, None, 0), (4, 9, 17, 3), (17, 1000, 1008, 0),
    (33, 4099, None, 5), (2, 8192, None, 8), (64, 257, 264, 0), (700, 130, 131, 2), (3, 131072, None, 1),
    (1300, 515, 518, 1), (1217, 3, None, 0), (1251, 4099, None, 0),  # a warp per row
    (2501, 9001, None, 1),  # forward only, in 16 bits
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,stride,offset", SHAPES)
def test_token_logp_and_gradient(T, V, stride, offset, dtype):
    for temperature, with_entropy in ((1.0, False), (0.7, True)):
        x, flat = make_logits(T, V, dtype, 10 + T + V, stride, offset)
        y = make_targets(T, V, 3, masked=0.3 if T > 1 else 0.0)
        logq, lp, lse, ent = reference(x, y, temperature)
        E = bound(x, temperature)
        f = zg.token_logp(x, y, temperature=temperature, entropy=with_entropy)
        check(f.logp, lp, E, "logp")
        check(f.lse, lse, E, "lse")
        assert (f.entropy is not None) == with_entropy
        if with_entropy:
            check(f.entropy, ent, E * (1 + ent), "entropy")
        assert bool((f.logp[y < 0] == 0).all()) and bool((f.lse[y < 0] == 0).all())
        g = torch.randn(T, device=DEV, generator=gen(5))
        h = torch.randn(T, device=DEV, generator=gen(6)) if with_entropy else None
        want = reference_grad(logq, y, g.double(), None if h is None else h.double(), ent, temperature)
        args = (logq, y, g.double(), None if h is None else h.double(), ent, E, dtype, temperature)
        keep = x.clone()
        d = zg.token_logp_backward(x, y, f, g, h, temperature=temperature)
        assert d.shape == x.shape and d.dtype == x.dtype and (T <= 1 or d.stride() == x.stride())
        check_grad(d, want, *args)
        assert torch.equal(x, keep)
        # into a layout of another alignment, and in place: the same bits, and nothing beside the rows
        other, oflat = make_logits(T, V, dtype, 1, (stride or V) + 5, offset + 1)
        assert zg.token_logp_backward(x, y, f, g, h, temperature=temperature, out=other) is other
        assert torch.equal(other, d)
        inside = torch.zeros_like(oflat, dtype=torch.bool)
        inside[offset + 1:].as_strided((T, V), ((stride or V) + 5, 1)).fill_(True)
        assert bool(oflat[~inside].isnan().all())
        zg.token_logp_backward(x, y, f, g, h, temperature=temperature, out=x)
        assert torch.equal(x, d)
        inside = torch.zeros_like(flat, dtype=torch.bool)
        inside[offset:].as_strided((T, V), (stride or V, 1)).fill_(True)
        assert bool(flat[~inside].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [37, 4096, 50257])
def test_masked_vocabularies_and_extreme_rows(V, dtype):
    """-inf and lowest-value masks over part of a row and over all of it, one finite value, large
    equal offsets; and the rows that have no value: NaN, +inf, a target past the vocabulary."""
    low = torch.finfo(TYPES[dtype]).min
    x, _ = make_logits(10, V, dtype, 77)
    y = torch.randint(0, V, (10,), device=DEV, generator=gen(4))
    x[0, V // 2:] = -math.inf
    y[0] = 1
    x[1, 1:] = low
    x[2, :] = low                      # nothing allowed, by the lowest value: uniform
    x[3, :] = -math.inf                # nothing allowed, by -inf
    x[4, :] = -math.inf
    x[4, V - 1] = 2.0                  # one token allowed
    y[4] = V - 1
    x[5] += 20000.0                    # an offset common to the row (a multiple of the type's spacing there)
    x[6, V // 2:] = -math.inf
    y[6] = V - 1                       # the target itself is masked
    x[7, V // 3] = math.nan
    x[8, V // 3] = math.inf
    y[9] = V + 3
    f = zg.token_logp(x, y, entropy=True)
    logq, lp, lse, ent = reference(x, y.clamp(max=V - 1))
    E = bound(x)
    fine = [0, 1, 2, 4, 5]
    check(f.logp[fine], lp[fine], E[fine], "logp")
    check(f.entropy[fine], ent[fine], E[fine] * (1 + ent[fine]), "entropy")
    check(f.lse[[0, 1, 4, 5]], lse[[0, 1, 4, 5]], E[[0, 1, 4, 5]], "lse")
    assert f.logp[3] == -math.inf and f.lse[3] == -math.inf and f.entropy[3] == 0
    assert f.logp[6] == -math.inf
    check(f.lse[6:7], lse[6:7], E[6:7], "lse")
    assert bool(f.logp[7:9].isnan().all()) and bool(f.entropy[7:9].isnan().all())
    assert bool(f.logp[9].isnan()) and bool(f.lse[9].isfinite())
    g, h = torch.full((10,), 0.5, device=DEV), torch.full((10,), -0.25, device=DEV)
    d = zg.token_logp_backward(x, y, f, g, h)
    rows = [0, 1, 2, 4, 5, 6]
    gd, hd = g.double(), h.double()
    want = reference_grad(logq, y.clamp(max=V - 1), gd, hd, ent, 1.0)
    k = torch.tensor(rows, device=DEV)
    check_grad(d[k], want[k], logq[k], y[k], gd[k], hd[k], ent[k], E[k], dtype, 1.0)
    assert bool((d[3] == 0).all())
    assert bool(d[7].isnan().all()) and bool(d[8].isnan().all()) and bool(d[9].isnan().all())


def test_rows_without_a_target_are_not_read():
    x, _ = make_logits(6, 513, "bf16", 9)
    x[2] = math.nan
    x[5] = math.nan
    y = make_targets(6, 513, 1, masked=0.0)
    y[2] = y[5] = -100
    f = zg.token_logp(x, y, entropy=True)
    assert bool(f.logp.isfinite().all()) and bool(f.entropy.isfinite().all())
    d = zg.token_logp_backward(x, y, f, torch.ones(6, device=DEV), torch.ones(6, device=DEV))
    assert bool(d.isfinite().all()) and bool((d[2] == 0).all()) and bool((d[5] == 0).all())
    # nor a row whose coefficients are 0
    x[1] = math.nan
    g = torch.ones(6, device=DEV)
    g[1] = 0.0
    assert bool((zg.token_logp_backward(x, y, f, g)[1] == 0).all())


def test_gradient_against_differences():
    """Central differences of the fp64 formula's own values in every logit of a row, and the
    kernel's gradient in fp32: the difference quotient with step s is off by s^2 / 6 times the
    third derivative (below 2 for these coefficients and spreads) and 2^-52 / s."""
    V, s = 23, 1e-4
    x, _ = make_logits(2, V, "fp32", 3, spread=1.0)
    y = torch.tensor([4, 22], device=DEV)
    g, h = torch.tensor([0.8, -0.6], device=DEV), torch.tensor([0.3, 0.9], device=DEV)
    f = zg.token_logp(x, y, entropy=True, temperature=1.5)
    d = zg.token_logp_backward(x, y, f, g, h, temperature=1.5)

    def value(z):
        _, lp, _, ent = reference(z, y, 1.5)
        return g.double() * lp + h.double() * ent
    for j in range(V):
        up, down = x.double().clone(), x.double().clone()
        up[:, j] += s
        down[:, j] -= s
        diff = (value(up) - value(down)) / (2 * s)
        tol = s * s / 6 * 2 + 2.0 ** -50 / s + 2 * bound(x, 1.5) * 4
        assert bool(((d[:, j].double() - diff).abs() <= tol).all())


def make_offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int64, device=DEV)


PAIRS = [[700, 0, 311, 260], [1, 1], [5, 0], [0, 0], [3, 9, 1, 2], [40, 17, 0, 5, 64, 64, 2, 1], [300, 211], [7, 1, 0, 0, 130, 95, 211, 60, 0, 0, 1, 88]]


@pytest.mark.parametrize("lens", PAIRS)
@pytest.mark.parametrize("kind,smoothing,average", [("sigmoid", 0.0, False), ("sigmoid", 0.2, True), ("hinge", 0.0, False),
                                                    ("ipo", 0.0, True)])
def test_preference_loss(lens, kind, smoothing, average):
    dtype = ["bf16", "fp16", "fp32"][len(lens) % 3]
    T, V, beta = sum(lens) + 3, 515, 0.3     # three tokens of no pair at the end
    x, _ = make_logits(T, V, dtype, 5)
    y = make_targets(T, V, 8)
    ref = None if len(lens) == 4 else torch.randn(T, device=DEV, generator=gen(9)) - 6.0
    off = make_offsets(lens)
    r = zg.preference_loss(x, y, off, ref, beta=beta, kind=kind, label_smoothing=smoothing, average=average)
    logq, lp, _, ent = reference(x, y)
    E = bound(x)
    check(r.logp, lp, E, "logp")
    live = y >= 0
    delta = torch.where(live, lp - (0 if ref is None else ref.double()), torch.zeros_like(lp))
    P = len(lens) // 2
    g, losses, slack = torch.zeros_like(lp), [], []
    for i in range(P):
        d, n, e = [], [], []
        for k in (2 * i, 2 * i + 1):
            part = slice(int(off[k]), int(off[k + 1]))
            n.append(max(1, int(live[part].sum())) if average else 1)
            d.append(float(delta[part].sum()) / n[-1])
            e.append(float((E * (1 + lp.abs()) * live)[part].sum()) / n[-1])
        m = d[0] - d[1]
        s = beta * m
        if kind == "sigmoid":
            tail = math.log1p(math.exp(-abs(s)))       # log(1 + e^x) = max(x, 0) + this, at any margin
            loss = (1 - smoothing) * (max(-s, 0) + tail) + smoothing * (max(s, 0) + tail)
            sig = 1 / (1 + math.exp(-s)) if s > 0 else math.exp(s) / (1 + math.exp(s))
            dm = beta * (sig - (1 - smoothing))
            slope, curve = beta, beta * beta / 4
        elif kind == "hinge":
            loss, dm, slope, curve = max(0.0, 1 - s), -beta if s < 1 else 0.0, beta, 0.0
        else:
            loss, dm = (m - 0.5 / beta) ** 2, 2 * (m - 0.5 / beta)
            slope, curve = abs(dm), 2.0
        err = e[0] + e[1]
        assert abs(float(r.chosen_reward[i]) - beta * d[0]) <= beta * e[0] + 2.0 ** -23 * abs(beta * d[0]) + 1e-30
        assert abs(float(r.rejected_reward[i]) - beta * d[1]) <= beta * e[1] + 2.0 ** -23 * abs(beta * d[1]) + 1e-30
        slack.append(slope * err + curve * err * err + 2.0 ** -23 * loss)
        assert abs(float(r.pair_loss[i]) - loss) <= slack[-1]
        losses.append(loss)
        for sign, k, c in ((1, 2 * i, n[0]), (-1, 2 * i + 1, n[1])):
            g[int(off[k]):int(off[k + 1])] = sign * dm / P / c
        # the coefficient's own error, as a part of every entry of the pair's rows
        E[int(off[2 * i]):int(off[2 * i + 2])] += (curve * err + 2.0 ** -23 * abs(dm)) / max(abs(dm), 1e-300) if dm else 0.0
    assert abs(float(r.loss) - sum(losses) / P) <= sum(slack) / P + 2.0 ** -23 * sum(losses) / P
    g = torch.where(live, g, torch.zeros_like(g))
    want = reference_grad(logq, y, g, None, ent, 1.0)
    hot = torch.zeros_like(logq).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    tol = g.abs()[:, None] * (2 * E[:, None] * (torch.exp(logq) + hot)) + UNIT[dtype] * want.abs() + 2.0 ** -100
    if dtype == "fp16":
        tol = tol + 2.0 ** -25
    assert bool(((r.dlogits.double() - want).abs() <= tol).all())
    assert bool((r.dlogits[sum(lens):] == 0).all()) and bool((r.dlogits[~live] == 0).all())
    again = zg.preference_loss(x, y, off, ref, beta=beta, kind=kind, label_smoothing=smoothing, average=average)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
    inplace = zg.preference_loss(x, y, off, ref, beta=beta, kind=kind, label_smoothing=smoothing, average=average, out=x)
    assert torch.equal(x, r.dlogits) and torch.equal(inplace.loss, r.loss)


def test_infinite_margins():
    """A target that the model gives no probability (its logit masked by -inf) in one side of a pair:
    the margin is infinite, the loss its limit, and no gradient is NaN."""
    x, _ = make_logits(8, 64, "bf16", 4)
    y = torch.randint(0, 32, (8,), device=DEV, generator=gen(2))
    off = make_offsets([2, 2, 2, 2])
    x[3, y[3]] = -math.inf        # rejected of pair 0: margin +inf
    x[4, y[4]] = -math.inf        # chosen of pair 1: margin -inf
    for kind, limits in (("sigmoid", (0.0, math.inf)), ("hinge", (0.0, math.inf))):
        r = zg.preference_loss(x, y, off, beta=0.1, kind=kind)
        assert (float(r.pair_loss[0]), float(r.pair_loss[1])) == limits
        assert bool(r.dlogits.isfinite().all()) and bool((r.dlogits[:4] == 0).all()) and bool((r.dlogits[4:] != 0).any())


def policy_reference(x, y, adv, old, ref, off, lo, hi, dual, kl, kc, ec, reduce, temperature):
    logq, lp, lse, ent = reference(x, y, temperature)
    T = lp.shape[0]
    seq = torch.full((T,), -1, device=DEV)
    if off is not None:
        for s in range(off.numel() - 1):
            seq[int(off[s]):int(off[s + 1])] = s
    live = (y >= 0) & ((seq >= 0) if off is not None else torch.ones_like(y, dtype=torch.bool))
    A = adv.double()
    if A.numel() != T:
        A = torch.where(seq >= 0, A[seq.clamp(min=0)], torch.zeros_like(lp))
    r = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    loss = torch.maximum(-r * A, -r.clamp(1 - lo, 1 + hi) * A)
    on = ~(((A > 0) & (r > 1 + hi)) | ((A < 0) & (r < 1 - lo)))
    if dual:
        on &= ~((A < 0) & (r > dual))
        loss = torch.where(A < 0, torch.minimum(loss, -dual * A), loss)
    g = torch.where(on, -r * A, torch.zeros_like(r))
    k = torch.zeros_like(lp)
    if ref is not None:
        d = ref.double() - lp
        k, dk = {"k1": (-d, torch.ones_like(d)), "k2": (d * d / 2, -d), "k3": (torch.expm1(d) - d, -torch.expm1(d))}[kl]
        loss, g = loss + kc * k, g + kc * dk
    loss = loss - ec * ent
    n = max(1, int(live.sum()))
    w = torch.zeros_like(lp)
    if reduce == "token":
        w[live] = 1.0 / n
    elif reduce == "sum":
        w[live] = 1.0
    else:
        counts = [int((live & (seq == s)).sum()) for s in range(off.numel() - 1)]
        filled = max(1, sum(c > 0 for c in counts))
        for s, c in enumerate(counts):
            w[live & (seq == s)] = 1.0 / max(c, 1) / filled
    zero = torch.zeros_like(lp)
    term = torch.where(live, loss * w, zero)
    return dict(logq=logq, lp=torch.where(live, lp, zero), ent=ent, live=live, loss=term.sum(), r=r, A=A, w=w,
                clip=float((~on & live).sum()) / n, kl=float(torch.where(live, k, zero).sum()) / n, g=g * w, h=-ec * w)


POLICY = [  # lens, reduce, advantages per, old, ref, kl, kl_coef, entropy_coef, dual, temperature, V, dtype
    ([1], "token", "token", True, True, "k3", 0.1, 0.0, 0.0, 1.0, 333, "bf16"),
    ([4, 0, 9], "sequence", "sequence", True, True, "k2", 0.1, 0.05, 3.0, 0.8, 1024, "fp32"),
    ([31, 1, 77, 0, 0, 5], "sequence", "sequence", True, False, "k1", 0.0, 0.0, 0.0, 1.0, 4097, "fp16"),
    ([200, 130], "token", "sequence", True, True, "k1", 0.2, 0.01, 1.5, 1.0, 2051, "bf16"),
    ([64, 64, 64], "sum", "token", False, True, "k3", 0.02, 0.0, 0.0, 1.3, 513, "fp32"),
    (None, "token", "token", True, True, "k3", 0.1, 0.02, 0.0, 1.0, 50257, "bf16"),
    (None, "sum", "token", False, False, "k3", 0.0, 0.0, 0.0, 1.0, 130, "fp16"),
    ([700, 0, 640], "sequence", "sequence", True, True, "k3", 0.1, 0.02, 3.0, 0.9, 517, "bf16"),  # a warp per row
    ([700, 640], "token", "token", True, True, "k2", 0.1, 0.0, 0.0, 1.0, 1001, "fp32"),
    # rows cut over a cluster, and rows too long for one
    ([3, 2], "token", "token", True, True, "k3", 0.1, 0.02, 0.0, 1.0, 131073, "bf16"),
    ([3, 2], "sequence", "sequence", True, True, "k3", 0.1, 0.02, 3.0, 1.0, 300001, "fp32"),
    ([310], "token", "token", True, False, "k3", 0.0, 0.01, 0.0, 1.0, 60001, "bf16"),
    ([160], "sum", "sequence", True, True, "k3", 0.05, 0.01, 0.0, 1.0, 30011, "bf16"),  # one CTA per row, large and small
    ([160], "token", "sequence", True, True, "k3", 0.05, 0.0, 0.0, 1.0, 12007, "fp16"),
]


@pytest.mark.parametrize("case", POLICY)
def test_policy_loss(case):
    lens, reduce, per, with_old, with_ref, kl, kc, ec, dual, temperature, V, dtype = case
    T = 29 if lens is None else sum(lens) + 2      # two tokens of no sequence at the end
    lo, hi = 0.2, 0.28
    x, _ = make_logits(T, V, dtype, 21, stride=V + 3, offset=1)
    y = make_targets(T, V, 22)
    off = None if lens is None else make_offsets(lens)
    lp = reference(x, y, temperature)[1]
    # odd hundredths: off the clip's edges by more than the bound on log p
    step = torch.round(torch.randn(T, device=DEV, generator=gen(3)) * 10.0) + 0.5
    old = (lp - 0.02 * step).float() if with_old else None
    ref = (lp + 0.3 * torch.randn(T, device=DEV, generator=gen(4))).float() if with_ref else None
    adv = torch.randn(len(lens) if per == "sequence" else T, device=DEV, generator=gen(5)) + 0.3
    kw = dict(offsets=off, clip_low=lo, clip_high=hi, dual_clip=dual, kl=kl, kl_coef=kc, entropy_coef=ec, reduce=reduce,
              temperature=temperature)
    q = zg.policy_loss(x, y, adv, old, ref, **kw)
    w = policy_reference(x, y, adv, old, ref, off, lo, hi, dual, kl, kc, ec, reduce, temperature)
    E = bound(x, temperature) * (1 + w["lp"].abs())
    assert float(E.max()) < 2e-3
    live = w["live"]
    check(q.logp, w["lp"], bound(x, temperature), "logp")
    if ec:
        check(q.entropy[live], w["ent"][live], (bound(x, temperature) * (1 + w["ent"]))[live], "entropy")
    assert abs(float(q.clip_fraction) - w["clip"]) <= 2.0 ** -23
    # d loss / d logp times its error, the entropy's, and a few roundings of each term
    terms = w["w"] * (w["r"] * w["A"].abs() + kc * 4 + ec * w["ent"])
    tol = (w["w"] * (w["r"] * w["A"].abs() + kc * 4 + ec * (1 + w["ent"])) * 2 * E).sum() + 2.0 ** -21 * terms.sum()
    assert abs(float(q.loss) - float(w["loss"])) <= float(tol)
    if ref is not None:
        d = (ref.double() - w["lp"]).abs()
        tol = float((torch.where(live, (1 + torch.exp(d)) * E + 2.0 ** -20 * (1 + d), torch.zeros_like(E))).sum()) / max(1, int(live.sum()))
        assert abs(float(q.kl) - w["kl"]) <= tol
    else:
        assert float(q.kl) == 0.0
    g, h = w["g"], (w["h"] if ec else None)
    zero = torch.zeros_like(g)
    g = torch.where(live, g, zero)
    want = reference_grad(w["logq"], y, g, None if h is None else torch.where(live, h, zero), w["ent"], temperature)
    want = torch.where(live[:, None], want, torch.zeros_like(want))
    # the coefficients' own error: r and the KL's slope move with log p
    p = torch.exp(w["logq"])
    hot = torch.zeros_like(p).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    gerr = w["w"] * ((w["r"] * w["A"].abs() + kc * 4) * (E + 2.0 ** -21))
    size = g.abs() + (w["h"].abs() * (1 + w["ent"]) if ec else 0)
    plogp = torch.where(p > 0, p * w["logq"].abs(), torch.zeros_like(p))
    tol = ((2 * E * size + gerr)[:, None] * (p + hot) + (2 * E * w["h"].abs())[:, None] * plogp) / temperature
    tol = tol + UNIT[dtype] * want.abs() + 2.0 ** -100 + (2.0 ** -25 if dtype == "fp16" else 0.0)
    err = (q.dlogits.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err - tol).max()))
    assert bool((q.dlogits[~live] == 0).all())
    again = zg.policy_loss(x, y, adv, old, ref, **kw)
    assert all(torch.equal(a, b) for a, b in zip(q, again) if a is not None)
    inplace = zg.policy_loss(x, y, adv, old, ref, out=x, **kw)
    assert torch.equal(x, q.dlogits) and torch.equal(inplace.loss, q.loss)


MANY = [  # as POLICY, with more tokens than a CTA takes at a time: one sequence, a long one among short ones, none
    ((5001,), "sequence", "sequence", True, True, "k3", 0.05, 0.01, 0.0, 1.0, 40, "bf16"),
    ((3, 0, 9000, 1, 70, 0), "sequence", "token", True, False, "k1", 0.0, 0.0, 3.0, 0.8, 24, "fp32"),
    ((40,) * 130, "token", "sequence", False, True, "k2", 0.1, 0.0, 0.0, 1.0, 33, "fp16"),
]


@pytest.mark.parametrize("case", MANY)
def test_policy_loss_of_many_tokens(case):
    test_policy_loss(case)


@pytest.mark.parametrize("T", [61, 6000])
@pytest.mark.parametrize("reduce", ["token", "sequence", "sum"])
def test_tokens_of_no_sequence(T, reduce):
    """Tokens in front of the first sequence and behind the last change nothing: the same gradients as
    without them, bit for bit, and the same loss but for one rounding of each."""
    x, _ = make_logits(T, 33, "fp32", 5)
    y = make_targets(T, 33, 6)
    n = T - 8
    off = torch.tensor([3, 3, 10, 12, n + 3], device=DEV)
    adv = torch.rand(4, device=DEV, generator=gen(7)) + 0.5  # every term of the loss has one sign
    q = zg.policy_loss(x, y, adv, offsets=off, reduce=reduce)
    r = zg.policy_loss(x[3:n + 3], y[3:n + 3], adv, offsets=off - 3, reduce=reduce)
    assert torch.equal(q.dlogits[3:n + 3], r.dlogits)
    assert bool((q.dlogits[:3] == 0).all()) and bool((q.dlogits[n + 3:] == 0).all())
    assert abs(float(q.loss) - float(r.loss)) <= 2.0 ** -22 * abs(float(r.loss))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V", [(40, 50304), (1300, 600)])
def test_padding_with_the_lowest_value(T, V, dtype):
    """Over a vocabulary padded with the type's lowest value or with -inf the terms are the same zeros."""
    x, _ = make_logits(T, V, dtype, 9)
    y = make_targets(T, V - 100, 8)
    adv = torch.randn(T, device=DEV, generator=gen(3))
    results = []
    for mask in (torch.finfo(TYPES[dtype]).min, -math.inf):
        x[:, -100:] = mask
        f = zg.token_logp(x, y, entropy=True)
        q = zg.policy_loss(x, y, adv, entropy_coef=0.02)
        results.append([f.logp, f.lse, f.entropy, q.logp, q.entropy, q.loss, q.dlogits])
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(a.isfinite().all())


def test_policy_gradient_against_differences():
    """Central differences of the 64-bit loss in logits of both sequences; the loss is smooth
    here (no ratio near an edge), its third derivatives below 30."""
    V, T, s = 11, 7, 1e-4
    x, _ = make_logits(T, V, "fp32", 31, spread=1.0)
    y = torch.randint(0, V, (T,), device=DEV, generator=gen(1))
    off = make_offsets([4, 3])
    lp = reference(x, y)[1]
    old, ref = (lp - 0.01).float(), (lp + 0.2).float()
    adv = torch.tensor([0.7, -0.4], device=DEV)
    kw = dict(kl="k3", kc=0.1, ec=0.05, reduce="sequence", temperature=1.0)
    q = zg.policy_loss(x, y, adv, old, ref, offsets=off, kl="k3", kl_coef=0.1, entropy_coef=0.05, reduce="sequence")

    def value(z):
        return float(policy_reference(z, y, adv, old, ref, off, 0.2, 0.2, 0.0, **kw)["loss"])
    for t in (0, 3, 5):
        for j in range(V):
            up, down = x.double().clone(), x.double().clone()
            up[t, j] += s
            down[t, j] -= s
            diff = (value(up) - value(down)) / (2 * s)
            assert abs(float(q.dlogits[t, j]) - diff) <= s * s / 6 * 30 + 2.0 ** -48 / s + 4 * float(bound(x)[t])


def test_nothing_to_learn_from():
    """No target at all, and no tokens at all: losses of 0 (or a pair's at margin 0), zero gradients."""
    x, _ = make_logits(5, 40, "bf16", 2)
    y = torch.full((5,), -1, device=DEV)
    off = make_offsets([3, 2])
    q = zg.policy_loss(x, y, torch.ones(2, device=DEV), torch.zeros(5, device=DEV), offsets=off, reduce="sequence")
    assert float(q.loss) == 0 and float(q.clip_fraction) == 0 and bool((q.dlogits == 0).all())
    r = zg.preference_loss(x, y, off)
    assert abs(float(r.loss) - math.log(2)) <= 2.0 ** -24 and bool((r.dlogits == 0).all())
    e, ye = x[:0], y[:0]
    f = zg.token_logp(e, ye, entropy=True)
    assert f.logp.shape == (0,) and zg.token_logp_backward(e, ye, f, f.logp, f.logp).shape == (0, 40)
    z = make_offsets([0, 0])
    r = zg.preference_loss(e, ye, z)
    assert abs(float(r.loss) - math.log(2)) <= 2.0 ** -24 and r.dlogits.shape == (0, 40)
    q = zg.policy_loss(e, ye, torch.ones(2, device=DEV), offsets=z, reduce="sequence")
    assert float(q.loss) == 0 and float(q.kl) == 0


def test_long_offsets_pass_32_bits():
    """Rows whose element offsets pass 2^31: the last rows of 50257-wide logits of 4.4 GB."""
    T, V = 43000, 50257
    assert (T - 1) * V > 2 ** 31
    x = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    x[-2:].copy_(torch.randn((2, V), device=DEV, generator=gen(1)))
    y = torch.full((T,), -1, device=DEV)
    y[-2:] = torch.tensor([17, V - 1], device=DEV)
    f = zg.token_logp(x, y)
    logq, lp, _, ent = reference(x[-2:], y[-2:])
    check(f.logp[-2:], lp, bound(x[-2:]), "logp")
    g = torch.ones(T, device=DEV)
    want = reference_grad(logq, y[-2:], torch.ones(2, device=DEV, dtype=torch.float64), None, ent, 1.0)
    q = zg.policy_loss(x, y, -g, f.logp, reduce="sum")
    d = zg.token_logp_backward(x, y, f, g, out=x)
    ones = torch.ones(2, device=DEV, dtype=torch.float64)
    check_grad(d[-2:], want, logq, y[-2:], ones, None, ent, bound(torch.randn(2, V)).to(DEV) * 2, "bf16", 1.0)
    check_grad(q.dlogits[-2:], want, logq, y[-2:], ones, None, ent, bound(torch.randn(2, V)).to(DEV) * 4, "bf16", 1.0)
    assert float(d[:-2].abs().max()) == 0 and float(q.dlogits[:-2].abs().max()) == 0


def test_side_stream_and_graph():
    """A call on a stream of its own, and one captured in a CUDA graph and replayed on new values."""
    x, _ = make_logits(40, 1003, "bf16", 5)
    y = make_targets(40, 1003, 6)
    off = make_offsets([10, 10, 12, 8])
    ref = torch.randn(40, device=DEV, generator=gen(3)) - 6
    adv = torch.randn(4, device=DEV, generator=gen(4))
    want_f, want_p = zg.token_logp(x, y, entropy=True), zg.preference_loss(x, y, off, ref)
    want_q = zg.policy_loss(x, y, adv, ref, offsets=off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = zg.token_logp(x, y, entropy=True, stream=side)
    p = zg.preference_loss(x, y, off, ref, stream=side)
    q = zg.policy_loss(x, y, adv, ref, offsets=off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((f, want_f), (p, want_p), (q, want_q)):
        assert all(torch.equal(u, v) for u, v in zip(a, b) if u is not None)
    keep = x.clone()
    import gc
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf = zg.token_logp(x, y, entropy=True)
        gp = zg.preference_loss(x, y, off, ref)
        gq = zg.policy_loss(x, y, adv, ref, offsets=off)
    x.mul_(0.5)
    graph.replay()
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in ((gf, want_f), (gp, want_p), (gq, want_q)):
        assert all(torch.equal(u, v) for u, v in zip(a, b) if u is not None)


LINEAR = [  # T, V, D, ld_hidden, ld_weight
    (1, 1, 8, 8, 8), (1, 9, 3, 8, 8), (1, 50257, 768, 768, 768), (3, 127, 64, 64, 64), (5, 129, 72, 80, 88), (16, 1000, 8, 8, 16),
    (130, 300, 200, 200, 200), (257, 2049, 136, 136, 136), (64, 4096, 1024, 1024, 1024), (300, 777, 1000, 1000, 1008),
    (300, 20011, 264, 264, 264), (500, 20011, 520, 520, 520), (640, 9001, 64, 64, 64),  # tiles of 128 tokens, and of 256
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D,ldh,ldw", LINEAR)
def test_linear_logp(T, V, D, ldh, ldw, dtype):
    """The products are exact in fp32 and their sum of D terms is off by at most D + 16 roundings of
    the sum of magnitudes S = sum |h w|; this error of each logit enters log p twice (the
    target's and, averaged, the sum's), and the softmax adds E."""
    t = TYPES[dtype]
    hflat = torch.full((T, ldh), float("nan"), device=DEV, dtype=t)
    wflat = torch.full((V, ldw), float("nan"), device=DEV, dtype=t)
    hidden, weight = hflat[:, :D], wflat[:, :D]
    hidden.copy_(torch.randn((T, D), device=DEV, generator=gen(1)))
    weight.copy_(torch.randn((V, D), device=DEV, generator=gen(2)) * (2.0 / math.sqrt(D)))
    y = make_targets(T, V, 3, masked=0.2 if T > 1 else 0.0)
    for temperature, with_entropy in ((1.0, True), (1.4, False)):
        f = zg.linear_logp(hidden, weight, y, temperature=temperature, entropy=with_entropy)
        z = hidden.double() @ weight.double().T
        _, lp, lse, ent = reference(z, y, temperature)
        S = (hidden.double().abs() @ weight.double().abs().T).amax(1) / temperature
        E = bound(z, temperature) + 2 * (D + 16) * 2.0 ** -24 * S
        check(f.logp, lp, E, "logp")
        check(f.lse, lse, E, "lse")
        if with_entropy:
            check(f.entropy, ent, E * (2 + math.log(V) + 28), "entropy")
        again = zg.linear_logp(hidden, weight, y, temperature=temperature, entropy=with_entropy)
        assert torch.equal(f.logp, again.logp) and torch.equal(f.lse, again.lse)


def test_linear_logp_agrees_with_token_logp():
    """The frozen side's log-probabilities against those of the materialised logits in fp32."""
    T, V, D = 70, 1500, 256
    hidden = torch.randn((T, D), device=DEV, generator=gen(1)).to(torch.bfloat16)
    weight = (torch.randn((V, D), device=DEV, generator=gen(2)) / 8).to(torch.bfloat16)
    y = make_targets(T, V, 3)
    y[5] = V + 1
    a = zg.linear_logp(hidden, weight, y, entropy=True)
    b = zg.token_logp((hidden.double() @ weight.double().T).float(), y, entropy=True)
    ok = torch.arange(T, device=DEV) != 5
    assert bool(a.logp[5].isnan()) and bool(b.logp[5].isnan())
    assert bool(((a.logp - b.logp)[ok].abs() <= 1e-4).all()) and bool(((a.entropy - b.entropy)[ok].abs() <= 1e-4).all())
    empty = zg.linear_logp(hidden[:0], weight, y[:0])
    assert empty.logp.shape == (0,)


def test_refusals():
    x, _ = make_logits(4, 32, "bf16", 1)
    y = make_targets(4, 32, 2, masked=0.0)
    f = zg.token_logp(x, y)
    g = torch.ones(4, device=DEV)
    off = make_offsets([2, 2])
    bad = [
        lambda: zg.token_logp(x.cpu(), y), lambda: zg.token_logp(x, y.int()), lambda: zg.token_logp(x, y[:3]),
        lambda: zg.token_logp(x.double(), y), lambda: zg.token_logp(x.T, y), lambda: zg.token_logp(x[0], y),
        lambda: zg.token_logp(x[:1].expand(4, 32), y), lambda: zg.token_logp(x, y.cpu()),
        lambda: zg.token_logp_backward(x, y, f, g, g), lambda: zg.token_logp_backward(x, y, f, g.double()),
        lambda: zg.token_logp_backward(x, y, f, g, out=torch.empty(4, 31, device=DEV, dtype=torch.bfloat16)),
        lambda: zg.preference_loss(x, y, off[:2]), lambda: zg.preference_loss(x, y, off.int()),
        lambda: zg.preference_loss(x, y, off, g[:2]),
        lambda: zg.policy_loss(x, y, g[:3], offsets=off), lambda: zg.policy_loss(x, y, g, old_logp=g[:1]),
        lambda: zg.policy_loss(x, y, g[:2], per_sequence=True),
        lambda: zg.policy_loss(x, y, g, offsets=make_offsets([1, 1, 1, 1])),
        lambda: zg.linear_logp(x, x.half(), y), lambda: zg.linear_logp(x, x[:, :16], y),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was not refused")
    with pytest.raises(KeyError):
        zg.preference_loss(x, y, off, kind="other")
    coded = [
        (-1, lambda: zg.token_logp(x, y, temperature=0.0)), (-1, lambda: zg.token_logp(x, y, temperature=math.inf)),
        (-1, lambda: zg.token_logp(x, y, temperature=math.nan)),
        (-1, lambda: zg.preference_loss(x, y, off, beta=0.0)), (-1, lambda: zg.preference_loss(x, y, off, label_smoothing=0.7)),
        (-1, lambda: zg.policy_loss(x, y, g, clip_low=1.5)), (-1, lambda: zg.policy_loss(x, y, g, clip_high=-0.1)),
        (-1, lambda: zg.policy_loss(x, y, g, dual_clip=0.5)), (-1, lambda: zg.policy_loss(x, y, g, kl_coef=0.1)),
        (-1, lambda: zg.policy_loss(x, y, g, reduce="sequence")), (-1, lambda: zg.policy_loss(x, y, g, kl_coef=math.nan, ref_logp=g)),
        (-1, lambda: zg.linear_logp(x.float(), x.float(), y)), (-2, lambda: zg.linear_logp(x[:, 1:], x[:, 1:], y)),
        (-2, lambda: zg.linear_logp(torch.zeros(4, 30, device=DEV).half(), torch.zeros(9, 30, device=DEV).half(), y)),
        # in place needs the logits' own row stride
        (-1, lambda: zg.token_logp_backward(x, y, f, g, out=x.as_strided((4, 32), (33, 1)))),
    ]
    for code, call in coded:
        with pytest.raises(zg.ZeroError) as e:
            call()
        assert e.value.code == code

