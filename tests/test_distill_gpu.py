"""distill_loss against its definition in 64 bits, written here with elementary operations, and its gradient
against the formula's and against differences.

Tolerances. u = 2^-24. As for the other losses a log-probability log q is within E = 2^-22 (8 + R) + 2^-24 n / 256
of its value, R = max |z - max z| that matters (cut at 28) plus log V, times 1 + |log q|; so is the rest's, whose
sum is formed over its own terms. With l = E (2 + |log p| + |log q|) an entry's r = log p - log q is within l (the
teacher's numbers are exact, exp(log p) is within u (2 + |log p|)). D's terms p r, q r are then within
p (l + |r| 2^-22 (2 + |log p|)) and q (l + |r| l); the js terms lie between those. The sums of at most 513 terms
over 32 lanes add 22 u of their magnitudes. A gradient entry c - q C, with c of the size of p, q (1 + |r|) or less,
takes the same bounds once more, E for its own q. p_rest from 1 - sum p is off by 600 u absolutely (sums of
513 numbers of at most 1), which for D counts with 1 + |r|. Gradients are rounded once to their type.
"""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
U = 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def place(x, stride=None, offset=0):
    T, V = x.shape
    stride = stride or V
    flat = torch.full((offset + max(T, 1) * stride + 16,), math.nan, device=DEV, dtype=x.dtype)
    out = flat[offset:].as_strided((T, V), (stride, 1))
    out.copy_(x)
    return out, flat


def data(T, V, k, dtype, seed, noise=0.7, masked=0.25, short=True):
    """Student logits, targets, and the lists of a teacher that the student differs from."""
    g = gen(seed)
    z = torch.randn((T, V), device=DEV, generator=g) * 2
    x = (z + noise * torch.randn((T, V), device=DEV, generator=g)).to(TYPES[dtype])
    y = torch.randint(0, V, (T,), device=DEV, generator=g)
    if masked and T > 1:
        y = torch.where(torch.rand(T, device=DEV, generator=g) < masked, -1, y)
    logp = torch.log_softmax(z.double(), 1)
    top = torch.topk(logp, k, dim=1)
    index, lp = top.indices, top.values.float()
    if short and k > 2:  # lists of any length, with holes
        gone = torch.rand((T, k), device=DEV, generator=g) < 0.2
        index = index.masked_fill(gone, -1)
        lp = lp.masked_fill(torch.rand((T, k), device=DEV, generator=g) < 0.1, -math.inf)
    index = index.contiguous()
    there = (index >= 0) & (lp > -math.inf)
    left = logp.clone()
    left.scatter_(1, index.clamp(min=0), torch.where(there, -math.inf, left.gather(1, index.clamp(min=0))))
    left = torch.cat([left, left.new_full((T, 1), -math.inf)], 1)
    rest = torch.logsumexp(left, 1).float()
    return x, y, index, lp.contiguous(), rest


def weights(y, offsets, reduce):
    T = y.shape[0]
    live = (y >= 0).double()
    seq = None
    if offsets is not None:
        seq = torch.searchsorted(offsets[1:].contiguous(), torch.arange(T, device=DEV), right=True)
        live = live * ((torch.arange(T, device=DEV) >= offsets[0]) & (seq < offsets.numel() - 1)).double()
    if reduce == "token":
        return live / max(1.0, float(live.sum()))
    if reduce == "sum":
        return live
    n = torch.zeros(offsets.numel(), dtype=torch.float64, device=DEV).index_add_(0, seq, live)
    return live / n.clamp(min=1)[seq] / max(1, int((n > 0).sum()))


def reference(x, y, index, lp, rest, w, kind, tail, mix, kl_coef, ce_coef, temperature):
    """(D, logp, gradient, and the bounds of D, logp and the gradient without its last rounding)."""
    T, V = x.shape
    k = index.shape[1]
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    logq = (z - m) - torch.log(torch.exp(z - m).sum(1, keepdim=True))
    there = (index >= 0) & (lp > -math.inf)
    at = index.clamp(min=0)
    member = torch.zeros((T, V + 1), dtype=torch.bool, device=DEV).scatter_(1, torch.where(there, index, V), True)[:, :V]
    outside = torch.where(member, -math.inf, logq)
    top = outside.amax(1, keepdim=True).clamp(min=-1e300)
    lqr = top[:, 0] + torch.log(torch.exp(outside - top).sum(1))
    lq = torch.where(there, logq.gather(1, at), -math.inf)
    P = torch.where(there, lp.double(), -math.inf)
    loose = torch.zeros(T, dtype=torch.float64, device=DEV)
    if tail == "renormalise":
        P = P - torch.log(torch.exp(P).sum(1, keepdim=True))
        P = torch.where(there, P, -math.inf)
    if tail == "rest":
        if rest is not None:
            pr = rest.double()
        else:
            pr = torch.log((1 - torch.exp(P).sum(1)).clamp(min=2.0 ** -24))
            loose = 600 * U / torch.exp(pr)  # relative to p_rest
    else:
        pr, lqr = torch.full_like(lqr, -math.inf), torch.full_like(lqr, -math.inf)
    whole = there.sum(1) == V
    pr = torch.where(whole, -math.inf, pr)
    P, lq = torch.cat([P, pr[:, None]], 1), torch.cat([lq, lqr[:, None]], 1)
    p, q = torch.exp(P), torch.exp(lq)
    both = (P == -math.inf) & (lq == -math.inf)
    r = torch.where(both, 0.0, P - lq)
    fin = lambda v: torch.where(v.isfinite(), v, 0.0)  # noqa: E731
    if kind == "forward":
        d, c = torch.where(p > 0, p * r, 0.0), -p
        size = p
    elif kind == "reverse":
        d = torch.where(q > 0, -q * r, 0.0)
        c, size = d, q
    else:
        lm = torch.log(mix * p + (1 - mix) * q)
        c = torch.where(q > 0, (1 - mix) * q * (lq - lm), 0.0)
        d = torch.where(p > 0, mix * p * (P - lm), 0.0) + c
        size = p + q
    D = d.sum(1)
    C = c.sum(1, keepdim=True)
    live = y >= 0
    yy = y.clamp(min=0)[:, None]
    logp = logq.gather(1, yy)[:, 0]
    prob = torch.exp(logq)
    entry = torch.full((T, V), k, dtype=torch.int64, device=DEV)
    rows, cols = there.nonzero(as_tuple=True)
    entry[rows, index[rows, cols]] = cols
    cond = torch.where(entry < k, 1.0, torch.exp(logq - lqr[:, None]).nan_to_num(0.0))  # a place's share of its entry
    grad = kl_coef * (c.gather(1, entry) * cond - C * prob) + ce_coef * prob
    grad.scatter_add_(1, yy, torch.full_like(logp[:, None], -ce_coef))
    scale = torch.where(live, w, 0.0)[:, None] / temperature
    grad = torch.where(scale == 0, 0.0, grad * scale)

    R = torch.clamp((m - torch.where(z.isfinite(), z, m).amin(1, keepdim=True))[:, 0], max=28.0) + math.log(V)
    E = (2.0 ** -22 * (8 + R) + 2.0 ** -24 * V / 256)[:, None]
    l = E * (2 + fin(P).abs() + fin(lq).abs())
    extra = torch.zeros_like(l)
    extra[:, k] = loose
    ar = fin(r).abs()
    each = size * (l * (1 + ar) + ar * 2.0 ** -22 * (2 + fin(P).abs()) + extra * (1 + ar)) + 22 * U * fin(d).abs()
    dtol = each.sum(1) + U * D.abs()
    # a place takes its share of its entry's bounds, and its probability's of the sum's
    entry_tol = each + fin(c).abs() * (2.0 ** -22 * (2 + fin(P).abs()) + extra + 2 * E) + E * size
    sum_tol = entry_tol.sum(1, keepdim=True)
    gtol = abs(kl_coef) * (cond * entry_tol.gather(1, entry) + prob * (sum_tol + 2 * E * C.abs())) + 2 * E * abs(ce_coef) * prob
    hot = torch.zeros_like(prob).scatter_(1, yy, abs(ce_coef))
    gtol = (gtol + hot * 2.0 ** -22) * scale.abs() + 2.0 ** -110
    return torch.where(live, D, 0.0), torch.where(live, logp, 0.0), grad, dtol, E[:, 0] * (1 + fin(logp).abs()), gtol


def close(got, want, tol, what):
    same = got.double() == want
    near = (got.double() - want).abs() <= tol
    bad = ~(same | near)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist(), tol.expand_as(want)[bad][:3].tolist())


def check(x, y, index, lp, rest, dtype, offsets=None, kind="forward", tail="rest", mix=0.5, kl_coef=1.0, ce_coef=0.0, reduce="token",
          temperature=1.0, out=None):
    keep = x.clone()
    w = weights(y, offsets, reduce)
    D, logp, grad, dtol, ltol, gtol = reference(keep, y, index, lp, rest, w, kind, tail, mix, kl_coef, ce_coef, temperature)
    r = zg.distill_loss(x, y, index, lp, rest, offsets=offsets, kind=kind, tail=tail, mix=mix, kl_coef=kl_coef, ce_coef=ce_coef,
                        reduce=reduce, temperature=temperature, out=out)
    on = w > 0
    D, logp = torch.where(on, D, 0.0), torch.where(on, logp, 0.0)
    close(r.token_kl, D, dtol, "token_kl")
    close(r.logp, logp, ltol, "logp")
    tol = 0.0
    for coef, v, t in ((kl_coef, D, dtol), (ce_coef, logp, ltol)):
        if coef:
            tol = tol + abs(coef) * (w * (t + 2 * U * v.abs())).sum()
    want = (w * ((kl_coef * D if kl_coef else 0.0) - (ce_coef * logp if ce_coef else 0.0))).sum()
    close(r.loss, want, tol, "loss")
    n = max(1, int(on.sum()))
    close(r.kl, D.sum() / n, dtol[on].sum() / n + 2 * U * D.abs().sum() / n, "kl")
    close(r.dlogits, grad, gtol + UNIT[dtype] * grad.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0), "dlogits")
    assert bool((r.dlogits[~on] == 0).all())
    return r


SHAPES = [  # T, V, k, stride, offset
    (1, 1, 1, None, 0), (1, 50257, 32, None, 0), (3, 7, 7, None, 1), (5, 8, 3, None, 0), (4, 9, 1, 17, 3), (2, 600, 512, 601, 5),
    (17, 1000, 64, 1008, 0), (33, 4099, 65, None, 5), (64, 257, 5, 264, 0), (2, 151936, 300, None, 1), (330, 50257, 64, None, 0),
    (310, 9001, 20, 9002, 1), (1300, 515, 64, 518, 1), (1217, 3, 2, None, 0), (400, 30011, 8, None, 2), (310, 80001, 40, None, 0),
    (160, 151937, 24, None, 0), (310, 50257, 512, None, 1), (700, 20011, 500, None, 0), (1300, 8001, 3, None, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,k,stride,offset", SHAPES)
def test_shapes(T, V, k, stride, offset, dtype):
    x, y, index, lp, rest = data(T, V, k, dtype, T + V)
    x, _ = place(x, stride, offset)
    check(x, y, index, lp, rest, dtype, ce_coef=0.3)
    out, flat = place(torch.zeros_like(x), (stride or V) + 3, offset + 1)  # another alignment
    check(x, y, index, lp, None, dtype, tail="renormalise", temperature=0.7, out=out)
    assert int(flat.isnan().sum()) == flat.numel() - T * V
    own, _ = place(x, stride, offset)
    r = check(own, y, index, lp, rest, dtype, kind="reverse")
    again = zg.distill_loss(own, y, index, lp, rest, kind="reverse", out=own)  # in place
    assert torch.equal(again.dlogits, r.dlogits) and again.dlogits.data_ptr() == own.data_ptr()


@pytest.mark.parametrize("V,dtype", [(3001, "bf16"), (50257, "bf16"), (50257, "fp32"), (140001, "bf16")])
@pytest.mark.parametrize("kind,tail,known", [("forward", "rest", True), ("forward", "rest", False), ("forward", "drop", True),
                                             ("forward", "renormalise", True), ("reverse", "rest", True), ("reverse", "rest", False),
                                             ("js", "rest", True), ("js", "rest", False)])
def test_kinds(kind, tail, known, V, dtype):
    T = 61
    x, y, index, lp, rest = data(T, V, 48, dtype, V)
    off = torch.tensor([2, 2, 20, 41, 41, 58], device=DEV)
    for reduce, kl_coef, ce_coef, temperature, mix in (("token", 1.0, 0.0, 1.0, 0.5), ("sequence", 0.7, 0.5, 1.5, 0.1), ("sum", 0.0, 1.0, 0.6, 0.9)):
        check(x, y, index, lp, rest if known else None, dtype, offsets=off, kind=kind, tail=tail, mix=mix, kl_coef=kl_coef,
              ce_coef=ce_coef, reduce=reduce, temperature=temperature)


@pytest.mark.parametrize("T,V", [(6, 5000), (6, 50257), (320, 20001), (3, 160001)])
def test_by_differences(T, V):
    """The gradient in fp32 against central differences of the 64-bit definition along random directions: the
    definition is smooth, with step 1e-4 the third derivative's share is below 1e-7 of |d|^3-sized terms."""
    x, y, index, lp, rest = data(T, V, 16, "fp32", 5)
    w = weights(y, None, "token")
    g = gen(9)
    for kind in ("forward", "reverse", "js"):
        r = zg.distill_loss(x, y, index, lp, rest, kind=kind, ce_coef=0.2)
        d = torch.randn((T, V), device=DEV, generator=g, dtype=torch.float64)
        d.scatter_(1, index.clamp(min=0), 3.0)

        def loss(e):
            D, logp, *_ = reference(x.double() + e * d, y, index, lp, rest, w, kind, "rest", 0.5, 1.0, 0.2, 1.0)
            return float((w * (D - 0.2 * logp)).sum())

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        got = float((r.dlogits.double() * d).sum())
        assert abs(slope - got) <= 1e-5 * float((r.dlogits.double() * d).abs().sum()) + 1e-7


@pytest.mark.parametrize("V,dtype", [(5000, "fp32"), (50257, "bf16"), (160001, "fp16")])
def test_a_rest_of_little_probability(V, dtype):
    """A student that is nearly sure of the list: the rest's probability, 1e-11 and 1e-30 of all, and its
    gradient keep their full precision."""
    T, k = 4, 5
    for gap in (25.0, 69.0):
        x = torch.randn((T, V), device=DEV, generator=gen(1)).clamp(-2, 2)
        index = torch.stack([torch.randperm(V, device=DEV, generator=gen(i))[:k] for i in range(T)])
        x.scatter_(1, index, gap + math.log(V) + torch.randn((T, k), device=DEV, generator=gen(3)))
        x = x.to(TYPES[dtype])
        lp = torch.log_softmax(torch.randn((T, k), device=DEV, generator=gen(4)), 1) - 0.05
        y = index[:, 0].clone()
        y[1] = int((index[1].max() + 1) % V)
        for kind in ("forward", "reverse", "js"):
            check(x, y, index, lp, None, dtype, kind=kind)
            check(x, y, index, lp, torch.full((T,), -3.0, device=DEV), dtype, kind=kind, ce_coef=0.1)


@pytest.mark.parametrize("V,T", [(3000, 9), (50257, 9), (50257, 400), (150000, 9)])
def test_masked_logits(V, T):
    """-inf in the vocabulary: at its end, everywhere but in a few places, in the list, in all of the rest."""
    for dtype in ("bf16", "fp32"):
        x, y, index, lp, rest = data(T, V, 12, dtype, 3, masked=0.0, short=False)
        x[0, V - V // 50:] = -math.inf
        x[1] = torch.where(torch.rand(V, device=DEV, generator=gen(1)) < 0.99, -math.inf, x[1])
        x[2].scatter_(0, index[2, 3:4], -math.inf)  # forward: infinite
        x[3].scatter_(0, index[3], -math.inf)
        only = torch.full((V,), -math.inf, device=DEV, dtype=x.dtype)
        only[index[4]] = x[4, index[4]]
        x[4] = only
        x[5] = torch.finfo(x.dtype).min
        x[5, index[5]] = x[4, index[4]]  # the rest is at the lowest value
        y[0], y[3], y[4] = 5, index[3, 0], index[4, 1]
        y[5] = index[5, 2]
        for kind in ("reverse", "js"):
            check(x, y, index, lp, rest, dtype, kind=kind)
        D, logp, grad, dtol, ltol, gtol = reference(x, y, index, lp, rest, weights(y, None, "token"), "forward", "rest", 0.5, 1.0, 0.0, 1.0)
        r = zg.distill_loss(x, y, index, lp, rest)
        fin = D.isfinite()
        assert torch.equal(r.token_kl.isfinite(), fin) and bool((r.token_kl[~fin] == math.inf).all())
        close(r.token_kl[fin], D[fin], dtol[fin], "token_kl")
        ok = fin & grad.isfinite().all(1)
        close(r.dlogits[ok], grad[ok], (gtol + UNIT[dtype] * grad.abs())[ok], "dlogits")
        assert bool(r.dlogits.isfinite().all())  # an infinite divergence has a finite gradient


@pytest.mark.parametrize("V,T", [(900, 5), (50257, 5), (50257, 330), (150001, 5)])
def test_rows_without_a_result(V, T):
    x, y, index, lp, rest = data(T, V, 8, "bf16", 3, masked=0.0, short=False)
    good = zg.distill_loss(x, y, index, lp, rest, reduce="sum", ce_coef=0.1)
    index[0, 7] = index[0, 2]      # twice
    index[1, 0] = V                # past the vocabulary
    y[2] = V + 3
    x[3, V // 2] = math.nan
    r = zg.distill_loss(x, y, index, lp, rest, reduce="sum", ce_coef=0.1)
    for i in range(4):
        assert bool(r.dlogits[i].isnan().all()) and r.token_kl[i].isnan() and r.logp[i].isnan() == (i != 0 or True)
    for i in range(4, T):
        assert torch.equal(r.dlogits[i], good.dlogits[i]) and r.token_kl[i] == good.token_kl[i]
    assert r.loss.isnan()
    # an entry that is not there may name any place, also one that is there
    index[0, 7], lp[0, 7] = index[0, 2], -math.inf
    one = zg.distill_loss(x[:1], y[:1], index[:1], lp[:1], rest[:1])
    index[0, 7] = -5
    two = zg.distill_loss(x[:1], y[:1], index[:1], lp[:1], rest[:1])
    assert torch.equal(one.dlogits, two.dlogits) and bool(one.dlogits.isfinite().all())
    lp[0, 3] = math.nan
    assert bool(zg.distill_loss(x[:1], y[:1], index[:1], lp[:1], rest[:1]).dlogits.isnan().all())
    x[0] = -math.inf
    lp[0, 3] = -1.0
    none = zg.distill_loss(x[:1], y[:1], index[:1], lp[:1], rest[:1], ce_coef=0.5)
    assert bool((none.dlogits == 0).all()) and none.logp[0] == -math.inf and none.token_kl[0] == math.inf


def test_the_whole_vocabulary_as_a_list():
    """No rest: the divergence of two full softmaxes."""
    T, V = 30, 300
    z, x = (torch.randn((T, V), device=DEV, generator=gen(s)) for s in (1, 2))
    lp = torch.log_softmax(z, 1)
    index = torch.stack([torch.randperm(V, device=DEV, generator=gen(i)) for i in range(T)])
    y = torch.zeros(T, dtype=torch.int64, device=DEV)
    check(x, y, index, lp.gather(1, index).contiguous(), None, "fp32")
    top = zg.top_logits(z, V)
    r = zg.distill_loss(x, y, top.index, top.logp, top.rest, kind="reverse")
    want = (torch.softmax(x.double(), 1) * (torch.log_softmax(x.double(), 1) - torch.log_softmax(z.double(), 1))).sum(1)
    assert bool(((r.token_kl - want).abs() <= 2.0 ** -18 * (1 + want)).all())


def test_a_teacher_of_itself():
    """Lists of the student's own logits: no divergence, and no gradient beyond roundings."""
    x = (torch.randn((50, 50257), device=DEV, generator=gen(1)) * 2)
    y = torch.zeros(50, dtype=torch.int64, device=DEV)
    top = zg.top_logits(x, 64, y)
    for kind in ("forward", "reverse", "js"):
        r = zg.distill_loss(x, y, top.index, top.logp, top.rest, kind=kind, reduce="sum")
        q = torch.softmax(x.double(), 1)
        assert float(r.token_kl.abs().max()) <= 2.0 ** -18
        assert bool((r.dlogits.double().abs() <= 2.0 ** -18 * q + 2.0 ** -110).all())


def test_empty_calls_and_masked_batches():
    x, y, index, lp, rest = data(6, 500, 8, "bf16", 3)
    r = zg.distill_loss(x[:0], y[:0], index[:0], lp[:0], rest[:0])
    assert r.loss == 0 and r.kl == 0 and r.dlogits.shape == (0, 500)
    r = zg.distill_loss(torch.full_like(x, math.nan), torch.full_like(y, -1), index, lp, rest)
    assert r.loss == 0 and bool((r.dlogits == 0).all()) and bool((r.token_kl == 0).all())
    # lists of nothing: the rest is all, on both sides
    r = zg.distill_loss(x, y, torch.full_like(index, -1), lp, None)
    assert float(r.token_kl.abs().max()) <= 2.0 ** -20 and float(r.dlogits.float().abs().max()) <= 2.0 ** -20
    for tail in ("drop", "renormalise"):
        r = zg.distill_loss(x, y, torch.full_like(index, -1), lp, None, tail=tail)
        assert bool((r.token_kl == 0).all()) and bool((r.dlogits == 0).all())


@pytest.mark.parametrize("V", [2000, 50257, 140000])
def test_equal_calls_streams_and_graphs(V):
    x, y, index, lp, rest = data(200, V, 32, "bf16", 1)
    first = zg.distill_loss(x, y, index, lp, rest, ce_coef=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = zg.distill_loss(x, y, index, lp, rest, ce_coef=0.1, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = zg.distill_loss(x, y, index, lp, rest, ce_coef=0.1)
    g.replay()
    for r in (other, held, zg.distill_loss(x, y, index, lp, rest, ce_coef=0.1)):
        assert all(torch.equal(a, b) for a, b in zip(r, first))
    x.copy_(x.roll(1, 0))
    y.copy_(y.roll(3))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, zg.distill_loss(x, y, index, lp, rest, ce_coef=0.1)))


def test_rows_past_two_to_the_31_elements():
    T, V, k = 43001, 50257, 4
    x = torch.zeros((T, V), device=DEV, dtype=torch.bfloat16)
    x[-3:] = torch.randn((3, V), device=DEV, generator=gen(1)).bfloat16()
    y = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    y[-3:] = torch.tensor([5, 50256, 77], device=DEV)
    top = zg.top_logits(x, k, y)
    z = torch.log_softmax(x[-3:].double(), 1)
    want = torch.sort(z, dim=1, descending=True, stable=True)
    # log-probabilities near 10, off by E = 2^-22 (8 + R + log V) with R below 10
    assert torch.equal(top.index[-3:], want.indices[:, :k]) and bool((top.index[:-3] == -1).all())
    assert float((top.logp[-3:] - want.values[:, :k]).abs().max()) <= 2.0 ** -22 * 29 * 13
    index, lp = top.index, (top.logp - 0.1).contiguous()
    r = zg.distill_loss(x, y, index, lp)
    w = torch.full((3,), 1.0 / 3, dtype=torch.float64, device=DEV)
    D, _, grad, dtol, _, gtol = reference(x[-3:], y[-3:], index[-3:], lp[-3:], None, w, "forward", "rest", 0.5, 1.0, 0.0, 1.0)
    close(r.token_kl[-3:], D, dtol, "token_kl")
    close(r.dlogits[-3:], grad, gtol + UNIT["bf16"] * grad.abs(), "dlogits")
    assert int(r.dlogits[:-3].count_nonzero()) == 0


def test_two_calls_at_once():
    """On two streams, each with what it allocates for itself."""
    x, y, index, lp, rest = data(900, 50257, 32, "bf16", 1)
    x2, y2, index2, lp2, rest2 = data(500, 30011, 100, "bf16", 2)
    want, want2 = zg.distill_loss(x, y, index, lp, rest), zg.distill_loss(x2, y2, index2, lp2, rest2, kind="js")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = zg.distill_loss(x, y, index, lp, rest, stream=a)
        got2 = zg.distill_loss(x2, y2, index2, lp2, rest2, kind="js", stream=b)
        top = zg.top_logits(x2, 50, stream=b)
        top2 = zg.top_logits(x, 50, stream=a)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and all(torch.equal(u, v) for u, v in zip(got2, want2))
        assert torch.equal(top.index, zg.top_logits(x2, 50).index) and torch.equal(top2.logp, zg.top_logits(x, 50).logp)


def test_refusals():
    x, y, index, lp, rest = data(6, 500, 8, "bf16", 3)
    good = dict(logits=x, targets=y, index=index, teacher_logp=lp, teacher_rest=rest)
    wide = torch.zeros((6, 16), dtype=torch.int64, device=DEV)
    for kw in (dict(index=index.int()), dict(index=index[:5]), dict(index=index.cpu()), dict(index=wide[:, ::2]), dict(index=index[0]),
               dict(index=index[:, :0]), dict(index=torch.zeros((6, 513), dtype=torch.int64, device=DEV)), dict(teacher_logp=lp.double()),
               dict(teacher_logp=lp[:, :7]), dict(teacher_rest=rest[:5]), dict(teacher_rest=rest.cpu()), dict(targets=y.int()),
               dict(logits=x.double()), dict(kind="up"), dict(tail="up"), dict(reduce="up"), dict(kind="reverse", tail="drop"),
               dict(kind="js", tail="renormalise"), dict(offsets=torch.tensor(3, device=DEV)), dict(out=x[:, :499]), dict(out=x.float())):
        with pytest.raises(ValueError):
            zg.distill_loss(**{**good, **kw})
    for kw in (dict(mix=0.0), dict(mix=1.0), dict(mix=math.nan), dict(kl_coef=math.inf), dict(ce_coef=math.nan), dict(ce_coef=1e39),
               dict(temperature=0.0), dict(reduce="sequence")):
        with pytest.raises(zg.ZeroError):
            zg.distill_loss(**{**good, **kw})
    with pytest.raises(zg.ZeroError):
        zg.distill_loss(torch.zeros((1, 2 ** 20 + 1), device=DEV), y[:1], index[:1], lp[:1])
