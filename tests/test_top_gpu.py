"""top_logits against a stable sort and 64-bit formulas written here with elementary operations.

Tolerances. The indices are exact. For the rest u = 2^-24: a term's exponent carries three roundings of a
number of at most R = max z - min z that matters (cut at 28, smaller terms are lost in the sum), the
exponential 2^-22, and a thread's sum n / 128 roundings: log-probabilities, lse and rest are within
E = 2^-22 (8 + R + log V) + 2^-24 n / 128, times 1 + |value| for the final roundings. The rest is relative to
its own largest term, so the same bound holds for it however small it is.
"""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def place(x, stride=None, offset=0):
    """The matrix inside a larger allocation, NaN around its rows, which no call may read."""
    T, V = x.shape
    stride = stride or V
    flat = torch.full((offset + max(T, 1) * stride + 16,), math.nan, device=DEV, dtype=x.dtype)
    out = flat[offset:].as_strided((T, V), (stride, 1))
    out.copy_(x)
    return out


def check(x, k, temperature=1.0, targets=None):
    got = zg.top_logits(x, k, targets, temperature=temperature)
    T, V = x.shape
    assert got.index.shape == got.logp.shape == (T, k) and got.lse.shape == got.rest.shape == (T,)
    for i in range(0, T, 512):  # rows at a time
        rows = slice(i, i + 512)
        z = x[rows].double() / temperature
        v, at = torch.sort(z, dim=1, descending=True, stable=True)
        m = torch.where(v[:, :1] == -math.inf, 0.0, v[:, :1])
        e = torch.exp(v - m)
        total = torch.log(e.sum(1, keepdim=True))
        lse, logp = (m + total)[:, 0], torch.where(v[:, :k] == -math.inf, -math.inf, (v[:, :k] - m) - total)
        logp = torch.where(lse[:, None] == -math.inf, -math.inf, logp)
        if k < V:
            mr = torch.where(v[:, k:k + 1] == -math.inf, 0.0, v[:, k:k + 1])
            rest = (mr - m)[:, 0] + torch.log(torch.exp(v[:, k:] - mr).sum(1)) - total[:, 0]
            rest = torch.where(v[:, k] == -math.inf, -math.inf, rest)
        else:
            rest = torch.full_like(lse, -math.inf)
        fin = torch.where(z.isfinite(), z, m)
        R = torch.clamp(fin.amax(1) - fin.amin(1), max=28.0) + math.log(V)
        E = 2.0 ** -22 * (8 + R) + 2.0 ** -24 * V / 128
        on = torch.ones(z.shape[0], dtype=torch.bool, device=DEV) if targets is None else targets[rows] >= 0
        assert torch.equal(got.index[rows], torch.where(on[:, None], at[:, :k], -1))
        for what, a, b, tol in (("logp", got.logp[rows], logp, E[:, None]), ("lse", got.lse[rows], lse, E), ("rest", got.rest[rows], rest, E)):
            o = on[:, None] if b.dim() == 2 else on
            b = torch.where(o, b, 0.0)
            same = a.double() == b  # infinities among them
            near = (a.double() - b).abs() <= tol * (1 + b.abs())
            assert bool((same | near).all()), (what, (a.double() - b).abs().nan_to_num(0).max().item(), (~(same | near)).nonzero()[:3].tolist())
    return got


SHAPES = [  # T, V, k, stride, offset
    (1, 1, 1, None, 0), (1, 50257, 20, None, 0), (1, 50257, 512, None, 1), (3, 7, 7, None, 1), (5, 8, 3, None, 0), (4, 9, 1, 17, 3),
    (2, 500, 500, None, 0), (2, 600, 512, 601, 5), (17, 1000, 64, 1008, 0), (33, 4099, 65, None, 5), (2, 8192, 128, None, 8),
    (2, 8192, 129, None, 8), (64, 257, 5, 264, 0), (3, 131072, 300, None, 1), (700, 50257, 64, None, 0), (400, 9001, 200, 9002, 1),
    (1300, 515, 64, 518, 1), (1217, 3, 2, None, 0), (1251, 4099, 40, None, 0), (1300, 240, 33, None, 0), (1300, 257, 64, None, 3),
    (2, 3000001, 100, None, 1), (2, 3000001, 512, None, 0),
    (1300, 8192, 60, None, 0), (1300, 4096, 64, None, 0), (1250, 8190, 7, None, 0), (1250, 8191, 33, 8200, 0),  # a warp each
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,k,stride,offset", SHAPES)
def test_top(T, V, k, stride, offset, dtype):
    x = place((torch.randn((T, V), device=DEV, generator=gen(T + V)) * 3).to(TYPES[dtype]), stride, offset)
    check(x, k)
    targets = torch.randint(-1, 2, (T,), device=DEV, generator=gen(2))
    check(x, k, 0.7, targets)


ROWS = ["equal", "zeros", "few values", "rising", "falling", "mostly -inf", "-inf first", "-inf alone", "lowest", "one high", "far apart", "half full"]


def hard(kind, T, V, dtype, seed):
    x = torch.randn((T, V), device=DEV, generator=gen(seed)) * 3
    low = torch.finfo(dtype).min
    if kind == "equal":
        x = torch.full((T, V), 1.25, device=DEV)
    elif kind == "zeros":  # of both signs
        x = torch.where(x > 0, 0.0, -0.0)
        x[:, ::1001] = 1.0
    elif kind == "few values":
        x = x.round()
    elif kind == "rising":
        x = torch.arange(V, device=DEV, dtype=torch.float32)[None].expand(T, V) / max(1, V // 100)
    elif kind == "falling":
        x = -torch.arange(V, device=DEV, dtype=torch.float32)[None].expand(T, V) / max(1, V // 100)
    elif kind == "mostly -inf":
        x[:, 7:] = torch.where(torch.rand((T, V - 7), device=DEV, generator=gen(seed + 1)) < 20 / V, x[:, 7:], -math.inf)
    elif kind == "-inf first":
        x[:, : V // 2] = -math.inf
    elif kind == "-inf alone":
        x.fill_(-math.inf)
    elif kind == "lowest":
        x.fill_(low)
        x[:, V // 3] = 0.0
        x[:, V - 1] = low / 2
    elif kind == "one high":
        x[:, V // 2] = 200.0
    elif kind == "far apart":
        x = x * 3000
    elif kind == "half full":
        x[T // 2:] = -math.inf
    return x.to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ROWS)
@pytest.mark.parametrize("T,V,k", [(2, 50257, 64), (2, 50257, 400), (160, 20011, 3), (1300, 3001, 30), (9, 300, 100)])
def test_hard_rows(T, V, k, kind, dtype):
    check(hard(kind, T, V, TYPES[dtype], 11), k)


@pytest.mark.parametrize("temperature", [2.0 ** -64, 1e-3, 1e3, 2.0 ** 64])
def test_temperatures(temperature):
    x = torch.randn((3, 5000), device=DEV, generator=gen(1))
    check(x, 40, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V,k", [(3, 50257, 64), (3, 5000, 200), (1300, 500, 20)])
def test_nan_and_infinity(T, V, k, dtype):
    x = (torch.randn((T, V), device=DEV, generator=gen(4)) * 3).to(TYPES[dtype])
    x[0, V // 2] = math.nan
    x[1, V - 1] = math.inf
    if T > 3:
        x[3, 5:] = math.nan
        x[4, 0] = math.nan
    good = x.clone()
    good[0, V // 2] = -math.inf
    r = zg.top_logits(x, k)
    rows = [0, 1] + ([3, 4] if T > 3 else [])
    for a in (r.logp, r.lse, r.rest):
        assert bool(a[rows].isnan().all())
    assert torch.equal(r.index[:2], torch.sort(good[:2].double(), dim=1, descending=True, stable=True).indices[:, :k])
    if T > 3:
        assert set(r.index[3].tolist()) == {-1, 0, 1, 2, 3, 4}
    others = [2] + list(range(5, T))
    check(x[others], k)


def test_wide_fp32_and_many_chunks():
    x = torch.randn((40, 151936), device=DEV, generator=gen(3)) * 2
    for k in (1, 128, 129, 512):
        check(x, k, 2.0)


def test_equal_calls_streams_and_graphs():
    x = (torch.randn((300, 50257), device=DEV, generator=gen(1)) * 2).bfloat16()
    first = zg.top_logits(x, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = zg.top_logits(x, 64, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = zg.top_logits(x, 64)
    g.replay()
    for r in (other, held, zg.top_logits(x, 64)):
        assert all(torch.equal(a, b) for a, b in zip(r, first))
    x.copy_(x.roll(5, 1))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, zg.top_logits(x, 64)))


def test_no_rows_and_refusals():
    x = torch.randn((4, 100), device=DEV)
    r = zg.top_logits(x[:0], 5)
    assert r.index.shape == (0, 5) and r.lse.shape == (0,)
    for k in (0, -1, 101, 513):
        with pytest.raises(ValueError):
            zg.top_logits(x, k)
    with pytest.raises(ValueError):
        zg.top_logits(torch.randn((4, 1000), device=DEV), 513)
    for bad in (x.cpu(), x.double(), x[0], x.T):
        with pytest.raises(ValueError):
            zg.top_logits(bad, 3)
    for bad in (torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            zg.top_logits(x, 3, bad)
    for t in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(zg.ZeroError):
            zg.top_logits(x, 3, temperature=t)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("k", [1, 7, 31, 32, 64])
def test_a_warps_row_of_equal_maxima(k, dtype):
    """Rows of a warp each in which all of its 32 lanes find the same largest value, so that their threshold is known
    without a step of search; each row over another base."""
    T, V = 1300, 2048
    x = torch.randn((T, V), device=DEV, generator=gen(5)).clamp(-3, 3) + torch.arange(T, device=DEV)[:, None] % 50
    per = 16 // torch.empty(0, dtype=TYPES[dtype]).element_size()
    x[:, per - 1:32 * per:per] = (4.0 + torch.arange(T, device=DEV) % 50)[:, None]  # in every lane's first 16 bytes
    check(x.to(TYPES[dtype]), k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,live,k", [(8, 50257, 5, 64), (8, 3000, 5, 400), (1300, 3001, 3, 30), (8, 50257, 5, 400), (8, 300, 1, 2)])
def test_nan_and_infinity_beside_masked_places(T, V, live, k, dtype):
    """Lists that reach into the places at -inf: a row that holds NaN or +inf has no results there either, one
    that does not has -inf."""
    x = torch.full((T, V), -math.inf, device=DEV)
    at = torch.stack([torch.randperm(V, device=DEV, generator=gen(i))[:live] for i in range(T)])
    x.scatter_(1, at, torch.randn((T, live), device=DEV, generator=gen(7)))
    x[0, V // 2] = math.nan
    x[1, V - 1] = math.inf
    x[2, 0], x[2, V // 3] = math.inf, math.nan
    x[3] = -math.inf
    x[3, V // 2] = math.nan
    x = x.to(TYPES[dtype])
    r = zg.top_logits(x, k)
    for a in (r.logp, r.lse, r.rest):
        assert bool(a[:4].isnan().all())
    check(x[4:], k)
    loss = zg.distill_loss(x, torch.zeros(T, dtype=torch.int64, device=DEV), r.index, r.logp, r.rest)
    assert bool(loss.dlogits[:4].isnan().all()) and bool(loss.token_kl[:4].isnan().all())
