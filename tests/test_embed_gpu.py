"""The embedding of tokens and its gradient against 64-bit formulas written here with elementary
operations.

Tolerances. u = 2^-24. A forward value is one product in fp32 with the scale's own rounding, then one
rounding to the type: |w| (3 u + unit). A gradient entry is a sum that passes at most 32 additions in a
block, 32 over a group's blocks, one for each group of 1024 rows of its token, one for the old value and
one product: with n rows of a token, (70 + n / 256) u times the sum of the magnitudes (a quarter of the
longest group covers blocks of 8), then one rounding to the type. Half the smallest fp16 number, 2^-25,
where that type underflows.
"""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def guarded(rows, cols, dtype, seed, stride=None, offset=0, values=True):
    """A matrix inside a larger allocation, NaN before, between and behind its rows."""
    stride = stride or cols
    flat = torch.full((offset + max(rows, 1) * stride + 16,), math.nan, device=DEV, dtype=dtype)
    x = flat[offset:].as_strided((rows, cols), (stride, 1))
    if values:
        x.copy_(torch.randn((rows, cols), device=DEV, generator=gen(seed)))
    return x, flat


def untouched(flat, x, offset):
    """Whether everything around the matrix is still NaN."""
    mask = torch.ones_like(flat, dtype=torch.bool)
    mask[offset:].as_strided(x.shape, x.stride()).fill_(False)
    return bool(flat[mask].isnan().all())


def small(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140


SHAPES = [  # T, V, D, stride, offset
    (1, 1, 1, None, 0), (1, 7, 768, None, 0), (3, 5, 8, None, 1), (17, 100, 257, 260, 3), (300, 50257, 64, None, 0),
    (129, 33, 1000, 1008, 8), (40, 11, 4104, None, 0), (2100, 900, 24, None, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,D,stride,offset", SHAPES)
def test_embedding(T, V, D, stride, offset, dtype):
    w, _ = guarded(V, D, TYPES[dtype], T + V, stride, offset)
    t = torch.randint(0, V, (T,), device=DEV, generator=gen(1))
    if T > 2:
        t[1] = -1
        t[-1] = -2 ** 40
    for scale in (1.0, -math.sqrt(D)):
        got = zg.embedding(w, t, scale=scale)
        want = torch.where((t >= 0)[:, None], w.double()[t.clamp(min=0)] * scale, 0.0)
        assert got.dtype == w.dtype and got.shape == (T, D)
        assert bool(((got.double() - want).abs() <= want.abs() * (3 * U + UNIT[w.dtype]) + small(w.dtype)).all())
    out, flat = guarded(T, D, TYPES[dtype], 0, stride, offset, values=False)
    assert zg.embedding(w, t, scale=scale, out=out) is out and torch.equal(out, got) and untouched(flat, out, offset)


def test_tokens_past_the_matrix_are_not_followed():
    w = torch.randn((10, 64), device=DEV)
    t = torch.tensor([3, 10, -1, 2 ** 62, 9], device=DEV)
    out = zg.embedding(w, t)
    assert bool(out[[1, 3]].isnan().all()) and torch.equal(out[[0, 4]], w[[3, 9]]) and bool((out[2] == 0).all())
    d = zg.embedding_backward(t, torch.ones((5, 64), device=DEV), 10)
    want = torch.zeros((10, 64), device=DEV)
    want[[3, 9]] = 1.0
    assert torch.equal(d, want)


def tokens(kind, T, V, seed):
    if kind == "uniform":
        return torch.randint(0, V, (T,), device=DEV, generator=gen(seed))
    if kind == "one":
        return torch.full((T,), V // 2, device=DEV)
    if kind == "masked":
        return torch.full((T,), -1, device=DEV)
    if kind == "two":  # two tokens in turn, so that every block holds both
        return torch.arange(T, device=DEV) % 2 * (V - 1)
    u = torch.rand(T, device=DEV, generator=gen(seed), dtype=torch.float64)  # text: 1 / rank
    t = (torch.exp(u * math.log(V + 1.0)) - 1).long().clamp(0, V - 1)
    t[::7] = -1
    t[3::11] = V + 5
    return t


def reference(t, dh, V, scale, old):
    live = (t >= 0) & (t < V)
    at = torch.where(live, t, V)
    x = torch.where(live[:, None], dh.double(), 0.0)
    grad = torch.zeros((V + 1, dh.shape[1]), dtype=torch.float64, device=DEV).index_add_(0, at, x)[:V] * scale
    size = torch.zeros((V + 1, dh.shape[1]), dtype=torch.float64, device=DEV).index_add_(0, at, x.abs())[:V] * abs(scale)
    count = torch.zeros(V + 1, dtype=torch.float64, device=DEV).index_add_(0, at, live.double())[:V]
    if old is not None:
        grad, size = grad + old.double(), size + old.double().abs()
    return grad, (70 + count[:, None] / 256) * U * size


BACKWARD = [  # T, V, D, kind, row strides and offsets of dhidden and of the gradient
    (0, 7, 8, "uniform", None, 0, None, 0), (1, 1, 1, "one", None, 0, None, 0), (1, 50257, 768, "uniform", None, 0, None, 0),
    (7, 3, 264, "two", None, 0, None, 0), (9, 40, 8, "uniform", None, 1, None, 0), (64, 1000, 100, "text", 101, 0, 104, 4),
    (65, 9, 72, "one", 80, 8, None, 0), (513, 3, 257, "uniform", 259, 3, None, 1), (1000, 5, 16, "masked", None, 0, None, 0),
    (4096, 2, 40, "one", None, 0, None, 0), (4097, 2, 40, "one", None, 0, None, 0), (5000, 2, 24, "two", None, 0, None, 0),
    (9001, 1500, 130, "text", None, 0, 136, 0), (40000, 300, 8, "text", None, 0, None, 0), (70001, 3, 3, "one", 4, 1, None, 0),
    (3000, 200003, 8, "text", None, 0, None, 0),
]


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp32"), ("fp32", "bf16"), ("bf16", "fp16")])
@pytest.mark.parametrize("T,V,D,kind,stride,offset,ostride,ooffset", BACKWARD)
def test_gradient(T, V, D, kind, stride, offset, ostride, ooffset, dtype, out_dtype):
    dh, _ = guarded(T, D, TYPES[dtype], 5, stride, offset)
    t = tokens(kind, T, V, 3)
    dh[(t < 0) | (t >= V)] = math.nan  # not read
    O = TYPES[out_dtype]
    for accumulate, scale in ((False, 1.0), (True, -2.75)):
        out, flat = guarded(V, D, O, 9, ostride, ooffset, values=accumulate)
        old = out.clone() if accumulate else None
        got = zg.embedding_backward(t, dh, V, scale=scale, out=out, accumulate=accumulate)
        want, tol = reference(t, dh, V, scale, old)
        assert got is out and untouched(flat, out, ooffset)
        bad = ~((got.double() - want).abs() <= tol + UNIT[O] * want.abs() + small(O))
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), (got.double() - want).abs().max().item())
        if accumulate:  # rows of no token keep their bits
            none = torch.ones(V, dtype=torch.bool, device=DEV)
            none[t[(t >= 0) & (t < V)]] = False
            assert torch.equal(out[none], old[none])
    new = zg.embedding_backward(t, dh, V)
    want, tol = reference(t, dh, V, 1.0, None)
    assert new.dtype == dh.dtype and bool(((new.double() - want).abs() <= tol + UNIT[dh.dtype] * want.abs() + small(dh.dtype)).all())


def test_gradient_is_that_of_the_forward():
    """By differences: sum(g * embedding(w + e d)) is linear in e, so one difference gives the slope."""
    V, D, T, scale = 37, 24, 200, 1.5
    w = torch.randn((V, D), device=DEV, generator=gen(1))
    d = torch.randn((V, D), device=DEV, generator=gen(2))
    g = torch.randn((T, D), device=DEV, generator=gen(3))
    t = tokens("text", T, V, 4)
    t[t >= V] = 0
    f = lambda x: (g.double() * zg.embedding(x, t, scale=scale).double()).sum()  # noqa: E731
    slope = f(w + d) - f(w)
    got = (zg.embedding_backward(t, g, V, scale=scale).double() * d.double()).sum()
    # 2 T D products off by 3 u of numbers of about 1, and the gradient's entries by 72 u
    assert abs(float(slope - got)) <= 80 * U * 4 * T * D


def test_equal_calls_give_equal_bits():
    t = tokens("text", 20000, 5000, 8)
    dh = torch.randn((20000, 136), device=DEV, generator=gen(9))
    first = zg.embedding_backward(t, dh, 5000)
    for _ in range(5):
        assert torch.equal(zg.embedding_backward(t, dh, 5000), first)


def test_another_stream_and_a_graph():
    V, D, T = 1000, 64, 6000
    t, dh = tokens("text", T, V, 8), torch.randn((T, D), device=DEV, generator=gen(9))
    w = torch.randn((V, D), device=DEV, generator=gen(2)).bfloat16()
    t[t >= V] = 1
    want = zg.embedding_backward(t, dh, V, scale=0.5)
    rows = zg.embedding(w, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = zg.embedding_backward(t, dh, V, scale=0.5, stream=side)
    emb = zg.embedding(w, t, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(emb, rows)
    # two graphs of their own workspaces, replayed in turn with new contents
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(zg.embedding_backward(t, dh, V, scale=0.5))
        graphs.append(g)
    for seed in (20, 21):
        dh.copy_(torch.randn((T, D), device=DEV, generator=gen(seed)))
        t.copy_(t.roll(seed))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = zg.embedding_backward(t, dh, V, scale=0.5)
        assert all(torch.equal(o, want) for o in outs)


def test_into_the_flat_gradient():
    """A tied matrix: the output product's gradient first, the embedding's added in the rank's buffer."""
    V, D, T = 500, 40, 300
    opt = zg.ZeroOptimizer([V * D, 77], M=1, stage=2, master_init=torch.zeros(V * D + 77, device=DEV))
    flat = opt.new_grad_buffers()[0]
    flat.zero_()
    view = opt.tensor_view(flat, 0).view(V, D)
    t = tokens("uniform", T, V, 1)
    a, b = (torch.randn((T, D), device=DEV, generator=gen(s)).bfloat16() for s in (2, 3))
    zg.embedding_backward(t, a, V, out=view)
    first = view.clone()
    zg.embedding_backward(t, b, V, out=view, accumulate=True)
    want, tol = reference(t, b, V, 1.0, first)
    assert bool(((view.double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())
    assert bool((opt.tensor_view(flat, 1) == 0).all())


def test_offsets_past_two_to_the_31_elements():
    V, D = 70001, 32768
    w = torch.zeros((V, D), device=DEV, dtype=torch.bfloat16)
    w[-1] = torch.randn(D, device=DEV, generator=gen(1)).bfloat16()
    w[-2] = 3.0
    t = torch.tensor([V - 1, 0, V - 2, V - 1], device=DEV)
    out = zg.embedding(w, t)
    assert torch.equal(out, w[t])
    d = zg.embedding_backward(t, out, V, out=w)
    assert torch.equal(d[-1], 2 * out[0]) and bool((d[-2] == 3).all()) and int(d[:-2].count_nonzero()) == 0
    del w, d
    dh = torch.zeros((V, D), device=DEV, dtype=torch.bfloat16)  # as many tokens
    dh[-1] = 1.0
    dh[-2, 1] = 2.0
    d = zg.embedding_backward(torch.arange(V, device=DEV) % 3, dh, 4)
    want = torch.zeros((4, D), device=DEV, dtype=torch.bfloat16)
    want[(V - 1) % 3] = 1.0
    want[(V - 2) % 3, 1] = 2.0
    assert torch.equal(d, want)


def test_refusals():
    w = torch.zeros((10, 16), device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    dh = torch.zeros((4, 16), device=DEV)
    for bad in (t.int(), t.cpu(), t[None], None, torch.zeros(8, dtype=torch.int64, device=DEV)[::2]):
        with pytest.raises(ValueError):
            zg.embedding(w, bad)
        with pytest.raises(ValueError):
            zg.embedding_backward(bad, dh, 10)
    for bad in (w.cpu(), w.double(), w.T, w[0]):
        with pytest.raises(ValueError):
            zg.embedding(bad, t)
    for bad in (torch.zeros((4, 15), device=DEV), torch.zeros((3, 16), device=DEV), torch.zeros((4, 16), device=DEV).half()):
        with pytest.raises(ValueError):
            zg.embedding(w, t, out=bad)
    for kw in (dict(accumulate=True), dict(out=torch.zeros((9, 16), device=DEV)), dict(out=torch.zeros((10, 16)))):
        with pytest.raises(ValueError):
            zg.embedding_backward(t, dh, 10, **kw)
    with pytest.raises(ValueError):
        zg.embedding_backward(t, dh, 0)
    with pytest.raises(ValueError):
        zg.embedding_backward(t[:3], dh, 10)
    for scale in (math.inf, math.nan, 1e300):
        with pytest.raises(zg.ZeroError):
            zg.embedding(w, t, scale=scale)
        with pytest.raises(zg.ZeroError):
            zg.embedding_backward(t, dh, 10, scale=scale)


def depth_rows(T, D, n):
    """1 and then rows of a little less than half its last bit, n to a block: added one by one they are all lost."""
    dh = torch.full((T, D), 2.0 ** -24 * 0.99, device=DEV)
    dh[::n] = 1.0
    return dh


@pytest.mark.parametrize("D,ld", [(2048, 2048), (2047, 2047)])
def test_sums_are_no_deeper_than_stated(D, ld):
    """Sums of 32 rows at most, then of such sums: of 128 rows of a block 31 are added to the 1 in it, where a chain of all
    would lose 127. One token with rows in one block, and one with rows in all."""
    T, V = 33000, 5
    dh = depth_rows(T, D, 128)
    for t in (torch.zeros(T, dtype=torch.int64, device=DEV), torch.arange(T, device=DEV) // 8192):
        got = zg.embedding_backward(t, dh, V)
        want, tol = reference(t, dh, V, 1.0, None)
        assert bool(((got.double() - want).abs() <= tol + U * want.abs()).all())
    one = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    one[:128] = 3
    got = zg.embedding_backward(one, dh, V)
    want, tol = reference(one, dh, V, 1.0, None)
    assert bool(((got.double() - want).abs() <= tol + U * want.abs()).all())
