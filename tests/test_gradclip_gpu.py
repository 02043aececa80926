"""GradClip (global norm over many tensors, clipping) against 64-bit sums.

Tolerances: a tensor's sum of squares is formed in fp32 over at most a few dozen squares and in
fp64 beyond, so norms are within 2^-24 (32 + 2) of themselves, and rounded once more to fp32;
scale = max_norm / norm inherits that; a clipped value is one product (2^-24), the scale's error,
and one rounding to its type.
"""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg

pytestmark = pytest.mark.gpu

DEV = "cuda"
NORM = 2.0 ** -24 * 36
UNIT = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}  # half a spacing
B, H, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def make(sizes, types, seed, odd=False, std=1e-2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = types[i % len(types)]
        x = (torch.randn(n, device=DEV, generator=g) * std).to(t)
        if odd:  # a view at an odd element offset of a larger tensor
            big = torch.full((n + 9,), float("nan"), device=DEV, dtype=t)
            big[1 + i % 5:1 + i % 5 + n].copy_(x)
            x = big[1 + i % 5:1 + i % 5 + n]
        out.append(x)
    return out


def exact(grads, max_norm):
    norms = [float(x.double().pow(2).sum().sqrt()) if x.numel() else 0.0 for x in grads]
    norm = math.sqrt(sum(v * v for v in norms))
    return norms, norm, (max_norm / norm if norm > max_norm else 1.0)


def check(r, grads64, dst, max_norm):
    norms = [float(x.pow(2).sum().sqrt()) if x.numel() else 0.0 for x in grads64]
    norm = math.sqrt(sum(v * v for v in norms))
    scale = max_norm / norm if norm > max_norm else 1.0
    assert abs(float(r.norm) - norm) <= NORM * norm
    assert abs(float(r.scale) - scale) <= 2 * NORM * scale and (scale < 1 or float(r.scale) == 1.0)
    for got, want in zip(r.norms.tolist(), norms):
        assert abs(got - want) <= NORM * want
    for d, x in zip(dst, grads64):
        want = x * scale
        tol = (UNIT[d.dtype] + 3 * NORM) * want.abs() + (2.0 ** -25 if d.dtype == H else 2.0 ** -140)
        assert bool(((d.double().reshape(-1) - want.reshape(-1)).abs() <= tol.reshape(-1)).all())


SETS = [
    ([1], [F]), ([0, 0, 5], [B]), ([0], [F]), ([7, 0, 1, 130, 3, 0], [B, F, H]), ([4096], [B]), ([4097, 8191, 2, 65536], [F, B]),
    ([768] * 130, [F]), (list(range(0, 400)), [B, H, F]), ([1000003, 17, 250001, 1, 64], [B]), ([3000001, 5, 2000000], [F, B]),
    ([1] * 3001, [F, B]),
]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("sizes,types", SETS)
def test_norm_and_clip(sizes, types, odd):
    for max_norm in (1e-3, 1e6):
        grads = make(sizes, types, 3, odd)
        exact64 = [x.double().clone() for x in grads]
        # into tensors of other types, guard values around them
        dst, guards = [], []
        for i, x in enumerate(grads):
            t = (B, F, H)[i % 3]
            big = torch.full((x.numel() + 8,), 7.0, device=DEV, dtype=t)
            o = 0 if not odd else 1 + i % 3
            dst.append(big[o:o + x.numel()])
            guards.append((big, o, x.numel()))
        plan = zg.GradClip(grads, dst)
        r = plan.clip(max_norm)
        check(r, exact64, dst, max_norm)
        assert all(torch.equal(x.double(), e) for x, e in zip(grads, exact64))
        assert all(bool((b[:o] == 7).all()) and bool((b[o + n:] == 7).all()) for b, o, n in guards)
        again = plan.clip(max_norm)
        assert torch.equal(r.norm, again.norm) and torch.equal(r.norms, again.norms) and torch.equal(r.scale, again.scale)
        plan.close()
        # in place
        plan = zg.GradClip(grads)
        r2 = plan.clip(max_norm)
        assert torch.equal(r.norm, r2.norm) and torch.equal(r.norms, r2.norms)
        check(r2, exact64, grads, max_norm)
        if max_norm > 1:
            assert all(torch.equal(x.double(), e) for x, e in zip(grads, exact64))
        plan.close()


def test_values_whose_squares_leave_fp32():
    """Gradients of 1e30 and of 1e-30: their squares are no fp32 numbers, their norm is one."""
    for std in (1e30, 1e-30):
        grads = make([3001, 70000, 5], [F, B, F], 9, std=std)
        r = zg.GradClip(grads, [torch.empty_like(x) for x in grads]).clip(math.inf)
        norms, norm, _ = exact(grads, math.inf)
        assert abs(float(r.norm) - norm) <= NORM * norm
        for got, want in zip(r.norms.tolist(), norms):
            assert abs(got - want) <= NORM * want
    mixed = make([5000], [F], 2, std=1e-25) + make([3], [F], 3, std=1e25)
    norms, norm, _ = exact(mixed, math.inf)
    r = zg.GradClip(mixed).clip(math.inf)
    assert abs(float(r.norm) - norm) <= NORM * norm and abs(float(r.norms[0]) - norms[0]) <= NORM * norms[0]


def test_many_values_at_the_ends_of_fp32():
    """Sums of squares that pass fp32 by their number: 2^20 values of 2^58, and of 2^-62. A norm that
    is no fp32 number counts as not finite."""
    for x in (2.0 ** 58, 2.0 ** -62, 2.0 ** 39):
        grads = [torch.full((1 << 20,), x, device=DEV), torch.full((3,), x, device=DEV, dtype=B)]
        r = zg.GradClip(grads).clip(math.inf)
        want = x * math.sqrt((1 << 20) + 3)
        assert abs(float(r.norm) - want) <= NORM * want and abs(float(r.norms[0]) - x * 1024) <= NORM * x * 1024
    grads = [torch.full((4096,), 3e38, device=DEV)]
    r = zg.GradClip(grads).clip(1.0)
    assert float(r.norm) == math.inf and float(r.scale) == 1.0 and bool((grads[0] == 3e38).all())


def test_more_values_than_32_bits_count():
    n = 2 ** 31 + 12345
    x = torch.zeros(n, dtype=B, device=DEV)
    x[-3:] = 4.0
    x[:2] = 2.0
    r = zg.GradClip([x]).clip(1.0)
    want = math.sqrt(3 * 16 + 2 * 4)
    assert abs(float(r.norm) - want) <= NORM * want
    s = float(r.scale)
    assert bool((x[-3:] == torch.tensor(4.0 * s, device=DEV).to(B)).all()) and bool((x[:2] == torch.tensor(2.0 * s, device=DEV).to(B)).all())
    assert int((x != 0).sum()) == 5


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_leaves_the_values(value):
    grads = make([100, 3000], [F, B], 4)
    grads[1][1234] = value
    keep = [x.clone() for x in grads]
    dst = [torch.zeros_like(x) for x in grads]
    r = zg.GradClip(grads, dst).clip(1e-3)
    assert not math.isfinite(float(r.norm)) and float(r.scale) == 1.0
    assert math.isfinite(float(r.norms[0])) and not math.isfinite(float(r.norms[1]))
    for d, k in zip(dst, keep):
        assert torch.equal(d.isnan(), k.isnan()) and torch.equal(d[~d.isnan()], k[~k.isnan()])
    zg.GradClip(grads).clip(1e-3)
    for x, k in zip(grads, keep):
        assert torch.equal(x.isnan(), k.isnan()) and torch.equal(x[~x.isnan()], k[~k.isnan()])


def test_zero_gradients_and_infinite_threshold():
    grads = [torch.zeros(1000, device=DEV), torch.zeros(3, device=DEV, dtype=B)]
    r = zg.GradClip(grads).clip(1.0)
    assert float(r.norm) == 0.0 and float(r.scale) == 1.0 and bool((r.norms == 0).all())
    grads = make([500], [F], 5)
    keep = grads[0].clone()
    r = zg.GradClip(grads).clip(math.inf)
    assert float(r.scale) == 1.0 and torch.equal(grads[0], keep)


def test_into_the_optimizers_gradient_buffer():
    """Separate fp32 gradients clipped into a rank's padded buffer, then the step, against a step on
    the same values rounded by hand; the padding lanes keep what they held."""
    numel = [4096, 1000, 3, 77]
    w0 = torch.randn(sum(numel), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 0.02
    opts = [zg.ZeroOptimizer(numel, M=2, stage=2, master_init=w0) for _ in range(2)]
    bufs, want = opts[0].new_grad_buffers(), opts[1].new_grad_buffers()
    lanes = torch.zeros(bufs[0].numel(), dtype=torch.bool, device=DEV)
    for i in range(len(numel)):
        opts[0].tensor_view(lanes, i).fill_(True)
    for r in range(2):
        grads = make(numel, [F], 10 + r)
        bufs[r].fill_(3.0)
        c = zg.GradClip.into(opts[0], grads, bufs[r]).clip(0.25)
        assert float(c.scale) < 1
        for i, x in enumerate(grads):
            opts[1].tensor_view(want[r], i).copy_((x * c.scale).to(B))
        assert torch.equal(bufs[r][lanes], want[r][lanes]) and bool((bufs[r][~lanes] == 3).all())
    for o, g in zip(opts, (bufs, want)):
        o.step(g, zg.Hyper(lr=1e-3))
    assert torch.equal(opts[0].params(), opts[1].params()) and torch.equal(opts[0].master, opts[1].master)


def test_side_stream_and_graph():
    grads = make([70001, 5, 30000], [F, B], 6)
    dst = [torch.zeros(x.numel(), device=DEV, dtype=B) for x in grads]
    plan = zg.GradClip(grads, dst)
    want = plan.clip(0.1)
    keep = [d.clone() for d in dst]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = plan.clip(0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    import gc
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = plan.clip(0.1)
    for k in range(2):
        for d in dst:
            d.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, want)) and all(torch.equal(a, b) for a, b in zip(dst, keep))


def test_refusals():
    x = torch.ones(10, device=DEV)
    for call in (lambda: zg.GradClip([]), lambda: zg.GradClip([x.cpu()]), lambda: zg.GradClip([x.double()]),
                 lambda: zg.GradClip([x[::2]]), lambda: zg.GradClip([x], [x[:5]]), lambda: zg.GradClip([x], [])):
        with pytest.raises(ValueError):
            call()
    plan = zg.GradClip([x])
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(zg.ZeroError) as e:
            plan.clip(bad)
        assert e.value.code == -1
    plan.close()
    with pytest.raises(zg.ZeroError) as e:
        plan.clip(1.0)
    assert e.value.code == -7
    opt = zg.ZeroOptimizer([10, 5], M=1, stage=1, master_init=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        zg.GradClip.into(opt, [x], opt.new_grad_buffers()[0])
