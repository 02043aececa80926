"""The embedding's gradient written into a bucket directly before that bucket's step, on one stream with launch
overlap: a bucket kernel that follows a call without a context waits for it. The results are those of
ordinary launches, bit for bit."""
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


@pytest.mark.parametrize("form", ["written", "added", "clipped"])
@pytest.mark.parametrize("own_stream", [False, True])
def test_buckets_behind_an_embedding_gradient(form, own_stream):
    V, D, T, n = 1500, 264, 6000, 6
    init = torch.randn(n * V * D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    opts = []
    for mode in ("none", "launch", "buckets"):
        opt = zg.ZeroOptimizer([V * D] * n, M=1, stage=2, master_init=init.clone(), bucket_bytes=2 * V * D)
        opt.set_launch_overlap(mode)
        assert len(opt.buckets) == n
        opts.append((opt, opt.new_grad_buffers()[0].zero_()))
    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
    for step in range(3):
        g = torch.Generator(device=DEV).manual_seed(10 + step)
        tokens = [torch.randint(0, V, (T,), device=DEV, generator=g) for _ in range(n)]
        dh = [torch.randn((T, D), device=DEV, generator=g).bfloat16() for _ in range(n)]
        for opt, flat in opts:
            views = [opt.tensor_view(flat, i).view(V, D) for i in range(n)]
            news = [torch.empty_like(v) for v in views]
            plans = [zg.GradClip([a], [v]) for a, v in zip(news, views)]
            torch.cuda.synchronize()
            for b in reversed(range(n)):
                if form == "clipped":
                    zg.embedding_backward(tokens[b], dh[b], V, out=news[b], stream=stream)
                    with torch.cuda.stream(stream):
                        plans[b].clip(0.5)
                else:
                    zg.embedding_backward(tokens[b], dh[b], V, out=views[b], accumulate=form == "added", stream=stream)
                off = opt.buckets[b][0]
                opt.step_bucket(b, [flat[off:off + opt.bucket_lanes(b)]], zg.Hyper(lr=1e-2), stream=stream)
            torch.cuda.synchronize()
    (one, flat1), *others = opts
    for other, flat in others:
        assert torch.equal(flat, flat1) and torch.equal(other.master, one.master) and torch.equal(other.params(), one.params())
        assert torch.equal(other.m, one.m) and torch.equal(other.v, one.v)
    assert not torch.equal(one.master, init)
