"""A GradClip plan used on another stream than the one it was made on, and dropped while that is busy."""
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


@pytest.mark.parametrize("named", [False, True])
def test_a_plan_dropped_while_its_stream_is_busy(named):
    """What the allocator hands out before the other stream is done does not reach into the plan's
    workspace, and the clipping that waited there is right."""
    grads = [torch.randn(n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(n)) for n in (5000, 7, 30000)]
    dst = [torch.zeros_like(x) for x in grads]
    want = [torch.zeros_like(x) for x in grads]
    w = zg.GradClip(grads, want).clip(0.5)
    plan = zg.GradClip(grads, dst)
    lo = plan.workspace.data_ptr()
    size = plan.workspace.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    if named:
        r = plan.clip(0.5, stream=side)
    else:
        with torch.cuda.stream(side):
            r = plan.clip(0.5)
    del plan
    others = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(64)]
    busy = not side.query()
    assert busy and all(o.data_ptr() + o.numel() <= lo or lo + size <= o.data_ptr() for o in others)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r.norm, w.norm) and torch.equal(r.norms, w.norms) and all(torch.equal(a, b) for a, b in zip(dst, want))
