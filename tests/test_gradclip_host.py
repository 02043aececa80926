"""Host-only checks of GradClip (no GPU): the library and torch's streams are stood in for."""
import types

import pytest

from zero_gradient_reduce_scatter_gb300 import _build


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Workspace:
    """Remembers the streams that it was recorded on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream.cuda_stream)

    def data_ptr(self):
        return 1 << 20


class Tensor(types.SimpleNamespace):
    at = 1 << 16

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return True

    def numel(self):
        return 10


@pytest.fixture
def world(monkeypatch):
    """A GradClip whose tensors, workspace and library are stand-ins; current[0] is the current stream."""
    _build.build()
    import torch
    from zero_gradient_reduce_scatter_gb300 import gradclip, losses
    current, used, made = [0], [], []
    lib = types.SimpleNamespace(
        zero_grads_workspace=lambda n: 4096, zero_grads_destroy=lambda p: 0,
        zero_grads_init=lambda *a: 0,
        zero_grads_clip=lambda plan, m, a, b, c, handle: used.append(handle) or 0)

    def empty(*a, **kw):
        made.append(Workspace())
        return made[-1]
    fake = types.SimpleNamespace(empty=empty, uint8=None, Tensor=Tensor, cuda=types.SimpleNamespace(current_stream=lambda device=None: Stream(current[0])))
    monkeypatch.setattr(gradclip, "torch", fake)
    monkeypatch.setattr(gradclip, "_lib", lambda: lib)
    monkeypatch.setattr(gradclip, "_on", lambda stream: losses._NOTHING)
    monkeypatch.setattr(gradclip, "_floats", lambda device, *shape: Tensor())
    monkeypatch.setattr(gradclip, "_handle", lambda stream, device: current[0] if stream is None else stream.cuda_stream)
    grad = Tensor(is_cuda=True, dtype=torch.float32, device=types.SimpleNamespace(index=0))
    return types.SimpleNamespace(make=lambda **kw: gradclip.GradClip([grad], **kw), current=current, used=used, made=made, grad=grad)


def test_the_workspace_is_recorded_on_every_stream_that_uses_it(world):
    """A plan made on one stream and used on another, named or current: the allocator must not hand its
    table out before the kernels that follow it are done."""
    plan = world.make()
    plan.clip(1.0)
    assert world.used == [0] and world.made[0].streams == []
    plan.clip(1.0, stream=Stream(7))
    assert world.made[0].streams == [7]
    world.current[0] = 9                       # with torch.cuda.stream(...): plan.clip(1.0)
    plan.clip(1.0)
    assert world.used == [0, 7, 9] and world.made[0].streams == [7, 9]
    side = world.make(stream=Stream(5))        # made on a stream of its own, used on the current one
    side.clip(1.0)
    side.clip(1.0, stream=Stream(5))
    assert world.made[1].streams == [9]


def test_gradients_made_anew_are_noticed(world):
    """zero_grad() sets gradients to None and the next backward makes others: handed to clip, they are refused."""
    plan = world.make()
    kw = dict(is_cuda=True, dtype=world.grad.dtype, device=world.grad.device)
    plan.clip(1.0, grads=[world.grad])
    plan.clip(1.0, grads=(g for g in [Tensor(**kw)]))      # a view of the same values
    assert world.used == [0, 0]
    for grads in ([Tensor(at=1 << 18, **kw)], [None], [], [world.grad, world.grad]):
        with pytest.raises(ValueError):
            plan.clip(1.0, grads=grads)
    assert world.used == [0, 0]
