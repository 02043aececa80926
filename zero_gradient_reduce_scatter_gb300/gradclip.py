"""Global norm and clipping of gradients that are still separate tensors.

``ZeroOptimizer.step`` clips by the norm of the averaged gradient. ``GradClip`` serves the step
before that: a rank's own gradients, as autograd leaves them (any mix of bfloat16, float16 and
float32, any sizes), are measured and clipped in place or straight into the rank's flat bf16
gradient buffer, with no host synchronisation.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _lib
from .losses import TYPES, _floats, _handle, _on


class GradTensor(ctypes.Structure):
    """zero_grad_tensor."""

    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64), ("src_type", ctypes.c_int32),
                ("dst_type", ctypes.c_int32)]


class Clipped(NamedTuple):
    norm: torch.Tensor    # fp32, 0-dim: the norm before clipping
    scale: torch.Tensor   # fp32, 0-dim
    norms: torch.Tensor   # fp32 [n]: every tensor's own norm


class GradClip:
    """A plan over a fixed list of CUDA tensors; ``clip`` is one call on their current values.

    grads: contiguous tensors of one device. dst: where the clipped values go, one tensor of the
    same size each (any of the three types), or None for in place. The plan keeps references to
    both, and their addresses: gradients must stay the same tensors from call to call, which
    ``optimizer.zero_grad(set_to_none=False)`` or ``p.grad.zero_()`` does and torch's default,
    gradients set to None and made anew, does not (``clip(..., grads=)`` checks it).
    A dst tensor must not overlap any gradient but its own. A plan may be dropped right after
    ``clip``, on whatever stream that ran; one captured in a CUDA graph must live as long as the graph.
    """

    def __init__(self, grads, dst=None, stream=None):
        self.grads = list(grads)
        self.dst = self.grads if dst is None else list(dst)
        if not self.grads:
            raise ValueError("GradClip needs at least one tensor")
        if len(self.dst) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients, {len(self.dst)} destinations")
        dev = self.grads[0].device
        for name, ts in (("grads", self.grads), ("dst", self.dst)):
            for i, t in enumerate(ts):
                if not (t.is_cuda and t.dtype in TYPES and t.is_contiguous() and t.device == dev and t.numel() == self.grads[i].numel()):
                    raise ValueError(f"{name}[{i}] must be a contiguous CUDA tensor on {dev} in bfloat16, float16 or float32, "
                                     "of its gradient's size")
        self.device = dev
        n = len(self.grads)
        rows = (GradTensor * n)(*[GradTensor(g.data_ptr(), d.data_ptr(), g.numel(), TYPES[g.dtype], TYPES[d.dtype])
                                  for g, d in zip(self.grads, self.dst)])
        size = _lib().zero_grads_workspace(n)
        with _on(stream):
            self.workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        self._home = _handle(stream, dev)  # the stream that the workspace was allocated on
        plan = ctypes.c_void_p()
        _check(_lib().zero_grads_init(ctypes.byref(plan), ctypes.cast(rows, ctypes.c_void_p), n, self.workspace.data_ptr(),
                                      size, self._home), "zero_grads_init")
        self._plan = plan

    @classmethod
    def into(cls, opt, grads, buf, stream=None):
        """Clip into `buf`, a padded bf16 gradient buffer of the optimizer `opt` (one of
        ``new_grad_buffers``), tensor i into its place; the padding lanes are not touched."""
        if len(grads) != len(opt.numel):
            raise ValueError(f"the optimizer has {len(opt.numel)} tensors, got {len(grads)}")
        return cls(grads, [opt.tensor_view(buf, i) for i in range(len(opt.numel))], stream=stream)

    def clip(self, max_norm: float, stream=None, grads=None) -> Clipped:
        """Measure, and write gradient * min(1, max_norm / norm). A norm that is not finite leaves
        the values as they are (scale 1). max_norm may be infinite: then the values are only
        measured and packed. grads: the gradients as the caller holds them now (``[p.grad for p in
        params]``); ValueError where one is not the plan's, whose old values would be clipped instead."""
        if grads is not None:
            now = list(grads)
            if len(now) != len(self.grads):
                raise ValueError(f"the plan has {len(self.grads)} gradients, got {len(now)}")
            for i, (a, b) in enumerate(zip(now, self.grads)):
                if a is not b and not (isinstance(a, torch.Tensor) and a.data_ptr() == b.data_ptr() and a.dtype == b.dtype
                                       and a.numel() == b.numel() and a.is_contiguous()):
                    raise ValueError(f"grads[{i}] is not the tensor that the plan was made for")
        with _on(stream):
            norm, scale, norms = _floats(self.device), _floats(self.device), _floats(self.device, len(self.grads))
        handle = _handle(stream, self.device)
        if handle != self._home:  # the kernels follow the workspace's table: not handed out again before this call is done
            self.workspace.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
        _check(_lib().zero_grads_clip(self._plan, max_norm, norm.data_ptr(), scale.data_ptr(), norms.data_ptr(), handle),
               "zero_grads_clip")
        return Clipped(norm, scale, norms)

    def close(self):
        if getattr(self, "_plan", None) is not None and self._plan.value:
            _lib().zero_grads_destroy(self._plan)
            self._plan = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
