"""Distillation: a teacher's most likely tokens, and a student's loss on them.

``top_logits`` reads a teacher's logits once and gives the k most likely tokens of every position with
their log-probabilities and the log of the probability outside them: what is kept of a teacher instead
of its logits. ``distill_loss`` is the loss of a student's logits against such lists with its gradient on the
logits, which ``logits.backward(result.dlogits)`` carries into a model. The calls follow those of losses.py in memory, streams, errors, masked tokens and
autograd (none). include/zero_gb300.h states the formulas.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _lib
from .losses import REDUCE, TYPES, Logits, _bytes, _floats, _gradient, _handle, _logits, _matrix, _on, _vector


KIND = {"forward": 0, "reverse": 1, "js": 2}
TAIL = {"rest": 0, "drop": 1, "renormalise": 2}
MOST = 512  # entries of a list

_P, _I32, _I64, _D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class Distill(ctypes.Structure):
    """zero_distill."""

    _fields_ = [("index", _P), ("teacher_logp", _P), ("teacher_rest", _P), ("offsets", _P), ("seqs", _I64), ("k", _I64), ("mix", _D),
                ("kl_coef", _D), ("ce_coef", _D), ("kind", _I32), ("tail", _I32), ("reduce", _I32), ("loss", _P), ("kl", _P),
                ("token_kl", _P), ("logp", _P), ("dlogits", _P), ("dstride", _I64)]


class TopLogits(NamedTuple):
    index: torch.Tensor   # int64 [T, k]
    logp: torch.Tensor    # fp32 [T, k]
    lse: torch.Tensor     # fp32 [T]
    rest: torch.Tensor    # fp32 [T]: log of the probability outside the k


class DistillLoss(NamedTuple):
    loss: torch.Tensor       # fp32, 0-dim
    kl: torch.Tensor         # fp32, 0-dim: the mean divergence over the targets
    token_kl: torch.Tensor   # fp32 [T]
    logp: torch.Tensor       # fp32 [T]: the targets' log-probabilities
    dlogits: torch.Tensor    # [T, V] of the logits' type


def top_logits(logits, k: int, targets=None, *, temperature: float = 1.0, stream=None) -> TopLogits:
    """The k most likely tokens under logits [T, V] / temperature, the likeliest first, 1 <= k <= min(V, 512).
    targets: int64 [T], of which those below 0 mark rows that are not read (index -1, results 0)."""
    rows, cols, stride = _matrix(logits, "logits")
    dev = logits.device
    at = None if targets is None else _vector(targets, "targets", rows, torch.int64, dev)
    a = Logits(logits.data_ptr(), at, rows, cols, stride, TYPES[logits.dtype], temperature)
    k = int(k)
    if not 1 <= k <= min(cols, MOST):
        raise ValueError(f"k must be in 1 .. min(vocabulary, {MOST})")
    with _on(stream):
        index, logp = torch.empty((rows, k), dtype=torch.int64, device=dev), _floats(dev, rows, k)
        lse, rest = _floats(dev, rows), _floats(dev, rows)
    _check(_lib().zero_top_logits(ctypes.byref(a), k, index.data_ptr(), logp.data_ptr(), lse.data_ptr(), rest.data_ptr(),
                                  _handle(stream, dev)), "zero_top_logits")
    return TopLogits(index, logp, lse, rest)


def _lists(x, name, rows, k, dtype, device):
    if not (isinstance(x, torch.Tensor) and x.dtype == dtype and x.device == device and tuple(x.shape) == (rows, k) and x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of [{rows}, {k}] on {device}")
    return x.data_ptr()


def distill_loss(logits, targets, index, teacher_logp, teacher_rest: Optional[torch.Tensor] = None, *, offsets=None, kind: str = "forward",
                 tail: str = "rest", mix: float = 0.5, kl_coef: float = 1.0, ce_coef: float = 0.0, reduce: str = "token",
                 temperature: float = 1.0, out=None, stream=None) -> DistillLoss:
    """Divergence of the student's logits [T, V] from a teacher's lists index (int64 [T, k]) and teacher_logp (fp32
    [T, k]) at the same temperature, 1 <= k <= min(V, 512); entries with an index below 0 or a log-probability of
    -inf are not there. kind: "forward" KL(teacher | student), "reverse", or "js" with the teacher's share mix.
    tail: what becomes of the vocabulary outside a list: one more entry ("rest", with its log-probability
    teacher_rest [T] or what the list leaves), "drop" or "renormalise". ce_coef adds -log q of the targets;
    a target below 0 marks a token without a loss. offsets (int64 [S + 1]) and reduce as for policy_loss."""
    a = _logits(logits, targets, temperature)
    dev, f32 = logits.device, torch.float32
    if kind not in KIND or tail not in TAIL or reduce not in REDUCE:
        raise ValueError(f"kind is one of {list(KIND)}, tail of {list(TAIL)}, reduce of {list(REDUCE)}")
    if kind != "forward" and tail != "rest":
        raise ValueError('kind "reverse" and "js" need tail="rest"')
    k = index.shape[1] if isinstance(index, torch.Tensor) and index.dim() == 2 else 0
    if not 1 <= k <= min(a.vocab, MOST):
        raise ValueError(f"index must be [T, k] with k in 1 .. min(vocabulary, {MOST})")
    at, lp = _lists(index, "index", a.rows, k, torch.int64, dev), _lists(teacher_logp, "teacher_logp", a.rows, k, f32, dev)
    rest = None if teacher_rest is None else _vector(teacher_rest, "teacher_rest", a.rows, f32, dev)
    seqs, off = 0, None
    if offsets is not None:
        if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.shape[0] >= 1):
            raise ValueError("offsets must hold the number of sequences + 1 values")
        seqs = offsets.shape[0] - 1
        off = _vector(offsets, "offsets", seqs + 1, torch.int64, dev)
    lib = _lib()
    size = lib.zero_distill_workspace(a.rows)
    with _on(stream):
        out, dstride = _gradient(logits, a, out)
        loss, kl, ws = _floats(dev), _floats(dev), _bytes(dev, size)
        token_kl, logp = _floats(dev, a.rows), _floats(dev, a.rows)
    p = Distill(at, lp, rest, off, seqs, k, mix, kl_coef, ce_coef, KIND[kind], TAIL[tail], REDUCE[reduce], loss.data_ptr(), kl.data_ptr(),
                token_kl.data_ptr(), logp.data_ptr(), out.data_ptr(), dstride)
    _check(lib.zero_distill_loss(ctypes.byref(a), ctypes.byref(p), ws.data_ptr(), size, _handle(stream, dev)), "zero_distill_loss")
    return DistillLoss(loss, kl, token_kl, logp, out)
