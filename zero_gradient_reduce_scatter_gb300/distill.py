"""Distillation: a teacher's most likely tokens, and a student's loss on them.

``top_logits`` reads a teacher's logits once and gives the k most likely tokens of every position with
their log-probabilities and the log of the probability outside them: what is kept of a teacher instead
of its logits. The calls follow those of losses.py in memory, streams, errors, masked tokens and
autograd (none). include/zero_gb300.h states the formulas.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _lib
from .losses import TYPES, Logits, _floats, _handle, _matrix, _on, _vector


class TopLogits(NamedTuple):
    index: torch.Tensor   # int64 [T, k]
    logp: torch.Tensor    # fp32 [T, k]
    lse: torch.Tensor     # fp32 [T]
    rest: torch.Tensor    # fp32 [T]: log of the probability outside the k


def top_logits(logits, k: int, targets=None, *, temperature: float = 1.0, stream=None) -> TopLogits:
    """The k most likely tokens under logits [T, V] / temperature, the likeliest first, 1 <= k <= min(V, 512).
    targets: int64 [T], of which those below 0 mark rows that are not read (index -1, results 0)."""
    rows, cols, stride = _matrix(logits, "logits")
    dev = logits.device
    at = None if targets is None else _vector(targets, "targets", rows, torch.int64, dev)
    a = Logits(logits.data_ptr(), at, rows, cols, stride, TYPES[logits.dtype], temperature)
    k = int(k)
    if not 1 <= k <= min(cols, 512):
        raise ValueError("k must be in 1 .. min(vocabulary, 512)")
    with _on(stream):
        index, logp = torch.empty((rows, k), dtype=torch.int64, device=dev), _floats(dev, rows, k)
        lse, rest = _floats(dev, rows), _floats(dev, rows)
    _check(_lib().zero_top_logits(ctypes.byref(a), k, index.data_ptr(), logp.data_ptr(), lse.data_ptr(), rest.data_ptr(),
                                  _handle(stream, dev)), "zero_top_logits")
    return TopLogits(index, logp, lse, rest)
