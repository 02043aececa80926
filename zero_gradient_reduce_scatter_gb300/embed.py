"""The embedding of tokens: rows of the vocabulary matrix, and their gradient.

``embedding`` gathers and scales a batch's rows. ``embedding_backward`` turns the gradient on them
into the matrix' gradient, tokens in sorted order and every row written once: as a new tensor, into
one that is given (a view of the optimizer's flat gradient, ``opt.tensor_view(grads[0], i)``, is one),
or added to what that holds, as a matrix needs that is also the output matrix. Both follow the calls
of losses.py in memory, streams, errors and autograd (none). include/zero_gb300.h states the formulas.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _lib
from .losses import TYPES, _bytes, _handle, _matrix, _on, _vector

_P, _I32, _I64, _D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class Embed(ctypes.Structure):
    """zero_embed."""

    _fields_ = [("weight", _P), ("tokens", _P), ("rows", _I64), ("vocab", _I64), ("dim", _I64), ("ld_weight", _I64),
                ("type", _I32), ("scale", _D)]


class EmbedGrad(ctypes.Structure):
    """zero_embed_grad."""

    _fields_ = [("tokens", _P), ("dhidden", _P), ("dweight", _P), ("rows", _I64), ("vocab", _I64), ("dim", _I64),
                ("ld_hidden", _I64), ("ld_weight", _I64), ("type", _I32), ("out_type", _I32), ("scale", _D),
                ("accumulate", _I32)]


def _tokens(tokens, device):
    if not (isinstance(tokens, torch.Tensor) and tokens.dim() == 1):
        raise ValueError("tokens must be a 1-D tensor")
    return _vector(tokens, "tokens", tokens.shape[0], torch.int64, device)


def embedding(weight, tokens, *, scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """scale * weight[tokens]: [T, D] of weight's type, from weight [V, D] and tokens [T] (int64). A token
    below 0 gets a row of zeros, one past the matrix a row of NaN. out: where to write it."""
    vocab, dim, ld = _matrix(weight, "weight")
    at = _tokens(tokens, weight.device)
    rows = tokens.shape[0]
    if out is None:
        with _on(stream):
            out, ld_out = torch.empty((rows, dim), dtype=weight.dtype, device=weight.device), dim
    else:
        r, c, ld_out = _matrix(out, "out")
        if (r, c, out.dtype, out.device) != (rows, dim, weight.dtype, weight.device):
            raise ValueError("out must be [tokens, dim] of the weight's type and device")
    x = Embed(weight.data_ptr(), at, rows, vocab, dim, ld, TYPES[weight.dtype], scale)
    _check(_lib().zero_embedding(ctypes.byref(x), out.data_ptr(), ld_out, _handle(stream, weight.device)), "zero_embedding")
    return out


def embedding_backward(tokens, dhidden, vocab: int, *, scale: float = 1.0, out=None, accumulate: bool = False,
                       stream=None) -> torch.Tensor:
    """The gradient [V, D] on embedding's weight of a function whose gradient on its result is dhidden
    [T, D]. out: where to write it, in any of the three types (default: a new tensor of dhidden's
    type); with accumulate it is added to what out holds."""
    rows, dim, ld = _matrix(dhidden, "dhidden")
    dev = dhidden.device
    at = _vector(tokens, "tokens", rows, torch.int64, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if vocab < 1:
            raise ValueError("vocab must be at least 1")
        with _on(stream):
            out, ld_out = torch.empty((vocab, dim), dtype=dhidden.dtype, device=dev), dim
    else:
        r, c, ld_out = _matrix(out, "out")
        if (r, c, out.device) != (vocab, dim, dev):
            raise ValueError("out must be [vocab, dim] on dhidden's device")
    lib = _lib()
    size = lib.zero_embedding_backward_workspace(rows, vocab, dim, TYPES[dhidden.dtype])
    with _on(stream):
        ws = _bytes(dev, max(size, 0))
    x = EmbedGrad(at, dhidden.data_ptr(), out.data_ptr(), rows, vocab, dim, ld, ld_out, TYPES[dhidden.dtype], TYPES[out.dtype],
                  scale, 1 if accumulate else 0)
    _check(lib.zero_embedding_backward(ctypes.byref(x), ws.data_ptr(), size, _handle(stream, dev)), "zero_embedding_backward")
    return out
