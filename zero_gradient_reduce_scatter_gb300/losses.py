"""Training losses that stand before an optimizer step, as calls of their own.

``token_logp`` / ``token_logp_backward``: log-probabilities (and entropies) of given tokens
from logits, and the gradient of any function of them on the logits. ``linear_logp``: the same
results straight from hidden states and the vocabulary matrix, with no logits in memory and
without a gradient (the frozen sides of the losses). ``preference_loss`` and ``policy_loss``:
a whole loss with its gradient on the logits, which ``logits.backward(result.dlogits)`` carries
into a model.

The calls marshal arguments; the arithmetic runs in the library's kernels (there is no CPU
fallback). They allocate their results with torch on the stream they run on and return once the
work is enqueued. ``stream`` is a torch.cuda.Stream (default: the current one of the logits'
device); inputs made on another stream need the usual event or stream wait, and have to live until
the work is done (or record_stream); results belong to the stream the call ran on. No call takes
part in autograd: results carry no graph, whether or not the logits require a gradient.
include/zero_gb300.h states every formula and what the calls do with masked tokens, infinities
and NaN.

A target below 0 marks a token without a loss: its row of logits is not read and its gradient
row is zero.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _RAW_STREAM, _check, _lib

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
PREFERENCE = {"sigmoid": 0, "hinge": 1, "ipo": 2}
KL = {"k1": 0, "k2": 1, "k3": 2}
REDUCE = {"token": 0, "sequence": 1, "sum": 2}

_P, _I32, _I64, _D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class Logits(ctypes.Structure):
    """zero_logits."""

    _fields_ = [("logits", _P), ("targets", _P), ("rows", _I64), ("vocab", _I64), ("stride", _I64), ("type", _I32),
                ("temperature", _D)]


class Preference(ctypes.Structure):
    """zero_preference."""

    _fields_ = [("offsets", _P), ("ref_logp", _P), ("pairs", _I64), ("beta", _D), ("label_smoothing", _D),
                ("kind", _I32), ("average", _I32), ("loss", _P), ("pair_loss", _P), ("chosen_reward", _P),
                ("rejected_reward", _P), ("logp", _P), ("dlogits", _P), ("dstride", _I64)]


class Policy(ctypes.Structure):
    """zero_policy."""

    _fields_ = [("advantages", _P), ("old_logp", _P), ("ref_logp", _P), ("offsets", _P), ("seqs", _I64),
                ("clip_low", _D), ("clip_high", _D), ("dual_clip", _D), ("kl_coef", _D), ("entropy_coef", _D),
                ("kl", _I32), ("reduce", _I32), ("per_sequence", _I32), ("loss", _P), ("clip_fraction", _P),
                ("kl_mean", _P), ("logp", _P), ("entropy", _P), ("dlogits", _P), ("dstride", _I64)]


class Linear(ctypes.Structure):
    """zero_linear."""

    _fields_ = [("hidden", _P), ("weight", _P), ("targets", _P), ("rows", _I64), ("vocab", _I64), ("dim", _I64),
                ("ld_hidden", _I64), ("ld_weight", _I64), ("type", _I32), ("temperature", _D)]


class TokenLogp(NamedTuple):
    logp: torch.Tensor                 # fp32 [T]
    lse: torch.Tensor                  # fp32 [T]
    entropy: Optional[torch.Tensor]    # fp32 [T], where asked for


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor                 # fp32, 0-dim: the mean over pairs
    pair_loss: torch.Tensor            # fp32 [P]
    chosen_reward: torch.Tensor        # fp32 [P]
    rejected_reward: torch.Tensor      # fp32 [P]
    logp: torch.Tensor                 # fp32 [T]
    dlogits: torch.Tensor              # [T, V] of the logits' type


class PolicyLoss(NamedTuple):
    loss: torch.Tensor                 # fp32, 0-dim
    clip_fraction: torch.Tensor        # fp32, 0-dim
    kl: torch.Tensor                   # fp32, 0-dim: mean over the targets
    logp: torch.Tensor                 # fp32 [T]
    entropy: Optional[torch.Tensor]    # fp32 [T], where it has a coefficient
    dlogits: torch.Tensor              # [T, V] of the logits' type


_NOTHING = contextlib.nullcontext()


def _on(stream):
    return _NOTHING if stream is None else torch.cuda.stream(stream)


def _floats(device, *shape):
    return torch.empty(shape, dtype=torch.float32, device=device)


def _bytes(device, size):
    return torch.empty(size, dtype=torch.uint8, device=device)


def _handle(stream, device) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    if _RAW_STREAM is not None:
        return int(_RAW_STREAM(device.index))
    return int(torch.cuda.current_stream(device).cuda_stream)


def _vector(x, name, n, dtype, device):
    if not (isinstance(x, torch.Tensor) and x.dtype == dtype and x.device == device and x.dim() == 1 and x.shape[0] == n
            and (n <= 1 or x.stride(0) == 1)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of [{n}] on {device}")
    return x.data_ptr()


def _matrix(x, name):
    """(rows, columns, row stride) of a CUDA matrix whose rows are contiguous."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2 and x.dtype in TYPES):
        raise ValueError(f"{name} must be a 2-D CUDA tensor in bfloat16, float16 or float32")
    rows, cols = x.shape
    if cols < 1 or (cols > 1 and x.stride(1) != 1) or (rows > 1 and x.stride(0) < cols):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return rows, cols, x.stride(0) if rows > 1 else cols


def _logits(logits, targets, temperature):
    rows, cols, stride = _matrix(logits, "logits")
    return Logits(logits.data_ptr(), _vector(targets, "targets", rows, torch.int64, logits.device), rows, cols, stride,
                  TYPES[logits.dtype], temperature)


def _gradient(logits, a, out):
    """The gradient's tensor: `out`, or a new one laid out like the logits (the same row stride,
    so that both sides of a row have the same alignment)."""
    if out is None:
        if a.stride == a.vocab:
            out = torch.empty_like(logits, memory_format=torch.contiguous_format)
        else:
            out = torch.empty(max(a.rows - 1, 0) * a.stride + a.vocab, dtype=logits.dtype, device=logits.device)
            out = out.as_strided((a.rows, a.vocab), (a.stride, 1))
        return out, a.stride
    rows, cols, stride = _matrix(out, "out")
    if (rows, cols, out.dtype, out.device) != (a.rows, a.vocab, logits.dtype, logits.device):
        raise ValueError("out must have the logits' shape, type and device")
    return out, stride if rows > 1 else a.stride


def token_logp(logits, targets, *, temperature: float = 1.0, entropy: bool = False, stream=None) -> TokenLogp:
    """Log-probabilities of targets [T] (int64) under logits [T, V] / temperature."""
    a = _logits(logits, targets, temperature)
    dev = logits.device
    with _on(stream):  # a tensor each: views of one allocation cost more host time than the allocations
        logp, lse = _floats(dev, a.rows), _floats(dev, a.rows)
        ent = _floats(dev, a.rows) if entropy else None
    _check(_lib().zero_token_logp(ctypes.byref(a), logp.data_ptr(), lse.data_ptr(), ent.data_ptr() if entropy else None,
                                  _handle(stream, dev)), "zero_token_logp")
    return TokenLogp(logp, lse, ent)


def token_logp_backward(logits, targets, forward: TokenLogp, dlogp, dentropy=None, *, temperature: float = 1.0, out=None,
                        stream=None) -> torch.Tensor:
    """The gradient on the logits of a function whose gradients on token_logp's results are
    dlogp and dentropy (fp32 [T]). out: where to write it; the logits themselves are allowed."""
    a = _logits(logits, targets, temperature)
    dev, f32 = logits.device, torch.float32
    logp = _vector(forward.logp, "forward.logp", a.rows, f32, dev)
    lse = _vector(forward.lse, "forward.lse", a.rows, f32, dev)
    g = _vector(dlogp, "dlogp", a.rows, f32, dev)
    h = ent = None
    if dentropy is not None:
        h = _vector(dentropy, "dentropy", a.rows, f32, dev)
        if forward.entropy is None:
            raise ValueError("dentropy needs a forward call with entropy=True")
        ent = _vector(forward.entropy, "forward.entropy", a.rows, f32, dev)
    with _on(stream):
        out, dstride = _gradient(logits, a, out)
    _check(_lib().zero_token_logp_backward(ctypes.byref(a), logp, lse, ent, g, h, out.data_ptr(), dstride,
                                           _handle(stream, dev)),
           "zero_token_logp_backward")
    return out


def linear_logp(hidden, weight, targets, *, temperature: float = 1.0, entropy: bool = False, stream=None) -> TokenLogp:
    """token_logp of hidden [T, D] @ weight [V, D].T (bfloat16 or float16, D and the row strides
    multiples of 8) without writing the logits; no gradient."""
    rows, dim, ld_h = _matrix(hidden, "hidden")
    vocab, wdim, ld_w = _matrix(weight, "weight")
    if weight.dtype != hidden.dtype or weight.device != hidden.device or wdim != dim:
        raise ValueError("hidden and weight must have the same type, device and last dimension")
    dev = hidden.device
    ld_h = ld_h if rows > 1 else -(-dim // 8) * 8  # of a single row: no stride is used
    ld_w = ld_w if vocab > 1 else -(-dim // 8) * 8
    a = Linear(hidden.data_ptr(), weight.data_ptr(), _vector(targets, "targets", rows, torch.int64, dev), rows, vocab, dim,
               ld_h, ld_w, TYPES[hidden.dtype], temperature)
    size = _lib().zero_linear_logp_workspace(rows, vocab)
    with _on(stream):
        logp, lse, ws = _floats(dev, rows), _floats(dev, rows), _bytes(dev, max(size, 0))
        ent = _floats(dev, rows) if entropy else None
    _check(_lib().zero_linear_logp(ctypes.byref(a), logp.data_ptr(), lse.data_ptr(), ent.data_ptr() if entropy else None,
                                   ws.data_ptr(), size, _handle(stream, dev)), "zero_linear_logp")
    return TokenLogp(logp, lse, ent)


def preference_loss(logits, targets, offsets, ref_logp=None, *, beta: float = 0.1, kind: str = "sigmoid",
                    label_smoothing: float = 0.0, average: bool = False, temperature: float = 1.0, out=None,
                    stream=None) -> PreferenceLoss:
    """Preference loss over packed pairs: sequence 2i of offsets [2P + 1] (int64) was chosen over
    2i + 1. kind: "sigmoid" (with label_smoothing), "hinge" or "ipo". ref_logp: fp32 [T]."""
    a = _logits(logits, targets, temperature)
    dev, f32 = logits.device, torch.float32
    if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.shape[0] >= 3 and offsets.shape[0] % 2 == 1):
        raise ValueError("offsets must hold 2 * pairs + 1 values, pairs >= 1")
    pairs = (offsets.shape[0] - 1) // 2
    off = _vector(offsets, "offsets", 2 * pairs + 1, torch.int64, dev)
    ref = None if ref_logp is None else _vector(ref_logp, "ref_logp", a.rows, f32, dev)
    size = _lib().zero_preference_workspace(a.rows)
    with _on(stream):
        out, dstride = _gradient(logits, a, out)
        loss, logp, ws = _floats(dev), _floats(dev, a.rows), _bytes(dev, size)
        pair_loss, chosen, rejected = _floats(dev, pairs), _floats(dev, pairs), _floats(dev, pairs)
    p = Preference(off, ref, pairs, beta, label_smoothing, PREFERENCE[kind], 1 if average else 0, loss.data_ptr(),
                   pair_loss.data_ptr(), chosen.data_ptr(), rejected.data_ptr(), logp.data_ptr(), out.data_ptr(), dstride)
    _check(_lib().zero_preference_loss(ctypes.byref(a), ctypes.byref(p), ws.data_ptr(), size, _handle(stream, dev)),
           "zero_preference_loss")
    return PreferenceLoss(loss, pair_loss, chosen, rejected, logp, out)


def policy_loss(logits, targets, advantages, old_logp=None, ref_logp=None, *, offsets=None, clip_low: float = 0.2,
                clip_high: float = 0.2, dual_clip: float = 0.0, kl: str = "k3", kl_coef: float = 0.0,
                entropy_coef: float = 0.0, reduce: str = "token", per_sequence: Optional[bool] = None,
                temperature: float = 1.0, out=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term and an entropy bonus. advantages: fp32 [T], or one per
    sequence [S] with offsets [S + 1] (int64); their size says which, or per_sequence where S = T.
    old_logp None: the current policy's own (a ratio of 1)."""
    a = _logits(logits, targets, temperature)
    dev, f32 = logits.device, torch.float32
    seqs, off = 0, None
    if offsets is not None:
        if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.shape[0] >= 1):
            raise ValueError("offsets must hold the number of sequences + 1 values")
        seqs = offsets.shape[0] - 1
        off = _vector(offsets, "offsets", seqs + 1, torch.int64, dev)
        if per_sequence is None:
            if seqs == a.rows:
                raise ValueError("as many sequences as tokens: say per_sequence")
            per_sequence = isinstance(advantages, torch.Tensor) and tuple(advantages.shape) == (seqs,)
    if per_sequence and offsets is None:
        raise ValueError("per_sequence needs offsets")
    adv = _vector(advantages, "advantages", seqs if per_sequence else a.rows, f32, dev)
    old = None if old_logp is None else _vector(old_logp, "old_logp", a.rows, f32, dev)
    ref = None if ref_logp is None else _vector(ref_logp, "ref_logp", a.rows, f32, dev)
    with_entropy = entropy_coef != 0.0
    size = _lib().zero_policy_workspace(a.rows)
    with _on(stream):
        out, dstride = _gradient(logits, a, out)
        loss, clip_fraction, kl_mean, ws = _floats(dev), _floats(dev), _floats(dev), _bytes(dev, size)
        logp = _floats(dev, a.rows)
        entropy = _floats(dev, a.rows) if with_entropy else None
    p = Policy(adv, old, ref, off, seqs, clip_low, clip_high, dual_clip, kl_coef, entropy_coef, KL[kl], REDUCE[reduce],
               1 if per_sequence else 0, loss.data_ptr(), clip_fraction.data_ptr(), kl_mean.data_ptr(), logp.data_ptr(), entropy.data_ptr() if with_entropy else None,
               out.data_ptr(), dstride)
    _check(_lib().zero_policy_loss(ctypes.byref(a), ctypes.byref(p), ws.data_ptr(), size, _handle(stream, dev)),
           "zero_policy_loss")
    return PolicyLoss(loss, clip_fraction, kl_mean, logp, entropy, out)
