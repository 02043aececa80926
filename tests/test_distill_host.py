"""Host-only checks of the distillation calls (no GPU): argument errors are found before anything touches
CUDA, and workspaces are sized as documented."""
import ctypes
import math

import pytest

from zero_gradient_reduce_scatter_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    import zero_gradient_reduce_scatter_gb300 as zg
    return zg._lib()


def logits(**kw):
    from zero_gradient_reduce_scatter_gb300.losses import Logits
    a = dict(logits=None, targets=None, rows=4, vocab=8, stride=8, type=0, temperature=1.0)
    a.update(kw)
    return Logits(*a.values())


@pytest.mark.parametrize("kw,k,code", [
    (dict(rows=-1), 2, -1), (dict(vocab=0), 1, -1), (dict(stride=7), 2, -1), (dict(type=3), 2, -1), (dict(temperature=0.0), 2, -1), (dict(), 0, -1),
    (dict(), -3, -1), (dict(), 9, -1), (dict(vocab=1000, stride=1000), 513, -1), (dict(rows=0), 2, 0), (dict(), 2, -1)])
def test_top_arguments(lib, kw, k, code):
    a = logits(**kw)
    assert lib.zero_top_logits(ctypes.byref(a), k, None, None, None, None, None) == code


def distill(**kw):
    from zero_gradient_reduce_scatter_gb300.distill import Distill
    a = dict(index=None, teacher_logp=None, teacher_rest=None, offsets=None, seqs=0, k=2, mix=0.5, kl_coef=1.0, ce_coef=0.0, kind=0, tail=0,
             reduce=0, loss=None, kl=None, token_kl=None, logp=None, dlogits=None, dstride=8)
    a.update(kw)
    return Distill(*a.values())


@pytest.mark.parametrize("kw,size,code", [
    (dict(k=0), 1 << 20, -1), (dict(k=9), 1 << 20, -1), (dict(mix=0.0), 1 << 20, -1), (dict(mix=1.0), 1 << 20, -1), (dict(mix=math.nan), 1 << 20, -1),
    (dict(kl_coef=math.inf), 1 << 20, -1), (dict(ce_coef=math.nan), 1 << 20, -1), (dict(kl_coef=1e39), 1 << 20, -1), (dict(kind=3), 1 << 20, -1),
    (dict(kind=-1), 1 << 20, -1), (dict(tail=3), 1 << 20, -1), (dict(kind=1, tail=1), 1 << 20, -1), (dict(kind=2, tail=2), 1 << 20, -1),
    (dict(reduce=1), 1 << 20, -1), (dict(reduce=3), 1 << 20, -1), (dict(offsets=16, seqs=-1), 1 << 20, -1), (dict(dstride=7), 1 << 20, -1),
    (dict(), 8, -3), (dict(), 1 << 20, -1)])
def test_distill_arguments(lib, kw, size, code):
    a, p = logits(), distill(**kw)
    assert lib.zero_distill_loss(ctypes.byref(a), ctypes.byref(p), None, size, None) == code


def test_wide_vocabularies_and_null(lib):
    a, p = logits(vocab=2 ** 20 + 1, stride=2 ** 20 + 1), distill(dstride=2 ** 20 + 1)
    assert lib.zero_distill_loss(ctypes.byref(a), ctypes.byref(p), None, 1 << 20, None) == -1
    assert lib.zero_distill_loss(None, ctypes.byref(p), None, 1 << 20, None) == -1
    assert lib.zero_distill_loss(ctypes.byref(a), None, None, 1 << 20, None) == -1
    assert lib.zero_top_logits(None, 2, None, None, None, None, None) == -1
    f = lib.zero_distill_workspace
    assert f(-1) < 0 and f(2 ** 62) < 0 and 0 < f(0) <= f(10) < f(1000)


def test_python_checks_come_first():
    """What needs no GPU to be refused."""
    import torch
    import zero_gradient_reduce_scatter_gb300 as zg
    x = torch.zeros((4, 8))
    i = torch.zeros((4, 2), dtype=torch.int64)
    with pytest.raises(ValueError):
        zg.top_logits(x, 2)
    with pytest.raises(ValueError):
        zg.distill_loss(x, i[:, 0], i, x[:, :2])
    with pytest.raises(ValueError):
        zg.embedding(x, i[:, 0])
    with pytest.raises(ValueError):
        zg.embedding_backward(i[:, 0], x, 8)
