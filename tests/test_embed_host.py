"""Host-only checks of the embedding calls (no GPU): argument errors are found before anything touches
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


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(rows=2 ** 31), -1), (dict(vocab=0), -1), (dict(vocab=2 ** 31), -1), (dict(dim=0), -1), (dict(ld_weight=15), -1),
    (dict(type=3), -1), (dict(scale=math.nan), -1), (dict(scale=1e39), -1), (dict(ld_weight=2 ** 60), -1), (dict(rows=0), 0), (dict(), -1)])
def test_embedding_arguments(lib, kw, code):
    from zero_gradient_reduce_scatter_gb300.embed import Embed
    a = dict(weight=None, tokens=None, rows=4, vocab=8, dim=16, ld_weight=16, type=0, scale=1.0)
    a.update(kw)
    x = Embed(*a.values())
    assert lib.zero_embedding(ctypes.byref(x), None, 16, None) == code


@pytest.mark.parametrize("kw,size,code", [
    (dict(rows=-1), 1 << 20, -1), (dict(vocab=0), 1 << 20, -1), (dict(dim=0), 1 << 20, -1), (dict(ld_hidden=15), 1 << 20, -1),
    (dict(ld_weight=15), 1 << 20, -1), (dict(type=-1), 1 << 20, -1), (dict(out_type=3), 1 << 20, -1), (dict(scale=math.inf), 1 << 20, -1),
    (dict(accumulate=2), 1 << 20, -1), (dict(), 8, -3), (dict(rows=0, accumulate=1), 1 << 20, 0), (dict(), 1 << 20, -1)])
def test_gradient_arguments(lib, kw, size, code):
    from zero_gradient_reduce_scatter_gb300.embed import EmbedGrad
    a = dict(tokens=None, dhidden=None, dweight=None, rows=4, vocab=8, dim=16, ld_hidden=16, ld_weight=16, type=0, out_type=0, scale=1.0,
             accumulate=0)
    a.update(kw)
    x = EmbedGrad(*a.values())
    assert lib.zero_embedding_backward(ctypes.byref(x), None, size, None) == code


def test_null_and_workspace(lib):
    assert lib.zero_embedding(None, None, 16, None) == -1
    assert lib.zero_embedding_backward(None, None, 1 << 20, None) == -1
    f = lib.zero_embedding_backward_workspace
    assert f(-1, 8, 8, 0) < 0 and f(8, 0, 8, 0) < 0 and f(8, 8, 0, 0) < 0 and f(8, 8, 8, 3) < 0
    assert 0 < f(0, 8, 8, 0) <= f(100, 8, 8, 0) < f(100, 50257, 8, 0)
    assert f(2 ** 31 - 1, 2 ** 30, 2 ** 28, 2) > 0  # no overflow in between
