"""Host-only checks of the loss and gradient-clipping calls (no GPU): argument errors are found
before anything touches CUDA, workspaces are sized as documented, and no entry throws."""
import ctypes
import math

import pytest

from zero_gradient_reduce_scatter_gb300 import _build


@pytest.fixture(scope="module")
def zg():
    _build.build()
    import zero_gradient_reduce_scatter_gb300 as zg
    zg._lib()
    return zg


def logits(**kw):
    from zero_gradient_reduce_scatter_gb300.losses import Logits
    a = dict(logits=None, targets=None, rows=4, vocab=8, stride=8, type=0, temperature=1.0)
    a.update(kw)
    return Logits(*a.values())


BAD_LOGITS = [dict(rows=-1), dict(vocab=0), dict(vocab=2 ** 31), dict(stride=7), dict(type=3), dict(type=-1), dict(temperature=0.0),
              dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf), dict(rows=2 ** 40, stride=2 ** 40)]


@pytest.mark.parametrize("kw", BAD_LOGITS)
def test_bad_logits(zg, kw):
    lib, a = zg._lib(), logits(**kw)
    assert lib.zero_token_logp(ctypes.byref(a), None, None, None, None) == -1
    assert lib.zero_token_logp_backward(ctypes.byref(a), None, None, None, None, None, None, 8, None) == -1


def test_null_pointers(zg):
    lib, a = zg._lib(), logits()
    assert lib.zero_token_logp(None, None, None, None, None) == -1
    assert lib.zero_token_logp(ctypes.byref(a), None, None, None, None) == -1
    assert lib.zero_token_logp_backward(ctypes.byref(a), None, None, None, None, None, None, 7, None) == -1
    assert lib.zero_preference_loss(ctypes.byref(a), None, None, 1 << 20, None) == -1
    assert lib.zero_policy_loss(ctypes.byref(a), None, None, 1 << 20, None) == -1
    assert lib.zero_linear_logp(None, None, None, None, None, 0, None) == -1
    empty = logits(rows=0)
    assert lib.zero_token_logp(ctypes.byref(empty), None, None, None, None) == 0


def preference(**kw):
    from zero_gradient_reduce_scatter_gb300.losses import Preference
    a = dict(offsets=None, ref_logp=None, pairs=1, beta=0.1, label_smoothing=0.0, kind=0, average=0, loss=None, pair_loss=None,
             chosen_reward=None, rejected_reward=None, logp=None, dlogits=None, dstride=8)
    a.update(kw)
    return Preference(*a.values())


@pytest.mark.parametrize("kw,size,code", [
    (dict(pairs=0), 1 << 20, -1), (dict(beta=0.0), 1 << 20, -1), (dict(beta=math.inf), 1 << 20, -1), (dict(beta=math.nan), 1 << 20, -1),
    (dict(label_smoothing=-0.1), 1 << 20, -1), (dict(label_smoothing=0.6), 1 << 20, -1), (dict(kind=3), 1 << 20, -1),
    (dict(average=2), 1 << 20, -1), (dict(), 8, -3), (dict(), 1 << 20, -1)])
def test_preference_arguments(zg, kw, size, code):
    a, p = logits(), preference(**kw)
    if not kw and size > 8:
        p.dstride = 7
    assert zg._lib().zero_preference_loss(ctypes.byref(a), ctypes.byref(p), None, size, None) == code


def policy(**kw):
    from zero_gradient_reduce_scatter_gb300.losses import Policy
    a = dict(advantages=None, old_logp=None, ref_logp=None, offsets=None, seqs=0, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
             kl_coef=0.0, entropy_coef=0.0, kl=2, reduce=0, per_sequence=0, loss=None, clip_fraction=None, kl_mean=None, logp=None,
             entropy=None, dlogits=None, dstride=8)
    a.update(kw)
    return Policy(*a.values())


@pytest.mark.parametrize("kw,size,code", [
    (dict(clip_low=-0.1), 1 << 20, -1), (dict(clip_low=1.1), 1 << 20, -1), (dict(clip_high=-1.0), 1 << 20, -1),
    (dict(clip_high=math.inf), 1 << 20, -1), (dict(dual_clip=1.0), 1 << 20, -1), (dict(dual_clip=math.inf), 1 << 20, -1),
    (dict(kl_coef=math.nan), 1 << 20, -1), (dict(kl_coef=0.1), 1 << 20, -1), (dict(entropy_coef=0.1), 1 << 20, -1),
    (dict(kl=3), 1 << 20, -1), (dict(reduce=3), 1 << 20, -1), (dict(reduce=1), 1 << 20, -1), (dict(per_sequence=1), 1 << 20, -1),
    (dict(offsets=16, seqs=-1), 1 << 20, -1), (dict(), 8, -3)])
def test_policy_arguments(zg, kw, size, code):
    a, p = logits(), policy(**kw)
    assert zg._lib().zero_policy_loss(ctypes.byref(a), ctypes.byref(p), None, size, None) == code


@pytest.mark.parametrize("kw,size,code", [
    (dict(rows=-1), 1 << 20, -1), (dict(vocab=0), 1 << 20, -1), (dict(dim=0), 1 << 20, -1), (dict(ld_hidden=8), 1 << 20, -1),
    (dict(ld_weight=8), 1 << 20, -1), (dict(type=2), 1 << 20, -1), (dict(temperature=0.0), 1 << 20, -1),
    (dict(ld_hidden=20), 1 << 20, -2), (dict(ld_weight=20), 1 << 20, -2), (dict(), 8, -3), (dict(rows=0), 0, 0),
    (dict(), 1 << 20, -1)])
def test_linear_arguments(zg, kw, size, code):
    from zero_gradient_reduce_scatter_gb300.losses import Linear
    a = dict(hidden=None, weight=None, targets=None, rows=4, vocab=8, dim=16, ld_hidden=16, ld_weight=16, type=0, temperature=1.0)
    a.update(kw)
    x = Linear(*a.values())
    assert zg._lib().zero_linear_logp(ctypes.byref(x), None, None, None, None, size, None) == code


def test_workspaces(zg):
    lib = zg._lib()
    for f in (lib.zero_preference_workspace, lib.zero_policy_workspace):
        assert f(-1) < 0 and f(0) >= 0 and f(1000) >= f(10) > 0
    assert lib.zero_linear_logp_workspace(-1, 5) < 0 and lib.zero_linear_logp_workspace(5, 0) < 0
    assert lib.zero_linear_logp_workspace(100, 50257) > 0
    assert lib.zero_grads_workspace(0) < 0 and lib.zero_grads_workspace(10) > 0


def test_gradient_plans(zg):
    lib = zg._lib()
    plan = ctypes.c_void_p(0x77)
    assert lib.zero_grads_init(ctypes.byref(plan), None, 1, None, 1 << 20, None) == -1 and not plan.value
    from zero_gradient_reduce_scatter_gb300.gradclip import GradTensor
    rows = (GradTensor * 1)(GradTensor(None, None, 5, 0, 0))
    at = ctypes.cast(rows, ctypes.c_void_p)
    assert lib.zero_grads_init(ctypes.byref(plan), at, 0, None, 1 << 20, None) == -1
    assert lib.zero_grads_init(ctypes.byref(plan), at, 1, None, 8, None) == -3
    assert lib.zero_grads_init(ctypes.byref(plan), at, 1, None, 1 << 20, None) == -1
    for bogus in (None, ctypes.c_void_p(0x1234)):
        assert lib.zero_grads_clip(bogus, 1.0, None, None, None, None) == -7
        assert lib.zero_grads_destroy(bogus) == -7
