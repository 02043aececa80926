"""distill_loss on lists at the edge of what the call allows: renormalised lists whose probabilities, or whose sum, pass fp32.
Against test_distill_gpu's reference; its tolerances, in which a renormalised log-probability lp - log sum exp is off by
its own rounding and that of lp at its distance from the list's largest, which count as |log p| does."""
import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_distill_gpu import UNIT, close, data, reference, weights

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("T,V,k,dtype", [(12, 3000, 20, "fp32"), (1300, 3000, 64, "bf16"), (12, 50257, 300, "bf16"), (320, 20011, 64, "fp16"),
                                         (8, 150001, 512, "bf16")])
@pytest.mark.parametrize("offset", [-500.0, -104.0, -90.0, -64.0, -30.0, 0.0, 60.0, 64.0, 95.0, 600.0])
def test_renormalised_lists_of_any_size(T, V, k, dtype, offset):
    """Lists of a distribution's far tail, and of a teacher's unnormalised logits: a constant leaves them as they are."""
    x, y, index, lp, _ = data(T, V, k, dtype, 3)
    lp = (lp + offset).contiguous()
    index[0] = -1  # a list of nothing
    w = weights(y, None, "sum")
    D, logp, grad, dtol, ltol, gtol = reference(x, y, index[:], lp, None, w, "forward", "renormalise", 0.5, 1.0, 0.2, 1.0)
    D[0], grad[0] = 0.0, 0.0
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise", ce_coef=0.2, reduce="sum")
    close(r.token_kl[1:], D[1:], dtol[1:], "token_kl")
    close(r.logp, logp, ltol, "logp")
    close(r.dlogits[1:], grad[1:], (gtol + UNIT[dtype] * grad.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0))[1:], "dlogits")
    assert r.token_kl[0] == 0 and bool(r.dlogits[0].isfinite().all())


def test_renormalised_lists_of_unequal_parts():
    """Entries that lie hundreds apart, in any order and in every warp's part of a list."""
    T, V, k = 40, 9001, 200
    x, y, index, _, _ = data(T, V, k, "fp32", 5, short=False)
    g = torch.Generator(device=DEV).manual_seed(4)
    lp = (torch.rand((T, k), device=DEV, generator=g) * 800 - 400).contiguous()
    lp[1] -= 400
    lp[2] += 500
    lp[3, :100] = -1000.0
    w = weights(y, None, "token")
    far = lp.double() - lp.double().amax(1, keepdim=True)  # the reference's exponentials end at e^709
    D, _, grad, dtol, _, gtol = reference(x, y, index, far, None, w, "forward", "renormalise", 0.5, 1.0, 0.0, 1.0)
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise")
    close(r.token_kl, D, dtol, "token_kl")
    close(r.dlogits, grad, gtol + UNIT["fp32"] * grad.abs(), "dlogits")
    lp[4, 7] = float("inf")
    lp[5, 7] = float("nan")
    y[4] = y[5] = 3
    r = zg.distill_loss(x, y, index, lp, None, tail="renormalise")
    assert bool(r.dlogits[4:6].isnan().all()) and bool(r.token_kl[4:6].isnan().all()) and bool(r.dlogits[6:].isfinite().all())
