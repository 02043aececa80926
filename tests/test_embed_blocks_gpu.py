"""embedding_backward where a training batch takes it: blocks of 16 to 128 positions, whose rows, tokens and ends of runs fill every
word of a block, joins of long blocks and of groups of them, and clusters that own a wide vocabulary's tokens. Random
rows in every place, tokens as text has them, masked and invalid ones among them. Formula and tolerances of test_embed_gpu.py."""
import math

import pytest
import torch

import zero_gradient_reduce_scatter_gb300 as zg
from test_embed_gpu import TYPES, UNIT, reference, small, tokens

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def block_of(T, D, size):
    """Positions of a block (zero_embed.cu)."""
    slices, block = -(-D // (32 * (16 // size))), 8
    while block < 128 and T * slices // (2 * block) >= 4096:
        block *= 2
    return block


CASES = [  # T, V, D, dtype, out_dtype, kind, block
    (20000, 50257, 520, "fp32", "fp32", "text", 16), (30000, 50257, 1100, "bf16", "fp32", "text", 32), (16384, 50257, 2048, "fp32", "fp32", "text", 64),
    (40000, 50257, 2048, "bf16", "bf16", "text", 64), (65536, 50257, 2048, "bf16", "bf16", "text", 128), (65536, 50257, 2048, "bf16", "fp32", "text", 128),
    (70001, 151936, 1600, "fp16", "fp16", "text", 64), (70001, 3000, 1024, "fp32", "bf16", "uniform", 128), (65537, 7, 2048, "bf16", "bf16", "two", 128),
    (66001, 5, 2056, "fp32", "fp32", "one", 128), (65536, 700, 2048, "bf16", "bf16", "few", 128),
    # rows of any alignment
    (20000, 50257, 521, "fp32", "fp32", "text", 16), (30000, 50257, 1101, "bf16", "bf16", "text", 32), (40001, 50257, 2047, "bf16", "bf16", "text", 64),
    (33000, 50257, 2047, "fp32", "fp32", "text", 128), (66001, 5, 2047, "bf16", "fp32", "one", 128), (66001, 700, 2049, "fp16", "fp16", "few", 128),
]


@pytest.mark.parametrize("T,V,D,dtype,out_dtype,kind,block", CASES)
def test_blocks(T, V, D, dtype, out_dtype, kind, block):
    assert block_of(T, D, TYPES[dtype].itemsize) == block
    g = torch.Generator(device=DEV).manual_seed(T + D)
    dh = torch.randn((T, D), device=DEV, generator=g).to(TYPES[dtype])
    if kind == "few":  # runs of about a block, so that their ends are anywhere in one
        t = torch.randint(0, V, (T,), device=DEV, generator=g)
        t[::5] = -1
    else:
        t = tokens(kind, T, V, 3)
    dh[(t < 0) | (t >= V)] = math.nan  # not read
    O = TYPES[out_dtype]
    for accumulate, scale in ((False, 1.0), (True, -1.75)):
        out = torch.randn((V, D), device=DEV, generator=g).to(O)
        old = out.clone() if accumulate else None
        assert zg.embedding_backward(t, dh, V, scale=scale, out=out, accumulate=accumulate) is out
        want, tol = reference(t, dh, V, scale, old)
        tol += UNIT[O] * want.abs() + small(O)
        off = want.sub_(out).abs_()
        bad = ~(off <= tol)
        assert not bad.any(), (accumulate, int(bad.sum()), bad.nonzero()[:3].tolist(), off.max().item())
        if accumulate:
            none = torch.ones(V, dtype=torch.bool, device=DEV)
            none[t[(t >= 0) & (t < V)]] = False
            assert torch.equal(out[none], old[none])
        again = old.clone() if accumulate else torch.empty_like(out)
        zg.embedding_backward(t, dh, V, scale=scale, out=again, accumulate=accumulate)
        assert torch.equal(again, out)  # equal calls, equal bits
        del out, old, want, tol, off, bad, again
