"""Causal attention of packed sequences where its calls touch other data: results in place of the queries, rows outside all
sequences, scratch memory that held something else; and rows whose scores are partly -infinity.

Both forms of the kernels: with few blocks four waves share a tile, with many they do not. Bounds as in the oracle's module.
"""
import math

import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B
from test_gpu_causal import DT, HALF, W, _close, _gen, _many, _np, _starts

pytestmark = pytest.mark.gpu


def _inputs(g, T, hq, hk, D, dt):
    return [torch.randn((T, h, D), generator=g, device=DEV).to(dt) for h in (hq, hk, hk, hq)]


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_in_place(act, many, D):
    """out may be q: the bits of a call with a result of its own, also where a tile holds a NaN that a row does not see, and the
    row is summed again over what it sees alone."""
    T, lens, first, dt = 170, [40, 70, 50], 3, DT[act]
    m = _many(T, 4) if many else 1
    q, k, v, _ = _inputs(_gen(D), T, 4 * m, 2 * m, D, dt)
    starts = _starts(lens, first)
    for bad in (None, math.nan, math.inf):
        if bad is not None:
            at = first + 40 + 37
            q[at], k[at, :, 5], v[at] = bad, bad, bad
            for t in (q, k, v):
                t[:first], t[first + 160:] = bad, bad
        want, want_lse = q.clone(), torch.full((T, 4 * m), 7.0, device=DEV)
        B.moe_causal_attention(q, k, v, starts, want, lse=want_lse)
        if bad is not None:
            assert torch.isfinite(want[first:at]).all() and torch.isfinite(want[first + 110:first + 160]).all()
        own, lse = q.clone(), torch.full((T, 4 * m), 7.0, device=DEV)
        B.moe_causal_attention(own, k, v, starts, own, lse=lse)
        assert _same_bits(own, want) and _same_bits(lse, want_lse), bad
