"""Causal attention of packed sequences and its gradient against the fp64 oracle, whose module derives the bounds used here.

To a bound of the sums in fp32 comes the rounding of the result: half a unit (fp32 2^-24, bf16 2^-8) of it.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
W = {"f32": 0.0, "bf16": 2.0 ** -8}


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _laid_out(g, T, H, D, dt, how):
    x = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)     # noqa: E731
    if how == "dense":
        return x(T, H, D)
    if how == "fused":                      # a slice of a wider projection
        return x(T, H + 3, D)[:, 2:2 + H]
    if how == "heads_first":                # [H, T, D]
        return x(H, T, D).transpose(0, 1)
    if how == "odd":                        # neither strides nor start fit a wide load
        return x(T * H * (D + 1) + 1)[1:].view(T, H, D + 1)[:, :, :D]
    if how == "one_head":                   # one row read for every head
        return x(T, 1, D).expand(T, H, D)
    raise ValueError(how)


def _outs(T, H, D, dt, how):
    return _laid_out(_gen(1), T, H, D, dt, "dense" if how == "one_head" else how).fill_(7.0)


def _starts(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def _close(got, ref, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / (tol + 1e-300)):.2f} tol"


def _check(act, T, hq, hk, D, lens, how="dense", first=0, scale=None, seed=0, edit=None, backward=True):
    """One forward and backward call against the oracle; rows outside the sequences keep what they held."""
    g, dt = _gen(seed + T * 7 + D), DT[act]
    q, k, v, d_out = (_laid_out(g, T, h, D, dt, how) for h in (hq, hk, hk, hq))
    if edit:
        q, k, v, d_out = (t.clone() for t in (q, k, v, d_out))
        edit(q, k, v, d_out)
    starts = _starts(lens, first)
    s_np = starts.cpu().numpy()
    scale_ = D ** -0.5 if scale is None else scale
    out, lse = _outs(T, hq, D, dt, how), torch.full((T, hq), 7.0, device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, scale=scale, lse=lse)
    ro, rl, to, tl = oracle.causal_attention(_np(q), _np(k), _np(v), s_np, scale_, W[act])
    inside = np.zeros(T, dtype=bool)
    inside[s_np[0]:s_np[-1]] = True
    at = torch.as_tensor(inside, device=DEV)
    assert (out[~at] == 7.0).all() and (lse[~at] == 7.0).all()
    tiny = 1e-37
    _close(out[at], ro[inside], (to + HALF[act] * np.abs(ro))[inside] + tiny, "out")
    _close(lse[at], rl[inside], tl[inside], "lse")
    if not backward:
        return
    dq, dk, dv = _outs(T, hq, D, dt, how), _outs(T, hk, D, dt, how), _outs(T, hk, D, dt, how)
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, dq, dk, dv, scale=scale)
    ref = oracle.causal_attention_grad(*map(_np, (q, k, v, out, d_out, lse)), s_np, scale_, W[act])
    for n, x, r, t in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[:3], ref[3:]):
        assert (x[~at] == 7.0).all()
        _close(x[at], r[inside], (t + HALF[act] * np.abs(r))[inside] + tiny, n)


CASES = [
    # T, hq, hk, D, lens, how, first row
    (1, 1, 1, 8, [1], "dense", 0),
    (2, 4, 2, 64, [1, 1], "dense", 0),
    (33, 2, 1, 64, [33], "fused", 0),
    (130, 6, 2, 80, [0, 31, 0, 0, 33, 1, 65], "dense", 0),
    (131, 3, 3, 72, [64, 64], "fused", 2),          # rows before and behind the sequences
    (300, 8, 1, 128, [300], "heads_first", 0),
    (257, 7, 1, 96, [129, 128], "dense", 0),
    (260, 4, 4, 128, [100, 3, 157], "odd", 0),
    (97, 10, 5, 192, [40, 57], "fused", 0),
    (200, 4, 2, 256, [150, 7, 43], "dense", 0),
    (161, 4, 2, 136, [161], "odd", 0),
    (70, 6, 3, 64, [35, 35], "one_head", 0),
    (640, 5, 1, 64, [1] * 100 + [2] * 50 + [0] * 70 + [440], "dense", 0),
]


def _many(T, hq):
    """How often hq heads give each CU a block of 128 tokens (with fewer, four waves share 32)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-cus // (-(-T // 128) * hq))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,lens,how,first", CASES)
def test_attention_and_gradient(act, T, hq, hk, D, lens, how, first, many):
    m = _many(T, hq) if many else 1
    _check(act, T, hq * m, hk * m, D, lens, how, first)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(2, 1), (30, 5)])
@pytest.mark.parametrize("D", [16, 64, 96, 128, 192, 256])
def test_longer(act, D, heads):
    """Several stages of keys, tiles without masks, sequences that end inside tiles; both forms of the kernels."""
    _check(act, 1100, *heads, D, [700, 1, 399], seed=D)
