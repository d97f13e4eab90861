"""Causal attention of packed sequences where its calls touch other data: results in place of the queries, rows outside all
sequences, scratch memory that held something else; and rows whose scores are partly -infinity.

Both forms of the kernels: with few blocks four waves share a tile, with many they do not. Bounds as in the oracle's module.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B
from test_gpu_causal import DT, HALF, W, _check, _close, _gen, _many, _np, _starts

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


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,many", [(4, 2, False), (8, 1, False), (4, 2, True)])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("lens,first,T", [([50, 71], 0, 128), ([33, 0, 40], 5, 300), ([100], 31, 140)])
def test_what_the_workspace_held_does_not_matter(act, hq, hk, many, D, lens, first, T):
    """Rows outside all sequences leave their places in the workspace as they were: zeros, NaN and infinities in them give the
    same bits."""
    m = _many(T, hq) if many else 1
    q, k, v, d_out = _inputs(_gen(D), T, hq * m, hk * m, D, DT[act])
    starts, out, lse = _starts(lens, first), torch.zeros_like(q), torch.zeros((T, hq * m), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, lse=lse)
    ws = torch.empty(B.moe_causal_attention_backward_workspace_bytes(T, D, hq * m, hk * m) // 4, dtype=torch.int32, device=DEV)
    want = None
    for held in (0, -1, 0x7F800000, -0x800000):      # 0, NaN, infinity, -infinity
        ws.fill_(held)
        grads = [torch.zeros_like(t) for t in (q, k, v)]
        B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, *grads, workspace=ws.view(torch.uint8))
        want = want or grads
        for n, a, b in zip(("dq", "dk", "dv"), grads, want):
            assert _same_bits(a, b), (hex(held), n)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("how", ["dense", "odd"])
def test_padding_takes_no_part(act, many, how):
    """NaN and infinities in the rows outside all sequences leave every bit of the results as it was."""
    T, lens, first, hq, hk, D, dt = 300, [50, 130, 61], 7, 4, 2, 96, DT[act]
    m = _many(T, hq) if many else 1
    pad = 0 if how == "dense" else 1      # rows on 16 bytes, and not
    x = [torch.randn((T, h * m, D + pad), generator=_gen(i), device=DEV).to(dt)[..., :D] for i, h in enumerate((hq, hk, hk, hq))]
    starts, rows = _starts(lens, first), slice(first, first + sum(lens))
    want = None
    for held in (0.0, math.nan, math.inf):
        for t in x:
            t[:first], t[rows.stop:] = held, -held
        q, k, v, d_out = x
        out, lse = torch.zeros_like(q), torch.zeros((T, hq * m), device=DEV)
        B.moe_causal_attention(q, k, v, starts, out, lse=lse)
        out[:first], out[rows.stop:], lse[:first], lse[rows.stop:] = held, held, held, held
        grads = [torch.zeros_like(t) for t in (q, k, v)]
        B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, *grads)
        got = [t[rows] for t in (out, lse, *grads)]
        want = want or got
        assert all(_same_bits(a, b) for a, b in zip(got, want)), held


@pytest.mark.parametrize("many", [False, True])
def test_rows_with_some_scores_of_minus_infinity(many):
    """Keys whose scores are -infinity weigh nothing: results, lse and gradients are those of the other keys alone. A gradient of
    dq is left out: its formula multiplies those keys' weights of 0 by their infinities."""
    T, D, n = 100, 64, 33
    m = _many(T, 1) if many else 1
    q, k, v, d_out = _inputs(_gen(3), T, m, m, D, torch.float32)
    q[..., 0], k[:, :, 0] = 1.0, 0.0
    k[:n, :, 0] = -math.inf
    few = min(m, 3)
    for t in (q, k, v, d_out):
        for h in range(few, m, few):
            t[:, h:h + few] = t[:, :min(few, m - h)].clone()
    starts, out, lse = _starts([T]), torch.empty_like(q), torch.empty((T, m), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, lse=lse)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, torch.empty_like(q), dk, dv)
    for t in (out, lse, dk, dv):
        for h in range(few, m, few):
            assert torch.equal(t[:, h:h + few], t[:, :min(few, m - h)]), h
    rest = [_np(t[n:, :few]) for t in (q, k, v, out, d_out, lse)]
    ro, rl, to, tl = oracle.causal_attention(*rest[:3], [0, T - n], D ** -0.5)
    # the sums run over the n other keys too: 4 u more of the weights for each, on either side of the division
    more = 8 * n * 2.0 ** -24
    size = oracle.causal_attention(*rest[:2], abs(rest[2]), [0, T - n], D ** -0.5)[0]
    _close(rest[3], ro, to + more * size + HALF["f32"] * abs(ro), "out")
    _close(rest[5], rl, tl + more, "lse")
    ref = oracle.causal_attention_grad(*rest, [0, T - n], D ** -0.5)
    for name, x, r, t in zip(("dk", "dv"), (dk, dv), ref[1:3], ref[4:]):
        _close(x[n:, :few], r, t + HALF["f32"] * abs(r) + 1e-37, name)
    assert (out[:n] == 0).all() and (lse[:n] == -math.inf).all() and (dk[:n] == 0).all() and (dv[:n] == 0).all()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_16_bits_in_tiles_with_masks(many, D):
    """In a sequence of one tile t enters dq and dk as two bf16 numbers, what is left off being 2^-8 of 2^-8 of it at most. Keys
    with an offset in common show that, since the t of a row cancel and their roundings do not: with t rounded once the oracle's
    own sums pass these bounds sixfold and more."""
    T = 32
    m = _many(T, 1) if many else 1
    q, k, v, d_out = _inputs(_gen(5 + D), T, m, m, D, torch.bfloat16)
    k = (k + 16.0 * torch.randn(D, generator=_gen(1), device=DEV).sign()).bfloat16()
    few = min(m, 3)
    for t in (q, k, v, d_out):
        for h in range(few, m, few):
            t[:, h:h + few] = t[:, :min(few, m - h)].clone()
    scale = 2.0 ** -10
    starts, out, lse = _starts([T]), torch.empty_like(q), torch.empty((T, m), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, scale=scale, lse=lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, *grads, scale=scale)
    ref = oracle.causal_attention_grad(*(_np(t[:, :few]) for t in (q, k, v, out, d_out, lse)), [0, T], scale, W["bf16"] ** 2)
    for name, x, r, t in zip(("dq", "dk"), grads, ref[:2], ref[3:5]):
        _close(x[:, :few], r, t + HALF["bf16"] * abs(r) + 1e-37, name)
        for h in range(few, m, few):
            assert torch.equal(x[:, h:h + few], x[:, :min(few, m - h)]), (name, h)


def _by_rows(q, k, v, d_out, starts, scale):
    """out, lse, dq, dk and dv of one head in fp64, every sum over the tokens that are seen and no others."""
    T, D = q.shape
    out, dq, dk, dv = np.zeros((4, T, D))
    lse = np.zeros(T)
    with np.errstate(all="ignore"):
        for a, b in zip(starts[:-1], starts[1:]):
            for i in range(a, b):
                kk, vv, g = k[a:i + 1], v[a:i + 1], d_out[i]
                s = scale * (kk @ q[i])
                m = s.max()
                p = np.exp(s - m)
                lse[i] = m + np.log(p.sum())
                p /= p.sum()
                out[i] = (p[:, None] * vv).sum(0)
                t = p * ((vv * g).sum(1) - (g * out[i]).sum())
                dq[i] = scale * (t[:, None] * kk).sum(0)
                dk[a:i + 1] += scale * t[:, None] * q[i]
                dv[a:i + 1] += p[:, None] * g
    return out, lse, dq, dk, dv


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_which_results_are_nan(act, many, D):
    """A NaN in one channel of a token makes exactly those results NaN whose formula holds it."""
    T, lens, first, dt = 230, [60, 150, 13], 4, DT[act]
    m = _many(T, 1) if many else 1
    starts = _starts(lens, first)
    s, rows = starts.cpu().numpy(), slice(first, first + sum(lens))
    for which in range(4):
        for bad in (first + 60 + 70, first + 60 + 149):      # amid its sequence, and its last token
            x = [t[:, :1].expand(T, m, D).clone() for t in _inputs(_gen(which), T, 1, 1, D, dt)]
            x[which][bad, :, 3] = math.nan
            q, k, v, d_out = x
            out, lse = torch.zeros_like(q), torch.zeros((T, m), device=DEV)
            B.moe_causal_attention(q, k, v, starts, out, lse=lse)
            grads = [torch.zeros_like(t) for t in (q, k, v)]
            B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, *grads)
            want = _by_rows(*(_np(t[:, 0]) for t in x), s, D ** -0.5)
            for n, a, b in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads), want):
                nan = torch.as_tensor(np.isnan(b), device=DEV)[:, None].expand(a.shape)
                assert torch.equal(a[rows].isnan(), nan[rows]), (which, bad, n)
                assert a[rows][~nan[rows]].isfinite().all(), (which, bad, n)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("lens", [[50] + [0] * 4000, [0] * 4000 + [50, 1],
                                  [5] + [0] * 3000 + [1, 0, 2] + [0] * 1000 + [40] + [0] * 200])
def test_thousands_of_empty_sequences(act, many, lens):
    """As padding of seq_start behind, in front of and between the others, beside rows that belong to none."""
    m = _many(100, 2) if many else 1
    _check(act, 100, 2 * m, m, 64, lens, first=3)
