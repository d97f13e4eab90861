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


def _check(act, T, hq, hk, D, lens, how="dense", first=0, scale=None, seed=0, edit=None):
    """One forward and backward call against the oracle; rows outside the sequences keep what they held. Of many key/value heads the
    first three (and their query heads) are compared with it, and the others, which repeat their inputs, with them, bit for bit."""
    g, dt, G, few = _gen(seed + T * 7 + D), DT[act], hq // hk, min(hk, 3)
    q, k, v, d_out = (_laid_out(g, T, h, D, dt, how) for h in (hq, hk, hk, hq))
    if edit:
        q, k, v, d_out = (t.clone() for t in (q, k, v, d_out))
        edit(q, k, v, d_out)
    if how != "one_head":
        for t, n in ((q, G * few), (k, few), (v, few), (d_out, G * few)):
            for h in range(n, t.shape[1], n):
                t[:, h:h + n] = t[:, :min(n, t.shape[1] - h)].clone()
    starts = _starts(lens, first)
    s_np = starts.cpu().numpy()
    scale_ = D ** -0.5 if scale is None else scale
    out, lse = _outs(T, hq, D, dt, how), torch.full((T, hq), 7.0, device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, scale=scale, lse=lse)
    dq, dk, dv = _outs(T, hq, D, dt, how), _outs(T, hk, D, dt, how), _outs(T, hk, D, dt, how)
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, dq, dk, dv, scale=scale)
    inside = np.zeros(T, dtype=bool)
    inside[s_np[0]:s_np[-1]] = True
    at = torch.as_tensor(inside, device=DEV)
    for t, n in ((out, G * few), (lse, G * few), (dq, G * few), (dk, few), (dv, few)):
        assert (t[~at] == 7.0).all()
        for h in range(n, t.shape[1], n):
            assert torch.equal(t[:, h:h + n], t[:, :min(n, t.shape[1] - h)]), h
    q, d_out, out, lse, dq, k, v, dk, dv = (*(t[:, :G * few] for t in (q, d_out, out, lse, dq)), *(t[:, :few] for t in (k, v, dk, dv)))
    ro, rl, to, tl = oracle.causal_attention(_np(q), _np(k), _np(v), s_np, scale_, W[act])
    tiny = 1e-37
    _close(out[at], ro[inside], (to + HALF[act] * np.abs(ro))[inside] + tiny, "out")
    _close(lse[at], rl[inside], tl[inside], "lse")
    ref = oracle.causal_attention_grad(*map(_np, (q, k, v, out, d_out, lse)), s_np, scale_, W[act])
    for n, x, r, t in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[:3], ref[3:]):
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
    """How often hq heads give each CU more than four blocks of 128 tokens (with fewer, four waves may share 32)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return (4 * cus) // (-(-T // 128) * hq) + 1


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,lens,how,first", CASES)
def test_attention_and_gradient(act, T, hq, hk, D, lens, how, first, many):
    m = _many(T, hq) if many else 1
    _check(act, T, hq * m, hk * m, D, lens, how, first)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(2, 1), (120, 10)])
@pytest.mark.parametrize("D", [16, 64, 96, 128, 192, 256])
def test_longer(act, D, heads):
    """Several stages of keys, tiles without masks, sequences that end inside tiles; both forms of the kernels."""
    _check(act, 1100, *heads, D, [700, 1, 399], seed=D)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_what_is_masked_does_not_matter(act, many, D):
    """Infinities and NaN in a token, and in rows outside all sequences, reach only the rows that see them."""
    lens, first, T = [40, 70, 50], 3, 170
    m = _many(T, 4) if many else 1
    hq, hk, dt = 4 * m, 2 * m, DT[act]
    g = _gen(D)
    q, k, v, d_out = (torch.randn((T, h, D), generator=g, device=DEV).to(dt) for h in (hq, hk, hk, hq))
    clean = [_np(t) for t in (q, k, v, d_out)]
    bad = first + 40 + 37
    for rows in (slice(bad, bad + 1), slice(0, first), slice(first + 160, T)):
        q[rows], k[rows, :, 5], v[rows], d_out[rows] = math.nan, math.nan, math.inf, -math.inf
    starts = _starts(lens, first)
    s = starts.cpu().numpy()
    out, lse = _outs(T, hq, D, dt, "dense"), torch.empty((T, hq), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, lse=lse)
    fine = np.zeros(T, dtype=bool)
    fine[s[0]:s[-1]] = True
    others = fine.copy()
    others[s[1]:s[2]] = False      # tokens of the other sequences
    fine[bad:s[2]] = False         # rows that do not see the bad token
    ro, rl, to, tl = oracle.causal_attention(*clean[:3], s, D ** -0.5, W[act])
    _close(_np(out)[fine], ro[fine], (to + HALF[act] * np.abs(ro))[fine], "out")
    _close(_np(lse)[fine], rl[fine], tl[fine], "lse")
    assert not torch.isfinite(out[bad:s[2]]).any()
    dq, dk, dv = (_outs(T, h, D, dt, "dense") for h in (hq, hk, hk))
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, dq, dk, dv)
    o, z = _np(out), _np(lse)
    o[~fine], z[~fine] = 0.0, 0.0
    ref = oracle.causal_attention_grad(*clean[:3], o, clean[3], z, s, D ** -0.5, W[act])
    for n, x, r, t, rows in (("dq", dq, ref[0], ref[3], fine), ("dk", dk, ref[1], ref[4], others), ("dv", dv, ref[2], ref[5], others)):
        _close(_np(x)[rows], r[rows], (t + HALF[act] * np.abs(r))[rows] + 1e-37, n)
        assert (x[:first] == 7.0).all() and (x[first + 160:] == 7.0).all()


@pytest.mark.parametrize("many", [False, True])
def test_scores_of_minus_infinity(many):
    """A row that sees nothing else gives zeros, and has no part in dk and dv."""
    T, D = 100, 64
    m = _many(T, 1) if many else 1
    g = _gen(3)
    q, k, v, d_out = (torch.randn((T, m, D), generator=g, device=DEV) for _ in range(4))
    q[..., 0], k[:, :, 0] = 1.0, 0.0
    k[:33, :, 0] = -math.inf
    starts, out, lse = _starts([T]), torch.empty_like(q), torch.empty((T, m), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, lse=lse)
    assert (out[:33] == 0).all() and (lse[:33] == -math.inf).all() and torch.isfinite(out[33:]).all()
    rest, rest_lse = torch.empty_like(q[33:]), torch.empty((T - 33, m), device=DEV)
    B.moe_causal_attention(q[33:], k[33:], v[33:], _starts([T - 33]), rest, lse=rest_lse)
    ref, _, tol, _ = oracle.causal_attention(_np(q[33:]), _np(k[33:]), _np(v[33:]), [0, T - 33], D ** -0.5)
    _close(out[33:], ref, 2 * tol, "out")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, dq, dk, dv)
    assert (dk[:33] == 0).all() and (dv[:33] == 0).all() and torch.isfinite(dk[33:]).all() and torch.isfinite(dv).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(act, many, scale):
    m = _many(150, 2) if many else 1
    _check(act, 150, 2 * m, m, 64, [150], scale=scale)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_rise_and_fall(act, many, sign):
    """Scores that grow (or fall) by hundreds along the keys: the running reference moves in tiles without masks."""
    T, D = 400, 64
    m = _many(T, 1) if many else 1

    def edit(q, k, v, d_out):
        q[..., 0] = 4.0
        k[:, :, 0] = sign * torch.arange(T, device=DEV)[:, None] / 2.0
    _check(act, T, m, m, D, [T], edit=edit)


def test_thousands_of_sequences():
    """One token each among empty ones: its row is its value (p v / p in fp32: the product, the reciprocal and their product round, three
    half units), its score is its lse, its keys have no gradient."""
    n, D = 5000, 64
    g = _gen(9)
    lens = torch.zeros(9300, dtype=torch.int64)
    lens[torch.randperm(9300, generator=torch.Generator().manual_seed(1))[:n]] = 1
    starts = _starts(lens.numpy())
    q, k, v, d_out = (torch.randn((n, 2, D), generator=g, device=DEV) for _ in range(4))
    out, lse = torch.empty_like(q), torch.empty((n, 2), device=DEV)
    B.moe_causal_attention(q, k, v, starts, out, lse=lse)
    assert ((out - v).abs() <= 3 * 2.0 ** -24 * v.abs() * (1 + 2.0 ** -20)).all()
    s = (q.double() * k.double()).sum(-1) * D ** -0.5
    bound = (D + 4) * 2 ** -23 * (q.double() * k.double()).abs().sum(-1) * D ** -0.5 + 2.0 ** -20
    assert ((lse - s).abs() <= bound).all()
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    B.moe_causal_attention_backward(d_out, q, k, v, out, lse, starts, dq, dk, dv)
    mag = (d_out * v).abs().sum(-1, keepdim=True).double()
    rel = (2 * bound + 2.0 ** -20 + 8 * 2 ** -24 * lse.abs())[..., None]
    assert ((dv - d_out).abs() <= rel * d_out.abs() + 1e-37).all()
    assert (dq.abs() <= 2 * (D + 4) * 2 ** -23 * mag * k.abs() * D ** -0.5 * 1.01 + 1e-37).all()


@pytest.mark.parametrize("starts", [[5, 3, 90, 20, 400], [-7, 40, 10 ** 9], [2 ** 31 - 1, -2 ** 31, 60], [50], [90, 90]])
@pytest.mark.parametrize("many", [False, True])
def test_starts_out_of_range_or_order(starts, many):
    """Unspecified results, but nothing outside the T rows is written."""
    T, D = 130, 64
    m = _many(T, 1) if many else 1
    g = _gen(2)
    big = [torch.full((T + 80, m, D), 3.0, device=DEV) for _ in range(4)]
    q, k, v, d = (torch.randn((T, m, D), generator=g, device=DEV) for _ in range(4))
    outs = [t[40:40 + T] for t in big]
    lse = torch.zeros((T + 80, m), device=DEV)
    st = torch.tensor(starts, dtype=torch.int64).to(torch.int32).to(DEV)
    B.moe_causal_attention(q, k, v, st, outs[0], lse=lse[40:40 + T])
    B.moe_causal_attention_backward(d, q, k, v, outs[0], lse[40:40 + T], st, *outs[1:])
    torch.cuda.synchronize()
    for t in big:
        assert (t[:40] == 3.0).all() and (t[40 + T:] == 3.0).all()
    assert (lse[:40] == 0).all() and (lse[40 + T:] == 0).all()
    if len(starts) == 1 or starts[0] == starts[-1]:
        assert all((t == 3.0).all() for t in big)


def test_nothing_to_do():
    z = torch.zeros((0, 2, 64), device=DEV)
    B.moe_causal_attention(z, z, z, _starts([]), z)
    B.moe_causal_attention_backward(z, z, z, z, z, torch.zeros((0, 2), device=DEV), _starts([0, 0]), z.clone(), z.clone(), z.clone())


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_offsets_past_32_bits(act):
    """Rows 2^31 elements and more into a buffer, and rows too far apart for the direct loads, give the bits of dense ones."""
    g, dt = _gen(4), DT[act]
    for T, stride, lens in ((70000, 33024 if act == "bf16" else 31232, [64] * 1093 + [48]), (40, 1 << 24, [40])):
        D = 64
        buf = torch.empty(T * stride, dtype=dt, device=DEV).view(T, stride)
        x = torch.randn((T, 3, D), generator=g, device=DEV).to(dt)
        at = [buf[:, i * D:(i + 1) * D].unflatten(1, (1, D)) for i in range(8)]
        for i in range(3):
            at[i].copy_(x[:, i:i + 1])
        starts, d_out = _starts(lens), torch.randn((T, 1, D), generator=g, device=DEV).to(dt)
        at[7].copy_(d_out)
        dense = [x[:, i:i + 1].contiguous() for i in range(3)]
        lse, want, want_lse = torch.empty((T, 1), device=DEV), torch.empty((T, 1, D), dtype=dt, device=DEV), torch.empty((T, 1), device=DEV)
        B.moe_causal_attention(*at[:3], starts, at[3], lse=lse)
        B.moe_causal_attention(*dense, starts, want, lse=want_lse)
        assert torch.equal(at[3], want) and torch.equal(lse, want_lse)
        grads = [torch.empty_like(want) for _ in range(3)]
        B.moe_causal_attention_backward(at[7], *at[:3], at[3], lse, starts, *at[4:7])
        B.moe_causal_attention_backward(d_out, *dense, want, want_lse, starts, *grads)
        for a, b in zip(at[4:7], grads):
            assert torch.equal(a, b)
        del buf, at


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,T", [(4, 2, 300), (128, 8, 1100), (6, 1, 1030)])
def test_equal_calls_graphs_and_streams(act, hq, hk, T):
    """Equal calls give equal bits: again, on a stream of their own, and replayed from a graph between eager work."""
    D, dt, g = 96, DT[act], _gen(T)
    q, k, v, d_out = (torch.randn((T, h, D), generator=g, device=DEV).to(dt) for h in (hq, hk, hk, hq))
    starts = _starts([T // 3, T - T // 3])
    new = lambda: (torch.empty_like(q), torch.empty((T, hq), device=DEV), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))  # noqa: E731

    def both(o, **kw):
        B.moe_causal_attention(q, k, v, starts, o[0], lse=o[1], **kw)
        B.moe_causal_attention_backward(d_out, q, k, v, o[0], o[1], starts, *o[2:], **kw)
        return o
    want = both(new())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = both(new(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, there))
    rec = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(rec)
    for step in range(3):
        for t in rec:
            t.fill_(float("nan"))
        q.mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        want = both(new())
        assert all(torch.equal(a, b) for a, b in zip(want, rec)), step


@pytest.mark.parametrize("many", [False, True])
def test_gradient_against_differences(many):
    """Along random directions e of q, k and v: (f(x + h e) - f(x - h e)) / 2h = grad . e, f = sum(d_out out). fp32, h = 2^-6: the
    third-order rest is h^2 / 6 f''', the rounding of f some 2^-20 of its terms' size over h; both far below 2% of |grad||e|."""
    T, D = 90, 64
    m = _many(T, 2) if many else 1
    g = _gen(11)
    x = [torch.randn((T, h * m, D), generator=g, device=DEV) for h in (2, 1, 1)]
    d_out = torch.randn((T, 2 * m, D), generator=g, device=DEV)
    starts = _starts([50, 40])

    def f(*t):
        out = torch.empty_like(t[0])
        lse = torch.empty(out.shape[:2], device=DEV)
        B.moe_causal_attention(*t, starts, out, lse=lse)
        return out, lse
    out, lse = f(*x)
    grads = [torch.empty_like(t) for t in x]
    B.moe_causal_attention_backward(d_out, *x, out, lse, starts, *grads)
    h = 2.0 ** -6
    for i in range(3):
        e = torch.randn(x[i].shape, generator=g, device=DEV)
        moved = [[t + s * h * e if j == i else t for j, t in enumerate(x)] for s in (1, -1)]
        diff = ((f(*moved[0])[0].double() - f(*moved[1])[0].double()) * d_out.double()).sum() / (2 * h)
        along = (grads[i].double() * e.double()).sum()
        assert abs(diff - along) <= 0.02 * grads[i].double().norm(), (i, diff, along)


def test_refused_by_the_binding():
    x = torch.zeros((4, 2, 64), device=DEV)
    st = _starts([4])
    with pytest.raises(ValueError, match="kv_heads"):
        B.moe_causal_attention(x, x[:3], x[:3], st, x.clone())
    with pytest.raises(TypeError, match="bfloat16"):
        B.moe_causal_attention(x, x, x.bfloat16(), st, x.clone())
    with pytest.raises(TypeError, match="int32"):
        B.moe_causal_attention(x, x, x, st.long(), x.clone())
    with pytest.raises(ValueError, match="current GPU|tensors on"):
        B.moe_causal_attention(x, x, x, st.cpu(), x.clone())
    with pytest.raises(ValueError, match="shape of q"):
        B.moe_causal_attention(x, x, x, st, x[:, :1].clone())
    with pytest.raises(TypeError, match="lse must be fp32"):
        B.moe_causal_attention(x, x, x, st, x.clone(), lse=torch.zeros((4, 2), dtype=torch.float64, device=DEV))
    with pytest.raises(B.MoEError, match="workspace"):
        B.moe_causal_attention_backward(x, x, x, x, x, x[..., 0].contiguous(), st, x.clone(), x.clone(), x.clone(),
                                        workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(B.MoEError, match="takes the place"):
        B.moe_causal_attention_backward(x, x, x, x, x, x[..., 0].contiguous(), st, x, x.clone(), x.clone())
