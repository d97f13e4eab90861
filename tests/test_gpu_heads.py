"""Rotary positions, the paged cache append and shared-prefix attention against the fp64 oracle.

Tolerances, from the arithmetic:
* u = 2^-24 is the fp32 and 2^-8 the bf16 half unit (relative; 23 and 7 stored bits).
* A rotated channel is two products and a sum in fp32: 3 u of the added magnitudes, then the output rounding.
* A score of D products summed in any order in fp32 is off by at most delta = (D + 4) 2u scale sum|q||k| (2u: a
  matrix unit may truncate), which moves every weight by a factor within e^(2 delta); exp itself by 2^-21 (argument
  and result rounding at |argument| <= 30; smaller weights do not matter more). n weights are summed in fp32: n 2u.
  bf16 rounds each weight (2^-8) for the product with v, and may use the rounded ones in the sum (2^-8 more).
  All of it multiplies sum_j p_j |v_j|.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dt=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dt)


def _laid_out(g, T, H, D, dt, how):
    """Random [T, H, D] rows in one of the layouts a caller has them in."""
    if how == "dense":
        return _randn(g, T, H, D, dt=dt)
    if how == "fused":                      # a slice of a wider projection
        return _randn(g, T, H + 3, D, dt=dt)[:, 2:2 + H]
    if how == "heads_first":                # [H, T, D]
        return _randn(g, H, T, D, dt=dt).transpose(0, 1)
    if how == "odd":                        # neither strides nor start fit a wide load
        return _randn(g, T * H * (D + 1) + 1, dt=dt)[1:].view(T, H, D + 1)[:, :, :D]
    if how == "one_head":                   # one row read for every head
        return _randn(g, T, 1, D, dt=dt).expand(T, H, D)
    raise ValueError(how)


def _table(R, n=512, seed=0):
    return torch.as_tensor(oracle.rope_table(R, n), dtype=torch.float32, device=DEV).contiguous()


def _close(got, ref, tol, what=""):
    got, ref = _np(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / (tol + 1e-300)):.2f} tol"


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("parts", dict(factor=32.0, orig_len=4096.0, slow=1.0, fast=32.0)),
])
def test_rope_table(scaling, kw):
    """fp64 angles p theta (p up to 2^17: off by 2^-33 at most), one rounding."""
    n, R = 131072, 96
    code = dict(plain=B.MOE_ROPE_PLAIN, linear=B.MOE_ROPE_LINEAR, base=B.MOE_ROPE_BASE, parts=B.MOE_ROPE_PARTS)
    got = B.moe_rope_table(R, n, base=50000.0, scaling=code[scaling], amplitude=1.25, **kw)
    ref = oracle.rope_table(R, n, amplitude=1.25, base=50000.0, scaling=scaling, **kw)
    _close(got, ref, np.abs(ref) * U32 + 1.25 * 2.0 ** -32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,hq,hk,D,R,inter,how", [
    (1, 1, 1, 2, 2, False, "dense"),
    (3, 4, 2, 64, 64, False, "dense"),
    (300, 7, 3, 128, 128, False, "fused"),
    (129, 5, 1, 128, 64, True, "fused"),
    (65, 4, 4, 80, 40, False, "dense"),
    (65, 4, 4, 80, 20, True, "heads_first"),
    (33, 3, 2, 66, 34, False, "odd"),
    (33, 3, 2, 67, 34, True, "odd"),
    (1000, 16, 4, 256, 256, True, "heads_first"),
    (17, 6, 2, 192, 96, False, "one_head"),
    (5, 2, 2, 1024, 1000, False, "dense"),
])
@pytest.mark.parametrize("back", [False, True])
def test_rotary(dt, T, hq, hk, D, R, inter, how, back):
    g = _gen(T * 1000 + D)
    q, k = _laid_out(g, T, hq, D, DT[dt], how), _laid_out(g, T, hk, D, DT[dt], how)
    pos = torch.randint(0, 512, (T,), generator=g, device=DEV, dtype=torch.int32)
    table = _table(R)
    qo = torch.full((T, hq, D), float("nan"), dtype=DT[dt], device=DEV)
    ko = torch.full((hk, T, D), float("nan"), dtype=DT[dt], device=DEV).transpose(0, 1)
    call = B.moe_rotary_backward if back else B.moe_rotary
    call(q, k, pos, table, qo, ko, layout=B.MOE_ROPE_INTERLEAVED if inter else B.MOE_ROPE_HALF)
    for x, y in ((q, qo), (k, ko)):
        ref, mag = oracle.rotate(_np(x), _np(table)[pos.cpu().numpy()], inter, back)
        _close(y, ref, 3 * U32 * mag + (U16 * np.abs(ref) if dt == "bf16" else 0) + 1e-37)
        assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rotary_in_place_and_q_alone(dt):
    g = _gen(5)
    x = _randn(g, 50, 9, 96, dt=DT[dt])
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    table = _table(64)
    for layout in (B.MOE_ROPE_HALF, B.MOE_ROPE_INTERLEAVED):
        want = torch.empty_like(x)
        B.moe_rotary(x, None, pos, table, want, layout=layout)
        both = x.clone()
        B.moe_rotary(both[:, :5], both[:, 5:], pos, table, both[:, :5], both[:, 5:], layout=layout)
        assert torch.equal(both, want)


def test_rotary_skips_positions_outside_the_table():
    g = _gen(6)
    q = _randn(g, 6, 2, 64)
    pos = torch.tensor([0, -1, 511, 512, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    B.moe_rotary(q, None, pos, _table(64), out)
    assert (out[[1, 3, 4, 5]] == 7.0).all() and not (out[[0, 2]] == 7.0).any()


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient_against_differences(inter):
    """The rotation is linear in x, so a difference quotient is exact up to rounding for any step: along random
    directions, (f(x + h e) - f(x)) . dy / h = backward(dy) . e. fp32, 64 x 3 x 80 terms."""
    g = _gen(7)
    layout = B.MOE_ROPE_INTERLEAVED if inter else B.MOE_ROPE_HALF
    x, e, dy = (_randn(g, 64, 3, 80) for _ in range(3))
    pos = torch.randint(0, 512, (64,), generator=g, device=DEV, dtype=torch.int32)
    f = lambda z: (lambda o: (B.moe_rotary(z, None, pos, _table(40), o, layout=layout), o)[1])(torch.empty_like(z))
    dx = torch.empty_like(dy)
    B.moe_rotary_backward(dy, None, pos, _table(40), dx, layout=layout)
    num = ((f(x + 2 * e).double() - f(x).double()) * dy.double()).sum() / 2
    ana = (dx.double() * e.double()).sum()
    scale = (f(x).double().abs() * dy.double().abs()).sum() + (f(e).double().abs() * dy.double().abs()).sum()
    assert abs(float(num - ana)) <= 8 * U32 * float(scale) * 2


def test_rotary_keeps_nan_and_infinities_in_their_pair():
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 3], x[0, 0, 5] = float("nan"), float("inf")
    out = torch.empty_like(x)
    B.moe_rotary(x, None, torch.tensor([3], dtype=torch.int32, device=DEV), _table(64), out)
    bad = ~torch.isfinite(out[0, 0])
    assert bad.nonzero().flatten().tolist() == [3, 5, 35, 37]
    assert torch.isnan(out[0, 0, [3, 35]]).all()


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("act,cache", [("f32", "f32"), ("bf16", "bf16"), ("f32", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("T,hk,hq,D,R,inter,page,how", [
    (1, 1, 0, 2, 2, False, 1, "dense"),
    (1, 8, 56, 128, 128, False, 64, "dense"),
    (37, 2, 6, 64, 64, True, 16, "fused"),
    (100, 3, 0, 128, 64, False, 32, "fused"),
    (70, 4, 4, 80, 40, True, 128, "heads_first"),
    (70, 4, 0, 67, 34, False, 16, "odd"),
    (300, 2, 5, 256, 256, False, 1, "dense"),
    (33, 2, 0, 320, 0, False, 16, "dense"),        # no rotation
    (9, 4, 0, 48, 24, False, 8, "one_head"),
])
def test_append(act, cache, T, hk, hq, D, R, inter, page, how):
    g = _gen(T * 100 + D)
    dt = DT[act]
    k, v = _laid_out(g, T, hk, D, dt, how), _laid_out(g, T, hk, D, dt, how)
    if how == "dense":
        v = v.clone()
        v[0, 0] = 0
    q = _laid_out(g, T, hq, D, dt, how) if hq else None
    n_pages = -(-2 * T // page) + 1
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].to(torch.int32)
    pos = torch.randint(0, 512, (T,), generator=g, device=DEV, dtype=torch.int32)
    if T > 30:                                   # not cached, past the cache, past the table
        slots[5], slots[11], slots[13], slots[20] = -1, n_pages * page, 2 ** 31 - 1, -2 ** 31
        if R:
            pos[17] = 512
    table = _table(R) if R else None
    cdt = torch.uint8 if cache == "e4m3" else dt
    kc, vc = (torch.full((n_pages, hk, page, D), 3, dtype=cdt, device=DEV) for _ in range(2))
    ks, vs = (torch.full((n_pages, hk, page), 5.0, device=DEV) for _ in range(2)) if cache == "e4m3" else (None, None)
    qo = torch.full((T, hq, D), 9.0, dtype=dt, device=DEV) if hq else None
    B.moe_kv_append(k, v, slots, kc, vc, ks, vs, pos if R else None, table,
                    B.MOE_ROPE_INTERLEAVED if inter else B.MOE_ROPE_HALF, q, qo)
    sl, ps = slots.cpu().numpy().astype(np.int64), pos.cpu().numpy()
    in_table = (ps < 512) if R else np.ones(T, bool)
    ok = (sl >= 0) & (sl < n_pages * page) & in_table
    cs = _np(table)[np.minimum(ps, 511)] if R else np.zeros((T, 0, 2))
    written = np.zeros((n_pages, page), bool)
    written[sl[ok] // page, sl[ok] % page] = True
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        ref, mag = oracle.rotate(_np(x), cs if x is k else np.zeros((T, 0, 2)), inter)
        got = c.cpu()[sl[ok] // page, :, sl[ok] % page]
        if cache != "e4m3":
            _close(got.double().numpy(), ref[ok], (3 * U32 * mag + (U16 * np.abs(ref) if act == "bf16" else 0))[ok] + 1e-37)
        else:
            sc = s.cpu().numpy()[sl[ok] // page, :, sl[ok] % page].astype(np.float64)
            _, want = oracle.quantize_rows(ref[ok])
            _close(sc, want, 8 * U32 * want)
            # value of a code: within half a step of x / scale (2^-4 relative, 2^-10 below the normal range)
            val = oracle.e4m3_decode(got.numpy())
            y = ref[ok] / want[..., None]
            _close(val, y, np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10) + 448 * 8 * U32)
            codes, _ = oracle.quantize_rows(ref[ok])
            assert np.mean(codes != got.numpy()) <= 0.01
        untouched = c.cpu().transpose(1, 2).numpy() if cache == "e4m3" else c.cpu().float().transpose(1, 2).numpy()
        assert (untouched[~written] == 3).all()
        if s is not None:
            assert (s.cpu().transpose(1, 2).numpy()[~written] == 5.0).all()
    if hq:
        ref, mag = oracle.rotate(_np(q), cs, inter)
        _close(_np(qo)[in_table], ref[in_table],
               (3 * U32 * mag + (U16 * np.abs(ref) if act == "bf16" else 0))[in_table] + 1e-37)
        assert (_np(qo)[~in_table] == 9.0).all()


def test_append_past_32_bit_offsets():
    """Slots whose bytes lie past 4 GiB of the cache."""
    hk, page, D = 8, 64, 128
    n_pages = (1 << 32) // (hk * page * D * 2) + 3
    kc = torch.empty((n_pages, hk, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    g = _gen(11)
    k, v = _randn(g, 3, hk, D, dt=torch.bfloat16), _randn(g, 3, hk, D, dt=torch.bfloat16)
    slots = torch.tensor([0, (n_pages - 2) * page + 5, n_pages * page - 1], dtype=torch.int32, device=DEV)
    B.moe_kv_append(k, v, slots, kc, vc)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], k[t]) and torch.equal(vc[s // page, :, s % page], v[t])


# ---------------------------------------------------------------- attention

def _attention_case(seed, act, cache, Bn, S, hkv, G, D, page, prefix, own_max, lens=None, scale=None, lse=True,
                    gain=1.0, poison=True, how="dense"):
    """Inputs with every slot that no row may use filled with NaN (codes 0x7F, NaN scales for E4M3)."""
    g = _gen(seed)
    dt = DT[act]
    n_pre, cols = -(-prefix // page), -(-own_max // page)
    n_pages = n_pre + Bn * cols + 2
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    pre, table = order[:n_pre].contiguous(), order[n_pre:n_pre + Bn * cols].view(Bn, cols).contiguous()
    if lens is None:
        lens = torch.randint(0, own_max + 1, (Bn,), generator=g, device=DEV)
    lens = torch.as_tensor(lens, dtype=torch.int32, device=DEV)
    kv = []
    used = torch.zeros((n_pages, page), dtype=torch.bool, device=DEV)
    if prefix:
        j = torch.arange(prefix, device=DEV)
        used[pre.long()[j // page], j % page] = True
    for b in range(Bn):
        j = torch.arange(int(lens[b].clamp(0, cols * page)), device=DEV)
        if len(j):
            used[table[b].long()[j // page], j % page] = True
    mask = ~used[:, None, :].expand(n_pages, hkv, page)
    for z in range(2):
        x = _randn(g, n_pages, hkv, page, D) * gain + 0.2
        if cache == "e4m3":
            s = x.abs().amax(-1) / 448.0
            c = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            val = c.view(torch.float8_e4m3fn).double() * s.double()[..., None]
            if poison:
                c[mask], s[mask] = 0x7F, float("nan")
            kv.append((c, s, val))
        else:
            c = x.to(dt)
            if poison:
                c[mask] = float("nan")
            kv.append((c, None, c.double()))
    q = _laid_out(g, Bn * S, hkv * G, D, dt, how)
    return dict(q=q, k=kv[0], v=kv[1], pre=pre, prefix=prefix, table=table if cols else None,
                lens=lens if cols else None, S=S, page=page, scale=D ** -0.5 if scale is None else scale, act=act,
                cache=cache)


def _run_attention(c, out=None, lse=None, **kw):
    q = c["q"]
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=DEV) if out is None else out
    B.moe_prefix_attention(q, c["k"][0], c["v"][0], c["pre"] if c["prefix"] else None, c["prefix"], c["table"], c["lens"],
                           out, q_len=c["S"], scale=c["scale"], k_scale=c["k"][1], v_scale=c["v"][1], lse=lse, **kw)
    return out


def _check_attention(c, out, lse=None, rows=None):
    """Against the oracle, every (row, head) or a sample of them."""
    q, S, page = _np(c["q"]), c["S"], c["page"]
    n, H, D = q.shape
    kv = [x[2] for x in (c["k"], c["v"])]
    hkv = kv[0].shape[1]
    got, glse = _np(out), None if lse is None else _np(lse).reshape(n, H)
    per_seq, pre = {}, {}
    every = [(t, h) for t in range(n) for h in range(H)]
    for t, h in every if rows is None else rows:
        b, i, hk = t // S, t % S, h // (H // hkv)
        if hk not in pre:
            pre[hk] = [_np(x[c["pre"].long(), hk].reshape(-1, D)[:c["prefix"]]) for x in kv]
        if (b, hk) not in per_seq:
            m = 0 if c["table"] is None else int(np.clip(int(c["lens"][b]), 0, c["table"].shape[1] * page))
            per_seq[b, hk] = [np.zeros((0, D))] * 2 if m == 0 else \
                [_np(x[c["table"][b].long(), hk].reshape(-1, D)[:m]) for x in kv]
        own = per_seq[b, hk]
        see = max(0, len(own[0]) - S + 1 + i)
        k, v = (np.concatenate([p, o[:see]]) for p, o in zip(pre[hk], own))
        ref, rlse, mag = oracle.attend(q[t, h], k, v, c["scale"])
        delta = (D + 4) * 2 * U32 * abs(c["scale"]) * (np.abs(k) @ np.abs(q[t, h])).max() if len(k) else 0.0
        rel = 2 * delta + 2.0 ** -20 + 2 * U32 * len(k) + (2 * U16 if c["act"] == "bf16" else 0)
        tol = rel * mag + (U16 if c["act"] == "bf16" else U32) * np.abs(ref)
        _close(got[t, h], ref, tol, f"row {t} head {h}")
        if glse is not None:
            if np.isinf(rlse):
                assert glse[t, h] == rlse
            else:
                _close(glse[t, h], rlse, delta + rel + 4 * U32 * abs(rlse), f"lse of row {t} head {h}")


KINDS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3")]


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("Bn,S,hkv,G,D,page,prefix,own_max", [
    (1, 1, 1, 1, 64, 16, 0, 1),
    (1, 1, 1, 1, 8, 1, 1, 0),           # nothing but one prefix token
    (2, 1, 4, 4, 128, 16, 100, 40),
    (3, 1, 2, 7, 128, 64, 65, 200),
    (5, 2, 1, 3, 80, 32, 33, 70),
    (2, 5, 2, 2, 64, 16, 17, 9),        # some queries have no own token
    (1, 70, 1, 2, 128, 16, 31, 130),    # a chunk of a prompt after the prefix
    (4, 1, 2, 1, 256, 128, 129, 300),
    (3, 3, 1, 16, 96, 1, 7, 50),
    (33, 1, 2, 4, 64, 16, 513, 64),
    (2, 1, 1, 5, 192, 64, 1000, 700),
    (2, 4, 2, 9, 24, 8, 0, 33),         # no prefix
    (7, 1, 1, 8, 128, 32, 2000, 0),     # no own tokens at all
    (1, 1, 3, 40, 136, 256, 255, 257),
])
def test_attention(act, cache, Bn, S, hkv, G, D, page, prefix, own_max):
    c = _attention_case(Bn * 7 + D, act, cache, Bn, S, hkv, G, D, page, prefix, own_max)
    lse = torch.full((Bn * S, hkv * G), 55.0, device=DEV)
    out = _run_attention(c, lse=lse)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("act,cache", KINDS)
def test_attention_lengths_around_tiles_and_splits(act, cache):
    """Own lengths 0, 1 and one around each power of two; the prefix ends inside a page."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1025, 2047]
    c = _attention_case(21, act, cache, len(lens), 1, 1, 2, 64, 16, 37, 2048, lens=lens)
    lse = torch.empty((len(lens), 2), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse)
    c["prefix"] = 0                          # the first row now sees nothing
    out = _run_attention(c, lse=lse)
    assert not out[0].any() and torch.isinf(lse[0]).all()
    _check_attention(c, out, lse)


@pytest.mark.parametrize("act,cache", KINDS)
def test_attention_long_prefix_and_long_own(act, cache):
    c = _attention_case(22, act, cache, 3, 2, 2, 4, 128, 64, 20011, 9000, lens=[9000, 1, 4097])
    rows = [(t, h) for t in range(6) for h in (0, 3, 7)]
    lse = torch.empty((6, 8), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse, rows)


@pytest.mark.parametrize("act,cache", KINDS)
def test_attention_of_a_large_batch(act, cache):
    """Enough rows on one prefix for many row tiles; a sample of them is checked."""
    c = _attention_case(23, act, cache, 200, 1, 2, 7, 128, 32, 3001, 96)
    rng = np.random.default_rng(0)
    rows = [(int(t), int(h)) for t, h in zip(rng.integers(0, 200, 150), rng.integers(0, 14, 150))]
    _check_attention(c, _run_attention(c), rows=rows)


@pytest.mark.parametrize("act,cache", KINDS)
def test_attention_large_scores(act, cache):
    """Scores up to several hundred: the running maximum moves far and most weights vanish."""
    c = _attention_case(24, act, cache, 3, 1, 1, 4, 64, 16, 700, 300, scale=2.0, gain=3.0)
    lse = torch.empty((3, 4), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse)


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("how", ["fused", "heads_first", "odd", "one_head"])
def test_attention_query_and_output_strides(act, cache, how):
    c = _attention_case(25, act, cache, 4, 3, 2, 3, 64, 16, 50, 60, how=how)
    out = torch.zeros((6, 12, 65), dtype=DT[act], device=DEV).transpose(0, 1)[:, :, 1:]
    _check_attention(c, _run_attention(c, out=out))


def test_attention_out_may_be_q():
    c = _attention_case(26, "bf16", "bf16", 5, 2, 2, 4, 128, 16, 300, 200)
    want = _run_attention(c)
    c["q"] = c["q"].clone()
    _run_attention(c, out=c["q"])
    assert torch.equal(c["q"], want)


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_rows_do_not_see_later_tokens_values(act, cache, bad):
    """A non-finite key or value reaches the queries that see it and no other."""
    S, own = 4, 40
    c = _attention_case(27, act, cache, 2, S, 1, 2, 64, 16, 20, own, lens=[own, own])
    clean = _run_attention(c)
    page, row = int(c["table"][0, (own - 2) // 16]), (own - 2) % 16
    for side in ("k", "v"):
        x, s, _ = c[side]
        t = s if cache == "e4m3" else x
        at = (page, 0, row) if cache == "e4m3" else (page, 0, row, 5)
        keep = t[at].clone()
        t[at] = bad
        out = _run_attention(c)
        t[at] = keep
        assert torch.equal(out[:2], clean[:2]) and torch.equal(out[4:], clean[4:])
        seen = out[2:4]
        assert not torch.isfinite(seen).all()


def test_attention_leaves_out_pages_outside_the_cache():
    c = _attention_case(28, "bf16", "bf16", 2, 1, 2, 2, 64, 16, 48, 64, lens=[64, 64])
    pre, table = c["pre"].clone(), c["table"].clone()
    c["pre"][1] = -1
    c["table"][0, 2], c["table"][1, 0] = 10 ** 9, c["k"][0].shape[0]
    out = _run_attention(c)
    for b in range(2):
        pages = [int(p) for p in pre[[0, 2]]] + [int(table[b, j]) for j in range(4) if j != (2 if b == 0 else 0)]
        for h in range(4):
            k, v = (_np(x[2][pages, h // 2].reshape(-1, 64)) for x in (c["k"], c["v"]))
            ref, _, mag = oracle.attend(_np(c["q"])[b, h], k, v, c["scale"])
            _close(_np(out)[b, h], ref, 3 * U16 * mag + U16 * np.abs(ref))


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("G,D,page,prefix,own_max,scale", [
    (20, 64, 1, 1500, 3, None),         # more page table entries than a wave holds at once
    (20, 128, 2, 1111, 3, None),
    (33, 128, 4, 2085, 0, None),
    (17, 80, 8, 1999, 40, None),        # head_dim inside the padded one
    (17, 72, 16, 1300, 40, None),       # no multiple of 16
    (40, 96, 32, 3333, 10, None),
    (19, 136, 16, 900, 5, None),
    (25, 192, 64, 1025, 5, None),
    (25, 256, 64, 2047, 5, None),
    (40, 128, 4096, 5000, 9, -0.09),    # pages longer than the prefix's parts; a negative scale
    (40, 128, 64, 1024, 9, 0.0),        # every token counts the same
])
def test_attention_many_rows_on_a_prefix(act, cache, G, D, page, prefix, own_max, scale):
    """Rows enough that the waves of a block share the prefix's tiles."""
    c = _attention_case(G + D + page, act, cache, 5, 1, 2, G, D, page, prefix, own_max, scale=scale)
    rng = np.random.default_rng(1)
    rows = [(int(t), int(h)) for t, h in zip(rng.integers(0, 5, 40), rng.integers(0, 2 * G, 40))]
    lse = torch.empty((5, 2 * G), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse, rows)


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [3, 40])
def test_attention_scores_that_grow_along_the_prefix(act, cache, D, G):
    """Scores up to several hundred more at the end than at the start, past every reference taken before."""
    prefix, page = 1400, 16
    c = _attention_case(31, act, cache, 2, 1, 1, G, D, page, prefix, 20, poison=False)
    j = torch.arange(prefix, device=DEV)
    at = (c["pre"].long()[j // page], 0, j % page)
    x, s, val = c["k"]
    grow = 2.0 ** torch.floor(8.0 * j / prefix)      # powers of two: the stored numbers stay exact
    if cache == "e4m3":
        s[at] *= grow
    else:
        x[at] *= grow[:, None].to(x.dtype)
    val[at] *= grow[:, None].double()
    lse = torch.empty((2, G), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse)


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("D,page", [(64, 2), (64, 8), (128, 4), (128, 8), (128, 16), (128, 64), (256, 2), (256, 32)])
@pytest.mark.parametrize("G", [24, 40])
@pytest.mark.parametrize("missing", ["first", "odd", "middle", "last"])
def test_attention_leaves_out_pages_of_a_shared_prefix(act, cache, D, page, missing, G):
    """Page numbers outside the cache on a prefix that many rows read; page 0 holds keys that would win every row."""
    prefix, own = 640, 5
    c = _attention_case(32, act, cache, 2, 1, 1, G, D, page, prefix, own, lens=[own, own], poison=False)
    pre, n = c["pre"], -(-prefix // page)
    first = int(pre[0])                                  # page 0 changes places with the prefix's first page
    for side in ("k", "v"):
        for x in c[side]:
            if x is not None:
                x[[0, first]] = x[[first, 0]]
    where = {0: first, first: 0}
    for t in (pre, c["table"]):
        t.copy_(torch.tensor([where.get(int(p), int(p)) for p in t.flatten()], device=DEV).view(t.shape))
    if cache == "e4m3":
        c["k"][1][0] *= 64.0
    else:
        c["k"][0][0] *= 64.0
    c["k"][2][0] *= 64.0
    gone = {"first": [0], "odd": [i for i in range(n) if i % 5 == 1 or i == 0], "middle": [0, n // 2], "last": [0, n - 1]}[missing]
    kept = [int(p) for i, p in enumerate(pre) if i not in gone]
    pre[gone] = torch.tensor([-1 if i % 2 else c["k"][0].shape[0] + i for i in gone], dtype=torch.int32, device=DEV)
    out = _run_attention(c)
    for b, h in ((0, 0), (0, G - 1), (1, 7)):
        k, v = (np.concatenate([_np(x[2][kept, 0].reshape(-1, D)), _np(x[2][c["table"][b].long(), 0].reshape(-1, D)[:own])])
                for x in (c["k"], c["v"]))
        ref, _, mag = oracle.attend(_np(c["q"])[b, h], k, v, c["scale"])
        u = U16 if act == "bf16" else U32
        delta = (D + 4) * 2 * U32 * c["scale"] * (np.abs(k) @ np.abs(_np(c["q"])[b, h])).max()
        rel = 2 * delta + 2.0 ** -20 + 2 * U32 * len(k) + (2 * U16 if act == "bf16" else 0)
        _close(_np(out)[b, h], ref, rel * mag + u * np.abs(ref), f"row {b} head {h}")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("G", [2, 40])
def test_attention_leading_scores_of_minus_infinity(act, G):
    """Tokens whose scores are -infinity weigh nothing, however low the scores after them are."""
    prefix, page, D = 400, 16, 64
    c = _attention_case(33, act, act, 2, 1, 1, G, D, page, prefix, 0, poison=False)
    c["q"] = c["q"].abs() + 0.25
    x, val = c["k"][0], c["k"][2]
    x.copy_((x.float() / 16 - 40.0).to(x.dtype))
    val.copy_(x.double())
    x[c["pre"][:3].long()] = -float("inf")
    out = _run_attention(c)
    for b, h in ((0, 0), (1, G - 1)):
        k, v = (_np(z[2][c["pre"].long(), 0].reshape(-1, D)[48:prefix]) for z in (c["k"], c["v"]))
        ref, _, mag = oracle.attend(_np(c["q"])[b, h], k, v, c["scale"])
        delta = (D + 4) * 2 * U32 * c["scale"] * (np.abs(k) @ np.abs(_np(c["q"])[b, h])).max()
        rel = 2 * delta + 2.0 ** -20 + 2 * U32 * len(k) + (2 * U16 if act == "bf16" else 0)
        _close(_np(out)[b, h], ref, rel * mag + (U16 if act == "bf16" else U32) * np.abs(ref), f"row {b} head {h}")


def test_attention_lens_outside_the_table_are_clamped():
    c = _attention_case(29, "bf16", "bf16", 3, 1, 1, 2, 64, 16, 5, 32, lens=[32, 0, 32])
    want = _run_attention(c)
    c["lens"] = torch.tensor([10 ** 9, -7, 32], dtype=torch.int32, device=DEV)
    assert torch.equal(_run_attention(c), want)


def test_attention_past_32_bit_offsets():
    """Pages whose bytes lie past 4 GiB of the cache."""
    hkv, page, D = 8, 64, 128
    n_pages = (1 << 32) // (hkv * page * D * 2) + 8
    kc = torch.empty((n_pages, hkv, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    g = _gen(12)
    pages = list(range(n_pages - 6, n_pages))
    kc[pages], vc[pages] = _randn(g, 6, hkv, page, D, dt=torch.bfloat16), _randn(g, 6, hkv, page, D, dt=torch.bfloat16)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    q = _randn(g, 2, 16, D, dt=torch.bfloat16)
    out = torch.empty_like(q)
    B.moe_prefix_attention(q, kc, vc, t(pages[:2]), 100, t([pages[2:4], pages[4:]]), t([128, 70]), out)
    for b, n in ((0, 128), (1, 70)):
        for h in (0, 9, 15):
            cat = [_np(torch.cat([x[pages[:2], h // 2].reshape(-1, D)[:100],
                                  x[pages[2 + 2 * b:4 + 2 * b], h // 2].reshape(-1, D)[:n]])) for x in (kc, vc)]
            ref, _, mag = oracle.attend(_np(q)[b, h], *cat, D ** -0.5)
            _close(_np(out)[b, h], ref, 3 * U16 * mag + U16 * np.abs(ref))


@pytest.mark.parametrize("act,cache", KINDS)
def test_attention_is_reproducible_and_runs_on_its_stream(act, cache):
    c = _attention_case(30, act, cache, 20, 1, 2, 4, 128, 16, 1500, 400)
    want = _run_attention(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            assert torch.equal(_run_attention(c), want)
    side.synchronize()
    n = B.moe_prefix_attention_workspace_bytes(c["k"][0], 20, 1, 8, c["prefix"], c["table"].shape[1])
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)      # whatever the workspace held
    assert torch.equal(_run_attention(c, workspace=ws), want)


def test_attention_on_a_given_stream_keeps_its_workspace():
    """stream= without workspace=: what the current stream allocates next is not the scratch of the running call."""
    c = _attention_case(35, "bf16", "bf16", 40, 1, 2, 8, 128, 16, 30000, 200)
    want = _run_attention(c)
    n = B.moe_prefix_attention_workspace_bytes(c["k"][0], 40, 1, 16, c["prefix"], c["table"].shape[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    for out in outs:
        _run_attention(c, out=out, stream=side)
        torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_decode_calls_in_a_graph():
    """Append and attention recorded once; three replays with other inputs and eager work between them."""
    g = _gen(31)
    Bn, hkv, G, D, page, prefix = 6, 2, 4, 128, 16, 200
    c = _attention_case(32, "bf16", "bf16", Bn, 1, hkv, G, D, page, prefix, 64, lens=[3, 60, 17, 32, 16, 1], poison=False)
    table = _table(D, 1024)
    q, k, v = (_randn(g, Bn, h, D, dt=torch.bfloat16) for h in (hkv * G, hkv, hkv))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    slots, pos = torch.empty(Bn, dtype=torch.int32, device=DEV), torch.empty(Bn, dtype=torch.int32, device=DEV)

    def place():
        last = c["lens"].long() - 1
        slots.copy_(c["table"].gather(1, (last // page)[:, None])[:, 0] * page + last % page)
        pos.copy_(prefix + last)

    def step():
        B.moe_kv_append(k, v, slots, c["k"][0], c["v"][0], positions=pos, table=table, q=q, q_out=qr)
        B.moe_prefix_attention(qr, c["k"][0], c["v"][0], c["pre"], prefix, c["table"], c["lens"], out, workspace=ws)

    ws = torch.empty(max(256, B.moe_prefix_attention_workspace_bytes(c["k"][0], Bn, 1, hkv * G, prefix, 4)),
                     dtype=torch.uint8, device=DEV)
    place()
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for r in range(3):
        for x in (q, k, v):
            x.copy_(_randn(g, *x.shape))
        c["lens"].add_(1)
        place()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, qr, c["k"][0], c["v"][0])]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, qr, c["k"][0], c["v"][0])):
            assert torch.equal(a, b)
