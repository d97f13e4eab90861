"""Attention over the paged cache where its loops hand over to each other: page tables that leave the cache inside a
part, references that move. Tolerances as derived in test_gpu_heads.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from test_gpu_heads import KINDS, U16, U32, _attention_case, _check_attention, _close, _np, _run_attention

pytestmark = pytest.mark.gpu


def _check_rows(c, out, lse, kept, rows):
    """Rows (t, h) of a call whose prefix consists of the pages `kept` and that has no own tokens, one kv head."""
    k, v = (_np(x[2][kept, 0].reshape(-1, c["q"].shape[2])) for x in (c["k"], c["v"]))
    D, u = k.shape[1], U16 if c["act"] == "bf16" else U32
    for t, h in rows:
        q = _np(c["q"])[t, h]
        ref, rlse, mag = oracle.attend(q, k, v, c["scale"])
        delta = (D + 4) * 2 * U32 * abs(c["scale"]) * (np.abs(k) @ np.abs(q)).max()
        rel = 2 * delta + 2.0 ** -20 + 2 * U32 * len(k) + (2 * U16 if c["act"] == "bf16" else 0)
        _close(_np(lse)[t, h], rlse, delta + rel + 4 * U32 * abs(rlse), f"lse of row {t} head {h}")
        _close(_np(out)[t, h], ref, rel * mag + u * np.abs(ref), f"row {t} head {h}")


@pytest.mark.parametrize("act,cache,D,page", [
    ("f32", "f32", 64, 4), ("f32", "f32", 128, 2), ("f32", "f32", 256, 2), ("bf16", "bf16", 128, 4),
    ("bf16", "bf16", 256, 2), ("bf16", "e4m3", 64, 16), ("bf16", "e4m3", 128, 8), ("bf16", "e4m3", 256, 4),
])
@pytest.mark.parametrize("G", [3, 40])
def test_attention_pages_that_leave_the_cache_inside_a_part(act, cache, D, page, G):
    """Runs of 64 pages in the cache and 64 outside it, in turn. A wave looks 64 table entries ahead, and the prefix is
    long enough for parts of 128 pages or a multiple: each one's first tile outside starts a new look ahead, and
    its last tile inside lies behind it. A tile counted twice, or not at all, shows in the lse."""
    prefix = 256 * 128 * page if page <= 4 else 128 * 128 * page
    c = _attention_case(41, act, cache, 2, 1, 1, G, D, page, prefix, 0, poison=False)
    i = torch.arange(prefix // page, device=DEV)
    inside = i % 128 < 64
    kept = c["pre"][inside].long()
    c["pre"][~inside] = torch.where(i % 2 == 0, -1, c["k"][0].shape[0] + i)[~inside].to(torch.int32)
    lse = torch.empty((2, G), device=DEV)
    out = _run_attention(c, lse=lse)
    _check_rows(c, out, lse, kept, [(0, 0), (1, G - 1)])


def _growing(seed, cache, D, G, page, prefix):
    """Two sequences on a prefix whose scores grow along it, by powers of two of the keys."""
    c = _attention_case(seed, "bf16", cache, 2, 1, 1, G, D, page, prefix, 0, poison=False)
    j = torch.arange(prefix, device=DEV)
    at = (c["pre"].long()[j // page], 0, j % page)
    x, s, val = c["k"]
    grow = 2.0 ** torch.floor(6.0 * j / prefix)
    if cache == "e4m3":
        s[at] *= grow
    else:
        x[at] *= grow[:, None].to(x.dtype)
    val[at] *= grow[:, None].double()
    return c


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_rows_reference_is_moved_by_its_own_scores_alone(cache, D):
    """Rows of one wave: one row's scores pass every reference by far, or stay at zero. The others give the same bits."""
    c = _growing(42, cache, D, 48, 16, 100 * 16)
    c["q"] *= 0.25      # the others pass their first reference too, but by little
    outs = []
    for gain in (0.0, 40.0):
        q = c["q"].clone()
        q[0, 5] *= gain
        lse = torch.empty((2, 48), device=DEV)
        outs.append((_run_attention({**c, "q": q}, lse=lse), lse))
    others = torch.ones((2, 48), dtype=torch.bool, device=DEV)
    others[0, 5] = False
    for a, b in zip(*outs):
        assert torch.equal(a[others], b[others]) and not torch.equal(a[~others], b[~others])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [3, 48])
def test_large_values_behind_growing_scores(cache, D, G):
    """Values of 2^100 and scores that end about 2^35 past the first reference: the sums stay finite, as the result is."""
    c = _growing(43, cache, D, G, 16, 100 * 16)
    c["q"] *= 0.25
    x, s, val = c["v"]
    (s if cache == "e4m3" else x).mul_(2.0 ** 100)
    val *= 2.0 ** 100
    lse = torch.empty((2, G), device=DEV)
    out = _run_attention(c, lse=lse)
    assert torch.isfinite(out).all()
    _check_rows(c, out, lse, c["pre"].long(), [(t, h) for t in range(2) for h in range(0, G, 5)])


def _sample(c, n, seed=0):
    """n rows (t, h), the first and the last token of every sequence among them."""
    rng = np.random.default_rng(seed)
    T, H, S = c["q"].shape[0], c["q"].shape[1], c["S"]
    ends = [(t, int(rng.integers(H))) for b in range(T // S) for t in (b * S, b * S + S - 1)]
    return ends + [(int(rng.integers(T)), int(rng.integers(H))) for _ in range(n)]


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("Bn,S,hkv,G,D,page,prefix,lens", [
    (3, 9, 2, 12, 128, 64, 500, [3300, 2047, 9]),       # one row tile: several parts of many whole tiles
    (2, 33, 1, 8, 128, 16, 0, [4100, 1031]),            # row tiles with ends of their own, no prefix
    (2, 70, 1, 3, 64, 32, 77, [2900, 69]),              # a sequence shorter than its queries
    (2, 20, 1, 7, 256, 128, 300, [2500, 1999]),
    (1, 25, 2, 5, 80, 16, 64, [3000]),                  # head_dim inside the padded one
    (1, 300, 1, 4, 128, 4, 100, [1777]),                # pages smaller than a tile
])
def test_attention_of_long_own_streams_with_many_rows(act, cache, Bn, S, hkv, G, D, page, prefix, lens):
    """More than 64 rows a kv head on a sequence's own tokens: their tiles are shared by the waves of a block."""
    c = _attention_case(44, act, cache, Bn, S, hkv, G, D, page, prefix, max(lens), lens=lens)
    lse = torch.empty((Bn * S, hkv * G), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse, _sample(c, 40))


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("S,hkv,G,D,prefix", [(2051, 2, 7, 128, 0), (1500, 1, 4, 64, 1024), (700, 1, 2, 256, 4096)])
def test_attention_of_a_chunk_of_a_prompt(act, cache, S, hkv, G, D, prefix):
    """One sequence whose queries are all of its own tokens, after the chunks before it."""
    c = _attention_case(45, act, cache, 1, S, hkv, G, D, 64, prefix, S, lens=[S])
    lse = torch.empty((S, hkv * G), device=DEV)
    _check_attention(c, _run_attention(c, lse=lse), lse, _sample(c, 60))


@pytest.mark.parametrize("act,cache", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_on_shared_tiles_do_not_see_later_tokens(act, cache, D, bad):
    """A non-finite key or value among the last tokens of a long own stream reaches the queries that see it and no other."""
    S, own, tok = 40, 700, 688
    c = _attention_case(46, act, cache, 2, S, 1, 3, D, 16, 20, own, lens=[own, own])
    clean = _run_attention(c)
    first = tok - (own - S)      # the first query that sees the token
    for side in ("k", "v"):
        x, s, _ = c[side]
        t = s if cache == "e4m3" else x
        at = (int(c["table"][0, tok // 16]), 0, tok % 16) + (() if cache == "e4m3" else (5,))
        keep = t[at].clone()
        t[at] = bad
        out = _run_attention(c)
        t[at] = keep
        assert torch.equal(out[:first], clean[:first]) and torch.equal(out[S:], clean[S:])
        finite = torch.isfinite(out[first:S]).all(-1)
        if side == "k" and bad == float("inf"):      # a score of -infinity weighs nothing
            q = c["q"][first:S].double()
            up = (q @ c["k"][2][at[:3]] if cache == "e4m3" else q[..., 5]) > 0
            assert torch.equal(finite, ~up) and up.any() and not up.all()
        else:
            assert not finite.any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("G,S", [(2, 1), (40, 2)])
def test_rows_with_no_score_above_minus_infinity(act, G, S):
    """Every key a row sees gives -infinity: zeros and an lse of -infinity, beside rows that see the same keys otherwise."""
    c = _attention_case(47, act, act, 2, S, 1, G, 64, 16, 200, 40, lens=[40, 40], poison=False)
    c["k"][0][..., 7] = float("inf")
    c["q"] = c["q"].abs() + 0.25
    c["q"][:, 1::2, 7] *= -1.0
    lse = torch.empty((2 * S, G), device=DEV)
    out = _run_attention(c, lse=lse)
    assert (out[:, 1::2] == 0).all() and (lse[:, 1::2] == -float("inf")).all()
    assert torch.isnan(out[:, ::2]).all()
