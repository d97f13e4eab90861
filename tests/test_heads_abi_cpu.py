"""Refusals of the rotary, cache-append and attention calls, on the host before any launch (runs without a GPU)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_gate_amd import binding as B

P = 0x1000   # never dereferenced: validation fails first


def _rows(**kw):
    a = dict(in_=P, in_t=512, in_h=128, out=2 * P, out_t=512, out_h=128, heads=4)
    a.update(kw)
    return B.moe_heads(*[a[n] for n, _ in B.moe_heads._fields_])


def _rope(**kw):
    a = dict(rot_dim=64, layout=B.MOE_ROPE_HALF, n_positions=100, table=P)
    a.update(kw)
    return B.moe_rope(*[a[n] for n, _ in B.moe_rope._fields_])


def _cache(**kw):
    a = dict(n_pages=8, page_size=16, kv_heads=4, head_dim=128, dtype=B.MOE_BF16, k=P, v=P, k_scale=None, v_scale=None)
    a.update(kw)
    return B.moe_kv_cache(*[a[n] for n, _ in B.moe_kv_cache._fields_])


def _msg():
    return B.lib().moe_last_error().decode()


@pytest.mark.parametrize("call", ["moe_rotary", "moe_rotary_backward"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(rope=None), B.MOE_E_INVALID, "NULL"),
    (dict(q=None), B.MOE_E_INVALID, "NULL"),
    (dict(act=B.MOE_F8E4M3), B.MOE_E_INVALID, "act"),
    (dict(T=-1), B.MOE_E_INVALID, "negative"),
    (dict(rope=dict(rot_dim=63)), B.MOE_E_INVALID, "rot_dim"),
    (dict(rope=dict(rot_dim=0)), B.MOE_E_INVALID, "rot_dim"),
    (dict(rope=dict(rot_dim=130)), B.MOE_E_INVALID, "rot_dim"),
    (dict(rope=dict(layout=2)), B.MOE_E_INVALID, "layout"),
    (dict(rope=dict(n_positions=0)), B.MOE_E_INVALID, "n_positions"),
    (dict(rope=dict(table=None)), B.MOE_E_INVALID, "table"),
    (dict(rope=dict(table=P + 4)), B.MOE_E_INVALID, "aligned"),
    (dict(positions=None), B.MOE_E_INVALID, "positions"),
    (dict(q=dict(heads=0)), B.MOE_E_INVALID, "head"),
    (dict(q=dict(in_=None)), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(out=None)), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(in_=P + 1)), B.MOE_E_INVALID, "aligned"),
    (dict(q=dict(out_t=0)), B.MOE_E_INVALID, "overlap"),
    (dict(q=dict(out_t=511)), B.MOE_E_INVALID, "overlap"),
    (dict(q=dict(out_h=127)), B.MOE_E_INVALID, "overlap"),
    (dict(q=dict(out_t=128, out_h=128 * 6)), B.MOE_E_INVALID, "overlap"),   # [heads, T, D] needs T = 7 rows
    (dict(q=dict(out=P, out_t=640)), B.MOE_E_INVALID, "in place"),
    (dict(q=dict(in_t=1 << 60)), B.MOE_E_INVALID, "stride"),
    (dict(k=dict(heads=0)), B.MOE_E_INVALID, "head"),
])
def test_rotary_refusals(call, kw, status, needle):
    a = dict(rope={}, act=B.MOE_BF16, T=7, D=128, q={}, k=None, positions=P)
    a.update(kw)
    made = lambda f, v: None if v is None else f(**v)
    st = getattr(B.lib(), call)(made(_rope, a["rope"]), a["act"], a["T"], a["D"], made(_rows, a["q"]),
                                made(_rows, a["k"]), a["positions"], None)
    assert st == status and needle in _msg(), _msg()


def test_empty_calls_do_nothing():
    L = B.lib()
    assert L.moe_rotary(_rope(), B.MOE_F32, 0, 128, _rows(), None, None, None) == B.MOE_OK
    assert L.moe_kv_append(_cache(), None, B.MOE_BF16, 0, _rows(), _rows(), None, None, None, None) == B.MOE_OK
    for b, s in ((0, 1), (3, 0)):
        assert L.moe_prefix_attention(_cache(), B.MOE_BF16, b, s, _rows(), 0.1, None, 0, None, 0, None, None, None, 0,
                                      None) == B.MOE_OK


@pytest.mark.parametrize("kw,needle", [
    (dict(R=3), "even"), (dict(R=0), "even"), (dict(n=0), "n_positions"), (dict(base=1.0), "base"),
    (dict(scaling=4), "scaling"), (dict(scaling=B.MOE_ROPE_LINEAR, factor=0.5), "factor"),
    (dict(scaling=B.MOE_ROPE_BASE, factor=2.0, R=2), "rot_dim > 2"),
    (dict(scaling=B.MOE_ROPE_PARTS, factor=2.0), "orig_len"),
    (dict(scaling=B.MOE_ROPE_PARTS, factor=2.0, orig=100.0, slow=32.0), "slow < fast"),
    (dict(amp=float("nan")), "amplitude"), (dict(table=None), "table"), (dict(table=P + 4), "aligned"),
])
def test_rope_table_refusals(kw, needle):
    a = dict(R=64, n=16, base=1e4, scaling=0, factor=1.0, orig=0.0, slow=1.0, fast=32.0, amp=1.0, table=P)
    a.update(kw)
    st = B.lib().moe_rope_table(a["R"], a["n"], a["base"], a["scaling"], a["factor"], a["orig"], a["slow"], a["fast"],
                                a["amp"], a["table"], None)
    assert st == B.MOE_E_INVALID and needle in _msg(), _msg()


_CACHE_BAD = [
    (dict(cache=None), B.MOE_E_INVALID, "NULL"),
    (dict(cache=dict(n_pages=0)), B.MOE_E_INVALID, "non-positive"),
    (dict(cache=dict(page_size=24)), B.MOE_E_UNSUPPORTED, "power of two"),
    (dict(cache=dict(page_size=1 << 17)), B.MOE_E_UNSUPPORTED, "power of two"),
    (dict(cache=dict(n_pages=1 << 27)), B.MOE_E_UNSUPPORTED, "2^31"),
    (dict(cache=dict(dtype=B.MOE_F4E2M1)), B.MOE_E_INVALID, "dtype"),
    (dict(cache=dict(k=None)), B.MOE_E_INVALID, "NULL"),
    (dict(cache=dict(dtype=B.MOE_F8E4M3)), B.MOE_E_INVALID, "k_scale"),
]


@pytest.mark.parametrize("kw,status,needle", _CACHE_BAD + [
    (dict(act=B.MOE_F32), B.MOE_E_INVALID, "must hold act"),
    (dict(act=7), B.MOE_E_INVALID, "act"),
    (dict(T=-1), B.MOE_E_INVALID, "negative"),
    (dict(k=None), B.MOE_E_INVALID, "NULL"),
    (dict(k=dict(heads=3)), B.MOE_E_INVALID, "heads"),
    (dict(slots=None), B.MOE_E_INVALID, "slots"),
    (dict(rope={}, positions=None), B.MOE_E_INVALID, "positions"),
    (dict(rope=dict(rot_dim=256)), B.MOE_E_INVALID, "rot_dim"),
    (dict(q={}), B.MOE_E_INVALID, "without a rotation"),
    (dict(rope={}, q=dict(out_h=0)), B.MOE_E_INVALID, "overlap"),
    (dict(v=dict(in_=P + 1)), B.MOE_E_INVALID, "aligned"),
])
def test_append_refusals(kw, status, needle):
    a = dict(cache={}, rope=None, act=B.MOE_BF16, T=7, k={}, v={}, q=None, positions=P, slots=P)
    a.update(kw)
    made = lambda f, v: None if v is None else f(**v)
    st = B.lib().moe_kv_append(made(_cache, a["cache"]), made(_rope, a["rope"]), a["act"], a["T"],
                               made(_rows, a["k"]), made(_rows, a["v"]), made(_rows, a["q"]), a["positions"],
                               a["slots"], None)
    assert st == status and needle in _msg(), _msg()


@pytest.mark.parametrize("kw,status,needle", _CACHE_BAD + [
    (dict(act=B.MOE_F32), B.MOE_E_INVALID, "fp32"),
    (dict(act=B.MOE_F8E4M3), B.MOE_E_INVALID, "act"),
    (dict(cache=dict(head_dim=100)), B.MOE_E_UNSUPPORTED, "head_dim"),
    (dict(cache=dict(head_dim=264)), B.MOE_E_UNSUPPORTED, "head_dim"),
    (dict(cache=dict(k=P + 8)), B.MOE_E_INVALID, "16-byte"),
    (dict(batch=-1), B.MOE_E_INVALID, "negative"),
    (dict(prefix=-1), B.MOE_E_INVALID, "negative"),
    (dict(scale=float("inf")), B.MOE_E_INVALID, "scale"),
    (dict(scale=float("nan")), B.MOE_E_INVALID, "scale"),
    (dict(q=None), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(heads=6)), B.MOE_E_INVALID, "multiple"),
    (dict(q=dict(out_t=0)), B.MOE_E_INVALID, "overlap"),
    (dict(prefix=5, pages=None), B.MOE_E_INVALID, "prefix_pages"),
    (dict(cols=2, table=None), B.MOE_E_INVALID, "page_table"),
    (dict(cols=2, lens=None), B.MOE_E_INVALID, "lens"),
    (dict(cols=1 << 28), B.MOE_E_UNSUPPORTED, "2^30"),
    (dict(prefix=(1 << 30) + 1), B.MOE_E_UNSUPPORTED, "2^30"),
    (dict(cache=dict(page_size=1 << 16, kv_heads=256), q=dict(heads=256)), B.MOE_E_UNSUPPORTED, "2^29"),
    (dict(batch=1 << 30), B.MOE_E_UNSUPPORTED, "2^31"),
    (dict(ws=None), B.MOE_E_WORKSPACE, "workspace"),
    (dict(nb=16), B.MOE_E_WORKSPACE, "workspace"),
    (dict(ws=P + 4), B.MOE_E_INVALID, "aligned"),
])
def test_attention_refusals(kw, status, needle):
    a = dict(cache={}, act=B.MOE_BF16, batch=2, q_len=1, q={}, scale=0.1, pages=P, prefix=20, table=P, cols=3, lens=P,
             ws=P, nb=1 << 40)
    a.update(kw)
    made = lambda f, v: None if v is None else f(**v)
    st = B.lib().moe_prefix_attention(made(_cache, a["cache"]), a["act"], a["batch"], a["q_len"], made(_rows, a["q"]),
                                      a["scale"], a["pages"], a["prefix"], a["table"], a["cols"], a["lens"], None,
                                      a["ws"], a["nb"], None)
    assert st == status and needle in _msg(), _msg()


def test_workspace_of_refused_sizes_is_zero():
    f = B.lib().moe_prefix_attention_workspace_bytes
    assert f(_cache(), 4, 1, 8, 1000, 3) > 0
    for bad in ((None, 4, 1, 8, 10, 3), (_cache(), -1, 1, 8, 10, 3), (_cache(), 4, 1, 6, 10, 3),
                (_cache(), 4, 1, 8, -1, 3), (_cache(), 1 << 30, 1, 8, 10, 3)):
        assert f(*bad) == 0


def test_binding_refuses_wrong_tensors():
    """Shapes, dtypes and devices the C side cannot see are checked before the call."""
    t = torch.zeros
    q, k, pos, tab = t(3, 4, 8), t(3, 2, 8), t(3, dtype=torch.int32), t(10, 2, 2)
    ok = dict(q=q, k=k, positions=pos, table=tab, q_out=t(3, 4, 8), k_out=t(3, 2, 8))
    for bad, exc in ((dict(q_out=t(3, 4, 9)), ValueError), (dict(q_out=t(3, 4, 8).bfloat16()), TypeError),
                     (dict(q_out=t(3, 8, 4).transpose(1, 2)), ValueError), (dict(k=t(2, 2, 8)), ValueError),
                     (dict(k_out=None), ValueError), (dict(positions=pos.long()), TypeError),
                     (dict(positions=pos[:2]), ValueError), (dict(table=t(10, 4)), ValueError),
                     (dict(table=tab.double()), ValueError), ({}, ValueError)):      # {}: tensors not on a GPU
        with pytest.raises(exc):
            B.moe_rotary(**{**ok, **bad})
    kc = t(4, 2, 16, 8)
    ok = dict(k=k, v=k, slots=pos, k_cache=kc, v_cache=kc, positions=pos, table=tab)
    for bad, exc in ((dict(v=t(2, 2, 8)), ValueError), (dict(v=k.bfloat16()), ValueError),
                     (dict(q=q), ValueError), (dict(positions=None), ValueError), (dict(slots=pos.long()), TypeError),
                     (dict(v_cache=t(4, 2, 16, 4)), ValueError),
                     (dict(k_cache=kc.to(torch.uint8), v_cache=kc.to(torch.uint8)), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            B.moe_kv_append(**{**ok, **bad})
    ok = dict(q=q, k_cache=kc, v_cache=kc, prefix_pages=pos, prefix_len=20, page_table=t(3, 2, dtype=torch.int32),
              lens=pos, out=t(3, 4, 8))
    for bad, exc in ((dict(q_len=2), ValueError), (dict(q_len=0), ValueError), (dict(out=None), ValueError),
                     (dict(page_table=t(2, 2, dtype=torch.int32)), ValueError), (dict(lens=None), ValueError),
                     (dict(lens=pos.long()), TypeError), (dict(prefix_pages=pos[:1]), ValueError),
                     (dict(prefix_pages=None), ValueError), (dict(lse=t(3)), ValueError),
                     (dict(q=t(3, 4, 16)), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            B.moe_prefix_attention(**{**ok, **bad})


def test_struct_sizes_match_the_header():
    """ctypes layouts of the three structs (offsets follow from the natural alignment of their fields)."""
    assert ctypes.sizeof(B.moe_heads) == 56 and ctypes.sizeof(B.moe_rope) == 24 and ctypes.sizeof(B.moe_kv_cache) == 56
