"""Refusals of the causal attention and layer norm calls, on the host before any launch (runs without a GPU)."""
import pytest

from mixture_experts_layer_gate_amd import binding as B

P = 0x1000   # never dereferenced: validation fails first


def _rows(**kw):
    a = dict(in_=P, in_t=512, in_h=128, out=64 * P, out_t=512, out_h=128, heads=4)
    a.update(kw)
    return B.moe_heads(*[a[n] for n, _ in B.moe_heads._fields_])


def _msg():
    return B.lib().moe_last_error().decode()


_ATTENTION_BAD = [
    (dict(act=B.MOE_F8E4M3), B.MOE_E_INVALID, "act"),
    (dict(T=-1), B.MOE_E_INVALID, "negative T"),
    (dict(D=0), B.MOE_E_INVALID, "head_dim"),
    (dict(D=68), B.MOE_E_UNSUPPORTED, "multiple of 8"),
    (dict(D=264), B.MOE_E_UNSUPPORTED, "at most 256"),
    (dict(T=(1 << 30) + 1), B.MOE_E_UNSUPPORTED, "2^30"),
    (dict(T=1 << 30), B.MOE_E_UNSUPPORTED, "2^30 rows or head rows"),
    (dict(T=(1 << 28) + 1), B.MOE_E_UNSUPPORTED, "2^30 rows or head rows"),
    (dict(q=dict(heads=65540, out_t=65540 * 128)), B.MOE_E_UNSUPPORTED, "65536"),
    (dict(n=-1), B.MOE_E_INVALID, "n_seqs"),
    (dict(starts=None), B.MOE_E_INVALID, "seq_start"),
    (dict(starts=P + 2), B.MOE_E_INVALID, "seq_start"),
    (dict(q=None), B.MOE_E_INVALID, "NULL"),
    (dict(k=None), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(heads=0)), B.MOE_E_INVALID, "heads"),
    (dict(k=dict(heads=3), v=dict(heads=3)), B.MOE_E_INVALID, "multiple of kv heads"),
    (dict(k=dict(heads=2)), B.MOE_E_INVALID, "k has 2 and v 4"),
    (dict(q=dict(in_=None)), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(out=None)), B.MOE_E_INVALID, "NULL"),
    (dict(q=dict(out_t=511)), B.MOE_E_INVALID, "overlap"),
    (dict(v=dict(in_=P + 1)), B.MOE_E_INVALID, "aligned"),
    (dict(k=dict(in_t=1 << 60)), B.MOE_E_INVALID, "stride"),
    (dict(scale=float("nan")), B.MOE_E_INVALID, "scale"),
    (dict(scale=float("inf")), B.MOE_E_INVALID, "scale"),
    (dict(lse=P + 2), B.MOE_E_INVALID, "lse"),
]


def _attention(back=False, **kw):
    a = dict(act=B.MOE_BF16, T=7, D=128, n=1, starts=P, q={}, k={}, v={}, out={}, d_out={}, scale=0.1, lse=2 * P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    made = lambda f, i: None if f is None else _rows(**{**dict(in_=(4 + i) * P, out=(64 + i) * P), **f})     # noqa: E731
    h = [made(a[n], i) for i, n in enumerate(("q", "k", "v"))]
    if not back:
        return B.lib().moe_causal_attention(a["act"], a["T"], a["D"], a["n"], a["starts"], *h, a["scale"], a["lse"], None)
    return B.lib().moe_causal_attention_backward(a["act"], a["T"], a["D"], a["n"], a["starts"], *h, made(a["out"], 3), made(a["d_out"], 4),
                                                 a["scale"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status,needle", _ATTENTION_BAD)
def test_attention_refusals(back, kw, status, needle):
    assert _attention(back, **kw) == status and needle in _msg(), _msg()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(out=None), B.MOE_E_INVALID, "NULL"),
    (dict(d_out=None), B.MOE_E_INVALID, "NULL"),
    (dict(out=dict(heads=2)), B.MOE_E_INVALID, "out has 2"),
    (dict(lse=None), B.MOE_E_INVALID, "lse"),
    (dict(k=dict(out=None)), B.MOE_E_INVALID, "NULL"),
    (dict(v=dict(out_h=64)), B.MOE_E_INVALID, "overlap"),
    (dict(k=dict(in_=9 * P, out=9 * P)), B.MOE_E_INVALID, "takes the place"),
    (dict(d_out=dict(in_=65 * P)), B.MOE_E_INVALID, "takes the place"),
    (dict(ws=None), B.MOE_E_WORKSPACE, "workspace"),
    (dict(ws_bytes=100), B.MOE_E_WORKSPACE, "workspace"),
    (dict(ws=P + 4), B.MOE_E_INVALID, "16-byte"),
])
def test_attention_backward_refusals(kw, status, needle):
    assert _attention(True, **kw) == status and needle in _msg(), _msg()


def test_empty_calls_do_nothing():
    for kw in (dict(T=0), dict(n=0, starts=None)):
        assert _attention(**kw) == B.MOE_OK and _attention(True, **kw) == B.MOE_OK
    assert _norm(rows=0, x=None, y=None) == B.MOE_OK
    assert _norm_back(rows=0, x=None, dy=None, dx=None, dw=None, db=None, ws=None) == B.MOE_OK


def test_workspace_sizes():
    L = B.lib()
    for bad in ((-1, 64, 4, 4), (8, 60, 4, 4), (8, 264, 4, 4), (8, 64, 4, 3), (1 << 30, 64, 4, 4)):
        assert L.moe_causal_attention_backward_workspace_bytes(*bad) == 0
    assert L.moe_layer_norm_backward_workspace_bytes(-1, 8) == 0 and L.moe_layer_norm_backward_workspace_bytes(8, 16385) == 0
    assert L.moe_causal_attention_backward_workspace_bytes(1000, 64, 4, 4) >= 1000 * 4 * 8
    assert L.moe_layer_norm_backward_workspace_bytes(10 ** 6, 16384) < 1 << 30


def _norm(**kw):
    a = dict(act=B.MOE_F32, rows=5, d=64, x=P, xs=64, w=P, b=P, eps=1e-5, y=9 * P, ys=64, mean=None, rstd=None)
    a.update(kw)
    return B.lib().moe_layer_norm(a["act"], a["rows"], a["d"], a["x"], a["xs"], a["w"], a["b"], a["eps"], a["y"], a["ys"], a["mean"],
                                  a["rstd"], None)


def _norm_back(**kw):
    a = dict(act=B.MOE_F32, rows=5, d=64, dy=P, dys=64, x=2 * P, xs=64, w=P, mean=P, rstd=P, dr=None, drs=0, dx=9 * P, dxs=64, dw=P, db=P,
             ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return B.lib().moe_layer_norm_backward(*[a[n] for n in ("act", "rows", "d", "dy", "dys", "x", "xs", "w", "mean", "rstd", "dr", "drs",
                                                            "dx", "dxs", "dw", "db", "ws", "ws_bytes")], None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(act=7), B.MOE_E_INVALID, "act"),
    (dict(rows=-1), B.MOE_E_INVALID, "negative rows"),
    (dict(d=0), B.MOE_E_INVALID, "non-positive d"),
    (dict(d=16385), B.MOE_E_UNSUPPORTED, "16384"),
    (dict(rows=1 << 40), B.MOE_E_UNSUPPORTED, "2^40"),
    (dict(x=None), B.MOE_E_INVALID, "x is NULL"),
    (dict(x=P + 2), B.MOE_E_INVALID, "aligned"),
    (dict(xs=1 << 50), B.MOE_E_INVALID, "stride"),
])
def test_norm_refusals_of_both(kw, status, needle):
    assert _norm(**kw) == status and needle in _msg(), _msg()
    assert _norm_back(**kw) == status and needle in _msg(), _msg()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(y=None), B.MOE_E_INVALID, "y is NULL"),
    (dict(ys=63), B.MOE_E_INVALID, "overlap"),
    (dict(eps=-1.0), B.MOE_E_INVALID, "eps"),
    (dict(eps=float("nan")), B.MOE_E_INVALID, "eps"),
    (dict(y=P, ys=128), B.MOE_E_INVALID, "in place"),
    (dict(w=P + 2), B.MOE_E_INVALID, "weight"),
])
def test_norm_refusals(kw, status, needle):
    assert _norm(**kw) == status and needle in _msg(), _msg()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dy=None), B.MOE_E_INVALID, "dy is NULL"),
    (dict(dx=None), B.MOE_E_INVALID, "dx is NULL"),
    (dict(dxs=10), B.MOE_E_INVALID, "overlap"),
    (dict(dx=P, dxs=80), B.MOE_E_INVALID, "in place"),
    (dict(dr=9 * P, drs=100), B.MOE_E_INVALID, "in place"),
    (dict(mean=None), B.MOE_E_INVALID, "mean"),
    (dict(rstd=P + 1), B.MOE_E_INVALID, "aligned"),
    (dict(ws=None), B.MOE_E_WORKSPACE, "workspace"),
    (dict(ws_bytes=64), B.MOE_E_WORKSPACE, "workspace"),
    (dict(ws=P + 8), B.MOE_E_INVALID, "16-byte"),
])
def test_norm_backward_refusals(kw, status, needle):
    assert _norm_back(**kw) == status and needle in _msg(), _msg()
