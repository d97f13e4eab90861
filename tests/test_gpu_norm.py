"""Layer norm and its gradient against the fp64 oracle, whose module derives the bounds used here; to them comes the rounding of the
result: half a unit (fp32 2^-24, bf16 2^-8) of it."""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, tol, what):
    got = _np(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / (tol + 1e-300)):.2f} tol"


def _rows(g, R, d, dt, how):
    x = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)     # noqa: E731
    if how == "dense":
        return x(R, d)
    if how == "wide":
        return x(R, d + 8)[:, :d]
    if how == "odd":
        return x(R * (d + 1) + 1)[1:].view(R, d + 1)[:, :d]
    if how == "one_row":
        return x(1, d).expand(R, d)
    raise ValueError(how)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("R,d,how", [
    (1, 1, "dense"), (1, 2048, "dense"), (5, 7, "dense"), (3, 64, "wide"), (130, 256, "dense"), (9, 250, "odd"), (33, 1000, "wide"),
    (17, 1001, "dense"), (6, 1030, "odd"), (20, 2056, "dense"), (2100, 40, "dense"), (37, 48, "wide"), (5000, 512, "dense"), (19, 33, "odd"), (7, 4100, "odd"), (11, 7168, "dense"),
    (3, 8200, "wide"), (2, 16384, "dense"), (3, 16383, "dense"), (1030, 512, "one_row"),
])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_gradient(act, R, d, how, residual):
    g, dt = torch.Generator(device=DEV).manual_seed(R + 3 * d), DT[act]
    x, dy, dr = (_rows(g, R, d, dt, how) for _ in range(3))
    w, b = 1 + 0.3 * torch.randn(d, generator=g, device=DEV), torch.randn(d, generator=g, device=DEV)
    out = "dense" if how == "one_row" else how
    y, dx = _rows(g, R, d, dt, out), _rows(g, R, d, dt, out)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    B.moe_layer_norm(x, w, b, y, eps=1e-5, mean=mean, rstd=rstd)
    ry, rm, rr, ty, tm, tr = oracle.layer_norm(_np(x), _np(w), _np(b), 1e-5)
    _close(mean, rm, tm, "mean")
    _close(rstd, rr, tr, "rstd")
    _close(y, ry, ty + HALF[act] * np.abs(ry) + 1e-37, "y")
    dw, db = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    B.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, d_residual=dr if residual else None)
    ref = oracle.layer_norm_grad(_np(dy), _np(x), _np(w), _np(mean), _np(rstd), _np(dr) if residual else None)
    _close(dx, ref[0], ref[3] + HALF[act] * np.abs(ref[0]) + 1e-37, "dx")
    _close(dw, ref[1], ref[4] + 1e-37, "dweight")
    _close(db, ref[2], ref[5] + 1e-37, "dbias")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_in_place_and_without_vectors(act):
    g, dt = torch.Generator(device=DEV).manual_seed(1), DT[act]
    for R, d in ((50, 96), (50, 3000), (7, 10000)):
        x, dy = torch.randn((R, d), generator=g, device=DEV).to(dt), torch.randn((R, d), generator=g, device=DEV).to(dt)
        one, zero = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
        y, mean, rstd = torch.empty_like(x), torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        B.moe_layer_norm(x, one, zero, y, mean=mean, rstd=rstd)
        z = x.clone()
        B.moe_layer_norm(z, None, None, z)
        assert torch.equal(y, z)
        dx, dw, db = torch.empty_like(x), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
        B.moe_layer_norm_backward(dy, x, one, mean, rstd, dx, dw, db, d_residual=x)
        for where in ("dy", "x", "d_residual"):
            a = {"dy": dy.clone(), "x": x.clone(), "d_residual": x.clone()}
            only = torch.empty(d, device=DEV)
            B.moe_layer_norm_backward(a["dy"], a["x"], None, mean, rstd, a[where], dbias=only, d_residual=a["d_residual"])
            assert torch.equal(a[where], dx) and torch.equal(only, db), where


def test_no_rows_and_one_channel():
    e = lambda *s: torch.full(s, 5.0, device=DEV)     # noqa: E731
    dw, db = e(40), e(40)
    B.moe_layer_norm(e(0, 40), None, None, e(0, 40))
    B.moe_layer_norm_backward(e(0, 40), e(0, 40), None, e(0), e(0), e(0, 40), dw, db)
    assert (dw == 0).all() and (db == 0).all()
    y = e(3, 1)
    B.moe_layer_norm(e(3, 1), e(1), e(1), y)
    assert (y == 5.0).all()


def test_rows_with_a_large_mean():
    """Deviations of 1 about 4096: their squares would lose 24 bits against the mean's."""
    g = torch.Generator(device=DEV).manual_seed(2)
    for d in (100, 5000):
        x = 4096 + torch.randn((20, d), generator=g, device=DEV)
        y = torch.empty_like(x)
        B.moe_layer_norm(x, None, None, y)
        ref, _, _, tol, _, _ = oracle.layer_norm(_np(x), np.ones(d), np.zeros(d), 1e-5)
        _close(y, ref, tol + HALF["f32"] * np.abs(ref), "y")


@pytest.mark.parametrize("d", [96, 2048, 9000])
def test_rows_that_are_not_finite_stay_alone(d):
    g = torch.Generator(device=DEV).manual_seed(3)
    x, dy = (torch.randn((40, d), generator=g, device=DEV) for _ in range(2))
    y, z = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    B.moe_layer_norm(x, None, None, y, mean=mean, rstd=rstd)
    bad = x.clone()
    bad[7, 3], bad[21, 0] = math_nan, float("inf")
    m, r = mean.clone(), rstd.clone()
    B.moe_layer_norm(bad, None, None, z, mean=m, rstd=r)
    rest = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(z[rest], y[rest]) and torch.equal(m[rest], mean[rest]) and torch.equal(r[rest], rstd[rest])
    assert torch.isnan(z[7]).all() and torch.isnan(r[[7, 21]]).all()
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    B.moe_layer_norm_backward(dy, x, None, mean, rstd, dx)
    B.moe_layer_norm_backward(dy, bad, None, m, r, dz)
    assert torch.equal(dz[rest], dx[rest]) and torch.isnan(dz[7]).all()


math_nan = float("nan")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("R,d", [(3, 64), (900, 300), (700, 2048), (520, 7168)])
def test_equal_calls_graphs_and_streams(act, R, d):
    g, dt = torch.Generator(device=DEV).manual_seed(4), DT[act]
    x, dy = torch.randn((R, d), generator=g, device=DEV).to(dt), torch.randn((R, d), generator=g, device=DEV).to(dt)
    w = torch.randn(d, generator=g, device=DEV)
    new = lambda: (torch.empty_like(x), *(torch.empty(R, device=DEV) for _ in range(2)), torch.empty_like(x),   # noqa: E731
                   *(torch.empty(d, device=DEV) for _ in range(2)))

    def both(o, **kw):
        B.moe_layer_norm(x, w, w, o[0], mean=o[1], rstd=o[2], **kw)
        B.moe_layer_norm_backward(dy, x, w, o[1], o[2], *o[3:], d_residual=dy, **kw)
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
            t.fill_(math_nan)
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(both(new()), rec)), step


def test_gradient_against_differences():
    """Along random directions: central differences in fp32 with h = 2^-5, whose rounding (2^-22 of the sum's terms over h) and third-
    order rest (h^2 / 6) are far below 2% of |grad||e|."""
    g = torch.Generator(device=DEV).manual_seed(5)
    R, d, h = 30, 200, 2.0 ** -5
    p = {"x": torch.randn((R, d), generator=g, device=DEV), "w": torch.randn(d, generator=g, device=DEV),
         "b": torch.randn(d, generator=g, device=DEV)}
    dy = torch.randn((R, d), generator=g, device=DEV)

    def f(p, **kw):
        y = torch.empty_like(p["x"])
        B.moe_layer_norm(p["x"], p["w"], p["b"], y, **kw)
        return y.double()
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    f(p, mean=mean, rstd=rstd)
    grads = {n: torch.empty_like(t) for n, t in p.items()}
    B.moe_layer_norm_backward(dy, p["x"], p["w"], mean, rstd, grads["x"], grads["w"], grads["b"])
    for n, t in p.items():
        e = torch.randn(t.shape, generator=g, device=DEV)
        diff = ((f({**p, n: t + h * e}) - f({**p, n: t - h * e})) * dy.double()).sum() / (2 * h)
        assert abs(diff - (grads[n].double() * e.double()).sum()) <= 0.02 * grads[n].double().norm(), n


def test_refused_by_the_binding():
    x, r = torch.zeros((4, 8), device=DEV), torch.zeros(4, device=DEV)
    with pytest.raises(ValueError, match="as x is"):
        B.moe_layer_norm(x, None, None, x[:3].clone())
    with pytest.raises(TypeError, match="weight must be fp32"):
        B.moe_layer_norm(x, torch.zeros(8, dtype=torch.bfloat16, device=DEV), None, x)
    with pytest.raises(ValueError, match="weight has 7"):
        B.moe_layer_norm(x, torch.zeros(7, device=DEV), None, x)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_layer_norm(x.t().contiguous().t(), None, None, x)
    with pytest.raises(ValueError, match="current GPU|tensors on"):
        B.moe_layer_norm(x, torch.zeros(8), None, x)
    with pytest.raises(B.MoEError, match="d \\(16385\\)"):
        B.moe_layer_norm(torch.zeros((2, 16385), device=DEV), None, None, torch.zeros((2, 16385), device=DEV))
    with pytest.raises(B.MoEError, match="workspace"):
        B.moe_layer_norm_backward(x, x, None, r, r, x.clone(), r.new_zeros(8), workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
