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
