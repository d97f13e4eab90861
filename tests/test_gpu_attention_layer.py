"""The training half of a block as a user runs it: norm, projections, rotary positions, causal attention, and all the way back.

Against a plain layer in fp64 with torch's own gradients, on the CPU. fp32: each result passes six products or sums of at most 256
terms, each off by 256 * 2^-23 of its terms' magnitudes at worst, in all 2e-4 of the norm. bf16: twelve roundings of 2^-8 on the way
forth and back, in all 5% of the norm at worst.
"""
import importlib.util
import os

import pytest
import torch

from gpu_common import DEV
from mixture_experts_layer_gate_amd import AttentionLayer, MOE_ROPE_INTERLEAVED

pytestmark = pytest.mark.gpu


def _weights(g, d, hq, hk, D, dt):
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)     # noqa: E731
    return {"w_qkv": (r((hq + 2 * hk) * D, d) * d ** -0.5).to(dt), "w_out": (r(d, hq * D) * (hq * D) ** -0.5).to(dt),
            "norm_weight": (1 + 0.1 * r(d)).float(), "norm_bias": (0.1 * r(d)).float()}


def _plain(x, w, starts, hq, hk, D, R, interleaved):
    """The layer in fp64 from its formulas."""
    T = len(x)
    n = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, correction=0, keepdim=True) + 1e-5) * w["norm_weight"] + w["norm_bias"]
    q, k, v = (n @ w["w_qkv"].t()).view(T, -1, D).split([hq, hk, hk], 1)
    theta = 10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)

    def turn(t, pos):
        c, s = torch.cos(pos[:, None] * theta)[:, None], torch.sin(pos[:, None] * theta)[:, None]
        a, b = (t[..., 0:R:2], t[..., 1:R:2]) if interleaved else (t[..., :R // 2], t[..., R // 2:R])
        both = (a * c - b * s, b * c + a * s)
        r = torch.stack(both, -1).flatten(-2) if interleaved else torch.cat(both, -1)
        return torch.cat([r, t[..., R:]], -1)
    out = [x[:starts[0]]]
    for a, b in zip(starts[:-1], starts[1:]):
        pos = torch.arange(b - a, dtype=torch.float64)
        qq, kk, vv = turn(q[a:b], pos), turn(k[a:b], pos).repeat_interleave(hq // hk, 1), v[a:b].repeat_interleave(hq // hk, 1)
        s = torch.einsum("ihd,jhd->hij", qq, kk) * D ** -0.5
        p = torch.softmax(s.masked_fill(~torch.ones((b - a, b - a), dtype=torch.bool).tril(), -torch.inf), -1)
        out.append(x[a:b] + torch.einsum("hij,jhd->ihd", p, vv).reshape(b - a, hq * D) @ w["w_out"].t())
    out.append(x[starts[-1]:])
    return torch.cat(out)


@pytest.mark.parametrize("dt,bound", [(torch.float32, 2e-4), (torch.bfloat16, 0.05)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layer_and_gradients(dt, bound, interleaved):
    T, d, hq, hk, D, R, starts = 190, 160, 6, 2, 64, 48, [4, 50, 50, 51, 183]
    g = torch.Generator().manual_seed(7)
    w = _weights(g, d, hq, hk, D, dt)
    x = torch.randn((T, d), generator=g, dtype=torch.float64).to(dt)
    d_out = torch.randn((T, d), generator=g, dtype=torch.float64).to(dt)
    layer = AttentionLayer(w, hq, hk, D, max_len=256, rot_dim=R, layout=MOE_ROPE_INTERLEAVED if interleaved else 0)
    seq = torch.tensor(starts, dtype=torch.int32, device=DEV)
    out = layer.forward(x.to(DEV), seq)
    dx = layer.backward(d_out.to(DEV))
    leaves = {n: t.double().requires_grad_() for n, t in {**w, "x": x}.items()}
    want = _plain(leaves["x"], leaves, starts, hq, hk, D, R, interleaved)
    want.backward(d_out.double())
    got = {"out": (out, want.detach()), "x": (dx, leaves["x"].grad),
           **{n: (layer.grads[n], leaves[n].grad) for n in w}}
    for n, (a, b) in got.items():
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off <= bound, (n, off)
    assert torch.equal(out[:4].cpu(), x[:4]) and torch.equal(dx[183:].cpu(), d_out[183:])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_outside_the_sequences_may_hold_anything(dt):
    T, d, hq, hk, D, starts = 75, 96, 4, 2, 32, [3, 40, 41, 70]
    g = torch.Generator().manual_seed(9)
    layer = AttentionLayer(_weights(g, d, hq, hk, D, dt), hq, hk, D, max_len=64)
    x, d_out = (torch.randn((T, d), generator=g).to(dt).to(DEV) for _ in range(2))
    seq = torch.tensor(starts, dtype=torch.int32, device=DEV)
    out, dx, grads = layer.forward(x, seq), layer.backward(d_out), dict(layer.grads)
    for bad in (float("nan"), float("inf"), 3e38):
        y, e = x.clone(), d_out.clone()
        for t in (y, e):
            t[:3] = bad
            t[70:] = -bad
        out2, dx2 = layer.forward(y, seq), layer.backward(e)
        assert torch.equal(out2[3:70], out[3:70]) and torch.equal(dx2[3:70], dx[3:70])
        assert torch.equal(out2[:3].isnan(), y[:3].isnan()) and torch.equal(dx2[70:].nan_to_num(), e[70:].nan_to_num())
        for n, t in layer.grads.items():
            assert torch.equal(t, grads[n]), n


def test_refusals():
    w = _weights(torch.Generator().manual_seed(1), 64, 2, 1, 64, torch.float32)
    layer = AttentionLayer(w, 2, 1, 64, max_len=16)
    with pytest.raises(RuntimeError, match="forward first"):
        layer.backward(torch.zeros((4, 64), device=DEV))
    with pytest.raises(ValueError, match="x must be"):
        layer.forward(torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="w_qkv must be"):
        AttentionLayer(w, 4, 1, 64, max_len=16)
    with pytest.raises(TypeError, match="both"):
        AttentionLayer({**w, "w_out": w["w_out"].half()}, 2, 1, 64, max_len=16)
    layer.forward(torch.zeros((4, 64), device=DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="d_out must be"):
        layer.backward(torch.zeros((3, 64), device=DEV))


def test_the_example_block():
    """Attention and experts, both ways: the gradients that the two layers exchange are those of the whole."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.TrainBlock(ex.get_config("c1", gemm="bf16", act="bf16"))
    x, d_out = block.x0, torch.randn(block.x0.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).bfloat16()
    assert torch.isfinite(block.forward(x)).all()
    dx = block.backward(d_out)
    assert torch.isfinite(dx).all() and dx.shape == x.shape
    du = block.moe.backward(d_out).to(x.dtype)
    assert torch.equal(block.attention.backward(du), dx)
