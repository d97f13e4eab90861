"""AttentionLayer where a caller's own program meets it: tensors that autograd follows, buffers that are filled again, sequences
longer than the rotary table, batches without tokens, gradients of any strides, recorded graphs."""
import math

import pytest
import torch

from gpu_common import DEV
from mixture_experts_layer_gate_amd import AttentionLayer
from test_gpu_attention_layer import _weights

pytestmark = pytest.mark.gpu


def _made(dt, d=96, hq=4, hk=2, D=32, max_len=64, T=75, seed=9, **kw):
    g = torch.Generator().manual_seed(seed)
    layer = AttentionLayer(_weights(g, d, hq, hk, D, dt), hq, hk, D, max_len=max_len, **kw)
    x, d_out = (torch.randn((T, d), generator=g).to(dt).to(DEV) for _ in range(2))
    return layer, x, d_out


def _starts(*at):
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _all(layer, x, seq, d_out, **kw):
    out = layer.forward(x, seq, **kw)
    return {"out": out, "dx": layer.backward(d_out), **layer.grads}


def _equal(got, want):
    for n, t in want.items():
        assert torch.equal(got[n], t), n


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_outside_autograd(dt):
    """Nothing of the layer enters autograd's graph, whatever requires grad: its gradients come from backward() alone."""
    layer, x, d_out = _made(dt)
    seq = _starts(0, 40, 75)
    want = _all(layer, x, seq, d_out)
    for t in (layer.w_qkv, layer.w_out, layer.norm_weight, layer.norm_bias):
        t.requires_grad_()
    got = _all(layer, x.clone().requires_grad_(), seq, d_out.clone().requires_grad_())
    assert not any(t.requires_grad for t in got.values())
    with pytest.raises(RuntimeError, match="does not require grad"):
        got["out"].sum().backward()
    _equal(got, want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_past_the_rotary_table(dt):
    """Tokens whose position lies past the table come out as NaN, with what sees them; the others as ever."""
    layer, x, d_out = _made(dt, max_len=33)
    fits = layer.forward(x, _starts(2, 35, 68))
    out = layer.forward(x, _starts(2, 36, 69))
    last = [35, 69 - 1]
    assert out[last[:1]].isnan().all() and out[2:35].isfinite().all() and torch.equal(out[:2], x[:2])
    assert out[36:68].isfinite().all() and out[69:].isfinite().all()
    bound = 1e-4 if dt == torch.float32 else 0.05      # sums in another order beside a NaN that is masked
    assert (out[2:35] - fits[2:35]).double().norm() <= bound * fits[2:35].double().norm()
    assert layer.backward(d_out)[35].isnan().all() and layer.grads["w_qkv"].isnan().any()
    at = layer.positions(75, _starts(2, 35, 68))
    assert torch.equal(layer.forward(x, _starts(2, 35, 68), positions=at), fits)
    at[20], at[40] = 33, 2 ** 31 - 1
    out = layer.forward(x, _starts(2, 35, 68), positions=at)
    assert out[20:35].isnan().all() and out[40:68].isnan().all() and out[:20].isfinite().all() and out[35:40].isfinite().all()
    at[20], at[40] = -1, -2      # no place: not rotated
    assert layer.forward(x, _starts(2, 35, 68), positions=at).isfinite().all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("given", [False, True])
def test_buffers_filled_again_before_backward(dt, given):
    """The caller may reuse x, seq_start and positions once forward has returned."""
    layer, x, d_out = _made(dt)
    seq = _starts(3, 40, 41, 70)
    kw = {"positions": layer.positions(75, seq)} if given else {}
    want = _all(layer, x, seq, d_out, **kw)
    out = layer.forward(x, seq, **kw)
    assert torch.equal(out, want["out"])
    seq.copy_(_starts(0, 1, 2, 3))
    x.fill_(5.0)
    for t in kw.values():
        t.fill_(1)
    dx = layer.backward(d_out)
    _equal({"dx": dx, **layer.grads}, {n: t for n, t in want.items() if n != "out"})


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-46])
def test_rows_outside_without_eps(dt, eps):
    """Without eps a constant row has no norm; rows outside the sequences take no part all the same."""
    layer, x, d_out = _made(dt, eps=eps)
    x[:3], x[70:] = 0.0, 2.0
    got = _all(layer, x, _starts(3, 40, 41, 70), d_out)
    alone = _all(layer, x[3:70].clone(), _starts(0, 37, 38, 67), d_out[3:70].clone())
    assert torch.equal(got["out"][:3], x[:3]) and torch.equal(got["out"][70:], x[70:])
    assert torch.equal(got["dx"][:3], d_out[:3]) and torch.equal(got["dx"][70:], d_out[70:])
    bound = 2e-4 if dt == torch.float32 else 0.05      # as in the layer's own test: sums in another order
    for n, t in alone.items():
        a = got[n][3:70] if n in ("out", "dx") else got[n]
        assert (a - t).double().norm() <= bound * t.double().norm(), n


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_no_tokens(dt):
    """A batch without tokens, and one without sequences: nothing comes back changed, and gradients are zeros."""
    layer, x, d_out = _made(dt)
    for rows, seq in ((0, _starts(0)), (0, _starts(0, 0, 0)), (75, _starts(0)), (75, _starts(30, 30))):
        got = _all(layer, x[:rows], seq, d_out[:rows])
        assert torch.equal(got["out"], x[:rows]) and torch.equal(got["dx"], d_out[:rows])
        assert all((layer.grads[n] == 0).all() and layer.grads[n].shape == getattr(layer, n).shape for n in layer.grads)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_of_any_strides(dt):
    """One number for every element (the gradient of a sum), one row for all tokens, a transposed tensor."""
    layer, x, d_out = _made(dt)
    seq = _starts(3, 40, 70)
    for t in (torch.ones((), dtype=dt, device=DEV).expand(x.shape), d_out[:1].expand(x.shape), d_out.t().contiguous().t()):
        assert not t.is_contiguous()
        _equal(_all(layer, x, seq, t), _all(layer, x, seq, t.contiguous()))


def test_weight_gradients_in_fp32():
    """The gradients of bf16 weights are fp32, as MoELayer's are: nearer to the products of the tensors they come from than bf16
    could hold them. T 2u of their terms' magnitudes from the sums (a matrix unit may truncate), 2^-24 from the result."""
    layer, x, d_out = _made(torch.bfloat16, T=400, max_len=400)
    layer.forward(x, _starts(0, 150, 400))
    a = layer._saved[5].reshape(400, -1).double()
    layer.backward(d_out)
    assert all(t.dtype == torch.float32 for t in layer.grads.values())
    want, mag = d_out.double().t() @ a, d_out.double().abs().t() @ a.abs()
    assert ((layer.grads["w_out"] - want).abs() <= 400 * 2.0 ** -23 * mag + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_recorded(dt):
    """Both directions replayed from a graph between eager work, on new inputs, lengths included."""
    layer, x, d_out = _made(dt, max_len=75, T=75)
    seq = _starts(3, 40, 41, 70)
    _all(layer, x, seq, d_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = _all(layer, x, seq, d_out)
    for step, at in enumerate(([3, 40, 41, 70], [0, 10, 75, 75], [5, 5, 6, 60])):
        for t in rec.values():
            t.fill_(math.nan)
        x.mul_(0.75)
        d_out.mul_(1.25)
        seq.copy_(_starts(*at))
        graph.replay()
        torch.cuda.synchronize()
        want = _all(layer, x, seq, d_out)
        torch.cuda.synchronize()
        for n, t in want.items():
            assert torch.equal(rec[n], t), (step, n)
