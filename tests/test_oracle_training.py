"""The fp64 oracle of causal attention and the layer norm: against torch's softmax and its gradients on whole sequences, differences,
and closed forms."""
import numpy as np
import torch

import oracle


def _case(seed=0, T=23, hq=4, hk=2, D=8):
    r = np.random.default_rng(seed)
    return [r.standard_normal((T, h, D)) for h in (hq, hk, hk, hq)]


STARTS = [2, 9, 9, 10, 21]


def _torch(q, k, v, starts, scale):
    G = q.shape[1] // k.shape[1]
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), dtype=q.dtype)
    rows = []
    for a, b in zip(starts[:-1], starts[1:]):
        if a == b:
            continue
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(G, 1)) * scale
        s = s.masked_fill(~torch.ones((b - a, b - a), dtype=torch.bool).tril(), -torch.inf)
        rows.append((a, b, torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[a:b].repeat_interleave(G, 1)),
                     torch.logsumexp(s, -1).t()))
    for a, b, o, z in rows:
        out[a:b], lse[a:b] = o, z
    return out, lse


def test_attention_and_gradients_against_torch():
    q, k, v, g = _case()
    leaves = [torch.tensor(t, requires_grad=True) for t in (q, k, v)]
    out, lse = _torch(*leaves, STARTS, 0.3)
    o, z, to, tl = oracle.causal_attention(q, k, v, STARTS, 0.3)
    inside = slice(2, 21)
    assert np.isnan(o[:2]).all() and np.isnan(o[21:]).all()
    assert np.allclose(o[inside], out.detach().numpy()[inside], rtol=1e-12, atol=1e-12)
    assert np.allclose(z[inside], lse.detach().numpy()[inside], rtol=1e-12, atol=1e-12)
    assert (to[inside] > 0).all() and (tl[inside] > 0).all()
    (out[inside] * torch.tensor(g)[inside]).sum().backward()
    ref = oracle.causal_attention_grad(q, k, v, o, g, z, STARTS, 0.3)
    for a, t in zip(ref[:3], leaves):
        assert np.allclose(a[inside], t.grad.numpy()[inside], rtol=1e-11, atol=1e-12)
        assert np.isnan(a[:2]).all() and np.isnan(a[21:]).all()


def test_one_token_is_its_value():
    q, k, v, g = _case(1, T=3)
    o, z, _, _ = oracle.causal_attention(q, k, v, [0, 1, 2, 3], 0.5)
    assert np.allclose(o, v.repeat(2, 1)) and np.allclose(z, 0.5 * (q * k.repeat(2, 1)).sum(-1))
    dq, dk, dv = oracle.causal_attention_grad(q, k, v, o, g, z, [0, 1, 2, 3], 0.5)[:3]
    assert np.allclose(dq, 0) and np.allclose(dk, 0) and np.allclose(dv, g.reshape(3, 2, 2, 8).sum(2))


def test_scores_of_minus_infinity():
    q, k, v, _ = _case(2, T=4, hq=1, hk=1)
    q[:, :, 0], k[0, :, 0] = 1.0, -np.inf
    o, z, _, _ = oracle.causal_attention(q, k, v, [0, 4], 1.0)
    assert (o[0] == 0).all() and z[0, 0] == -np.inf and np.isfinite(o[1:]).all()


def test_bounds_hold_for_fp32():
    """torch's own fp32 arithmetic stays within the derived bounds."""
    q, k, v, g = [t.astype(np.float32) for t in _case(3, T=200, D=64)]
    starts = [0, 150, 200]
    t = [torch.tensor(x) for x in (q, k, v)]
    out, lse = _torch(*t, starts, 0.125)
    o, z, to, tl = oracle.causal_attention(q, k, v, starts, 0.125)
    assert (np.abs(out.numpy() - o) <= to + 2.0 ** -24 * np.abs(o)).all() and (np.abs(lse.numpy() - z) <= tl).all()
    assert to.max() < 1e-3 * np.abs(o).max()


def test_sequence_of():
    assert oracle.sequence_of(12, [2, 9, 9, 10]).tolist() == [[-1, -1]] * 2 + [[2, 9]] * 7 + [[9, 10]] + [[-1, -1]] * 2


def test_norm_and_gradients_against_torch():
    r = np.random.default_rng(4)
    x, w, b, g, res = r.standard_normal((9, 31)) + 3, r.standard_normal(31), r.standard_normal(31), r.standard_normal((9, 31)), \
        r.standard_normal((9, 31))
    leaves = [torch.tensor(t, requires_grad=True) for t in (x, w, b)]
    y = torch.nn.functional.layer_norm(leaves[0], (31,), leaves[1], leaves[2], 1e-3)
    y.backward(torch.tensor(g))
    ry, mean, rstd = oracle.layer_norm(x, w, b, 1e-3)[:3]
    assert np.allclose(ry, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = oracle.layer_norm_grad(g, x, w, mean, rstd, res)[:3]
    for a, t in zip((dx - res, dw, db), leaves):
        assert np.allclose(a, t.grad.numpy(), rtol=1e-10, atol=1e-11)


def test_norm_gradient_against_differences():
    r = np.random.default_rng(5)
    x, w, b, g, e = (r.standard_normal(s) for s in ((6, 20), 20, 20, (6, 20), (6, 20)))
    f = lambda t: (oracle.layer_norm(t, w, b, 1e-5)[0] * g).sum()     # noqa: E731
    _, mean, rstd = oracle.layer_norm(x, w, b, 1e-5)[:3]
    dx = oracle.layer_norm_grad(g, x, w, mean, rstd)[0]
    assert abs((f(x + 1e-5 * e) - f(x - 1e-5 * e)) / 2e-5 - (dx * e).sum()) < 1e-7
