"""Attention of a decode batch on a shared prompt as a user runs it, and the example's block around it.

Tolerances, from the arithmetic (u = 2^-24): a rotated channel is off by 4u of its two products' magnitudes, at most
4 sqrt(2) u of its pair's norm, so a score by 2 * 4 sqrt(2) u scale |q| |k| more than the (D + 4) 2u scale sum|q||k| of
its products (|q| |k| >= sum|q||k|); the rest as for one attention call: weights within e^(2 delta), exp 2^-20, sums 2u n.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import MOE_ROPE_INTERLEAVED, PrefixAttention

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _heads(g, n, h, D):
    return torch.randn((n, h, D), generator=g, device=DEV)


def _want(q, k, v, scale):
    """Causal attention of the last rows q [n, hq, D] on k, v [m, hkv, D], rotated already; (result, tolerance)."""
    n, hq, D = q.shape
    m, hkv, _ = k.shape
    ref, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        see = m - n + 1 + i
        for h in range(hq):
            kk, vv = k[:see, h // (hq // hkv)], v[:see, h // (hq // hkv)]
            ref[i, h], _, mag = oracle.attend(q[i, h], kk, vv, scale)
            norm = scale * (np.linalg.norm(kk, axis=1) * np.linalg.norm(q[i, h])).max()
            delta = (2 * (D + 4) + 8 * 2 ** 0.5) * U32 * norm
            tol[i, h] = (2 * delta + 2.0 ** -20 + 2 * U32 * see) * mag + 5 * U32 * mag
    return ref, tol


@pytest.mark.parametrize("interleaved", [False, True])
def test_prompt_and_steps_against_the_oracle(interleaved):
    """A prompt in two chunks, then steps of one and of three tokens; every result against the whole history."""
    Bn, hq, hk, D, R = 3, 4, 2, 64, 48
    g = torch.Generator(device=DEV).manual_seed(5)
    att = PrefixAttention(Bn, hq, hk, D, 80, 40, dtype=torch.float32, page_size=16, rot_dim=R,
                          layout=MOE_ROPE_INTERLEAVED if interleaved else 0)
    cs = oracle.rope_table(R, 200)
    rot = lambda x, p0: oracle.rotate(x, cs[p0:p0 + len(x)], interleaved)[0]
    npy = lambda t: t.double().cpu().numpy()
    K, V = np.zeros((0, hk, D)), np.zeros((0, hk, D))
    for n in (32, 41):
        q, k, v = (_heads(g, n, h, D) for h in (hq, hk, hk))
        out = att.prefill(q, k, v)
        p0 = len(K)
        K, V = np.concatenate([K, rot(npy(k), p0)]), np.concatenate([V, npy(v)])
        ref, tol = _want(rot(npy(q), p0), K, V, D ** -0.5)
        assert (np.abs(npy(out) - ref) <= tol).all()
    own = [(K, V)] * Bn
    for n in (1, 3, 1):
        q, k, v = (_heads(g, Bn * n, h, D) for h in (hq, hk, hk))
        out = npy(att.step(q, k, v, n))
        for b in range(Bn):
            rows, p0 = slice(b * n, b * n + n), len(own[b][0])
            own[b] = (np.concatenate([own[b][0], rot(npy(k)[rows], p0)]), np.concatenate([own[b][1], npy(v)[rows]]))
            ref, tol = _want(rot(npy(q)[rows], p0), *own[b], D ** -0.5)
            assert (np.abs(out[rows] - ref) <= tol).all()
    assert att.lens.tolist() == [5] * Bn
    again = att.prefix_len
    att.reset()
    assert att.lens.tolist() == [0] * Bn and att.prefix_len == again


def test_refusals():
    att = PrefixAttention(2, 2, 1, 64, 32, 16, page_size=16)
    z = lambda n, h: torch.zeros((n, h, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="room for 32"):
        att.prefill(z(33, 2), z(33, 1), z(33, 1))
    att.prefill(z(7, 2), z(7, 1), z(7, 1))
    with pytest.raises(ValueError, match="inside a page"):
        att.prefill(z(1, 2), z(1, 1), z(1, 1))
    for _ in range(16):
        att.step(z(2, 2), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="room for 16"):
        att.step(z(2, 2), z(2, 1), z(2, 1))
    att.reset(keep_prompt=False)
    assert att.prefix_len == 0


@pytest.mark.parametrize("cache", [None, "e4m3"])
def test_the_example_block(cache):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    cfg = ex.get_config("c1", gemm="bf16", act="bf16")
    block = ex.DecodeBlock(cfg, prompt=2 * cfg.T, new_tokens=4, cache=cache)
    x = block.x0
    for _ in range(2):
        assert torch.isfinite(block.prefill(x)).all()
    first = block.step(x).clone()
    block.attention.reset()
    assert torch.equal(block.step(x), first)      # the prompt is still there, the own tokens are not
    assert torch.isfinite(block.step(first)).all()
    assert block.attention.lens.tolist() == [2] * cfg.T
