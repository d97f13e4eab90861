"""Pins of oracle/attention.py: rotations keep lengths and depend on position differences only, the scaled frequencies
meet their end points, the gradient is the derivative, and attention equals a library softmax."""
import numpy as np
import pytest
from scipy.special import logsumexp, softmax

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_sees_position_differences(interleaved):
    rng = np.random.default_rng(0)
    cs = oracle.rope_table(16, 64)
    q, k = rng.standard_normal((2, 1, 1, 24))
    turn = lambda x, p: oracle.rotate(x, cs[[p]], interleaved)[0]
    assert np.allclose(np.linalg.norm(turn(q, 37)), np.linalg.norm(q), rtol=1e-13)
    assert np.array_equal(turn(q, 37)[..., 16:], q[..., 16:])
    assert np.allclose(turn(q, 0), q)
    a = np.sum(turn(q, 12) * turn(k, 5))
    assert np.allclose(a, np.sum(turn(q, 60) * turn(k, 53)), rtol=1e-11)


def test_layouts_are_a_permutation_of_each_other():
    rng = np.random.default_rng(1)
    cs = oracle.rope_table(8, 16)[[3, 9]]
    x = rng.standard_normal((2, 3, 8))
    to_half = np.r_[0:8:2, 1:8:2]
    assert np.allclose(oracle.rotate(x, cs, True)[0][..., to_half], oracle.rotate(x[..., to_half], cs, False)[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_transposed_rotation_is_the_gradient(interleaved):
    rng = np.random.default_rng(2)
    cs = oracle.rope_table(6, 32, amplitude=1.3)[[5, 31]]
    x, dy = rng.standard_normal((2, 2, 2, 10))
    dx, _ = oracle.rotate(dy, cs, interleaved, transpose=True)
    num = np.zeros_like(x)
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = 1e-3
        f = lambda z: np.sum(oracle.rotate(z, cs, interleaved)[0] * dy)
        num[at] = (f(x + e) - f(x - e)) / 2e-3
    assert np.allclose(dx, num, atol=1e-10)


def test_scaled_frequencies():
    plain = oracle.rope_frequencies(64)
    assert np.allclose(plain[0], 1.0) and np.allclose(plain[-1], 10000.0 ** (-62 / 64))
    assert np.allclose(oracle.rope_frequencies(64, scaling="linear", factor=8), plain / 8)
    b = oracle.rope_frequencies(64, scaling="base", factor=8)
    assert np.allclose(b[0], plain[0]) and np.allclose(b[-1], plain[-1] / 8)
    p = oracle.rope_frequencies(64, scaling="parts", factor=8, orig_len=4096, slow=1, fast=32)
    turns = 4096 * plain / (2 * np.pi)
    assert np.allclose(p[turns > 32], plain[turns > 32]) and np.allclose(p[turns < 1], plain[turns < 1] / 8)
    assert np.all(np.diff(p) < 0)


def test_quantize_rows_is_the_tile_rule():
    rng = np.random.default_rng(3)
    x = np.float32(rng.standard_normal((5, 128)))
    x[2] = 0
    codes, scale = oracle.quantize_rows(x)
    ref_codes, ref_scale = oracle.quantize_tiles(x)
    assert np.allclose(scale, ref_scale[:, 0], rtol=1e-6)
    assert np.mean(codes != ref_codes) < 0.01 and not codes[2].any()


def test_attend_is_softmax():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal(16), rng.standard_normal((33, 16)), rng.standard_normal((33, 16))
    out, lse, _ = oracle.attend(q, k, v, 0.25)
    assert np.allclose(out, softmax(0.25 * k @ q) @ v) and np.allclose(lse, logsumexp(0.25 * k @ q))
    out, lse, _ = oracle.attend(q, k[:0], v[:0], 0.25)
    assert not out.any() and lse == -np.inf
