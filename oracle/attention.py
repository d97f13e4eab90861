"""Rotary positions, cache rows and attention in fp64 (oracle side), written from their formulas.

* Rotary positions: channel pair (a, b) of a head at position p turns by p * theta_i, theta_i = base^(-2i/R);
  pairs are (i, i + R/2) or (2i, 2i + 1). The gradient is the transposed rotation.
* Attention: a softmax over the keys a row sees, row by row.
* An E4M3 cache row follows the tile rule of ``moe.quantize_tiles`` with one scale per row.
"""
from __future__ import annotations

import math

import numpy as np

from .e4m3 import e4m3_encode


def rope_frequencies(R, base=10000.0, scaling="plain", factor=1.0, orig_len=0.0, slow=1.0, fast=32.0):
    """theta_i of the R/2 pairs."""
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (R / (R - 2))
    theta = base ** (-2.0 * i / R)
    if scaling == "linear":
        return theta / factor
    if scaling == "parts":
        keep = np.clip((orig_len * theta / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return keep * theta + (1.0 - keep) * theta / factor
    return theta


def rope_table(R, n_positions, amplitude=1.0, **kw):
    """[n_positions, R/2, 2]: amplitude * (cos, sin) of p * theta_i."""
    a = np.arange(n_positions, dtype=np.float64)[:, None] * rope_frequencies(R, **kw)
    return amplitude * np.stack([np.cos(a), np.sin(a)], -1)


def rotate(x, cs, interleaved, transpose=False):
    """x [T, H, D] with its leading channels turned by cs [T, R/2, 2]; (result, sum of the magnitudes added)."""
    x = np.asarray(x, dtype=np.float64)
    half = cs.shape[1]
    out, mag = x.copy(), np.abs(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cs[:, i, 0][:, None], cs[:, i, 1][:, None]
        if transpose:
            s = -s
        xa, xb = x[:, :, a], x[:, :, b]
        out[:, :, a], out[:, :, b] = xa * c - xb * s, xb * c + xa * s
        mag[:, :, a], mag[:, :, b] = np.abs(xa * c) + np.abs(xb * s), np.abs(xb * c) + np.abs(xa * s)
    return out, mag


def quantize_rows(x):
    """E4M3 codes and the scale of every row of x [..., D]: amax/448 (1 for a zero row)."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.max(np.abs(x), axis=-1)
    some = amax > 0
    scale = np.where(some, amax / 448.0, 1.0)
    return e4m3_encode(np.clip(x / scale[..., None], -448, 448)), scale


def attend(q, k, v, scale):
    """One row: q [D], k and v [n, D] (the keys it sees) -> (out [D], lse, sum_j p_j |v_j|); zeros and -inf if n = 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    if len(k) == 0:
        return np.zeros(v.shape[-1]), -math.inf, np.zeros(v.shape[-1])
    s = scale * (k @ q)
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    return p @ v / total, m + math.log(total), p @ np.abs(v) / total
