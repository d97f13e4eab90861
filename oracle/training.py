"""Causal attention of packed sequences and the layer norm, with their gradients, in fp64 (oracle side), written from their
formulas; and how far an fp32 evaluation of them may be off.

u = 2^-24 is the half unit of fp32; a matrix unit may truncate, so a product or sum counts 2 u. w is the half unit of the weights
that enter a matrix product: 2^-8 where they are rounded to bf16, else 0. A score of D products is off by at most
e_s = (D + 4) 2u |scale| sum |q||k| (in any order), its exponential by a factor within e^(2 e_s) and 2^-20 more (argument and
result rounding at arguments down to -64; smaller weights do not matter more). A number below TINY = 2^-126 has no normal fp32
value: a weight, a product of one, or a term of a sum that comes to less may be taken for 0, which is off by TINY at most.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126


def sequence_of(T, seq_start):
    """(first token, end) of each row's sequence; (-1, -1) for rows outside all of them."""
    out = np.full((T, 2), -1, dtype=np.int64)
    for a, b in zip(seq_start[:-1], seq_start[1:]):
        out[a:b] = a, b
    return out


def _head(q, k, scale):
    n, D = q.shape
    s = scale * (q @ k.T)
    seen = np.tril(np.ones((n, n), dtype=bool))
    e_s = (D + 4) * 2 * U * abs(scale) * (np.abs(q) @ np.abs(k).T)
    return np.where(seen, s, -np.inf), np.where(seen, e_s, 0.0), seen


def causal_attention(q, k, v, seq_start, scale, w=0.0):
    """q [T, hq, D], k and v [T, hk, D] -> (out, lse, bound of out, bound of lse); rows outside all sequences hold NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, hq, D = q.shape
    G = hq // k.shape[1]
    out, tol = np.full((2, T, hq, D), np.nan)
    lse, ltol = np.full((2, T, hq), np.nan)
    for a, b in zip(seq_start[:-1], seq_start[1:]):
        for h in range(hq):
            if a == b:
                continue
            s, e_s, _ = _head(q[a:b, h], k[a:b, h // G], scale)
            m = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            total = p.sum(1, keepdims=True)
            z = (m + np.log(total))[:, 0] if np.isfinite(m).all() else np.log(np.where(total > 0, total, 1.0))[:, 0] + m[:, 0]
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
            n = np.arange(1, b - a + 1)[:, None]
            rel = 2 * np.max(e_s, 1, keepdims=True) + 2.0 ** -20 + 4 * U * n + w
            out[a:b, h], lse[a:b, h] = p @ v[a:b, h // G], z
            with np.errstate(invalid="ignore"):      # rows of -infinity alone have no bound
                tol[a:b, h] = rel * (p @ np.abs(v[a:b, h // G]))
            ltol[a:b, h] = (rel - w)[:, 0] + 4 * U * np.abs(z) + 4 * U
    return out, lse, tol, ltol


def causal_attention_grad(q, k, v, out, d_out, lse, seq_start, scale, w=0.0):
    """(dq, dk, dv, their bounds) from the out and lse that are given; rows outside all sequences hold NaN."""
    q, k, v, out, d_out, lse = (np.asarray(x, dtype=np.float64) for x in (q, k, v, out, d_out, lse))
    T, hq, D = q.shape
    hk = k.shape[1]
    G = hq // hk
    dq, tq = np.full((2, T, hq, D), np.nan)
    dk, tk, dv, tv = np.full((4, T, hk, D), np.nan)
    for a, b in zip(seq_start[:-1], seq_start[1:]):
        if a == b:
            continue
        dk[a:b] = tk[a:b] = dv[a:b] = tv[a:b] = 0.0
        n = (b - a) * G
        for h in range(hq):
            qq, kk, vv, g = q[a:b, h], k[a:b, h // G], v[a:b, h // G], d_out[a:b, h]
            s, e_s, seen = _head(qq, kk, scale)
            z = lse[a:b, h][:, None]
            p = np.where(seen & np.isfinite(z), np.exp(s - np.where(np.isfinite(z), z, 0.0)), 0.0)
            e_p = p * (2 * e_s + 2.0 ** -20 + 8 * U * (np.abs(z) * np.isfinite(z) + np.where(seen, np.abs(s), 0.0))) + TINY * seen
            delta = (g * out[a:b, h]).sum(1, keepdims=True)
            dp = np.where(seen, g @ vv.T, 0.0)
            e_dp = (D + 4) * 2 * U * (np.abs(g) @ np.abs(vv).T + (np.abs(g) * np.abs(out[a:b, h])).sum(1, keepdims=True))
            t = p * (dp - delta)
            e_t = e_p * np.abs(dp - delta) + (p + e_p) * e_dp + 4 * U * np.abs(t) + TINY * seen
            more = w + (n + 4) * 2 * U      # rounding of the weights, and the sum
            dq[a:b, h] = scale * (t @ kk)
            tq[a:b, h] = abs(scale) * ((e_t * (1 + more) + more * np.abs(t)) @ np.abs(kk)) + n * TINY
            dk[a:b, h // G] += scale * (t.T @ qq)
            tk[a:b, h // G] += abs(scale) * ((e_t * (1 + more) + more * np.abs(t)).T @ np.abs(qq)) + n * TINY
            dv[a:b, h // G] += p.T @ g
            tv[a:b, h // G] += (e_p * (1 + more) + more * p).T @ np.abs(g) + n * TINY
    return dq, dk, dv, tq, tk, tv


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd, their bounds) of rows x [R, d]. The mean of fp32 numbers is off by d 2u mean|x| at most before it is corrected
    by the mean of what is left, and by d 2u of that after it."""
    x, weight, bias = (np.asarray(t, dtype=np.float64) for t in (x, weight, bias))
    d = x.shape[1]
    mean = x.mean(1, keepdims=True)
    c = x - mean
    var = (c * c).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    h = c * rstd
    e_m = 2 * U * (np.abs(mean) + d * np.abs(c).mean(1, keepdims=True) + (d * 2 * U) * d * np.abs(x).mean(1, keepdims=True))
    e_c = 2 * U * (np.abs(c) + d * 2 * U * np.abs(x).mean(1, keepdims=True)) + 2 * U * d * np.abs(c).mean(1, keepdims=True)
    e_r = rstd * ((d + 8) * 2 * U)      # half the relative error of the variance, whose d terms are positive, and roundings
    y = h * weight + bias
    e_y = np.abs(weight) * (e_c * rstd + np.abs(c) * e_r + 4 * U * np.abs(h)) + 2 * U * np.abs(y)
    return y, mean[:, 0], rstd[:, 0], e_y, e_m[:, 0], e_r[:, 0]


def layer_norm_grad(dy, x, weight, mean, rstd, d_residual=None):
    """(dx, dweight, dbias, their bounds) from the mean and rstd that are given."""
    dy, x, weight, mean, rstd = (np.asarray(t, dtype=np.float64) for t in (dy, x, weight, mean, rstd))
    R, d = x.shape
    r = rstd[:, None]
    h = (x - mean[:, None]) * r
    g = dy * weight
    m0, m1 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx = r * (g - m0 - h * m1)
    e_h = 4 * U * np.abs(h)
    e0 = (d + 2) * 2 * U * np.abs(g).mean(1, keepdims=True)
    e1 = (d + 6) * 2 * U * np.abs(g * h).mean(1, keepdims=True)
    e = r * (2 * U * np.abs(g) + e0 + np.abs(h) * e1 + e_h * np.abs(m1) + 6 * U * (np.abs(g) + np.abs(m0) + np.abs(h * m1)))
    if d_residual is not None:
        d_residual = np.asarray(d_residual, dtype=np.float64)
        dx = dx + d_residual
        e = e + 2 * U * (np.abs(dx) + np.abs(d_residual))
    return (dx, (dy * h).sum(0), dy.sum(0), e, (R + 6) * 2 * U * np.abs(dy * h).sum(0), R * 2 * U * np.abs(dy).sum(0))
