"""Measured cases of the training half of a transformer block: causal attention over whole prompts of packed sequences with
its gradient, and the layer norm with its gradient.

With ``own`` false, ``run`` computes each operator from elementary torch operations in fp32; with ``own`` true it makes the
library's calls.

Head counts follow the hidden sizes of the synthetic workloads: 7168 = 56 heads of 128 (with 8 key/value heads), 2048 = 16
heads of 128 (4 key/value heads) or 32 of 64, and the tiny fp32 layer's 256 = 4 heads of 64.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: two short sequences; launch latency is all there is
        dict(name="attend_few_tokens", op="attend", n=2, lo=1, hi=40, hkv=4, G=4, D=128, act="bf16"),
        # one prompt of 8192 tokens
        dict(name="attend_prompt", op="attend", n=1, lo=8192, hi=8192, hkv=8, G=7, D=128, act="bf16"),
        # a training batch of sequences of very different lengths, packed
        dict(name="attend_packed", op="attend", n=12, lo=1, hi=4000, hkv=4, G=4, D=128, act="bf16"),
        # the tiny fp32 layer's heads
        dict(name="attend_f32", op="attend", n=16, lo=1, hi=300, hkv=4, G=1, D=64, act="f32"),
        # the smallest gradient
        dict(name="attend_grad_few_tokens", op="attend_grad", n=2, lo=16, hi=64, hkv=4, G=4, D=128, act="bf16"),
        # the gradient of one long sequence
        dict(name="attend_grad_prompt", op="attend_grad", n=1, lo=8192, hi=8192, hkv=4, G=4, D=128, act="bf16"),
        # many short sequences, heads of 64
        dict(name="attend_grad_packed", op="attend_grad", n=300, lo=1, hi=120, hkv=8, G=4, D=64, act="bf16"),
        # fp32 training, heads of 80 channels, a key/value head for each query head
        dict(name="attend_grad_f32", op="attend_grad", n=5, lo=100, hi=1000, hkv=12, G=1, D=80, act="f32"),
        # the norm of a few decoded tokens
        dict(name="norm_few_tokens", op="norm", rows=4, d=2048, act="bf16", wide=False),
        # the norm in front of the large layer
        dict(name="norm_prompt", op="norm", rows=8192, d=7168, act="bf16", wide=False),
        # its gradient, joined with the one that comes along the residual path
        dict(name="norm_grad", op="norm_grad", rows=8192, d=7168, act="bf16", wide=False, residual=True),
        # fp32 rows of odd length, slices of a wider buffer
        dict(name="norm_grad_f32_odd", op="norm_grad", rows=4093, d=1001, act="f32", wide=True, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST: dict = {}


def _sizes(case):
    """What a pass costs: bytes, operations, and the scores that the plain form holds at once."""
    w = work(case)
    if case["op"].startswith("attend"):
        w["scores"] = case["n"] * case["hkv"] * case["G"] * max(_lens(case)) ** 2
    return w


def _fits(case):
    """No more than the largest listed case of the operator."""
    if not _MOST:
        for c in listed():
            m = _MOST.setdefault(c["op"], {})
            for k, v in _sizes(c).items():
                m[k] = max(m.get(k, 0), v)
    return all(v <= _MOST[case["op"]][k] for k, v in _sizes(case).items())


def draw(rng):
    op = rng.choice(["attend", "attend", "attend_grad", "attend_grad", "norm", "norm_grad"])
    act = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op.startswith("attend"):
            hi = _log(rng, 24, 8192)
            c = dict(op=op, n=_log(rng, 1, 300), lo=rng.choice([1, 1, max(1, hi // 2), hi]), hi=hi,
                     hkv=rng.choice([1, 2, 4, 8, 12]), G=rng.choice([1, 2, 4, 5, 7, 8]),
                     D=rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256]), act=act)
        else:
            c = dict(op=op, rows=_log(rng, 1, 32768), d=rng.choice([_log(rng, 64, 16384), 256, 2048, 7168]), act=act,
                     wide=rng.random() < 0.3)
            if op == "norm_grad":
                c["residual"] = rng.random() < 0.5
        if _fits(c):
            return c


# ---------------------------------------------------------------- inputs

def _lens(c):
    """Lengths spread evenly over lo .. hi: the same set for every seed."""
    return [c["lo"] + int(((i + 1) * 0.6180339887498949) % 1.0 * (c["hi"] - c["lo"] + 1)) for i in range(c["n"])]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    dt = TORCH[c["act"]]
    if c["op"].startswith("norm"):
        R, d = c["rows"], c["d"]
        # activations of a residual stream: a few strong channels, rows of different sizes and offsets
        gain = 1.0 + 9.0 * (torch.rand((d,), generator=g, device=DEV) < 0.01).float()
        x = _randn(g, R, d) * gain * (0.5 + torch.rand((R, 1), generator=g, device=DEV)) + 0.2 * _randn(g, R, 1)
        if c["wide"]:                   # rows of a wider buffer
            w = torch.zeros((R, d + 64), dtype=dt, device=DEV)
            w[:, :d] = x
            s["x"] = w[:, :d]
        else:
            s["x"] = x.to(dt)
        s["weight"], s["bias"] = 1.0 + 0.1 * _randn(g, d), 0.1 * _randn(g, d)
        if c["op"] == "norm":
            s["y"] = torch.empty((R, d), dtype=dt, device=DEV)
            s["mean"], s["rstd"] = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
            return s
        x = s["x"].float()
        var, mean = torch.var_mean(x, 1, correction=0)
        s["mean"], s["rstd"] = mean, torch.rsqrt(var + EPS)
        s["dy"] = _randn(g, R, d).to(dt)
        s["d_residual"] = _randn(g, R, d).to(dt) if c["residual"] else None
        s["dx"] = torch.empty((R, d), dtype=dt, device=DEV)
        s["dweight"], s["dbias"] = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
        return s
    hq, hk, D = c["hkv"] * c["G"], c["hkv"], c["D"]
    lens = torch.tensor(_lens(c), device=DEV)[torch.randperm(c["n"], generator=g, device=DEV)]
    s["seq_start"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    T = sum(_lens(c))
    # q, k and v are slices of one projection's output; keys with a few strong channels, values with a small mean
    gain = 1.0 + (torch.rand((D,), generator=g, device=DEV) < 0.05).float()
    x = torch.empty((T, hq + 2 * hk, D), dtype=dt, device=DEV)
    s["q"], s["k"], s["v"] = x.split([hq, hk, hk], 1)
    s["q"][:] = _randn(g, T, hq, D)
    s["k"][:] = _randn(g, T, hk, D) * gain
    s["v"][:] = _randn(g, T, hk, D) + 0.1
    s["out"] = torch.empty((T, hq, D), dtype=dt, device=DEV)
    s["lse"] = torch.empty((T, hq), device=DEV)
    if c["op"] == "attend_grad":
        o, lse = _plain_attend(s)
        s["out"].copy_(o)
        s["lse"].copy_(lse)
        s["d_out"] = _randn(g, T, hq, D).to(dt)
        dx = torch.empty_like(x)
        s["dq"], s["dk"], s["dv"] = dx.split([hq, hk, hk], 1)
    return s


# ---------------------------------------------------------------- one pass

def _padded(s):
    """Tokens of every sequence in rows of the longest length: (token numbers [n, L], which of them exist)."""
    start = s["seq_start"].long()
    L = max(_lens(s["case"]))
    at = start[:-1, None] + torch.arange(L, device=start.device)
    return at.clamp(max=s["q"].shape[0] - 1), at < start[1:, None]


def _rows(x, at, G):
    """Head rows of x [T, h, D] as fp32 [h * G, n, L, D], a head for each of its G query heads."""
    return x.float()[at].permute(2, 0, 1, 3).repeat_interleave(G, 0)


def _weights(s, at, q, k):
    """exp(s - m), its sum and m; a row sees its own sequence's tokens up to itself."""
    L = at.shape[1]
    seen = torch.ones((L, L), dtype=torch.bool, device=at.device).tril()
    p = (q @ k.transpose(2, 3)).mul_(s["case"]["D"] ** -0.5).masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    return p, p.sum(-1, keepdim=True), m


def _plain_attend(s):
    G = s["case"]["G"]
    at, there = _padded(s)
    q, k, v = _rows(s["q"], at, 1), _rows(s["k"], at, G), _rows(s["v"], at, G)
    p, total, m = _weights(s, at, q, k)
    o = (p @ v / total).permute(1, 2, 0, 3)[there]
    return o.to(s["q"].dtype), (m + total.log())[..., 0].permute(1, 2, 0)[there]


def _plain_attend_grad(s):
    c = s["case"]
    G, hk, D = c["G"], c["hkv"], c["D"]
    at, there = _padded(s)
    q, k, v = _rows(s["q"], at, 1), _rows(s["k"], at, G), _rows(s["v"], at, G)
    do = _rows(s["d_out"], at, 1) * there[..., None]
    p, total, _ = _weights(s, at, q, k)
    p /= total
    dv = p.transpose(2, 3) @ do
    ds = do @ v.transpose(2, 3)
    ds = ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    back = lambda x: x.permute(1, 2, 0, 3)[there].to(s["q"].dtype)          # noqa: E731
    group = lambda x: x.view(hk, G, *x.shape[1:]).sum(1)                    # noqa: E731
    return {"dq": back(dq), "dk": back(group(dk)), "dv": back(group(dv))}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    return {"y": (x * rstd * s["weight"] + s["bias"]).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"]
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["d_residual"] is not None:
        dx = dx + s["d_residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "attend":
            o, lse = _plain_attend(s)
            return {"out": o, "lse": lse}
        return {"attend_grad": _plain_attend_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[op](s)
    import mixture_experts_layer_gate_amd as moe
    if op == "attend":
        moe.moe_causal_attention(s["q"], s["k"], s["v"], s["seq_start"], s["out"], lse=s["lse"])
        return {n: s[n] for n in ("out", "lse")}
    if op == "attend_grad":
        moe.moe_causal_attention_backward(s["d_out"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["seq_start"], s["dq"],
                                          s["dk"], s["dv"])
        return {n: s[n] for n in ("dq", "dk", "dv")}
    if op == "norm":
        moe.moe_layer_norm(s["x"], s["weight"], s["bias"], s["y"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
        return {n: s[n] for n in ("y", "mean", "rstd")}
    moe.moe_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                d_residual=s["d_residual"])
    return {n: s[n] for n in ("dx", "dweight", "dbias")}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    e = 4 if c["act"] == "f32" else 2
    if c["op"].startswith("norm"):
        R, d = c["rows"], c["d"]
        if c["op"] == "norm":
            return {"bytes": 2 * e * R * d + 8 * R + 8 * d, "flops": 8 * R * d}
        return {"bytes": (3 + c["residual"]) * e * R * d + 8 * R + 12 * d, "flops": 14 * R * d}
    lens = _lens(c)
    T, hq, hk, D = sum(lens), c["hkv"] * c["G"], c["hkv"], c["D"]
    pairs = sum(n * (n + 1) // 2 for n in lens) * hq
    more = 4 * T * hq + 4 * (c["n"] + 1)
    if c["op"] == "attend":
        return {"bytes": 2 * e * T * D * (hq + hk) + more, "flops": 4 * D * pairs}
    return {"bytes": 4 * e * T * D * (hq + hk) + more, "flops": 10 * D * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s, c):
    x, w = s["x"].double(), s["weight"].double()
    if c["op"] == "norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), "mean": mean, "rstd": rstd}
    mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    h, dy = (x - mean) * rstd, s["dy"].double()
    g = dy * w
    n = x.shape[1]
    dx = rstd * g - rstd / n * (g.sum(1, keepdim=True) + h * torch.linalg.vecdot(g, h)[:, None])
    if s["d_residual"] is not None:
        dx += s["d_residual"].double()
    return {"dx": dx, "dweight": torch.linalg.vecdot(dy, h, dim=0), "dbias": dy.sum(0)}


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(s, c)
    G, D = c["G"], c["D"]
    names = ("out", "lse") if c["op"] == "attend" else ("dq", "dk", "dv")
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in names}
    start = s["seq_start"].tolist()
    for a, b in zip(start[:-1], start[1:]):
        future = torch.triu(torch.full((b - a, b - a), -math.inf, dtype=torch.float64, device=DEV), 1)
        for h in range(c["hkv"] * G):
            q, k, v = s["q"][a:b, h].double(), s["k"][a:b, h // G].double(), s["v"][a:b, h // G].double()
            score = torch.addmm(future, q, k.t(), alpha=1.0 / math.sqrt(D))
            w = torch.softmax(score, 1)
            if c["op"] == "attend":
                out["out"][a:b, h] = w @ v
                out["lse"][a:b, h] = torch.logsumexp(score, 1)
                continue
            do = s["d_out"][a:b, h].double()
            dw = do @ v.t()
            dscore = w * (dw - torch.linalg.vecdot(w, dw)[:, None]) / math.sqrt(D)
            out["dq"][a:b, h] = dscore @ k
            out["dk"][a:b, h // G] += dscore.t() @ q
            out["dv"][a:b, h // G] += w.t() @ do
    return out
