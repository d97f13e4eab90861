"""The attention half of a block: of a decode batch whose sequences continue one prompt (``PrefixAttention``), and of packed
training sequences with its gradient (``AttentionLayer``).

``PrefixAttention`` owns the paged cache, its page tables, the rotary table and the workspace, and composes

  moe_kv_append (rotate q and k, write k and v to their pages) -> moe_prefix_attention

for the shared prompt (``prefill``) and for one or a few new tokens of every sequence (``step``). Both run on
the current stream with no host synchronisation. A call that raises leaves the prompt's and the sequences' lengths as they were.
A step recorded into a graph keeps the prompt's length and the workspace of its recording, and its replays are not counted
against the capacity: record again after a prefill or a step of more tokens.
"""
from __future__ import annotations

import math
from typing import Dict, Optional

import torch

from . import binding as B


class PrefixAttention:
    """Attention state of `batch` sequences on the current device.

    The prompt has room for `prefix_capacity` tokens, every sequence for `own_capacity` of its own; a capacity far above what
    the sequences come to use slows each step down (the split of the work expects half of it). `dtype` is that of q, k
    and v: torch.float32 or torch.bfloat16. `cache` is what the keys and values are kept in: None or `dtype` itself, or, for
    bfloat16, "e4m3": 8-bit codes with one scale per token and head. rot_dim leading channels of a head are rotated
    (default: all); `scaling` holds moe_rope_table's scaling arguments. scale defaults to 1 / sqrt(head_dim).
    """

    def __init__(self, batch: int, q_heads: int, kv_heads: int, head_dim: int, prefix_capacity: int, own_capacity: int,
                 dtype=torch.bfloat16, cache=None, page_size: int = 64, rot_dim: Optional[int] = None,
                 layout: int = B.MOE_ROPE_HALF, base: float = 10000.0, scaling: Optional[dict] = None,
                 scale: Optional[float] = None, device="cuda"):
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dtype must be torch.float32 or torch.bfloat16 (got {dtype})")
        if cache not in (None, dtype, "e4m3"):
            raise ValueError(f"cache must be None, {dtype} or 'e4m3' (got {cache!r})")
        if cache == "e4m3" and dtype != torch.bfloat16:
            raise ValueError(f"an E4M3 cache is read by bfloat16 queries (dtype is {dtype})")
        rot_dim = head_dim if rot_dim is None else rot_dim
        if rot_dim <= 0 or rot_dim % 2 or rot_dim > head_dim:
            raise ValueError(f"rot_dim ({rot_dim}) must be positive, even and at most head_dim ({head_dim})")
        self.batch, self.page_size, self.layout, self.scale = batch, page_size, layout, scale
        self.dev, self.dtype = torch.device(device), dtype
        pre, own = -(-prefix_capacity // page_size), -(-own_capacity // page_size)
        self.prefix_capacity, self.own_capacity = pre * page_size, own * page_size
        n_pages = max(1, pre + batch * own)
        e4m3 = cache == "e4m3"
        kw = dict(dtype=torch.uint8 if e4m3 else dtype, device=self.dev)
        self.k_cache = torch.zeros((n_pages, kv_heads, page_size, head_dim), **kw)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.scales: Dict[str, torch.Tensor] = {}
        if e4m3:
            self.scales = {s: torch.ones((n_pages, kv_heads, page_size), dtype=torch.float32, device=self.dev)
                           for s in ("k_scale", "v_scale")}
        pages = torch.arange(n_pages, dtype=torch.int32, device=self.dev)
        self.prefix_pages = pages[:pre]
        self.page_table = pages[pre:pre + batch * own].view(batch, own)
        self.table = B.moe_rope_table(rot_dim, self.prefix_capacity + self.own_capacity, base,
                                      device=self.dev, **(scaling or {}))
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.lens = torch.zeros(batch, dtype=torch.int32, device=self.dev)      # own tokens of each sequence
        self.prefix_len = 0
        self._taken = 0                  # the most own tokens any sequence can have, kept on the host
        self._ws = torch.empty(256, dtype=torch.uint8, device=self.dev)

    def _workspace(self, batch, q_len, prefix_len, cols):
        n = B.moe_prefix_attention_workspace_bytes(self.k_cache, batch, q_len, self.q_heads, prefix_len, cols)
        if n > self._ws.numel():
            self._ws = torch.empty(n, dtype=torch.uint8, device=self.dev)
        return self._ws

    def _check(self, q, k, v, n):
        """Raises unless q, k and v are n tokens of this state's heads and dtype."""
        for name, x, h in (("q", q, self.q_heads), ("k", k, self.kv_heads), ("v", v, self.kv_heads)):
            if x.shape != (n, h, self.head_dim):
                raise ValueError(f"{name} must be [{n}, {h}, {self.head_dim}] (got {tuple(x.shape)})")
            if x.dtype != self.dtype:
                raise TypeError(f"{name} is {x.dtype}, the state {self.dtype}")

    def _append(self, q, k, v, slots, positions):
        q_rot = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        B.moe_kv_append(k, v, slots, self.k_cache, self.v_cache, positions=positions, table=self.table,
                        layout=self.layout, q=q, q_out=q_rot, **self.scales)
        return q_rot

    def prefill(self, q, k, v) -> torch.Tensor:
        """The next n tokens of the prompt (q [n, q_heads, D]; k, v [n, kv_heads, D], not rotated): appends them and
        returns their causal attention over the prompt so far. All but the last call end on a page's end."""
        n, p = q.shape[0], self.prefix_len
        self._check(q, k, v, n)
        if p % self.page_size:
            raise ValueError(f"the prompt ends inside a page ({p} tokens of pages of {self.page_size}): it cannot go on")
        if p + n > self.prefix_capacity:
            raise ValueError(f"{p + n} prompt tokens, room for {self.prefix_capacity}")
        if self._taken:
            raise ValueError("the sequences have tokens of their own after the prompt; reset() first")
        at = torch.arange(p, p + n, dtype=torch.int32, device=self.dev)
        slots = self.prefix_pages[(at // self.page_size).long()] * self.page_size + at % self.page_size
        q_rot = self._append(q, k, v, slots.to(torch.int32), at)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if n:
            first, cols = p // self.page_size, -(-n // self.page_size)
            B.moe_prefix_attention(q_rot, self.k_cache, self.v_cache, self.prefix_pages, p,
                                   self.prefix_pages[first:first + cols].view(1, cols), torch.full_like(self.lens[:1], n),
                                   out, q_len=n, scale=self.scale, workspace=self._workspace(1, n, p, cols), **self.scales)
        self.prefix_len = p + n
        return out

    def step(self, q, k, v, q_len: int = 1) -> torch.Tensor:
        """q_len new tokens of every sequence (q [batch * q_len, q_heads, D], sequence by sequence): appends them and
        returns their attention over the prompt and their sequence's own tokens up to themselves."""
        if q_len < 1:
            raise ValueError(f"q_len ({q_len}) must be at least 1")
        self._check(q, k, v, self.batch * q_len)
        if self._taken + q_len > self.own_capacity:
            raise ValueError(f"{self._taken + q_len} own tokens, room for {self.own_capacity}")
        at = self.lens[:, None] + torch.arange(q_len, dtype=torch.int32, device=self.dev)
        cols = self.page_table.shape[1]
        page = self.page_table.gather(1, (at // self.page_size).clamp(max=cols - 1).long())
        slots = torch.where(at < self.own_capacity, page * self.page_size + at % self.page_size, -1).to(torch.int32).flatten()
        q_rot = self._append(q, k, v, slots, (at + self.prefix_len).flatten())
        self.lens += q_len
        try:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            B.moe_prefix_attention(q_rot, self.k_cache, self.v_cache, self.prefix_pages, self.prefix_len, self.page_table,
                                   self.lens, out, q_len=q_len, scale=self.scale,
                                   workspace=self._workspace(self.batch, q_len, self.prefix_len, cols), **self.scales)
        except Exception:
            self.lens -= q_len      # the appended rows lie past every length again
            raise
        self._taken += q_len
        return out

    def reset(self, keep_prompt: bool = True) -> None:
        """Forget the sequences' own tokens (and the prompt)."""
        self.lens.zero_()
        self._taken = 0
        if not keep_prompt:
            self.prefix_len = 0


class AttentionLayer:
    """x + attention(norm(x)) of packed sequences and its gradient: the half of a block in front of MoELayer(train=True).

    Layer norm, rotary positions and causal attention, and their gradients, run in libmoe (moe_layer_norm, moe_rotary,
    moe_causal_attention); the projections around them are plain matrix products. Both directions run on the current stream with no
    host synchronisation, and outside autograd: their results belong to no graph, whatever requires grad, and gradients come from
    backward() alone.

    weights: w_qkv [(q_heads + 2 kv_heads) * head_dim, d] (the rows of q's heads, then k's, then v's) and w_out
    [d, q_heads * head_dim] in the dtype of x, fp32 or bf16; norm_weight and norm_bias [d] fp32, or absent (1, 0). rot_dim leading
    channels of a head are rotated (default: all); `scaling` holds moe_rope_table's scaling arguments; scale defaults to
    1 / sqrt(head_dim). max_len: the longest sequence; positions from it on lie past the rotary table.
    """

    def __init__(self, weights: Dict[str, torch.Tensor], q_heads: int, kv_heads: int, head_dim: int, max_len: int,
                 rot_dim: Optional[int] = None, layout: int = B.MOE_ROPE_HALF, base: float = 10000.0,
                 scaling: Optional[dict] = None, scale: Optional[float] = None, eps: float = 1e-5, device="cuda"):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.layout, self.scale, self.eps, self.max_len = layout, scale, eps, max_len
        self.dev = torch.device(device)
        self.w_qkv, self.w_out = (weights[n].to(self.dev).contiguous() for n in ("w_qkv", "w_out"))
        self.dtype, self.d = self.w_qkv.dtype, self.w_qkv.shape[1]
        if self.dtype not in (torch.float32, torch.bfloat16) or self.w_out.dtype != self.dtype:
            raise TypeError("w_qkv and w_out must be both torch.float32 or both torch.bfloat16 "
                            f"(got {self.dtype}, {self.w_out.dtype})")
        rows = (q_heads + 2 * kv_heads) * head_dim
        if self.w_qkv.shape != (rows, self.d) or self.w_out.shape != (self.d, q_heads * head_dim):
            raise ValueError(f"w_qkv must be [{rows}, d] and w_out [d, {q_heads * head_dim}] "
                             f"(got {tuple(self.w_qkv.shape)}, {tuple(self.w_out.shape)})")
        vec = {n: weights.get(n) for n in ("norm_weight", "norm_bias")}
        for n, t in vec.items():
            if t is not None and t.shape != (self.d,):
                raise ValueError(f"{n} must be [{self.d}] (got {tuple(t.shape)})")
        self.norm_weight, self.norm_bias = (None if t is None else t.to(self.dev, torch.float32).contiguous() for t in vec.values())
        table = B.moe_rope_table(head_dim if rot_dim is None else rot_dim, max_len, base, device=self.dev, **(scaling or {}))
        self.table = torch.cat([table, torch.full_like(table[:1], math.nan)])      # the last one for places past it
        self.grads: Dict[str, torch.Tensor] = {}
        self._saved = None

    def positions(self, T: int, seq_start: torch.Tensor) -> torch.Tensor:
        """Place of each of T rows in its sequence, -1 outside all sequences."""
        at = torch.arange(T, dtype=torch.int32, device=self.dev)
        seq = torch.searchsorted(seq_start, at, right=True) - 1
        inside = (seq >= 0) & (seq < seq_start.numel() - 1)
        return torch.where(inside, at - seq_start[seq.clamp(min=0)], -1).to(torch.int32)

    def _heads(self, x):
        """q, k and v of [T, (q_heads + 2 kv_heads) * head_dim], where they lie."""
        heads = [self.q_heads, self.kv_heads, self.kv_heads]
        return x.view(len(x), sum(heads), self.head_dim).split(heads, 1)

    @staticmethod
    def _weight_grad(dy, x):
        """dy^T x in fp32."""
        return dy.t() @ x if x.dtype == torch.float32 else torch.mm(dy.t(), x, out_dtype=torch.float32)

    @torch.no_grad()
    def forward(self, x: torch.Tensor, seq_start: torch.Tensor, positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [T, d]; sequence s is rows seq_start[s] .. seq_start[s + 1] - 1 (int32 [n + 1] on the GPU; rows outside come back as
        they are, whatever they hold, and take no part in the gradients of the weights). positions: int32 [T] in the rotary table
        (default: the places in the sequences); a negative one leaves its token unrotated, and a token past the table (in a
        sequence longer than max_len) comes out as NaN, with all that see it."""
        if x.dim() != 2 or x.shape[1] != self.d or x.dtype != self.dtype:
            raise ValueError(f"x must be [tokens, {self.d}] in {self.dtype} (got {tuple(x.shape)}, {x.dtype})")
        T = len(x)
        f32 = dict(dtype=torch.float32, device=self.dev)
        seq_start = seq_start.clone()      # backward's own: the caller may fill theirs again
        if positions is None:
            positions = self.positions(T, seq_start)
            inside = positions >= 0
            if T > self.max_len:
                positions.clamp_(max=self.max_len)
        else:
            if positions.numel() < T:
                raise ValueError(f"positions has {positions.numel()} elements, needs {T}")
            positions, at = positions.flatten()[:T].clamp(max=self.max_len), torch.arange(T, device=self.dev)
            inside = (at >= seq_start[0]) & (at < seq_start[-1])
        rows = torch.where(inside[:, None], x, 0)      # weight gradients sum over all of them
        n, mean, rstd = torch.empty((T, self.d), dtype=self.dtype, device=self.dev), torch.empty(T, **f32), torch.empty(T, **f32)
        B.moe_layer_norm(rows, self.norm_weight, self.norm_bias, n, eps=self.eps, mean=mean, rstd=rstd)
        if self.eps < torch.finfo(torch.float32).tiny:      # rows of zeros have no norm: 0 times infinity
            n, rstd = torch.where(inside[:, None], n, 0), torch.where(inside, rstd, 0)
        qkv = n @ self.w_qkv.t()
        q, k, v = self._heads(qkv)
        B.moe_rotary(q, k, positions, self.table, q, k, layout=self.layout)
        a = torch.zeros((T, self.q_heads, self.head_dim), dtype=self.dtype, device=self.dev)
        lse = torch.empty((T, self.q_heads), **f32)
        B.moe_causal_attention(q, k, v, seq_start, a, scale=self.scale, lse=lse)
        self._saved = (rows, n, mean, rstd, qkv, a, lse, seq_start, positions, inside)
        return torch.addmm(x, a.flatten(1), self.w_out.t())

    @torch.no_grad()
    def backward(self, d_out: torch.Tensor) -> torch.Tensor:
        """The gradient of the last forward's x from that of its result, [T, d]; fills self.grads (w_qkv, w_out, norm_weight,
        norm_bias), all fp32."""
        if self._saved is None:
            raise RuntimeError("backward: run forward first")
        x, n, mean, rstd, qkv, a, lse, seq_start, positions, inside = self._saved
        if d_out.shape != x.shape or d_out.dtype != x.dtype:
            raise ValueError(f"d_out must be {tuple(x.shape)} in {x.dtype} (got {tuple(d_out.shape)}, {d_out.dtype})")
        d_out = d_out.contiguous()
        d_rows = torch.where(inside[:, None], d_out, 0)
        da = (d_rows @ self.w_out).view(a.shape)
        dqkv = torch.zeros_like(qkv)
        (q, k, v), (dq, dk, dv) = self._heads(qkv), self._heads(dqkv)
        B.moe_causal_attention_backward(da, q, k, v, a, lse, seq_start, dq, dk, dv, scale=self.scale)
        B.moe_rotary_backward(dq, dk, positions, self.table, dq, dk, layout=self.layout)
        dn, dx = dqkv @ self.w_qkv, torch.empty_like(n)
        dw, db = (torch.empty(self.d, dtype=torch.float32, device=self.dev) for _ in range(2))
        B.moe_layer_norm_backward(dn, x, self.norm_weight, mean, rstd, dx, dw, db, d_residual=d_out)
        self.grads = {"w_qkv": self._weight_grad(dqkv, n), "w_out": self._weight_grad(d_rows, a.flatten(1)), "norm_weight": dw,
                      "norm_bias": db}
        return dx
