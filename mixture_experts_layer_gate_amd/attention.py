"""The attention of a decode batch whose sequences continue one prompt.

``PrefixAttention`` owns the paged cache, its page tables, the rotary table and the workspace, and composes

  moe_kv_append (rotate q and k, write k and v to their pages) -> moe_prefix_attention

for the shared prompt (``prefill``) and for one or a few new tokens of every sequence (``step``). Both run on
the current stream with no host synchronisation. A call that raises leaves the prompt's and the sequences' lengths as they were.
A step recorded into a graph keeps the prompt's length and the workspace of its recording, and its replays are not counted
against the capacity: record again after a prefill or a step of more tokens.
"""
from __future__ import annotations

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
