"""PrefixAttention on bf16 and E4M3 caches: a prompt in chunks, then steps, against the oracle on the rows that the cache holds.

The rows are looked up where the state's page tables put them, compared with the rotated inputs (half a unit of the
stored type; an E4M3 row's scale to fp32 rounding), and read by the oracle as they are stored. The rotated queries come from
a second append to a scratch cache. Tolerances of the attention as derived in test_gpu_heads.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV
from mixture_experts_layer_gate_amd import MOE_ROPE_INTERLEAVED, PrefixAttention
from mixture_experts_layer_gate_amd import binding as B
from test_gpu_heads import U16, U32, _close, _np

pytestmark = pytest.mark.gpu


def _stored(att, side, slots):
    """Cache rows [n, kv_heads, D] in fp64."""
    p, r = slots // att.page_size, slots % att.page_size
    x = (att.k_cache if side == "k" else att.v_cache)[p, :, r]
    if not att.scales:
        return _np(x)
    return _np(x.view(torch.float8_e4m3fn).float()) * _np(att.scales[side + "_scale"][p, :, r])[..., None]


def _rotated_queries(att, q, k, v, positions):
    kc, vc = (torch.zeros((len(q), k.shape[1], 1, q.shape[2]), dtype=q.dtype, device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    B.moe_kv_append(k, v, torch.arange(len(q), dtype=torch.int32, device=DEV), kc, vc, positions=positions, table=att.table,
                    layout=att.layout, q=q, q_out=out)
    return _np(out)


@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Bn,hq,hk,D,R,page,chunks,steps", [
    (3, 4, 2, 64, 64, 16, (32, 41), (1, 3, 1)),
    (2, 14, 2, 128, 64, 64, (256, 192, 100), (1, 1, 9)),
    (5, 6, 1, 80, 40, 32, (300,), (2, 17, 40)),
])
def test_prompt_and_steps(cache, interleaved, Bn, hq, hk, D, R, page, chunks, steps):
    g = torch.Generator(device=DEV).manual_seed(Bn * D)
    att = PrefixAttention(Bn, hq, hk, D, sum(chunks), sum(steps), cache=cache, page_size=page, rot_dim=R,
                          layout=MOE_ROPE_INTERLEAVED if interleaved else B.MOE_ROPE_HALF)
    cs = oracle.rope_table(R, att.table.shape[0])
    new = lambda n: [torch.randn((n, h, D), generator=g, device=DEV).bfloat16() for h in (hq, hk, hk)]
    pre_slots, own_slots = torch.empty(0, dtype=torch.long, device=DEV), torch.empty((Bn, 0), dtype=torch.long, device=DEV)

    def place(pages, at):
        return pages[at // page].long() * page + at % page

    def check_rows(slots, positions, k, v):
        for side, x, turn in (("k", k, True), ("v", v, False)):
            ref, mag = oracle.rotate(_np(x), cs[positions.cpu().numpy()] if turn else np.zeros((len(x), 0, 2)), interleaved)
            got = _stored(att, side, slots)
            if cache is None:
                _close(got, ref, 4 * U32 * mag + U16 * np.abs(ref) + 1e-37)
            else:
                step = np.abs(ref).max(-1, keepdims=True) / 448.0
                _close(got, ref, np.maximum(np.abs(ref) * 2.0 ** -4, step * 2.0 ** -10) + step * 448 * 10 * U32)

    def check_out(out, q, seen):
        """Row t of out: q[t] on the slots seen(t)."""
        for t in sorted({0, len(q) - 1, *np.random.default_rng(len(q)).integers(0, len(q), 12).tolist()}):
            kk, vv = (_stored(att, s, seen(t)) for s in ("k", "v"))
            for h in (0, hq - 1):
                k, v, x = kk[:, h // (hq // hk)], vv[:, h // (hq // hk)], q[t, h]
                ref, _, mag = oracle.attend(x, k, v, D ** -0.5)
                delta = (D + 4) * 2 * U32 * D ** -0.5 * (np.abs(k) @ np.abs(x)).max()
                rel = 2 * delta + 2.0 ** -20 + 2 * U32 * len(k) + 2 * U16
                _close(_np(out)[t, h], ref, rel * mag + U16 * np.abs(ref), f"row {t} head {h}")

    for n in chunks:
        q, k, v = new(n)
        p0 = att.prefix_len
        out = att.prefill(q, k, v)
        at = torch.arange(p0, p0 + n, device=DEV)
        pre_slots = torch.cat([pre_slots, place(att.prefix_pages, at)])
        check_rows(pre_slots[p0:], at, k, v)
        check_out(out, _rotated_queries(att, q, k, v, at.int()), lambda t: pre_slots[:p0 + t + 1])
    for n in steps:
        q, k, v = new(Bn * n)
        o0 = own_slots.shape[1]
        out = att.step(q, k, v, n)
        at = torch.arange(o0, o0 + n, device=DEV)
        own_slots = torch.cat([own_slots, torch.stack([place(att.page_table[b], at) for b in range(Bn)])], 1)
        positions = (att.prefix_len + at).repeat(Bn)
        check_rows(own_slots[:, o0:].flatten(), positions, k, v)
        check_out(out, _rotated_queries(att, q, k, v, positions.int()),
                  lambda t: torch.cat([pre_slots, own_slots[t // n, :o0 + t % n + 1]]))
    assert att.lens.tolist() == [sum(steps)] * Bn
