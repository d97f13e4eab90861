"""Sizes and arguments of the attention half that are refused before they reach a kernel (runs without a GPU)."""
import os
import subprocess
import sys

import pytest
import torch

from mixture_experts_layer_gate_amd import binding as B
from test_heads_abi_cpu import P, _cache, _msg, _rows

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("batch,q_len,heads", [
    (1 << 30, 1 << 30, 16),     # 2^64 rows: 0 in 64 bits
    (1 << 30, 1 << 30, 12),     # 3 * 2^62
    (1 << 16, 1 << 16, 4),      # batch * q_len: 0 in 32 bits
])
def test_row_counts_past_any_integer(batch, q_len, heads):
    """In a process of its own: a count that wraps to 0 ends in a division by it."""
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]\n"
            "from test_heads_abi_cpu import B, P, _cache, _rows\n"
            f"b, s, h = {batch}, {q_len}, {heads}\n"
            "print(B.lib().moe_prefix_attention_workspace_bytes(_cache(), b, s, h, 20, 3),\n"
            "      B.lib().moe_prefix_attention(_cache(), B.MOE_BF16, b, s, _rows(heads=h), 0.1, P, 20, P, 3, P, None, None, 0,\n"
            "                                   None))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split() == ["0", str(B.MOE_E_UNSUPPORTED)]


def test_rope_table_takes_only_memory_of_the_current_gpu():
    """Like its siblings: the address of another memory never reaches the kernel."""
    with pytest.raises(ValueError, match="current GPU"):
        B.moe_rope_table(64, 16, out=torch.zeros((16, 32, 2)))
    with pytest.raises(ValueError, match="current GPU"):
        B.moe_rope_table(64, 16, device="cpu")


@pytest.mark.parametrize("cache,kw", [
    (dict(head_dim=100), {}), (dict(head_dim=264), {}), (dict(page_size=24), {}), (dict(page_size=1 << 17), {}),
    (dict(n_pages=1 << 27), {}), (dict(dtype=B.MOE_F4E2M1), {}), (dict(n_pages=0), {}),
    (dict(page_size=1 << 16, kv_heads=256), dict(heads=256)), ({}, dict(heads=6)), ({}, dict(heads=0)),
    ({}, dict(prefix=(1 << 30) + 1)), ({}, dict(cols=1 << 28)), ({}, dict(prefix=-1)), ({}, dict(batch=1 << 30)),
])
def test_workspace_of_every_refused_size_is_zero(cache, kw):
    """0 exactly where the call itself refuses the sizes."""
    a = dict(batch=4, q_len=1, heads=8, prefix=1000, cols=3)
    size = B.lib().moe_prefix_attention_workspace_bytes
    assert size(_cache(k=None, v=None), *a.values()) > 0      # from sizes alone
    a.update(kw)
    assert size(_cache(**cache), *a.values()) == 0 and _msg()
    st = B.lib().moe_prefix_attention(_cache(**cache), B.MOE_BF16, a["batch"], a["q_len"], _rows(heads=a["heads"]), 0.1, P,
                                      a["prefix"], P, a["cols"], P, None, None, 0, None)
    assert st in (B.MOE_E_INVALID, B.MOE_E_UNSUPPORTED), _msg()


@pytest.mark.parametrize("batch,q_len", [(0, 1), (4, 0)])
def test_workspace_of_no_rows(batch, q_len):
    assert B.lib().moe_prefix_attention_workspace_bytes(_cache(), batch, q_len, 8, 1000, 3) > 0


def test_rope_table_refuses_a_base_that_its_factor_carries_out_of_range():
    """base * factor^(R / (R - 2)) past fp64 would fill the table with NaN."""
    with pytest.raises(B.MoEError, match="base"):
        st = B.lib().moe_rope_table(4, 16, 1e299, B.MOE_ROPE_BASE, 1e29, 0.0, 1.0, 32.0, 1.0, P, None)
        B._check(st)
