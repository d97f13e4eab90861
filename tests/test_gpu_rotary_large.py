"""Rotary positions of more head rows than one launch has threads for."""
import pytest
import torch

from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B

pytestmark = pytest.mark.gpu


def test_rotary_of_2_to_29_rows():
    """72 channels take 8 lanes of 16-byte pieces a row, 2^32 threads in all: the first and last rows against a small call."""
    T, R, D = 1 << 29, 16, 72
    g = torch.Generator(device=DEV).manual_seed(3)
    table = torch.randn((4, R // 2, 2), generator=g, device=DEV)
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    few = torch.randn((5, 1, D), generator=g, device=DEV).bfloat16()
    few_pos = torch.tensor([3, 1, 2, 3, 0], dtype=torch.int32, device=DEV)
    want = torch.empty_like(few)
    B.moe_rotary(few, None, few_pos, table, want)
    x = torch.zeros((T, 1, D), dtype=torch.bfloat16, device=DEV)
    positions = torch.zeros(T, dtype=torch.int32, device=DEV)
    x[at], positions[at] = few, few_pos
    B.moe_rotary(x, None, positions, table, x)
    got = x[at]
    del x, positions
    torch.cuda.empty_cache()
    assert torch.equal(got, want)
