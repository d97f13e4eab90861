"""Sizes that the C calls' 32-bit arguments do not hold are refused by the binding, not cut off (runs without a GPU)."""
import pytest
import torch

from mixture_experts_layer_gate_amd import binding as B

BIG = 2 ** 31


def _heads(T, h, D):
    return torch.empty(1, 1, D).expand(T, h, D)


@pytest.mark.parametrize("T", [BIG, 2 ** 32, 2 ** 32 + 5])
def test_tokens(T):
    q, k, starts = _heads(T, 2, 64), _heads(T, 1, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_causal_attention(q, k, k, starts, q)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_causal_attention_backward(q, q, k, k, q, torch.empty(1).expand(2 * T), starts, q, k, k)
    assert B.moe_causal_attention_backward_workspace_bytes(T, 64, 2, 1) == 0


@pytest.mark.parametrize("hq,hk", [(2 ** 32 + 2, 2), (2 ** 32 + 2, 2 ** 31 + 1)])
def test_heads(hq, hk):
    q, k, starts = _heads(1, hq, 8), _heads(1, hk, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_causal_attention(q, k, k, starts, q)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_causal_attention_backward(q, q, k, k, q, torch.empty(1).expand(hq), starts, q, k, k)


def test_sequences():
    q = torch.zeros((4, 1, 8))
    starts = torch.zeros(1, dtype=torch.int32).expand(2 ** 32 + 3)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_causal_attention(q, q, q, starts, q)


@pytest.mark.parametrize("d", [BIG, 2 ** 32 + 8])
def test_channels_of_the_norm(d):
    x = torch.empty(1, 1).expand(1, d)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_layer_norm(x, None, None, x)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_layer_norm_backward(x, x, None, torch.zeros(1), torch.zeros(1), x)
    assert B.moe_layer_norm_backward_workspace_bytes(1, d) == 0


@pytest.mark.parametrize("T", [BIG, 2 ** 32 + 5])
def test_tokens_of_the_rotary_and_append_calls(T):
    x, table = _heads(T, 1, 8), torch.zeros((4, 4, 2))
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_rotary(x, None, torch.zeros(1, dtype=torch.int32), table, x)
    with pytest.raises(ValueError, match="2\\^31"):
        B.moe_kv_append(x, x, torch.zeros(1, dtype=torch.int32), torch.zeros((2, 1, 4, 8)), torch.zeros((2, 1, 4, 8)))
