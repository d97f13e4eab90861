"""What PrefixAttention refuses, and that a refusal leaves its state as it was (the library calls are replaced: no GPU)."""
import pytest
import torch

from mixture_experts_layer_gate_amd import PrefixAttention
from mixture_experts_layer_gate_amd import binding as B


class Calls:
    """The library calls that PrefixAttention makes; `fail` names one that raises."""

    def __init__(self, monkeypatch):
        self.made, self.fail = [], None
        monkeypatch.setattr(B, "moe_rope_table", lambda R, n, *a, **kw: torch.zeros((n, R // 2, 2)))
        monkeypatch.setattr(B, "moe_prefix_attention_workspace_bytes", lambda *a: 256)
        for name in ("moe_kv_append", "moe_prefix_attention"):
            monkeypatch.setattr(B, name, lambda *a, _n=name, **kw: self._call(_n, a))

    def _call(self, name, args):
        if name == self.fail:
            raise B.MoEError(B.MOE_E_HIP, name)
        self.made.append(name)
        if name == "moe_prefix_attention":
            self.lens = args[6].clone()


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


def _attention(**kw):
    a = dict(batch=3, q_heads=4, kv_heads=2, head_dim=8, prefix_capacity=32, own_capacity=16, page_size=16, device="cpu")
    a.update(kw)
    return PrefixAttention(**a)


def _qkv(n, hq=4, hk=2, D=8, dt=torch.bfloat16):
    return torch.zeros((n, hq, D), dtype=dt), torch.zeros((n, hk, D), dtype=dt), torch.zeros((n, hk, D), dtype=dt)


def _state(att):
    return att.lens.tolist(), att.prefix_len, att._taken


def _wrong(n):
    """Tensors that are not q, k and v of one number of tokens, of 4 and 2 heads of 8 bf16 channels."""
    q, k, v = _qkv(n)
    yield _qkv(n, D=16)
    yield _qkv(n, dt=torch.float32)
    yield _qkv(n, hq=2)
    yield q[:-1], k, v
    yield q, k[:-1], v
    yield q, k, v[:-1]
    yield q, k[:, :1], v
    yield q, k, v.float()
    yield q[:, 0], k, v


@pytest.mark.parametrize("q_len", [1, 2])
def test_step_refuses_before_it_changes_anything(calls, q_len):
    att = _attention()
    att.prefill(*_qkv(7))
    att.step(*_qkv(3))
    calls.made.clear()
    before = _state(att)
    assert before == ([1, 1, 1], 7, 1)
    for bad in [_qkv(3 * q_len - 1), _qkv(3 * q_len + 1), *_wrong(3 * q_len)]:
        with pytest.raises((ValueError, TypeError)):
            att.step(*bad, q_len=q_len)
        assert not calls.made and _state(att) == before
    for n in (0, -1):
        with pytest.raises(ValueError):
            att.step(*_qkv(3), q_len=n)
        assert not calls.made and _state(att) == before
    with pytest.raises(ValueError, match="room for 16"):
        att.step(*_qkv(48), q_len=16)
    assert not calls.made and _state(att) == before
    att.step(*_qkv(3 * q_len), q_len=q_len)
    assert _state(att) == ([1 + q_len] * 3, 7, 1 + q_len) and calls.lens.tolist() == [1 + q_len] * 3


@pytest.mark.parametrize("fail", ["moe_kv_append", "moe_prefix_attention"])
def test_a_call_that_fails_leaves_the_lengths(calls, fail):
    att = _attention()
    att.prefill(*_qkv(16))
    att.step(*_qkv(3))
    before = _state(att)
    calls.fail = fail
    with pytest.raises(B.MoEError):
        att.step(*_qkv(3))
    assert _state(att) == before
    calls.fail = None
    att.step(*_qkv(3))
    assert _state(att) == ([2] * 3, 16, 2)


@pytest.mark.parametrize("fail", [None, "moe_kv_append", "moe_prefix_attention"])
def test_prefill_refuses_before_it_changes_anything(calls, fail):
    att = _attention()
    att.prefill(*_qkv(16))
    calls.made.clear()
    before = _state(att)
    for bad in _wrong(5):
        with pytest.raises((ValueError, TypeError)):
            att.prefill(*bad)
        assert not calls.made and _state(att) == before
    if fail:
        calls.fail = fail
        with pytest.raises(B.MoEError):
            att.prefill(*_qkv(5))
        assert _state(att) == before
        calls.fail = None
    att.prefill(*_qkv(5))
    assert _state(att) == ([0] * 3, 21, 0)


@pytest.mark.parametrize("kw", [
    dict(cache="fp8"), dict(cache="bf16"), dict(cache=torch.float8_e4m3fn), dict(cache=torch.float32),
    dict(cache=torch.bfloat16, dtype=torch.float32), dict(cache="e4m3", dtype=torch.float32), dict(cache=torch.uint8),
    dict(dtype=torch.float16), dict(dtype=torch.uint8), dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=5), dict(rot_dim=10),
])
def test_arguments_that_would_be_misread(calls, kw):
    """A cache that is neither the activations' type nor "e4m3", fp32 queries on 8-bit codes, a rotation of no channels."""
    with pytest.raises((ValueError, TypeError)):
        _attention(**kw)


@pytest.mark.parametrize("kw,cache,rot", [
    (dict(), torch.bfloat16, 8), (dict(cache=torch.bfloat16), torch.bfloat16, 8), (dict(cache="e4m3"), torch.uint8, 8),
    (dict(dtype=torch.float32), torch.float32, 8), (dict(dtype=torch.float32, cache=torch.float32, rot_dim=4), torch.float32, 4),
])
def test_arguments_that_are_taken(calls, kw, cache, rot):
    att = _attention(**kw)
    assert att.k_cache.dtype == att.v_cache.dtype == cache and bool(att.scales) == (cache == torch.uint8)
    assert att.table.shape[1] == rot // 2
