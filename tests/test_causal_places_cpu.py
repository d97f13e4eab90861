"""Where the results of causal attention may lie, on the host before any launch (runs without a GPU)."""
import pytest

from mixture_experts_layer_gate_amd import binding as B
from test_training_abi_cpu import P, _attention, _msg


@pytest.mark.parametrize("kw", [dict(q=dict(out=5 * P)), dict(q=dict(out=6 * P))])
def test_a_result_in_place_of_k_or_v_is_refused(kw):
    assert _attention(**kw) == B.MOE_E_INVALID and "takes the place of k or v" in _msg(), _msg()


def test_in_place_of_q_needs_its_strides():
    assert _attention(q=dict(out=4 * P, out_t=1024)) == B.MOE_E_INVALID and "in place" in _msg(), _msg()
    assert _attention(T=0, q=dict(out=5 * P)) == B.MOE_OK
