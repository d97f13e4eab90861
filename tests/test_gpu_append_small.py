"""E4M3 cache rows of magnitudes around the smallest normal fp32 number."""
import pytest
import torch

from gpu_common import DEV
from mixture_experts_layer_gate_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 67])      # whole 16-byte pieces of a row; element by element
def test_rows_of_tiny_values_are_stored_without_nan(dt, D):
    """448 / amax passes fp32 below amax = 448 / 2^128 = 1.32e-36. What such a row stands for is its values to within
    amax, and its zeros are zeros; above, half a step of a code (2^-4 relative, 2^-10 of amax / 448) and the rounding."""
    mags = torch.tensor([1e-30, 1.4e-36, 1.3e-36, 1e-37, 1.2e-38, 1e-39, 1e-40], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.rand((len(mags), 2, D), generator=g, device=DEV) * 2 - 1) * mags[:, None, None]
    x[:, :, ::5] = 0.0
    x = x.to(dt)
    codes = [torch.zeros((1, 2, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((1, 2, 16), device=DEV) for _ in range(2)]
    B.moe_kv_append(x, x, torch.arange(len(mags), dtype=torch.int32, device=DEV), *codes, *scales)
    for c, s in zip(codes, scales):
        got = (c.view(torch.float8_e4m3fn).double() * s.double()[..., None])[0].transpose(0, 1)[:len(mags)].cpu()
        want = x.double().cpu()
        amax = want.abs().amax(-1, keepdim=True)
        err, step = (got - want).abs(), torch.maximum(want.abs() * 2.0 ** -4, amax / 448 * 2.0 ** -10) + amax * 2.0 ** -20
        assert torch.isfinite(got).all()
        assert (got[want == 0] == 0).all()
        assert (err <= torch.where(amax > 1.33e-36, step, amax)).all()
