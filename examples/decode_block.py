"""One decoder block on a decode batch: attention over a shared prompt, then the mixture of experts.

The batch's sequences continue one prompt. The prompt goes through the block in chunks, then every sequence
decodes on its own: rotary positions, cache append and attention (PrefixAttention) and the experts (MoELayer) run in
the framework's kernels; the projections around them are plain matrix products. Weights and tokens are synthetic.

    python examples/decode_block.py [--steps 32] [--prompt-chunks 4] [--cache e4m3]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from mixture_experts_layer_gate_amd import MoELayer, PrefixAttention  # noqa: E402
from moe_inputs import generate, get_config  # noqa: E402


class DecodeBlock:
    """x + attention(norm x), then the MoE layer (which adds its own residual)."""

    def __init__(self, cfg, q_heads=8, kv_heads=2, head_dim=64, prompt=256, new_tokens=256, cache=None, device="cuda", seed=0):
        self.hq, self.hk, self.D = q_heads, kv_heads, head_dim
        inp = generate(cfg, device)
        self.moe = MoELayer(cfg, inp, device, keep_scores=False)
        self.x0 = inp["u"]
        dt = self.x0.dtype
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda n, m: (torch.randn((n, m), generator=g, device=device) * m ** -0.5).to(dt)
        self.w_qkv = w((q_heads + 2 * kv_heads) * head_dim, cfg.d)
        self.w_out = w(cfg.d, q_heads * head_dim)
        self.attention = PrefixAttention(cfg.T, q_heads, kv_heads, head_dim, prompt, new_tokens, dtype=dt, cache=cache,
                                         page_size=32, device=device)

    def _block(self, x, attend):
        n = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
        qkv = (n @ self.w_qkv.t()).view(len(x), -1, self.D)      # q, k, v heads: read where they lie
        a = attend(*qkv.split([self.hq, self.hk, self.hk], 1))
        return self.moe.forward(x + a.reshape(len(x), -1) @ self.w_out.t())

    def prefill(self, x):
        return self._block(x, self.attention.prefill)

    def step(self, x):
        return self._block(x, self.attention.step)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--prompt-chunks", type=int, default=4)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    cfg = get_config("c1", gemm="bf16", act="bf16")
    block = DecodeBlock(cfg, prompt=cfg.T * a.prompt_chunks, new_tokens=a.steps, cache=a.cache if a.cache == "e4m3" else None)
    x = block.x0
    for _ in range(a.prompt_chunks):
        block.prefill(x)
    x = block.step(x).clone()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps - 1):
        x = block.step(x).clone()
        x = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, a.steps - 1)
    print(f"{cfg.T} sequences on {block.attention.prefix_len} prompt tokens, {a.steps} new tokens each: "
          f"{t * 1e6:.0f} us a step, finite: {bool(torch.isfinite(x).all())}")


if __name__ == "__main__":
    main()
