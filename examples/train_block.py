"""One decoder block trained on packed sequences: attention (AttentionLayer), then the mixture of experts (MoELayer).

Both run their forward and backward passes in the framework's kernels; the block's step is plain gradient descent on the weights of
the attention half. Weights and tokens are synthetic.

    python examples/train_block.py [--steps 8]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from mixture_experts_layer_gate_amd import AttentionLayer, MoELayer  # noqa: E402
from moe_inputs import generate, get_config  # noqa: E402


class TrainBlock:
    """The MoE layer (which adds its own residual) of x + attention(norm x), on a batch of packed sequences."""

    def __init__(self, cfg, q_heads=8, kv_heads=2, head_dim=64, lens=None, device="cuda", seed=0):
        inp = generate(cfg, device)
        self.moe = MoELayer(cfg, inp, device, train=True)
        self.x0 = inp["u"]
        dt = self.x0.dtype
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda n, m: (torch.randn((n, m), generator=g, device=device) * m ** -0.5).to(dt)
        lens = lens or [cfg.T // 2, cfg.T // 4, cfg.T - cfg.T // 2 - cfg.T // 4]
        self.attention = AttentionLayer(
            {"w_qkv": w((q_heads + 2 * kv_heads) * head_dim, cfg.d), "w_out": w(cfg.d, q_heads * head_dim),
             "norm_weight": torch.ones(cfg.d), "norm_bias": torch.zeros(cfg.d)}, q_heads, kv_heads, head_dim, max(lens),
            device=device)
        self.seq_start = torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)

    def forward(self, x):
        return self.moe.forward_train(self.attention.forward(x, self.seq_start))

    def backward(self, d_out):
        return self.attention.backward(self.moe.backward(d_out).to(d_out.dtype))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = TrainBlock(get_config("c1", gemm="bf16", act="bf16"))
    x = block.x0
    target = torch.randn(x.shape, generator=torch.Generator(device=x.device).manual_seed(1), device=x.device)
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        off = block.forward(x).float() - target
        block.backward((off / off.numel()).to(x.dtype))
        for n in ("w_qkv", "w_out"):
            getattr(block.attention, n).sub_(block.attention.grads[n], alpha=10.0)
        torch.cuda.synchronize()
        print(f"step {step}: loss {off.square().mean().item() / 2:.4f}, {(time.perf_counter() - t) * 1e6:.0f} us")


if __name__ == "__main__":
    main()
