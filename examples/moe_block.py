"""The feed-forward half of a decoder block with experts, and the fp8 projection that comes after it.

One layer with random weights: residual addition and RMS norm, a router, 4-bit experts of which every token takes a few, a
shared expert in fp8 that every token takes, and the next block's projection in fp8.

    python examples/moe_block.py             # a prompt, then single tokens
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_only_awq_gb300 import awq  # noqa: E402


class Fp8Layer:
    """An fp8 linear layer from 16-bit weights [outputs, inputs]: e4m3 codes and a scale for each block of 128 x 128."""

    def __init__(self, weight: torch.Tensor):
        n, k = weight.shape
        w = torch.nn.functional.pad(weight.float(), (0, -k % 128, 0, -n % 128))
        blocks = w.view(w.shape[0] // 128, 128, w.shape[1] // 128, 128)
        self.scale = (blocks.abs().amax(dim=(1, 3)) / 448.0).clamp(min=1e-30)
        codes = (blocks / self.scale[:, None, :, None]).view(w.shape)[:n, :k]
        self.codes = codes.to(torch.float8_e4m3fn).contiguous()

    def __call__(self, x, out=None):
        return awq.awq_fp8_linear(x, self.codes, self.scale, out=out)


class Experts:
    """Random 4-bit weights of a layer's experts, gate and up side by side, laid out once."""

    def __init__(self, experts, width, inner, dtype, gen):
        def layer(k, n, gated):
            qweight = torch.randint(-2 ** 31, 2 ** 31, (experts, k, n // 8), generator=gen, device="cuda", dtype=torch.int32)
            scales = 0.2 / math.sqrt(k) * (0.5 + torch.rand(experts, k // 128, n, generator=gen, device="cuda"))
            return awq.awq_moe_prepack(qweight, None, scales.to(dtype), gated=gated)

        self.up, self.down = layer(width, 2 * inner, True), layer(inner, width, False)


class MoeBlock:
    def __init__(self, width=2048, inner=1408, experts=64, top_k=6, outputs=2560, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.top_k = top_k
        self.norm = (1 + 0.1 * normal(width)).to(dtype)
        self.router = (normal(width, experts) / math.sqrt(width)).to(dtype)
        self.experts = Experts(experts, width, inner, dtype, gen)
        self.shared_up = Fp8Layer((normal(2 * inner, width) / math.sqrt(width)).to(dtype))
        self.shared_down = Fp8Layer((normal(width, inner) / math.sqrt(inner)).to(dtype))
        self.next_norm = (1 + 0.1 * normal(width)).to(dtype)
        self.projection = Fp8Layer((normal(outputs, width) / math.sqrt(width)).to(dtype))

    def step(self, x, residual):
        """x, residual [tokens, width] -> (the next block's projection [tokens, outputs], the new residual)."""
        y, residual = awq.awq_rmsnorm(x, self.norm, residual=residual)
        weights, _, plan = awq.awq_moe_route(y @ self.router, self.top_k)
        gate, up = self.shared_up(y).chunk(2, dim=1)
        shared = self.shared_down(torch.nn.functional.silu(gate) * up)
        mixed = awq.awq_moe(y, self.experts.up, self.experts.down, weights, plan, residual=shared, out=shared)
        y, residual = awq.awq_rmsnorm(mixed, self.next_norm, residual=residual)
        return self.projection(y), residual


def main():
    block = MoeBlock()
    width = block.norm.shape[0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for turn, tokens in enumerate((3000, 17, 1, 1, 1, 1)):
        x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
        residual = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        out, residual = block.step(x, residual)
        end.record()
        torch.cuda.synchronize()
        print(f"turn {turn}: {tokens} tokens, {begin.elapsed_time(end) * 1e3:.0f} us, output rms {out.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
