"""The attention half of a decoder block on W4A8 layers and a 4-bit paged cache.

One layer with random weights: residual addition and RMS norm to int8 codes, W4A8 qkv projection, rotary append of
keys and values to the cache, attention over it, W4A8 output projection.  `AttentionBlock.step` takes the new tokens
of several sequences at once: whole prompts, pieces of them, or one token each.

    python examples/attention_block.py             # a prompt for each sequence, then some single tokens
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_only_awq_gb300 import awq  # noqa: E402


def rope_table(positions: int, dim: int, base: float = 10000.0, stretch: float = 1.0) -> torch.Tensor:
    """fp32 [positions, dim]: cosines, then sines.  Any rule for long contexts is a table of its own; here
    positions are divided by `stretch` (linear interpolation)."""
    freq = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] / stretch * freq
    return torch.cat((angle.cos(), angle.sin()), dim=1).float().cuda()


class W4A8Layer:
    """A W4A8 linear layer with random int4 weights and channel scales."""

    def __init__(self, inputs: int, outputs: int, gen: torch.Generator):
        codes = torch.randint(0, 16, (inputs, outputs), generator=gen, device="cuda", dtype=torch.uint8)
        self.wq = awq.awq_pack(codes)
        self.scale = (0.2 / math.sqrt(inputs) * (0.5 + torch.rand(outputs, generator=gen, device="cuda"))).half()

    def from_codes(self, xq, s_tok):
        return awq.w4a8_gemm(xq, s_tok, self.wq, self.scale)

    def __call__(self, x):
        return awq.w4a8_linear(x, self.wq, self.scale)[0]


class AttentionBlock:
    """Weights, cache and page bookkeeping of one layer."""

    def __init__(self, width=4096, heads=32, kv_heads=8, dim=128, pages=512, page_size=64, positions=8192, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        self.norm = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).half()
        self.next_norm = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).half()
        self.qkv = W4A8Layer(width, (heads + 2 * kv_heads) * dim, gen)
        self.out = W4A8Layer(heads * dim, width, gen)
        self.table = rope_table(positions, dim)
        self.cache = awq.kv4_cache(pages, kv_heads, dim, page_size)
        self.free = list(range(pages))[::-1]
        self.pages: dict[int, list[int]] = {}
        self.length: dict[int, int] = {}

    def plan(self, new: dict[int, int]):
        """Gives the sequences room for `new[sequence]` tokens: positions, slots, block table, lengths, q_start."""
        positions, slots, starts, lengths = [], [], [0], []
        for seq, count in new.items():
            pages, length = self.pages.setdefault(seq, []), self.length.get(seq, 0)
            while len(pages) * self.page_size < length + count:
                pages.append(self.free.pop())
            at = range(length, length + count)
            positions += at
            slots += [pages[p // self.page_size] * self.page_size + p % self.page_size for p in at]
            self.length[seq] = length + count
            starts.append(starts[-1] + count)
            lengths.append(length + count)
        most = max(len(self.pages[seq]) for seq in new)
        table = [self.pages[seq] + [0] * (most - len(self.pages[seq])) for seq in new]

        def on_gpu(values, dtype):
            return torch.tensor(values, dtype=dtype, device="cuda")

        return {"positions": on_gpu(positions, torch.int32), "slots": on_gpu(slots, torch.int64),
                "block_table": on_gpu(table, torch.int32), "kv_len": on_gpu(lengths, torch.int32),
                "q_start": on_gpu(starts, torch.int32), "max_q": max(new.values())}

    def step(self, x, residual, plan):
        """x, residual fp16 [tokens, width] -> (int8 codes and scales for the next layer, the new residual)."""
        xq, s_tok, residual = awq.w4a8_rmsnorm_quant(x, self.norm, residual=residual)
        heads = self.qkv.from_codes(xq, s_tok).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = heads.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q = awq.kv4_append(self.cache, k, v, plan["positions"], plan["slots"], self.table, q=q, q_out=q)
        mixed = awq.kv4_attention(q, self.cache, plan["block_table"], plan["kv_len"], q_start=plan["q_start"],
                                  max_q=plan["max_q"])
        y = self.out(mixed.view(x.shape[0], -1))
        xq, s_tok, residual = awq.w4a8_rmsnorm_quant(y, self.next_norm, residual=residual)
        return (xq, s_tok), residual


def main():
    block = AttentionBlock()
    width = block.norm.shape[0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    new = {0: 700, 1: 33, 2: 1500}  # prompts
    for turn in range(9):
        plan = block.plan(new)
        tokens = sum(new.values())
        x = torch.randn(tokens, width, generator=gen, device="cuda").half()
        residual = torch.randn(tokens, width, generator=gen, device="cuda").half()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        (xq, s_tok), residual = block.step(x, residual, plan)
        end.record()
        torch.cuda.synchronize()
        print(f"turn {turn}: {tokens} tokens, {sum(block.length[s] for s in new)} in the cache, "
              f"{begin.elapsed_time(end) * 1e3:.0f} us, codes {tuple(xq.shape)}, residual rms {residual.float().square().mean().sqrt():.3f}")
        new = {seq: 1 for seq in new}


if __name__ == "__main__":
    main()
