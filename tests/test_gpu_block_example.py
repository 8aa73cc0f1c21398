"""The attention block example end to end: prompts, a further piece of one, then single tokens, against the same
block in float64 on what the cache holds.

The reference takes the operators' outputs in turn (codes, rotated queries, gathered entries), each of which has a
test of its own, so what is compared here is that they fit together.  The attention's output agrees to the bound of
its own test at these sizes, well under 1 % of its largest value."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_weight_only_awq_gb300 import build as awq_build
    awq_build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 64, 16), (4, 4, 128, 64)])
def test_block_against_float64(example, heads, kv_heads, dim, page):
    awq = example.awq
    block = example.AttentionBlock(width=512, heads=heads, kv_heads=kv_heads, dim=dim, pages=40, page_size=page, positions=512)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    tokens_of = {}
    for new in ({0: 70, 1: 3}, {0: 21}, {0: 1, 1: 1}, {1: 2, 0: 1}, {2: 130, 1: 1}):
        plan = block.plan(new)
        n = sum(new.values())
        x = torch.randn(n, 512, generator=gen, device="cuda").half()
        res = torch.randn(n, 512, generator=gen, device="cuda").half()
        (xq, s_tok), residual = block.step(x, res, plan)
        # the same, operator by operator
        cq, cs, r1 = awq.w4a8_rmsnorm_quant(x, block.norm, residual=res)
        h = (x.float() + res.float()).double()
        y = h * block.norm.double() / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
        assert (cq.double() * cs[:, None].double() - y).abs().max() <= 0.51 * cs.max()
        qkv = block.qkv.from_codes(cq, cs).view(n, -1, dim)
        q, k, v = qkv.split((heads, kv_heads, kv_heads), dim=1)
        # appending the same entries again changes nothing
        before = block.cache.clone()
        q = awq.kv4_append(block.cache, k, v, plan["positions"], plan["slots"], block.table, q=q)
        assert torch.equal(before, block.cache)
        want = torch.empty(n, heads, dim, dtype=torch.float64, device="cuda")
        at = 0
        for seq, count in new.items():
            pages, length = block.pages[seq], block.length[seq]
            slots = torch.tensor([pages[p // page] * page + p % page for p in range(length)], device="cuda")
            gk, gv = (t.double().repeat_interleave(heads // kv_heads, 1) for t in awq.kv4_gather(block.cache, slots))
            score = torch.einsum("ihd,jhd->hij", q[at:at + count].double(), gk) / dim ** 0.5
            hidden = torch.arange(length, device="cuda")[None] > torch.arange(length - count, length, device="cuda")[:, None]
            weight = torch.softmax(score.masked_fill(hidden, -torch.inf), -1)
            want[at:at + count] = torch.einsum("hij,jhd->ihd", weight, gv)
            at += count
        got = awq.kv4_attention(q, block.cache, plan["block_table"], plan["kv_len"], q_start=plan["q_start"], max_q=plan["max_q"])
        assert (got.double() - want).abs().max() <= 0.01 * want.abs().max()
        o = block.out(got.view(n, -1))
        nq, ns, r2 = awq.w4a8_rmsnorm_quant(o, block.next_norm, residual=r1)
        assert torch.equal(nq, xq) and torch.equal(ns, s_tok) and torch.equal(r2, residual)
        for seq, count in new.items():
            tokens_of[seq] = tokens_of.get(seq, 0) + count
    assert tokens_of == block.length and awq.awq_last_device_error() == 0
