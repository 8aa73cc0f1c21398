"""The block with experts and fp8 layers end to end, against the same block operator by operator in float64.

Each operator's own test holds its bound; here the reference takes each operator's 16-bit inputs as they are (norm's rows,
the shared expert's sum, the experts' output), so what is compared is that they fit together.  fp8 layers: the reference
multiplies the codes' values, and an output is off by its own rounding and the sums', under 2 % of the largest value."""

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
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def dense(awq, weights):
    """float64 [experts, K, N] of prepared symmetric layers."""
    qweight, _, scales = awq.awq_moe_unprepack(weights)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=qweight.device)
    q = ((qweight[..., None] >> shift) & 15).flatten(-2).double() - 8
    return q * scales.double().repeat_interleave(128, 1)


def fp8(awq, layer, x):
    """float64 product of an fp8 layer with the codes that x quantizes to."""
    xq, s = awq.awq_fp8_quant_act(x)
    n, k = layer.codes.shape
    a = xq.double() * s.double().t().repeat_interleave(128, 1)[:, :k]
    w = layer.codes.double() * layer.scale.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return a @ w.t()


@pytest.mark.parametrize("tokens", [1, 7, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_block_against_float64(example, tokens, dtype):
    awq = example.awq
    block = example.MoeBlock(width=256, inner=384, experts=12, top_k=3, outputs=264, dtype=dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    x, residual = (torch.randn(tokens, 256, generator=gen, device="cuda").to(dtype) for _ in range(2))
    out, new_residual = block.step(x, residual)
    y, r1 = awq.awq_rmsnorm(x, block.norm, residual=residual)
    logits = y @ block.router
    weights, ids, plan = awq.awq_moe_route(logits, 3)
    p = torch.softmax(logits.double(), 1).gather(1, ids.long())
    assert (weights.double() - p / p.sum(1, keepdim=True)).abs().max() <= 1e-5
    g, u = block.shared_up(y).chunk(2, dim=1)
    act = torch.nn.functional.silu(g) * u
    shared = block.shared_down(act)
    want = fp8(awq, block.shared_down, act)
    assert (shared.double() - want).abs().max() <= 0.02 * want.abs().max()
    up, down = dense(awq, block.experts.up), dense(awq, block.experts.down)
    want = shared.double()
    for j in range(3):
        h = torch.einsum("tk,tkn->tn", y.double(), up[ids[:, j].long()])
        gate, lift = h.chunk(2, dim=1)
        h = gate * torch.sigmoid(gate) * lift
        want = want + weights[:, j : j + 1].double() * torch.einsum("tk,tkn->tn", h, down[ids[:, j].long()])
    mixed = awq.awq_moe(y, block.experts.up, block.experts.down, weights, plan, residual=shared)
    assert (mixed.double() - want).abs().max() <= 0.02 * want.abs().max()
    z, r2 = awq.awq_rmsnorm(mixed, block.next_norm, residual=r1)
    assert torch.equal(r2, new_residual) and torch.equal(block.projection(z), out)
    want = fp8(awq, block.projection, z)
    assert (out.double() - want).abs().max() <= 0.02 * want.abs().max()
    assert awq.awq_last_device_error() == 0
