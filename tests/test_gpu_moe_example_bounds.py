"""The example's block, each of its layers against float64 with the bounds of the operators' own tests.

Every reference takes the layer's 16-bit input as it is.  An e4m3 layer: (27 + K / 128) 2^-23 of the magnitudes and half a
step.  The experts: the products' bounds, silu's, and the rounding of the rows between them, carried through `down`.
"""

import pytest

from tests.test_gpu_moe_example import dense, example, fp8  # noqa: F401  (example is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rounding(dtype):
    return (2.0 ** -8, 2.0 ** -134) if dtype is torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)


def check(got, want, err, dtype):
    half, least = rounding(dtype)
    tol = err + half * (want.abs() + err) + least
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()


def check_fp8(awq, layer, x, got):
    """With the magnitudes: the same product of absolute values."""
    class Magnitudes:
        codes, scale = layer.codes.float().abs().to(torch.float8_e4m3fn), layer.scale.abs()

    k = layer.codes.shape[1]
    check(got, fp8(awq, layer, x), (27 + k / 128) * 2.0 ** -23 * fp8(awq, Magnitudes, x.abs()), x.dtype)


@pytest.mark.parametrize("tokens", [1, 2, 7, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_block_within_the_operators_bounds(example, tokens, dtype):  # noqa: F811
    awq = example.awq
    width, inner, top_k = 256, 384, 3
    block = example.MoeBlock(width=width, inner=inner, experts=12, top_k=top_k, outputs=264, dtype=dtype, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, residual = (torch.randn(tokens, width, generator=gen, device="cuda").to(dtype) for _ in range(2))
    out, _ = block.step(x, residual)
    y, r1 = awq.awq_rmsnorm(x, block.norm, residual=residual)
    weights, ids, plan = awq.awq_moe_route(y @ block.router, top_k)
    both = block.shared_up(y)
    check_fp8(awq, block.shared_up, y, both)
    gate, lift = both.chunk(2, dim=1)
    act = torch.nn.functional.silu(gate) * lift
    shared = block.shared_down(act)
    check_fp8(awq, block.shared_down, act, shared)

    up, down, a = dense(awq, block.experts.up), dense(awq, block.experts.down), y.double()
    half, least = rounding(dtype)
    want = shared.double()
    err = 2.0 ** -24 * want.abs()
    for j in range(top_k):
        e, w = ids[:, j].long(), weights[:, j : j + 1].double()
        g, u = torch.einsum("tk,tkn->tn", a, up[e]).chunk(2, dim=1)
        dg, du = ((8 + width / 8) * 2.0 ** -23 * torch.einsum("tk,tkn->tn", a.abs(), up[e].abs())).chunk(2, dim=1)
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * u.abs() * dg + (s.abs() + 1.1 * dg) * du + 2.0 ** -20 * h.abs()
        dh = dh + half * (h.abs() + dh) + least
        t = torch.einsum("tk,tkn->tn", h, down[e])
        dt = torch.einsum("tk,tkn->tn", dh + (8 + inner / 8) * 2.0 ** -23 * (h.abs() + dh), down[e].abs())
        want = want + w * t
        err = err + w * dt + 2.0 ** -20 * (w * t).abs()
    mixed = awq.awq_moe(y, block.experts.up, block.experts.down, weights, plan, residual=shared)
    check(mixed, want, err, dtype)
    z, _ = awq.awq_rmsnorm(mixed, block.next_norm, residual=r1)
    check_fp8(awq, block.projection, z, out)
    assert awq.awq_last_device_error() == 0
