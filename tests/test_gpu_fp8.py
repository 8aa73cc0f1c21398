"""fp8 linear layers against the oracle's float64.

Codes and scales are defined bit for bit.  The product: e4m3 products are exact in fp32 (8 significant bits), a block's
128 of them are added in the tensor cores with at most 8 + 128 / 8 roundings of 2^-23 of their magnitudes, each block's
sum is scaled and added with 3 more, so that the output is off by at most (8 + 16 + 3 + K / 128) 2^-23 mag plus half an
ulp of its type.
"""

import numpy as np
import pytest

from oracle import layer
from oracle.block_oracle import round16

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_weight_only_awq_gb300 import build as awq_build
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq as mod
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev16(a, bf16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16 if bf16 else torch.float16).cuda()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K", [(0, 64), (1, 16), (1, 128), (3, 144), (17, 1040), (130, 4096), (1, 14336), (1000, 272)])
def test_quant(awq, M, K, bf16):
    rng = np.random.default_rng(M + K)
    x = rng.normal(size=(M, K)).astype(np.float32)
    x[:, :: max(3, K // 7)] *= 30
    x *= np.exp(3 * rng.normal(size=(M, 1)))
    x = round16(x, bf16)
    if M > 2 and K > 128:
        x[0, :128] = 0
        x[1, 128:] = np.nan
        x[2, 3] = -np.inf
    wide = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float16, device="cuda")
    wide[:, :K] = dev16(x, bf16)
    xq, s_x = awq.awq_fp8_quant_act(wide[:, :K])
    want_q, want_s = layer.fp8_quant(x)
    assert np.array_equal(s_x.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(codes(xq) & 127, want_q & 127)
    # the sign of a code 0 is the value's
    assert np.array_equal(codes(xq), want_q)


@pytest.mark.parametrize("bf16", [False, True])
def test_quant_at_the_borders_of_codes_and_of_the_range(awq, bf16):
    """Every ratio of two 16-bit significands near the borders between codes, largest values from the smallest to the
    largest, scales that are subnormal."""
    rng = np.random.default_rng(1)
    table = layer.e4m3_values()[:127]
    tops = np.exp2(rng.integers(-20, 15, 400)) * (1 + rng.integers(0, 128 if bf16 else 1024, 400) / (128 if bf16 else 1024))
    if bf16:
        tops[:120] = np.exp2(rng.integers(-133, -90, 120)) * (1 + rng.integers(0, 128, 120) / 128)
        tops[120:160] = np.exp2(rng.integers(100, 127, 40))
    else:
        tops[:40] = rng.integers(1, 64, 40) * 2.0 ** -24
    tops = round16(tops.astype(np.float32), bf16)
    border = (table[1:] + table[:-1]) / 2
    x = np.empty((400, 128), np.float32)
    with np.errstate(over="ignore", under="ignore"):
        for r in range(400):
            pick = rng.choice(border, 127)
            x[r, 0] = tops[r]
            x[r, 1:] = round16((pick / 448 * np.float64(tops[r]) * rng.choice([-1, 1], 127)).astype(np.float32), bf16)
    want_q, want_s = layer.fp8_quant(x)
    xq, s_x = awq.awq_fp8_quant_act(dev16(x, bf16))
    assert np.array_equal(s_x.cpu().numpy(), want_s)
    assert np.array_equal(codes(xq), want_q)


class Problem:
    def __init__(self, M, K, N, seed=0):
        rng = np.random.default_rng(seed)
        self.M, self.K, self.N = M, K, N
        table = layer.e4m3_values()
        self.xq, self.wq = (layer.e4m3_codes(np.clip(120 * rng.normal(size=(n, K)), -448, 448).astype(np.float32)) for n in (M, N))
        assert not np.isnan(table[self.xq]).any()
        g = -(-K // 128)
        self.s_x = (np.exp(rng.normal(size=(g, M))) / 100).astype(np.float32)
        self.s_w = (np.exp(rng.normal(size=(-(-N // 128), g))) / 1000).astype(np.float32)

    def on_gpu(self):
        return (dev(self.xq).view(torch.float8_e4m3fn), dev(self.s_x), dev(self.wq).view(torch.float8_e4m3fn), dev(self.s_w))


def check(got, want, mag, K, bf16):
    err = (27 + K / 128) * 2.0 ** -23 * mag
    tol = err + (2.0 ** -8 if bf16 else 2.0 ** -11) * (np.abs(want) + err) + (2.0 ** -134 if bf16 else 2.0 ** -25)
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (1, 128, 128), (2, 144, 136), (5, 4096, 256), (16, 272, 1032), (17, 512, 128),
                                   (31, 1040, 264), (33, 640, 520), (64, 256, 4096), (65, 384, 72), (128, 1024, 512),
                                   (130, 2048, 248), (257, 528, 1160), (300, 128, 2056), (1, 14336, 512), (700, 1296, 400),
                                   (601, 1040, 8200), (384, 16384, 2040), (515, 4112, 4096)])
@pytest.mark.parametrize("bf16", [False, True])
def test_gemm(awq, M, K, N, bf16):
    p = Problem(M, K, N, seed=M + K + N)
    args = p.on_gpu()
    dtype = torch.bfloat16 if bf16 else torch.float16
    y = awq.awq_fp8_gemm(*args, dtype=dtype)
    assert torch.equal(y, awq.awq_fp8_gemm(*args, dtype=dtype))
    check(y, *layer.fp8_gemm(p.xq, p.s_x, p.wq, p.s_w), K, bf16)
    assert awq.awq_last_device_error() == 0


def test_gemm_scales_of_blocks(awq):
    """A block's scale of 0 takes its weights out, a NaN one shows in its columns or rows only."""
    p = Problem(40, 384, 256, seed=1)
    p.s_w[0, 1] = 0
    p.s_x[2, 5] = 0
    want, mag = layer.fp8_gemm(p.xq, p.s_x, p.wq, p.s_w)
    check(awq.awq_fp8_gemm(*p.on_gpu()), want, mag, 384, False)
    p.s_w[1, 0] = np.nan
    p.s_x[1, 7] = np.nan
    y = awq.awq_fp8_gemm(*p.on_gpu()).isnan().cpu()
    assert y[:, 128:].all() and y[7].all() and not y[:7, :128].any() and not y[8:, :128].any()


@pytest.mark.parametrize("M,K,N", [(0, 64, 64), (1, 4096, 512), (19, 1040, 1000), (200, 512, 384), (2, 1040, 1000), (3, 272, 264),
                                   (16, 1024, 136), (601, 1040, 8200)])
@pytest.mark.parametrize("bf16", [False, True])
def test_linear_is_quant_and_gemm(awq, M, K, N, bf16):
    p = Problem(max(M, 1), K, N, seed=3)
    _, _, wq, s_w = p.on_gpu()
    x = dev16(np.random.default_rng(4).normal(size=(M, K)), bf16)
    y = awq.awq_fp8_linear(x, wq, s_w)
    xq, s_x = awq.awq_fp8_quant_act(x)
    assert y.dtype == x.dtype and torch.equal(y, awq.awq_fp8_gemm(xq, s_x, wq, s_w, dtype=x.dtype))
    # layers of other sizes between its calls find the counters of the shared workspace as they left them
    q = Problem(7, 2048, 128, seed=5)
    _, _, wq2, s_w2 = q.on_gpu()
    x2 = dev16(np.random.default_rng(6).normal(size=(7, 2048)), bf16)
    first = awq.awq_fp8_linear(x2, wq2, s_w2)
    for _ in range(3):
        assert torch.equal(awq.awq_fp8_linear(x, wq, s_w), y) and torch.equal(awq.awq_fp8_linear(x2, wq2, s_w2), first)


def test_linear_in_a_graph(awq):
    M, K, N = 9, 2048, 384
    p = Problem(M, K, N, seed=3)
    _, _, wq, s_w = p.on_gpu()
    x = torch.zeros(M, K, device="cuda").half()
    ws = torch.zeros(awq.awq_fp8_linear_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    awq.awq_fp8_linear(x, wq, s_w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = awq.awq_fp8_linear(x, wq, s_w, workspace=ws)
    for seed in range(3):
        x.copy_(torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        assert torch.equal(y, awq.awq_fp8_linear(x, wq, s_w))
    with pytest.raises(RuntimeError, match="workspace of its own"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            awq.awq_fp8_linear(x, wq, s_w)
    torch.cuda.synchronize()


def test_binding_refusals(awq):
    p = Problem(4, 256, 128)
    xq, s_x, wq, s_w = p.on_gpu()
    x = torch.zeros(4, 256, device="cuda").half()
    for bad in (lambda: awq.awq_fp8_gemm(xq, s_x[:1], wq, s_w), lambda: awq.awq_fp8_gemm(xq[:3], s_x, wq, s_w),
                lambda: awq.awq_fp8_gemm(xq, s_x, wq, s_w[:, :1].contiguous()),
                lambda: awq.awq_fp8_linear(x[:, :128], wq, s_w), lambda: awq.awq_fp8_linear(x, wq, s_w, out=x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.awq_fp8_gemm(x, s_x, wq, s_w), lambda: awq.awq_fp8_gemm(xq, s_x, wq, s_w.double()),
                lambda: awq.awq_fp8_gemm(xq, s_x, wq, s_w, dtype=torch.float32), lambda: awq.awq_fp8_linear(x.float(), wq, s_w),
                lambda: awq.awq_fp8_linear(x.cpu(), wq, s_w), lambda: awq.awq_fp8_quant_act(x.float())):
        with pytest.raises(TypeError):
            bad()
