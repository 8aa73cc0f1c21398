"""The RMS norm with residual and int8 codes against the oracle.

Codes and res_out are compared bit for bit: their operations are defined one rounding at a time.  The sum of
squares adds non-negative terms in fp32: in a chain of n additions its relative error is at most n 2^-24, and
no summation of a row by at least a warp has chains longer than K / 32 + 16; the square root halves it, and six
more roundings follow (mean, eps, square root, reciprocal, products).
"""

import numpy as np
import pytest

from oracle import block

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


def tol(K):
    return ((K / 32 + 16) / 2 + 6) * 2.0 ** -24


def dev(a, bf16):
    return torch.from_numpy(a).cuda().to(torch.bfloat16 if bf16 else torch.float16)


def host(t):
    return t.float().cpu().numpy()


def problem(M, K, bf16, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, K)).astype(np.float32)
    x[:, :: max(1, K // 3)] *= 30
    r = 2 * rng.normal(size=(M, K)).astype(np.float32)
    w = (1 + 0.3 * rng.normal(size=K)).astype(np.float32)
    return tuple(block.round16(a, bf16) for a in (x, r, w))


def check(awq, x, r, w, bf16, eps=1e-6, xt=None, rt=None):
    M, K = x.shape
    xt = dev(x, bf16) if xt is None else xt
    rt = rt if rt is not None else None if r is None else dev(r, bf16)
    y = torch.full((M, K), 7.0, dtype=xt.dtype, device="cuda")
    xq, s, res = awq.w4a8_rmsnorm_quant(xt, dev(w, bf16), rt, eps=eps, y=y)
    codes, s64 = block.rmsnorm_codes(x, r, w, eps)
    y64, h64 = block.rmsnorm(x, r, w, eps)
    assert np.array_equal(xq.cpu().numpy(), codes)
    assert np.all(np.abs(s.cpu().numpy() - s64) <= (tol(K) + 2.0 ** -22) * s64)
    half_ulp = 2.0 ** -8 if bf16 else 2.0 ** -11
    assert np.all(np.abs(host(y) - y64) <= (tol(K) * 1.01 + half_ulp) * np.abs(y64) + 2.0 ** -25)
    if r is None:
        assert res is None
    else:
        assert np.array_equal(host(res), block.round16(x + r, bf16))
    y2, res2 = awq.awq_rmsnorm(xt, dev(w, bf16), rt, eps=eps)
    assert torch.equal(y, y2) and (r is None or torch.equal(res, res2))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K", [(1, 8), (2, 16), (3, 248), (1, 4096), (5, 1000), (33, 2056), (7, 8192), (2, 11016),
                                 (3, 16384), (1, 16392), (2, 65536), (700, 512), (1300, 264)])
def test_against_the_oracle(awq, M, K, bf16):
    x, r, w = problem(M, K, bf16, M * 1000 + K)
    check(awq, x, r, w, bf16)
    check(awq, x, None, w, bf16)


def test_strided_rows(awq):
    x, r, w = problem(6, 520, False, 1)
    wide, wider = torch.zeros(6, 1040, dtype=torch.float16, device="cuda"), torch.zeros(6, 3, 528, dtype=torch.float16, device="cuda")
    wide[:, 520:] = dev(x, False)
    wider[:, 1, :520] = dev(r, False)
    check(awq, x, r, w, False, xt=wide[:, 520:], rt=wider[:, 1, :520])


def test_ties_and_extremes_of_the_codes(awq):
    # scale 1 exactly: halves round to the even code; the largest value makes 127
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0, 126.5]], np.float32)
    xq, s, _ = awq.w4a8_rmsnorm_quant(dev(x, False), torch.ones(8, dtype=torch.float16, device="cuda"), eps=0.0)
    assert xq.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -127, 126]]
    assert abs(float(s) - 1 / np.sqrt(np.mean(x ** 2))) <= 1e-6


@pytest.mark.parametrize("bf16", [False, True])
def test_zero_rows_and_rows_that_are_not_finite(awq, bf16):
    x, r, w = problem(5, 640, bf16, 9)
    x[1], r[1] = 0, 0
    x[2, 77] = np.nan
    x[3, 5] = np.inf
    xq, s, res = awq.w4a8_rmsnorm_quant(dev(x, bf16), dev(w, bf16), dev(r, bf16))
    s = s.cpu().numpy()
    assert s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and np.all(np.isfinite(s[[0, 4]]))
    codes, _ = block.rmsnorm_codes(x[[0, 4]], r[[0, 4]], w, 1e-6)
    got = xq.cpu().numpy()
    assert not got[1:4].any() and np.array_equal(got[[0, 4]], codes)
    assert np.isnan(host(res)[2, 77]) and np.isinf(host(res)[3, 5])


def test_in_place_and_repeated(awq):
    x, r, w = problem(9, 1032, False, 3)
    want = awq.w4a8_rmsnorm_quant(dev(x, False), dev(w, False), dev(r, False))
    rt = dev(r, False)
    got = awq.w4a8_rmsnorm_quant(dev(x, False), dev(w, False), rt, res_out=rt)
    assert got[2] is rt and all(torch.equal(a, b) for a, b in zip(got, want))
    again = awq.w4a8_rmsnorm_quant(dev(x, False), dev(w, False), dev(r, False))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_feeds_w4a8_gemm_on_another_stream(awq):
    from bit_weight_only_awq_gb300 import synth
    import oracle
    p = synth.w4a8_problem(5, 512, 256, seed=4)
    x, r, w = problem(5, 512, False, 5)
    xt, wt, rt = dev(x, False), dev(w, False), dev(r, False)
    wq, sc = torch.from_numpy(p["wq"]).cuda(), torch.from_numpy(p["s_ch"]).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        xq, s, _ = awq.w4a8_rmsnorm_quant(xt, wt, rt)
        y = awq.w4a8_gemm(xq, s, wq, sc)
    side.synchronize()
    want, _ = oracle.w4a8_linear(block.rmsnorm_codes(x, r, w, 1e-6)[0], s.cpu().numpy(), p["wq"], p["s_ch"])
    assert np.array_equal(y.cpu().numpy().view(np.uint16), want.view(np.uint16))


def test_wrong_operands_are_refused(awq):
    x = torch.zeros(2, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for bad in (lambda: awq.awq_rmsnorm(x.float(), w.float()), lambda: awq.awq_rmsnorm(x, w.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: awq.awq_rmsnorm(x, w[:32]), lambda: awq.awq_rmsnorm(x.t()[:, :2].t().as_strided((2, 64), (1, 2)), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(awq.AwqError):
        awq.awq_rmsnorm(x[:, :60].contiguous(), w[:60].contiguous())
    y, _ = awq.awq_rmsnorm(x[:0], w)
    assert y.shape == (0, 64)
