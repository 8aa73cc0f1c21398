"""The norm's rows at the edges of its definition: rows of zeros without eps, weights that are not numbers."""

import numpy as np
import pytest

from oracle import block
from tests.test_gpu_rmsnorm import awq, dev, host, problem, tol  # noqa: F401  (awq is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K", [(3, 640), (700, 512), (2, 16392)])
def test_a_row_of_zeros_without_eps(awq, M, K, bf16):  # noqa: F811
    x, r, w = problem(M, K, bf16, 41)
    x[1], r[1] = 0, 0
    other = np.arange(M) != 1
    for res in (r, None):
        rt = None if res is None else dev(res, bf16)
        y = torch.full((M, K), 7.0, dtype=torch.bfloat16 if bf16 else torch.float16, device="cuda")
        xq, s, _ = awq.w4a8_rmsnorm_quant(dev(x, bf16), dev(w, bf16), rt, eps=0.0, y=y)
        assert float(s[1]) == 0 and not xq[1].any() and not y[1].any()
        codes, scale = block.rmsnorm_codes(x[other], None if res is None else res[other], w, 0.0)
        assert np.array_equal(xq.cpu().numpy()[other], codes)
        assert np.all(np.abs(s.cpu().numpy()[other] - scale) <= (tol(K) + 2.0 ** -22) * scale)
        y2, _ = awq.awq_rmsnorm(dev(x, bf16), dev(w, bf16), rt, eps=0.0)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K", [(3, 640), (700, 512), (400, 11016), (2, 16392)])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_weight_that_is_not_finite_shows(awq, M, K, value, bf16):  # noqa: F811
    """Every row's largest |y| is then not a number, or infinite: a NaN scale and codes 0, as for such a row."""
    x, r, w = problem(M, K, bf16, 42)
    w[K - 3] = value
    x[0, K - 3], r[0, K - 3] = 0, 0  # 0 * inf is a NaN too
    xq, s, _ = awq.w4a8_rmsnorm_quant(dev(x, bf16), dev(w, bf16), dev(r, bf16))
    assert torch.isnan(s).all() and not xq.any()
    y, _ = awq.awq_rmsnorm(dev(x, bf16), dev(w, bf16), dev(r, bf16))
    bad = ~np.isfinite(host(y))
    assert bad[:, K - 3].all() and bad.sum() == M
