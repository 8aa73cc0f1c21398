"""Host-side checks of the C ABI of the layers with experts and the e4m3 layers: memory that results share with operands,
sizes of workspaces.

No address is dereferenced: the refusals come before anything is launched, and what is not refused ends at the check for the
GPU, which is why these run where there is none.
"""

import pytest

from bit_weight_only_awq_gb300 import build as awq_build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would run")

EINVAL, TAKEN = -1, -4  # TAKEN: refused for want of a GPU alone
A, B = 1 << 40, 1 << 41  # far apart
SPACE = (1 << 42, 1 << 40)


@pytest.fixture(scope="module")
def lib():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq
    return awq.lib


def gemm(lib, x, y, stride=256, rows=8, R=16, N=512, gated=0, wide=0, order=B):
    return lib.awq_moe_gemm(x, stride, rows, B, B, order, 2, y, wide, R, 4, 256, N, gated, 0, *SPACE, None)


def test_grouped_product_refuses_rows_under_its_results(lib):
    assert gemm(lib, A, B) == TAKEN
    for at in (0, 16, 8 * 512 - 16, -16 * 1024 + 16):
        assert gemm(lib, A, A + at) == EINVAL, at
    for at in (8 * 512, -16 * 1024):
        assert gemm(lib, A, A + at) == TAKEN, at
    # half as many columns when gated, twice the bytes in fp32, rows or tokens
    assert gemm(lib, A, A - 16 * 512, gated=1) == TAKEN and gemm(lib, A, A - 16 * 512 + 16, gated=1) == EINVAL
    assert gemm(lib, A, A - 16 * 1024, wide=1) == EINVAL and gemm(lib, A, A - 16 * 2048, wide=1) == TAKEN
    assert gemm(lib, A, A + 15 * 512, order=None, rows=16) == EINVAL
    # results that lie between two rows of x, and one row further
    far = 1 << 16
    assert gemm(lib, A, A + 512, stride=far, rows=8) == TAKEN and gemm(lib, A, A + 496, stride=far, rows=8) == EINVAL
    assert gemm(lib, A, A + 2 * far * 5 - 16 * 1024, stride=far) == TAKEN
    assert gemm(lib, A, A + 2 * far * 5 - 16 * 1024 + 16, stride=far) == EINVAL
    assert gemm(lib, A, A + 2 * far * 7 + 512, stride=far) == TAKEN


def test_sum_may_be_its_residual_and_nothing_else(lib):
    def layer(res, rs, out, T=6, H=320):
        return lib.awq_moe(B, 256, B, B, B, B, B, B, res, rs, out, T, 2, 4, 256, 384, H, 0, *SPACE, None)

    for call in (layer, lambda *a, **k: combine(lib, *a, **k)):
        assert call(A, 320, A + 16) == EINVAL and call(A, 328, A) == EINVAL and call(A + 16, 328, A) == EINVAL
    assert layer(A, 320, A) == TAKEN and layer(A, 328, A, T=1) == TAKEN and layer(A, 320, A + 6 * 640) == TAKEN
    assert layer(None, 0, A) == TAKEN
    assert layer(A, 1 << 16, A + 640) == TAKEN  # between its rows
    # over the tokens themselves: read before
    assert lib.awq_moe(A, 320, B, B, B, B, B, B, None, 0, A, 6, 2, 4, 256, 384, 320, 0, *SPACE, None) == TAKEN


def combine(lib, res, rs, out, y=B, T=6, wide=0):
    return lib.awq_moe_combine(y, wide, B, B, res, rs, out, T, 2, 320, 2 * T, 0, None)


def test_sum_refuses_rows_under_its_results(lib):
    for wide in (0, 1):
        assert combine(lib, None, 0, A, y=A, wide=wide) == EINVAL
        assert combine(lib, None, 0, A + 12 * 640 * (1 + wide) - 16, y=A, wide=wide) == EINVAL


def test_e4m3_calls_refuse_operands_under_their_results(lib):
    q = lib.awq_fp8_quant_act  # x, stride, xq, s_x, M, K, dtype, stream
    assert q(A, 64, A, B, 4, 64, 0, None) == EINVAL and q(A, 64, A + 4 * 128 - 16, B, 4, 64, 0, None) == EINVAL
    f = lib.awq_fp8_gemm  # xq, s_x, wq, s_w, y, M, K, N, dtype, ws, bytes, stream
    assert f(A, B, B, B, A, 4, 256, 128, 0, *SPACE, None) == EINVAL
    assert f(A, B, B, B, A + 4 * 256 - 16, 4, 256, 128, 0, *SPACE, None) == EINVAL
    assert f(A, B, B, B, A + 4 * 256, 4, 256, 128, 0, *SPACE, None) == TAKEN
    # x of a whole layer may be overwritten
    assert lib.awq_fp8_linear(A, 256, B, B, A, 4, 256, 256, 0, *SPACE, None) == TAKEN


def test_a_layers_workspace_has_rows_in_order_for_up_alone(lib):
    """down finds its rows in order: 235 MB less for 8192 rows of 14336 channels."""
    for T, k, E, K, inner, H in ((4096, 2, 8, 4096, 14336, 4096), (4001, 8, 128, 2048, 768, 2048), (100, 2, 8, 256, 1024, 320)):
        R = T * k
        up = lib.awq_moe_gemm_workspace_bytes(R, E, K, 2 * inner, 1)
        parts = up - R * K * 2
        assert 0 < parts < 1 << 25
        aligned = lambda n: (n + 255) // 256 * 256
        assert lib.awq_moe_workspace_bytes(T, k, E, K, inner, H) == aligned(up) + aligned(R * inner * 2) + R * H * 4
