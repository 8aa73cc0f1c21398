"""Host-side checks of the C ABI of the layer with experts and the fp8 layers: refusals before anything is launched
(no GPU), sizes, and the oracle's own pins."""

import numpy as np
import pytest

from bit_weight_only_awq_gb300 import build as awq_build
from oracle import layer

EINVAL, EALIGN, EWORKSPACE, ENULL = -1, -2, -6, -7
FAKE = 1 << 40          # an aligned address that is never dereferenced (checks run first)
OFF = FAKE + 4


@pytest.fixture(scope="module")
def lib():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq
    return awq.lib


def test_plan_refusals(lib):
    f = lib.awq_moe_plan  # ids, R, experts, offsets, order, place, stream
    for bad in ((-1, 8), (2 ** 30 + 1, 8), (10, 0), (10, 513)):
        assert f(FAKE, *bad, FAKE, FAKE, FAKE, None) == EINVAL, bad
    for i in (0, 3, 4, 5):
        args = [FAKE, 10, 8, FAKE, FAKE, FAKE, None]
        args[i] = None
        assert f(*args) == ENULL, i
        args[i] = FAKE + 2
        assert f(*args) == EALIGN, i


def _route(lib, logits=FAKE, stride=8, T=5, experts=8, top_k=2, kind=0, ids=FAKE, w=FAKE, offsets=FAKE, order=FAKE, place=FAKE):
    return lib.awq_moe_route(logits, stride, T, experts, top_k, 1, kind, ids, w, offsets, order, place, None)


def test_route_refusals(lib):
    for bad in ({"experts": 0}, {"experts": 513, "stride": 600}, {"top_k": 0}, {"top_k": 9}, {"stride": 7}, {"T": -1},
                {"kind": 3}, {"kind": -1}, {"T": 2 ** 29 + 1}, {"experts": 64, "stride": 64, "top_k": 33}):
        assert _route(lib, **bad) == EINVAL, bad
    for name in ("logits", "ids", "w", "offsets", "order", "place"):
        assert _route(lib, **{name: None}) == ENULL, name
    for name in ("ids", "w", "offsets", "order", "place"):
        assert _route(lib, **{name: FAKE + 2}) == EALIGN, name
    assert _route(lib, logits=FAKE + 1) == EALIGN and _route(lib, logits=FAKE + 2, kind=2) == EALIGN
    assert _route(lib, T=0, logits=None, ids=None, w=None, offsets=None, order=None, place=None) == 0


def test_prepack_sizes_and_refusals(lib):
    size = lib.awq_moe_prepacked_bytes
    assert size(3, 256, 320, 0) == 3 * 2 * 2 * 17024
    assert size(3, 256, 320, 1) == 3 * 2 * 2 * 17024   # 160 columns of gate, as many of up
    assert size(1, 128, 32, 0) == 17024 and size(1, 128, 64, 1) == 17024
    for bad in ((0, 256, 256, 0), (513, 256, 256, 0), (1, 200, 256, 0), (1, 0, 256, 0), (1, 256, 48, 0), (1, 256, 0, 0),
                (1, 256, 96, 1), (1, 2 ** 20 + 128, 256, 0), (1, 256, 2 ** 20 + 32, 0)):
        assert size(*bad) == 0, bad
    f = lib.awq_moe_prepack  # qw, qz, sc, experts, K, N, group, gated, packed, bytes, stream
    need = size(2, 256, 512, 0)
    ok = [FAKE, FAKE, FAKE, 2, 256, 512, 128, 0, FAKE, need, None]

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[int(k[1:])] = v
        return f(*args)

    assert call(a9=need - 1) == EINVAL and call(a6=64) == EINVAL and call(a4=100) == EINVAL
    for i in (0, 2, 8):
        assert call(**{f"a{i}": None}) == ENULL
    for i in (0, 1, 2, 8):
        assert call(**{f"a{i}": OFF}) == EALIGN
    g = lib.awq_moe_unprepack  # packed, experts, K, N, gated, qw, qz, sc, stream
    assert g(FAKE, 2, 256, 500, 0, FAKE, FAKE, FAKE, None) == EINVAL
    assert g(None, 2, 256, 512, 0, FAKE, FAKE, FAKE, None) == ENULL
    assert g(FAKE, 2, 256, 512, 0, FAKE, OFF, FAKE, None) == EALIGN


def _gemm(lib, x=FAKE, xs=256, xr=8, packed=FAKE, offsets=FAKE, order=FAKE, top_k=2, y=FAKE, R=16, experts=4, K=256, N=512,
          gated=0, dtype=0, ws=FAKE, wsb=1 << 40):
    return lib.awq_moe_gemm(x, xs, xr, packed, offsets, order, top_k, y, 0, R, experts, K, N, gated, dtype, ws, wsb, None)


def test_gemm_refusals(lib):
    for bad in ({"R": -1}, {"R": 2 ** 30 + 1}, {"xr": 0}, {"xr": 2 ** 30 + 1}, {"K": 200}, {"N": 500}, {"N": 96, "gated": 1},
                {"xs": 248}, {"xs": 260}, {"dtype": 2}, {"top_k": 0}, {"top_k": 33}, {"experts": 0}, {"experts": 513}):
        assert _gemm(lib, **bad) == EINVAL, bad
    for name in ("x", "packed", "offsets", "y"):
        assert _gemm(lib, **{name: None}) == ENULL, name
    for name in ("x", "packed", "y"):
        assert _gemm(lib, **{name: OFF}) == EALIGN, name
    for name in ("offsets", "order"):
        assert _gemm(lib, **{name: FAKE + 2}) == EALIGN, name
    assert _gemm(lib, R=0, x=None, packed=None, y=None) == 0
    need = lib.awq_moe_gemm_workspace_bytes(16, 4, 256, 512, 0)
    if need:
        assert _gemm(lib, ws=None) == EWORKSPACE and _gemm(lib, wsb=need - 1) == EWORKSPACE
        assert _gemm(lib, ws=FAKE + 16) == EALIGN
    assert lib.awq_moe_gemm_workspace_bytes(16, 4, 250, 512, 0) == 0


def test_combine_refusals(lib):
    def call(y=FAKE, place=FAKE, w=FAKE, res=FAKE, rs=64, out=FAKE, T=3, k=2, H=64, R=6, dtype=0):
        return lib.awq_moe_combine(y, 1, place, w, res, rs, out, T, k, H, R, dtype, None)

    for bad in ({"k": 0}, {"k": 33}, {"T": -1}, {"R": -1}, {"H": 60}, {"H": 0}, {"rs": 56}, {"rs": 68}, {"dtype": 5}):
        assert call(**bad) == EINVAL, bad
    for name in ("y", "place", "w", "out"):
        assert call(**{name: None}) == ENULL, name
    for name in ("y", "res", "out"):
        assert call(**{name: OFF}) == EALIGN, name
    for name in ("place", "w"):
        assert call(**{name: FAKE + 2}) == EALIGN, name
    assert call(T=0, y=None, place=None) == 0


def test_layer_refusals(lib):
    def call(x=FAKE, xs=256, up=FAKE, down=FAKE, offsets=FAKE, order=FAKE, place=FAKE, w=FAKE, res=FAKE, rs=320, out=FAKE, T=6,
             k=2, E=4, K=256, inner=384, H=320, dtype=0, ws=FAKE, wsb=1 << 40):
        return lib.awq_moe(x, xs, up, down, offsets, order, place, w, res, rs, out, T, k, E, K, inner, H, dtype, ws, wsb, None)

    for bad in ({"xs": 248}, {"xs": 260}, {"rs": 312}, {"rs": 324}, {"T": -1}, {"T": 2 ** 29 + 1}, {"k": 0}, {"k": 33}, {"E": 0},
                {"E": 513}, {"K": 250}, {"inner": 96}, {"inner": 0}, {"inner": 2 ** 62}, {"H": 300}, {"dtype": 3}):
        assert call(**bad) == EINVAL, bad
    for name in ("x", "up", "down", "offsets", "order", "place", "w", "out"):
        assert call(**{name: None}) == ENULL, name
    for name in ("x", "up", "down", "res", "out"):
        assert call(**{name: OFF}) == EALIGN, name
    for name in ("offsets", "order", "place", "w"):
        assert call(**{name: FAKE + 2}) == EALIGN, name
    assert call(T=0, x=None, out=None) == 0
    need = lib.awq_moe_workspace_bytes(6, 2, 4, 256, 384, 320)
    assert need >= lib.awq_moe_gemm_workspace_bytes(12, 4, 256, 768, 1) + 12 * 384 * 2 + 12 * 320 * 4
    assert call(ws=None) == EWORKSPACE and call(wsb=need - 1) == EWORKSPACE and call(ws=FAKE + 16) == EALIGN
    assert lib.awq_moe_workspace_bytes(6, 2, 4, 256, 100, 320) == 0


def test_fp8_refusals(lib):
    q = lib.awq_fp8_quant_act  # x, stride, xq, s_x, M, K, dtype, stream
    for bad in ((4, 4100, 4104, 0), (4, 8, 8, 0), (-1, 64, 64, 0), (4, 64, 56, 0), (4, 64, 68, 0), (4, 64, 64, 2),
                (4, 2 ** 20 + 16, 2 ** 20 + 16, 0)):
        M, K, stride, dtype = bad
        assert q(FAKE, stride, FAKE, FAKE, M, K, dtype, None) == EINVAL, bad
    assert q(None, 64, FAKE, FAKE, 4, 64, 0, None) == ENULL and q(FAKE, 64, OFF, FAKE, 4, 64, 0, None) == EALIGN
    assert q(FAKE, 64, FAKE, FAKE + 2, 4, 64, 0, None) == EALIGN and q(None, 64, None, None, 0, 64, 0, None) == 0

    def gemm(xq=FAKE, sx=FAKE, wq=FAKE, sw=FAKE, y=FAKE, M=4, K=256, N=512, dtype=0, ws=FAKE, wsb=1 << 40):
        return lib.awq_fp8_gemm(xq, sx, wq, sw, y, M, K, N, dtype, ws, wsb, None)

    for bad in ({"M": -1}, {"K": 8}, {"K": 250}, {"N": 4}, {"N": 500 + 2}, {"dtype": 2}, {"M": 2 ** 30 + 1}):
        assert gemm(**bad) == EINVAL, bad
    for name in ("xq", "sx", "wq", "sw", "y"):
        assert gemm(**{name: None}) == ENULL, name
    for name in ("xq", "wq", "y"):
        assert gemm(**{name: OFF}) == EALIGN, name
    for name in ("sx", "sw"):
        assert gemm(**{name: FAKE + 2}) == EALIGN, name
    assert gemm(M=0, xq=None, y=None) == 0
    f = lib.awq_fp8_linear  # x, stride, wq, s_w, y, M, K, N, dtype, ws, bytes, stream
    need = lib.awq_fp8_linear_workspace_bytes(4, 256, 512)
    assert need >= 65536 + 4 * 256 + 4 * 2 * 4  # counters that stay zero, codes, scales
    assert f(FAKE, 256, FAKE, FAKE, FAKE, 4, 256, 512, 0, None, 0, None) == EWORKSPACE
    assert f(FAKE, 256, FAKE, FAKE, FAKE, 4, 256, 512, 0, FAKE, need - 1, None) == EWORKSPACE
    assert f(FAKE, 256, FAKE, FAKE, FAKE, 4, 256, 512, 0, FAKE + 16, need, None) == EALIGN
    assert f(FAKE, 250, FAKE, FAKE, FAKE, 4, 256, 512, 0, FAKE, need, None) == EINVAL
    assert f(None, 256, FAKE, FAKE, FAKE, 4, 256, 512, 0, FAKE, need, None) == ENULL


# ---- the oracle

def test_plans_and_weights_of_other_sizes_are_refused(lib):
    import torch
    from bit_weight_only_awq_gb300 import awq
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    assert awq.MoePlan(i32(5), i32(6), i32(6), 2).rows == 6
    for bad in ((i32(5).long(), i32(6), i32(6), 2), (i32(5), i32(12)[::2], i32(6), 2), (i32(5), i32(6), i32((6, 1)), 2)):
        with pytest.raises(TypeError):
            awq.MoePlan(*bad)
    for bad in ((i32(1), i32(6), i32(6), 2), (i32(5), i32(6), i32(5), 2), (i32(5), i32(6), i32(6), 4), (i32(5), i32(6), i32(6), 0)):
        with pytest.raises(ValueError):
            awq.MoePlan(*bad)
    data = torch.zeros(2 * 17024, dtype=torch.uint8)
    assert awq.MoeWeights(data, 2, 128, 256, True, torch.float16).outputs == 128
    for bad in ((data, 2, 256, 256, False), (data[:-1], 2, 128, 256, False), (data[:0], 2, 128, 100, False)):
        with pytest.raises(ValueError):
            awq.MoeWeights(*bad, torch.float16)
    for bad in ((data.char(), torch.float16), (data, torch.float32)):
        with pytest.raises(TypeError):
            awq.MoeWeights(bad[0], 2, 128, 256, False, bad[1])


def test_oracle_plan_and_route_by_hand():
    offsets, order, place = layer.plan([[2, 0], [0, 9], [2, -1]], 3)
    assert offsets.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 2, 0, 4, -1, -1] and place.tolist() == [2, 0, 1, -1, 3, -1]
    w, ids = layer.route(np.array([[1.0, 3.0, 3.0, -np.inf]]), 3, True)
    assert ids.tolist() == [[1, 2, 0]]
    assert np.allclose(w, np.array([[1, 1, np.exp(-2)]]) / (2 + np.exp(-2)))
    assert layer.route(np.full((1, 4), -np.inf), 2, False)[0].tolist() == [[0.0, 0.0]]


def test_oracle_e4m3():
    v = layer.e4m3_values()
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and np.isnan(v[0xFF])
    finite = v[~np.isnan(v)]
    assert (layer.e4m3_values()[layer.e4m3_codes(finite.astype(np.float32))] == finite).all()
    # half way between two codes: to the even one
    assert layer.e4m3_codes(np.float32([17.0 / 16, 19.0 / 16, -2.0 ** -10, 460.0])).tolist() == [0x38, 0x3A, 0x80, 0x7E]


def test_oracle_prepack_holds_the_layer():
    rng = np.random.default_rng(0)
    qw = rng.integers(0, 2 ** 32, (2, 128, 8), dtype=np.uint32).view(np.int32)
    sc = rng.integers(0, 2 ** 16, (2, 1, 64), dtype=np.uint16)
    p = layer.prepack(qw, None, sc, True)
    assert p.shape == (2, 1, 1, 17024)
    from oracle import unpack
    q = unpack(qw[1])
    # column 3 of up (layer column 35), row 77 = chunk 2, word 1, k 5 of 8: place 3 ^ 4, word place 1 ^ 1, nibble 6 of the order
    word = p[1, 0, 0, 8192 + 2 * 2048 + 7 * 16 + 0:][:4].copy().view(np.uint32)[0]
    assert word >> (4 * 6) & 15 == q[77, 35]
    assert p[1, 0, 0, 16384 + 64 + 1] >> 4 == 8 and p[1, 0, 0, 16384 + 20] == 0
    assert p[1, 0, 0, 16512 + 2 * (128 + 3):][:2].copy().view(np.uint16)[0] == sc[1, 0, 35]
