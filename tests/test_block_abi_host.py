"""Host-side checks of the block operators' C ABI: refusals before anything is launched (no GPU)."""

import pytest

from bit_weight_only_awq_gb300 import build as awq_build

EINVAL, EALIGN, EWORKSPACE, ENULL = -1, -2, -6, -7
FAKE = 1 << 40          # an aligned address that is never dereferenced (checks run first)
OFF = FAKE + 4


@pytest.fixture(scope="module")
def lib():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq
    return awq.lib


def _norm(lib, x=FAKE, res=FAKE, w=FAKE, ro=FAKE, y=None, xq=FAKE, s=FAKE, M=4, K=4096, xs=None, rs=None, eps=1e-6,
          dtype=0):
    return lib.w4a8_rmsnorm_quant(x, res, w, ro, y, xq, s, M, K, K if xs is None else xs, K if rs is None else rs, eps,
                                  dtype, None)


def test_rmsnorm_refusals(lib):
    for bad in ({"M": -1}, {"K": 0}, {"K": 4100}, {"K": 65544}, {"xs": 4088}, {"xs": 4100}, {"rs": 8}, {"rs": 4097},
                {"eps": -1.0}, {"eps": float("nan")}, {"dtype": 2}):
        assert _norm(lib, **bad) == EINVAL, bad
    for name in ("x", "w", "xq", "s"):
        assert _norm(lib, **{name: None}) == ENULL, name
    for name in ("x", "res", "w", "ro", "y", "xq"):
        assert _norm(lib, **{name: OFF}) == EALIGN, name
    assert _norm(lib, s=FAKE + 2) == EALIGN
    assert _norm(lib, M=0, x=None, xq=None, s=None) == 0
    f = lib.awq_rmsnorm
    assert f(FAKE, None, FAKE, None, None, 4, 64, 64, 0, 1e-6, 0, None) == ENULL
    assert f(FAKE, None, FAKE, None, FAKE, 4, 60, 64, 0, 1e-6, 0, None) == EINVAL


def _append(lib, q=FAKE, k=FAKE, v=FAKE, qs=4096, ks=1024, vs=1024, pos=FAKE, slots=FAKE, table=FAKE, max_pos=100,
            rot=128, il=0, qo=FAKE, qos=4096, cache=FAKE, pages=9, T=3, heads=32, kv_heads=8, dim=128, page=64, dtype=0):
    return lib.kv4_append(q, k, v, qs, ks, vs, pos, slots, table, max_pos, rot, il, qo, qos, cache, pages, T, heads,
                          kv_heads, dim, page, dtype, None)


def test_append_refusals(lib):
    for bad in ({"dim": 96}, {"dim": 256}, {"page": 8}, {"page": 48}, {"page": 2048}, {"heads": -1}, {"kv_heads": -1},
                {"rot": 136}, {"rot": 4}, {"rot": -8}, {"qs": 4088}, {"ks": 1020}, {"vs": 1028}, {"qos": 8}, {"T": -1},
                {"pages": -1}, {"dtype": 7}, {"max_pos": -1}):
        assert _append(lib, **bad) == EINVAL, bad
    for name in ("q", "k", "v", "pos", "slots", "table", "qo", "cache"):
        assert _append(lib, **{name: None}) == ENULL, name
    for name in ("q", "k", "v", "table", "qo", "cache", "slots"):
        assert _append(lib, **{name: OFF}) == EALIGN, name
    assert _append(lib, pos=FAKE + 2) == EALIGN
    assert _append(lib, T=0, q=None, k=None) == 0
    assert _append(lib, heads=0, kv_heads=0, q=None, k=None, v=None) == 0


def test_gather_refusals(lib):
    f = lib.kv4_gather  # cache, slots, k, v, pages, T, kv_heads, dim, page, dtype, stream
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 2, 8, 100, 64, 0, None) == EINVAL
    assert f(FAKE, FAKE, FAKE, FAKE, 4, -2, 8, 128, 64, 0, None) == EINVAL
    assert f(None, FAKE, FAKE, FAKE, 4, 2, 8, 128, 64, 0, None) == ENULL
    assert f(FAKE, None, FAKE, FAKE, 4, 2, 8, 128, 64, 0, None) == ENULL
    assert f(FAKE, FAKE, OFF, FAKE, 4, 2, 8, 128, 64, 0, None) == EALIGN
    assert f(FAKE, FAKE, None, None, 4, 2, 8, 128, 64, 0, None) == 0


def _attention(lib, q=FAKE, qs=4096, cache=FAKE, table=FAKE, ts=64, kv=FAKE, start=FAKE, out=FAKE, lse=None, T=5, B=3,
               max_q=4, heads=32, kv_heads=8, dim=128, pages=100, page=64, max_pages=64, scale=0.1, window=0, dtype=0,
               ws=FAKE, wsb=1 << 40):
    return lib.kv4_attention(q, qs, cache, table, ts, kv, start, out, lse, T, B, max_q, heads, kv_heads, dim, pages, page,
                             max_pages, scale, window, dtype, ws, wsb, None)


def test_attention_refusals(lib):
    for bad in ({"heads": 30}, {"heads": 0}, {"kv_heads": 0}, {"dim": 80}, {"B": 4097}, {"B": -1}, {"T": -1}, {"max_q": 0},
                {"qs": 4000}, {"qs": 4100}, {"max_pages": 0}, {"ts": 63}, {"scale": float("inf")},
                {"scale": float("nan")}, {"window": -1}, {"dtype": -1}, {"pages": 0}, {"page": 24},
                {"max_pages": 1 << 30, "ts": 1 << 30}, {"start": None}, {"start": None, "T": 3}):
        assert _attention(lib, **bad) == EINVAL, bad
    for name in ("q", "cache", "table", "kv", "out"):
        assert _attention(lib, **{name: None}) == ENULL, name
    for name in ("q", "cache", "out"):
        assert _attention(lib, **{name: OFF}) == EALIGN, name
    for name in ("table", "kv", "start", "lse"):
        assert _attention(lib, **{name: FAKE + 2}) == EALIGN, name
    assert _attention(lib, T=0, q=None) == 0
    assert _attention(lib, B=0, q=None) == 0
    need = lib.kv4_attention_workspace_bytes(5, 3, 4, 32, 8, 128)
    if need:
        assert _attention(lib, ws=None) == EWORKSPACE
        assert _attention(lib, wsb=need - 1) == EWORKSPACE
        assert _attention(lib, ws=FAKE + 16) == EALIGN
    assert lib.kv4_attention_workspace_bytes(5, 3, 4, 30, 8, 128) == 0


def test_cache_bytes(lib):
    assert lib.kv4_cache_bytes(10, 8, 128, 64) == 10 * 8 * 4 * (16 * 128 + 128)
    assert lib.kv4_cache_bytes(3, 2, 64, 16) == 3 * 2 * (16 * 64 + 128)
    for bad in ((1, 8, 96, 64), (1, 0, 128, 64), (-1, 8, 128, 64), (1, 8, 128, 40)):
        assert lib.kv4_cache_bytes(*bad) == 0
