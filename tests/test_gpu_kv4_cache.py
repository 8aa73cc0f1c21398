"""Append to and read-back from the 4-bit cache, bit for bit against the oracle (every operation of the
definition is rounded by itself, so there is no tolerance)."""

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


def t16(a, bf16):
    return torch.from_numpy(a).cuda().to(torch.bfloat16 if bf16 else torch.float16)


def host(t):
    return t.float().cpu().numpy()


def expect(cache, q, k, v, positions, slots, table, interleaved, bf16):
    """The oracle's cache and rotated queries; cache is changed in place."""
    total = cache.shape[0] * cache.shape[2] * 16
    q = q.copy()
    for t, slot in enumerate(slots):
        ok = table is None or 0 <= positions[t] < len(table)
        turn = (lambda x: block.rope(x, table[positions[t]], interleaved)) if table is not None and ok else (lambda x: x)
        for h in range(q.shape[1]):
            q[t, h] = block.round16(turn(q[t, h]), bf16) if ok else 0
        if not ok or not 0 <= slot < total:
            continue
        for h in range(k.shape[1]):
            ku, ks, kz = block.kv4_quantize(turn(k[t, h]))
            vu, vs, vz = block.kv4_quantize(v[t, h])
            block.kv4_write(cache, int(slot), h, ku, ks, kz, vu, vs, vz)
    return q


CASES = [  # T, heads, kv_heads, dim, page, rot, interleaved, bf16
    (1, 1, 1, 64, 16, 64, False, False), (1, 32, 8, 128, 64, 128, False, False), (5, 4, 2, 128, 32, 64, True, True),
    (17, 6, 3, 64, 16, 32, False, True), (33, 2, 2, 128, 128, 128, True, False), (40, 5, 1, 64, 64, 64, True, False),
    (3, 8, 8, 128, 16, 96, False, True), (19, 3, 1, 128, 1024, 8, False, False), (7, 4, 4, 64, 32, 0, False, True),
    (129, 2, 1, 128, 64, 128, False, True),
]


@pytest.mark.parametrize("T,heads,kv_heads,dim,page,rot,interleaved,bf16", CASES)
def test_append_and_gather(awq, T, heads, kv_heads, dim, page, rot, interleaved, bf16):
    rng = np.random.default_rng(T * 7 + dim + rot)
    pages = -(-(T + 40) // page) + 1
    q, k, v = (block.round16(3 * rng.normal(size=(T, h, dim)).astype(np.float32), bf16) for h in (heads, kv_heads, kv_heads))
    k[..., 3] *= 16
    positions = rng.integers(0, 300, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    table = block.rope_table(300, rot) if rot else None
    before = rng.integers(0, 256, (pages, kv_heads, page // 16, 16 * dim + 128), dtype=np.uint8)
    cache = torch.from_numpy(before).cuda()
    got_q = awq.kv4_append(cache, t16(k, bf16), t16(v, bf16), torch.from_numpy(positions).cuda(),
                           torch.from_numpy(slots).cuda(), None if table is None else torch.from_numpy(table).cuda(),
                           q=t16(q, bf16), interleaved=interleaved)
    want_q = expect(before, q, k, v, positions, slots, table, interleaved, bf16)
    assert np.array_equal(host(got_q), want_q)
    assert np.array_equal(cache.cpu().numpy(), before)  # the other entries are as they were
    gk, gv = awq.kv4_gather(cache, torch.from_numpy(slots).cuda(), dtype=torch.bfloat16 if bf16 else torch.float16)
    for h in range(kv_heads):
        ku, ks, kz, vu, vs, vz = block.kv4_read(before, slots, h)
        assert np.array_equal(host(gk)[:, h], block.round16(block.kv4_dequant(ku, ks, kz), bf16))
        assert np.array_equal(host(gv)[:, h], block.round16(block.kv4_dequant(vu, vs, vz), bf16))


@pytest.mark.parametrize("T,heads,kv_heads,dim,rot,interleaved", [
    (6001, 1, 1, 64, 64, False), (6001, 2, 1, 64, 64, True), (300, 40, 23, 128, 48, False), (3000, 0, 3, 128, 128, False),
    (5000, 9, 0, 64, 32, True)])
def test_long_calls_are_their_pieces(awq, T, heads, kv_heads, dim, rot, interleaved):
    """Calls whose warps take parts of several tokens, some of them padding, against short calls of the same tokens."""
    gen = torch.Generator(device="cuda").manual_seed(T + heads)
    page, pages = 32, T // 32 + 9
    q, k, v = (torch.randn(T, h, dim, generator=gen, device="cuda").half() for h in (heads, kv_heads, kv_heads))
    positions = torch.randint(-5, 300, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T].contiguous()
    slots[torch.randint(0, T, (T // 10,), generator=gen, device="cuda")] = -1
    table = torch.from_numpy(block.rope_table(290, rot)).cuda()
    caches, outs = [], []
    for piece in (T, 64):
        cache = awq.kv4_cache(pages, max(kv_heads, 1), dim, page)
        out = torch.full_like(q, 7.0)
        for at in range(0, T, piece):
            to = min(T, at + piece)
            if kv_heads:
                awq.kv4_append(cache, k[at:to], v[at:to], positions[at:to], slots[at:to], table,
                               q=q[at:to] if heads else None, q_out=out[at:to] if heads else None, interleaved=interleaved)
            else:
                awq.lib.kv4_append(q[at:to].data_ptr(), None, None, heads * dim, 0, 0, positions[at:to].data_ptr(), None,
                                   table.data_ptr(), 290, rot, int(interleaved), out[at:to].data_ptr(), heads * dim, None,
                                   0, to - at, heads, 0, dim, page, 0, torch.cuda.current_stream().cuda_stream)
        caches.append(cache)
        outs.append(out)
    assert torch.equal(caches[0], caches[1]) and torch.equal(outs[0], outs[1])
    assert caches[0].any() == (kv_heads > 0) and (not heads or not (outs[0] == 7.0).all(dim=2).any())


def test_consecutive_prompt_tokens_from_one_projection(awq):
    """Columns of one qkv projection, queries in place, tokens of one page and across pages, an odd first slot."""
    rng = np.random.default_rng(1)
    T, heads, kv_heads, dim, page = 75, 4, 2, 128, 32
    qkv = block.round16(rng.normal(size=(T, heads + 2 * kv_heads, dim)).astype(np.float32), False)
    slots = np.concatenate([np.arange(2 * 32 + 5, 3 * 32), np.arange(0, 32), np.arange(4 * 32, 4 * 32 + T - 59)])
    positions = np.arange(9, 9 + T, dtype=np.int32)
    table = block.rope_table(100, dim)
    before = np.zeros((5, kv_heads, 2, 16 * dim + 128), np.uint8)
    cache = torch.from_numpy(before.copy()).cuda()
    dev = t16(qkv, False)
    q, k, v = dev.split((heads, kv_heads, kv_heads), dim=1)
    out = awq.kv4_append(cache, k, v, torch.from_numpy(positions).cuda(), torch.from_numpy(slots).cuda(),
                         torch.from_numpy(table).cuda(), q=q, q_out=q)
    want = expect(before, qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], positions, slots,
                  table, False, False)
    assert out.data_ptr() == dev.data_ptr() and np.array_equal(host(dev)[:, :heads], want)
    assert np.array_equal(host(dev)[:, heads:], qkv[:, heads:])
    assert np.array_equal(cache.cpu().numpy(), before)


def test_padding_and_positions_outside_the_table(awq):
    rng = np.random.default_rng(2)
    T, heads, kv_heads, dim, page, pages = 6, 2, 2, 64, 16, 3
    q, k, v = (block.round16(rng.normal(size=(T, h, dim)).astype(np.float32), False) for h in (heads, kv_heads, kv_heads))
    slots = np.array([-1, 48, 5, 6, 7, 1 << 40], np.int64)
    positions = np.array([3, 4, -1, 20, 19, 0], np.int32)
    table = block.rope_table(20, 64)
    before = rng.integers(0, 256, (pages, kv_heads, 1, 16 * dim + 128), dtype=np.uint8)
    cache = torch.from_numpy(before).cuda()
    got = awq.kv4_append(cache, t16(k, False), t16(v, False), torch.from_numpy(positions).cuda(),
                         torch.from_numpy(slots).cuda(), torch.from_numpy(table).cuda(), q=t16(q, False))
    want = expect(before, q, k, v, positions, slots, table, False, False)
    assert np.array_equal(host(got), want) and not want[2].any() and not want[3].any() and want[0].any()
    assert np.array_equal(cache.cpu().numpy(), before)
    gk, gv = awq.kv4_gather(cache, torch.from_numpy(slots).cuda())
    assert not host(gk)[[0, 1, 5]].any() and not host(gv)[[0, 1, 5]].any() and host(gk)[4].any()


@pytest.mark.parametrize("bf16", [False, True])
def test_extreme_heads(awq, bf16):
    """Equal channels, tiny and huge ranges, a NaN and infinities."""
    dim = 128
    rng = np.random.default_rng(3)
    k = np.zeros((8, 1, dim), np.float32)
    k[1] = 2.5
    k[2, 0] = np.linspace(-1e-6, 1e-6, dim)
    k[3, 0] = np.linspace(-60000, 60000, dim)
    k[4, 0, :] = rng.normal(size=dim)
    k[4, 0, 9] = np.nan
    k[5, 0, 100] = np.inf
    k[6, 0, 1] = -np.inf
    k[7, 0] = 1e30 if bf16 else 65504
    k[7, 0, 5] = -k[7, 0, 5]
    k = t16(k, bf16)
    k32 = host(k)
    v = k.flip(0).contiguous()
    cache = awq.kv4_cache(1, 1, dim, 16)
    slots = torch.arange(8, device="cuda")
    awq.kv4_append(cache, k, v, None, slots, None)
    want = np.zeros(tuple(cache.shape), np.uint8)
    for t in range(8):
        a, b = block.kv4_quantize(np.nan_to_num(k32[t, 0])), block.kv4_quantize(np.nan_to_num(k32[7 - t, 0]))
        block.kv4_write(want, t, 0, a[0], a[1], a[2], b[0], b[1], b[2])
    got = cache.cpu().numpy()
    fine = [0, 1, 2, 3, 7]
    g, w = block.kv4_read(got, np.arange(8), 0), block.kv4_read(want, np.arange(8), 0)
    for i in range(3):
        assert np.array_equal(g[i][fine], w[i][fine])
        assert np.array_equal(g[3 + i][[7 - t for t in fine]], w[3 + i][[7 - t for t in fine]])
    gk, gv = awq.kv4_gather(cache, slots, dtype=k.dtype)
    for t in (4, 5, 6):
        assert np.isnan(host(gk)[t]).all() and np.isnan(host(gv)[7 - t]).all()
        assert not g[0][t].any()


def test_a_cache_beyond_32_bit_offsets(awq):
    """Entries more than 4 GiB into the cache."""
    kv_heads, dim, page = 8, 128, 128
    pages = (5 << 30) // (kv_heads * (page // 16) * (16 * dim + 128))
    cache = torch.empty((pages, kv_heads, page // 16, 16 * dim + 128), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * page - 1, 3, (pages - 2) * page + 17], device="cuda")
    rng = np.random.default_rng(4)
    k, v = (block.round16(rng.normal(size=(3, kv_heads, dim)).astype(np.float32), False) for _ in range(2))
    awq.kv4_append(cache, t16(k, False), t16(v, False), None, slots, None)
    gk, gv = awq.kv4_gather(cache, slots)
    for got, x in ((gk, k), (gv, v)):
        u, s, z = block.kv4_quantize(x)
        want = z.astype(np.float32)[..., None] + u.astype(np.float32) * s.astype(np.float32)[..., None]
        assert np.array_equal(host(got), block.round16(want, False))


def test_wrong_operands_are_refused(awq):
    cache = awq.kv4_cache(2, 2, 64, 16)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: awq.kv4_append(cache.view(torch.int8), k, k, None, slots, None),
                lambda: awq.kv4_append(cache, k, k.bfloat16(), None, slots, None),
                lambda: awq.kv4_append(cache, k, k, None, slots.int(), None),
                lambda: awq.kv4_append(cache, k, k, slots, slots, torch.zeros(4, 64, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: awq.kv4_append(cache, k[:, :1], k[:, :1], None, slots, None),
                lambda: awq.kv4_append(cache, k, k, None, slots[:2], None),
                lambda: awq.kv4_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, None, slots, None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(awq.AwqError):
        awq.kv4_cache(2, 2, 80, 16)
    assert awq.kv4_append(cache, k[:0], k[:0], None, slots[:0], None) is None
