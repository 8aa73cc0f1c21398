"""Pins of the block operators' oracle: hand-worked values, closed forms, brute force (no GPU)."""

import numpy as np
import pytest

from oracle import block, pack

f32 = np.float32


def test_rmsnorm_hand_worked():
    x = np.array([[3.0, 4.0, 0.0, 0.0]], f32)           # mean of squares 25 / 4
    w = np.array([1.0, 2.0, 5.0, 1.0], f32)
    y, h = block.rmsnorm(x, None, w, 0.0)
    assert np.allclose(y, [[1.2, 3.2, 0.0, 0.0]], atol=1e-15) and np.array_equal(h, x)
    codes, s = block.rmsnorm_codes(x, None, w, 0.0)
    assert codes.tolist() == [[48, 127, 0, 0]]          # 1.2 / (3.2 / 127) = 47.625
    assert np.allclose(s, 3.2 / 127, rtol=1e-7)


def test_rmsnorm_residual_and_zero_row():
    x = np.array([[1.0, -2.0], [0.5, 0.5]], f32)
    r = np.array([[2.0, -2.0], [-0.5, -0.5]], f32)
    codes, s = block.rmsnorm_codes(x, r, np.ones(2, f32), 1e-6)
    assert codes.tolist() == [[95, -127], [0, 0]] and s[1] == 0.0   # 3 * 127 / 4 = 95.25


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_quarter_turn_and_rest(interleaved):
    x = np.arange(1.0, 9.0, dtype=f32)
    row = np.array([0, 1, 1, 0], f32)  # pair 0 turns by 90 degrees, pair 1 stays
    got = block.rope(x, row, interleaved)
    want = [-2, 1, 3, 4] if interleaved else [-3, 2, 1, 4]
    assert got.tolist() == want + [5, 6, 7, 8]


def test_rope_keeps_inner_products_of_equal_shifts():
    rng = np.random.default_rng(0)
    table = block.rope_table(64, 32)
    q, k = rng.normal(size=32).astype(f32), rng.normal(size=32).astype(f32)
    a = block.rope(q, table[9], False).astype(np.float64) @ block.rope(k, table[2], False)
    b = block.rope(q, table[47], False).astype(np.float64) @ block.rope(k, table[40], False)
    assert abs(a - b) < 1e-4


def test_quantize_hand_worked():
    x = np.array([-1.0, 0.0, 0.4, 14.0, 13.5, 6.49], f32)  # scale 1, zero -1
    codes, s, z = block.kv4_quantize(x)
    assert (float(s), float(z)) == (1.0, -1.0)
    assert codes.tolist() == [0, 1, 1, 15, 14, 7]           # 14.5 rounds to the even 14
    codes, s, z = block.kv4_quantize(np.full(4, 2.5, f32))
    assert codes.tolist() == [0] * 4 and (float(s), float(z)) == (0.0, 2.5)


@pytest.mark.parametrize("dim", [64, 128])
def test_places_are_a_permutation_and_keys_are_awq_words(dim):
    seen = set()
    for value in (False, True):
        for t in range(16):
            for c in range(dim):
                byte, shift = block.kv4_place(dim, t, c, value)
                assert (8 * dim if value else 0) <= byte < (16 * dim if value else 8 * dim)
                seen.add((byte, shift))
    assert len(seen) == 2 * 16 * dim
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (1, 1, 16, dim), dtype=np.uint8)
    cache = block.kv4_pack(codes, codes[..., ::-1].copy(), np.zeros((1, 1, 16, 4), np.float16))
    words = np.ascontiguousarray(cache[0, 0, 0, :8 * dim]).view(np.int32).reshape(16, dim // 8)
    assert np.array_equal(words, pack(codes[0, 0]))


def test_value_halves_hand_worked():
    # dim 64: 8 channels for each group of lanes; token 11, channel 21: half index [1][2][1][1], parity 1
    assert block.kv4_place(64, 11, 21, True) == (8 * 64 + 4 * (((8 + 2) * 4 + 1) * 2 + 1) + 2, 4)
    assert block.kv4_place(128, 0, 0, True) == (1024, 0)
    assert block.kv4_place(128, 15, 127, True) == (2047, 4)


def test_write_equals_pack_and_reads_back():
    rng = np.random.default_rng(2)
    dim, pages, heads, size = 64, 2, 3, 32
    k, v = (rng.integers(0, 16, (pages, heads, size, dim), dtype=np.uint8) for _ in range(2))
    meta = rng.normal(size=(pages, heads, size, 4)).astype(np.float16)
    cache = block.kv4_pack(k, v, meta)
    other = rng.integers(0, 256, cache.shape, dtype=np.uint8)
    for p in range(pages):
        for h in range(heads):
            for t in range(size):
                m = meta[p, h, t]
                block.kv4_write(other, p * size + t, h, k[p, h, t], m[0], m[1], v[p, h, t], m[2], m[3])
    assert np.array_equal(cache, other)
    ku, ks, kz, vu, vs, vz = block.kv4_read(cache, [37, 0, 63], 1)
    for i, (p, t) in enumerate(((1, 5), (0, 0), (1, 31))):
        assert np.array_equal(ku[i], k[p, 1, t]) and np.array_equal(vu[i], v[p, 1, t])
        assert [ks[i], kz[i], vs[i], vz[i]] == meta[p, 1, t].astype(f32).tolist()


def test_attention_special_cases():
    rng = np.random.default_rng(3)
    dim, size = 64, 16
    k, v = (rng.integers(0, 16, (3, 1, size, dim), dtype=np.uint8) for _ in range(2))
    meta = np.ones((3, 1, size, 4), np.float16)
    cache = block.kv4_pack(k, v, meta)
    table = np.array([[2, 0]], np.int32)
    flat = np.concatenate([v[2, 0], v[0, 0]]) + 1.0
    q = np.zeros((3, 2, dim), f32)
    # queries of zeros weigh every visible value alike; the first of three sees two keys fewer
    out, lse, _, _ = block.kv4_attention(q, cache, table, [20], [0, 3], 0.125)
    for i in range(3):
        assert np.allclose(out[i, 0], flat[:18 + i].mean(axis=0)) and np.allclose(lse[i], np.log(18 + i))
    out, _, _, _ = block.kv4_attention(q, cache, table, [20], [0, 3], 0.125, window=4)
    assert np.allclose(out[2, 1], flat[16:20].mean(axis=0))
    # a length below the number of queries leaves the first rows empty
    out, lse, _, _ = block.kv4_attention(q, cache, table, [1], [0, 3], 0.125)
    assert not out[:2].any() and np.all(lse[:2] == -np.inf) and np.allclose(out[2, 0], flat[0])
    # a brute-force softmax
    q = rng.normal(size=(1, 2, dim)).astype(f32)
    out, lse, _, _ = block.kv4_attention(q, cache, table, [29], [0, 1], 0.05)
    keys = (np.concatenate([k[2, 0], k[0, 0]]) + 1.0)[:29]
    e = np.array([np.exp(0.05 * sum(float(q[0, 1, d]) * keys[j, d] for d in range(dim))) for j in range(29)])
    assert np.allclose(out[0, 1], (e[:, None] * flat[:29]).sum(0) / e.sum()) and np.isclose(lse[0, 1], np.log(e.sum()))


# mistakes planted in the restatement: each one has to change a pinned result

def _no_offset(dim, token, channel, value):
    byte, shift = PLACE(dim, token, channel, value)
    return byte, 4 - shift


PLACE = block.kv4_place


@pytest.mark.parametrize("plant", ["nibble", "half_up", "window", "group"])
def test_planted_mistakes_are_seen(plant, monkeypatch):
    rng = np.random.default_rng(4)
    if plant == "nibble":
        monkeypatch.setattr(block, "kv4_place", _no_offset)
        codes = rng.integers(0, 16, (1, 1, 16, 64), dtype=np.uint8)
        cache = block.kv4_pack(codes, codes, np.zeros((1, 1, 16, 4), np.float16))
        assert not np.array_equal(np.ascontiguousarray(cache[0, 0, 0, :512]).view(np.int32).reshape(16, 8), pack(codes[0, 0]))
    elif plant == "half_up":
        monkeypatch.setattr(block.np, "rint", lambda a: np.floor(a + 0.5))
        assert block.kv4_quantize(np.array([-1.0, 14.0, 13.5], f32))[0].tolist() != [0, 15, 14]
    else:
        k, v = (rng.integers(0, 16, (1, 2, 32, 64), dtype=np.uint8) for _ in range(2))
        cache = block.kv4_pack(k, v, np.ones((1, 2, 32, 4), np.float16))
        q = rng.normal(size=(1, 4, 64)).astype(f32)
        table = np.zeros((1, 1), np.int32)
        right = block.kv4_attention(q, cache, table, [32], [0, 1], 0.1, window=8)[0]
        if plant == "window":
            wrong = block.kv4_attention(q, cache, table, [32], [0, 1], 0.1, window=9)[0]
        else:
            wrong = block.kv4_attention(q, cache[:, ::-1].copy(), table, [32], [0, 1], 0.1, window=8)[0]
        assert np.abs(right - wrong).max() > 1e-3
