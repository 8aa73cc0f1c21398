"""Attention over the 4-bit cache where a row's neighbours, the cache's signs and the arguments' limits could reach into
its result.  Bounds: those of test_gpu_kv4_attention, with the largest value taken over the compared rows alone.
"""

import numpy as np
import pytest

from oracle import block
from tests.test_gpu_kv4_attention import Problem, awq  # noqa: F401  (awq is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def meta_of(p):
    """float16 [pages, kv_heads, page_size, 4] over the cache: key scale, key zero, value scale, value zero."""
    meta = p.cache[..., 16 * p.dim:].view(np.float16)
    return meta.reshape(*p.cache.shape[:2], p.page, 4)


def put_meta(p, meta):
    p.cache[..., 16 * p.dim:] = np.ascontiguousarray(meta.reshape(*p.cache.shape[:3], 64)).view(np.uint8)


def check_rows(awq, p, rows, window=0, cache=None):  # noqa: F811
    """The rows (a boolean for each query token) against float64; `cache` has other values where they do not see."""
    out, lse = p.run(awq, window)
    cache = p.cache if cache is None else cache
    want, want_lse, mag, reach = block.kv4_attention(p.q, cache, p.table, p.lens, p.start, p.scale, window)
    got, got_lse = out.float().cpu().numpy()[rows], lse.cpu().numpy()[rows]
    want, want_lse, mag, reach = want[rows], want_lse[rows], mag[rows], reach[rows]
    assert np.all(np.isfinite(want))
    delta = reach * (8 + p.dim / 8) * 2.0 ** -23
    half_ulp = 2.0 ** -8 if p.bf16 else 2.0 ** -11
    bound = mag * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -17) + half_ulp * np.abs(want) + 2.0 ** -24 * (1 + mag.max())
    worst = np.max(np.abs(got - want) / bound)
    assert worst <= 1.0, worst
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(np.abs(got_lse - want_lse)[~empty] <= (delta + 2.0 ** -17 + 2.0 ** -22 * np.abs(want_lse))[~empty])
    assert awq.awq_last_device_error() == 0


def test_places_beyond_32_bits(awq):  # noqa: F811
    """A prompt whose column blocks times tiles of the cache are more than 2^31, and its rows more than 2^20; a window
    keeps the work small.  Rows all over it against float64 on the pages that they see."""
    heads, dim, page, T, before, window = 1, 64, 1024, 1_500_001, 37, 100
    length = T + before
    assert -(-T // 16) * -(-length // 64) > 2 ** 31
    pages = -(-length // page)
    gen = torch.Generator(device="cuda").manual_seed(36)
    cache = torch.randint(0, 256, (pages, 1, page // 16, 16 * dim + 128), generator=gen, device="cuda", dtype=torch.uint8)
    meta = cache[..., 16 * dim:].view(torch.float16).unflatten(-1, (16, 2, 2))
    sigma = torch.exp(0.3 * torch.randn(meta.shape[:-1], generator=gen, device="cuda"))
    meta[..., 0] = (sigma / 4.6).half()
    meta[..., 1] = (-7.5 * sigma / 4.6).half()
    table = torch.randperm(pages, generator=gen, device="cuda").int()[None]
    q = (2 * torch.randn(T, heads, dim, generator=gen, device="cuda")).half()
    lens, start = torch.tensor([length], dtype=torch.int32).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda()
    lse = torch.full((T, heads), 5.0, device="cuda")
    out = torch.full_like(q, float("nan"))
    awq.kv4_attention(q, cache, table, lens, q_start=start, max_q=T, window=window, out=out, lse=lse)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    rng = np.random.default_rng(37)
    for row in [0, 1, 62, 63, 255, 256, T - 1, T - 2, T - 256, 1 << 20, (1 << 20) - 1, *rng.integers(0, T, 60)]:
        pos = before + int(row)
        first = max(0, pos - window + 1) // page
        need = table[0, first:pos // page + 1].long()
        args = (q[row:row + 1].float().cpu().numpy(), cache[need].cpu().numpy(), np.arange(len(need))[None],
                np.array([pos + 1 - first * page]), np.array([0, 1]), dim ** -0.5, window)
        want, want_lse, mag, reach = block.kv4_attention(*args)
        delta = reach * (8 + dim / 8) * 2.0 ** -23
        bound = mag * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -17) + 2.0 ** -11 * np.abs(want) + 2.0 ** -24 * (1 + mag.max())
        assert np.all(np.abs(out[row:row + 1].float().cpu().numpy() - want) <= bound), row
        assert np.all(np.abs(lse[row:row + 1].cpu().numpy() - want_lse) <= delta + 2.0 ** -17 + 2.0 ** -22 * np.abs(want_lse))
    assert awq.awq_last_device_error() == 0


@pytest.mark.parametrize("lens,news,heads,kv_heads,dim", [([5, 40], [9, 3], 2, 1, 64), ([60], [140], 8, 2, 128), ([3], [9], 8, 2, 128)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 1 << 30])
def test_windows_up_to_the_largest_integer(awq, lens, news, heads, kv_heads, dim, window):  # noqa: F811
    """A window wider than any sequence hides nothing, also where there are more queries than tokens."""
    p = Problem(lens, news, heads, kv_heads, dim, 16, seed=31)
    out, lse = p.run(awq, window)
    want, want_lse = p.run(awq, 0)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    p.check(awq, window=window)


@pytest.mark.parametrize("new", [1, 3, 12, 70])
@pytest.mark.parametrize("small", [-0.001, -8.0])
def test_scales_of_either_sign(awq, new, small):  # noqa: F811
    """Scales as a cache of the caller's own may have them: every second eight tokens have negative ones, small or large."""
    p = Problem([200, 90], [new, new], 8, 2, 128, 64, seed=32, q_scale=0.2)
    meta = meta_of(p).copy()
    odd = np.arange(p.page) // 8 % 2 == 1
    for at, scale in ((0, 0.3), (2, 8.0)):
        meta[..., at] = np.where(np.isnan(meta[..., at]), meta[..., at], np.float16(scale))
        meta[:, :, odd, at] *= np.float16(small / 8.0)
        meta[..., at + 1] = np.where(np.isinf(meta[..., at + 1]), meta[..., at + 1], meta[..., at] * np.float16(-7.0))
    put_meta(p, meta)
    assert (meta[..., 2] < 0).any() and (meta[..., 2] > 0).any()
    p.check(awq)
    p.check(awq, window=33)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("heads", [2, 6, 16])
@pytest.mark.parametrize("new", [2, 5, 120])
@pytest.mark.parametrize("scale", [np.nan, np.inf, -np.inf, 65504.0])
def test_a_hidden_scale_takes_no_bits_from_a_row(awq, new, heads, scale, bf16):  # noqa: F811
    """Value scales near 0.003 beside one that is not finite, or the largest there is: rows that do not see it are as
    exact as without it, whether it lies after them or has left their window."""
    p = Problem([200, 150], [new, new], heads, 2, 64, 16, bf16=bf16, seed=33, q_scale=0.5)
    meta = meta_of(p).copy()
    meta[..., 2:] = np.where(np.isfinite(meta[..., 2:]), meta[..., 2:] * np.float16(0.01), meta[..., 2:])
    put_meta(p, meta)
    check_rows(awq, p, np.ones(2 * new, bool))
    cache = p.cache.copy()
    last = meta.copy()
    last[p.table[0, 199 // 16], :, 199 % 16, 2] = scale
    put_meta(p, last)
    rows = np.arange(2 * new) != new - 1
    check_rows(awq, p, rows, cache=cache)
    if np.isnan(scale):
        assert np.isnan(p.run(awq)[0].float().cpu().numpy()[new - 1]).all()
    # with a window, the oldest token that the first query sees is seen by no other
    window = 80 - new // 2
    at = 200 - new - window + 1
    if at >= 0:
        first = meta.copy()
        first[p.table[0, at // 16], :, at % 16, 2] = scale
        put_meta(p, first)
        check_rows(awq, p, np.arange(2 * new) != 0, window, cache)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("new", [1, 5, 100])
def test_small_query_elements_keep_their_bits(awq, new, bf16):  # noqa: F811
    """Elements of 2^-24 of the row's largest, where the largest meets keys that are 0: the score is theirs alone, and
    is to be as exact as fp32 sums are."""
    p = Problem([150], [new], 4, 2, 128, 64, bf16=bf16, seed=38, junk=False)
    meta = meta_of(p).copy()
    meta[..., 0], meta[..., 1] = 8.0, 0.0
    put_meta(p, meta)
    # channel 0's codes are 0: nibble 0 of the first word of each token's key
    keys = p.cache[..., :8 * p.dim].reshape(*p.cache.shape[:3], 16, p.dim // 2)
    keys[..., 0] &= 0xF0
    p.cache[..., :8 * p.dim] = keys.reshape(*p.cache.shape[:3], 8 * p.dim)
    rng = np.random.default_rng(39)
    digits = 2 ** 7 if bf16 else 2 ** 10
    small = (1 + rng.integers(0, digits, p.q.shape) / digits) * rng.choice([-1, 1], p.q.shape)
    p.q = (small * 2.0 ** -10).astype(np.float32)
    p.q[..., 0] = 2.0 ** 14
    assert np.array_equal(p.q, block.round16(p.q, bf16))
    p.scale = 1.0
    out, lse = p.run(awq, scale=1.0)
    want, want_lse, mag, reach = block.kv4_attention(p.q, p.cache, p.table, p.lens, p.start, 1.0)
    delta = reach * (8 + p.dim / 8) * 2.0 ** -23
    assert reach.max() < 40
    assert np.all(np.abs(lse.cpu().numpy() - want_lse) <= delta + 2.0 ** -17 + 2.0 ** -22 * np.abs(want_lse))
    half_ulp = 2.0 ** -8 if bf16 else 2.0 ** -11
    bound = mag * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -17) + half_ulp * np.abs(want) + 2.0 ** -24 * (1 + mag.max())
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= bound)
