"""Attention over the 4-bit cache against the oracle's float64.

Tolerance, element by element.  The score of a key is a sum of D products in fp32, at most 8 + D / 8 roundings of
at most 2^-23 of reach = |scale| max_j sum_d |q_d| (u scale + |zero|): every weight is off by at most delta =
reach (8 + D / 8) 2^-23 relative, in the numerator and in the denominator.  A weight times a value's scale is
rounded to fp16 (2^-11), the exponential and the fp32 sums cost less than 2^-17 together.  So the output is off by
at most mag (2 delta + 2^-11 + 2^-17), mag = sum_j p_j (u scale + |zero|), plus half an ulp of its type; weights
too small for fp16 add less than 2^-24 of the largest value.
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


class Problem:
    def __init__(self, lens, news, heads, kv_heads, dim, page, bf16=False, seed=0, q_scale=2.0, spread=0.3, junk=True):
        rng = np.random.default_rng(seed)
        self.bf16, self.dim, self.page = bf16, dim, page
        need = [max(1, -(-n // page)) for n in lens]
        pool = sum(need) + 2
        order = rng.permutation(pool).astype(np.int32)
        width = max(need) + 1
        # entries that no token needs are outside the pool
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        kc, vc = (np.clip(np.rint(rng.normal(7.5, 2.7, (pool, kv_heads, page, dim))), 0, 15).astype(np.uint8) for _ in range(2))
        sigma = np.exp(spread * rng.normal(size=(pool, kv_heads, page, 2)))
        meta = np.empty((pool, kv_heads, page, 4), np.float16)
        meta[..., 0::2] = sigma / 2.7
        meta[..., 1::2] = -7.5 * sigma / 2.7 + 0.1 * rng.normal(size=sigma.shape)
        if junk:  # what lies behind a sequence's last token must not matter
            used = np.zeros((pool, page), bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    used[self.table[b, j // page], j % page] = True
            for p in range(pool):
                meta[p, :, ~used[p]] = np.array([np.nan, np.inf, np.nan, -np.inf], np.float16)
        self.cache = block.kv4_pack(kc, vc, meta)
        self.lens = np.array(lens, np.int32)
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.q = block.round16(q_scale * rng.normal(size=(int(self.start[-1]), heads, dim)).astype(np.float32), bf16)
        self.max_q = max(list(news) + [1])
        self.scale = dim ** -0.5

    def run(self, awq, window=0, start=True, **kw):
        q = torch.from_numpy(self.q).cuda().to(torch.bfloat16 if self.bf16 else torch.float16)
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        out = awq.kv4_attention(q, torch.from_numpy(self.cache).cuda(), torch.from_numpy(self.table).cuda(),
                                torch.from_numpy(self.lens).cuda(),
                                q_start=torch.from_numpy(self.start).cuda() if start else None,
                                max_q=self.max_q if start else 1, window=window, lse=lse, **kw)
        return out, lse

    def check(self, awq, window=0, start=True):
        out, lse = self.run(awq, window, start)
        want, want_lse, mag, reach = block.kv4_attention(self.q, self.cache, self.table, self.lens, self.start,
                                                         self.scale, window)
        got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
        delta = reach * (8 + self.dim / 8) * 2.0 ** -23
        half_ulp = 2.0 ** -8 if self.bf16 else 2.0 ** -11
        largest = mag.max() if mag.size else 0.0
        bound = mag * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -17) + half_ulp * np.abs(want) + 2.0 ** -24 * (1 + largest)
        assert np.all(np.isfinite(got))
        worst = np.max((np.abs(got - want) / bound)) if got.size else 0.0
        assert worst <= 1.0, worst
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        assert np.all(np.abs(got_lse - want_lse)[~empty] <= (delta + 2.0 ** -17 + 2.0 ** -22 * np.abs(want_lse))[~empty])
        assert not got[empty].any()
        again, lse2 = self.run(awq, window, start)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert awq.awq_last_device_error() == 0


DECODE = [  # lens, heads, kv_heads, dim, page, bf16
    ([1], 1, 1, 64, 16, False), ([177], 8, 2, 128, 16, False), ([64], 4, 4, 128, 64, True), ([65], 2, 1, 64, 32, False),
    ([0, 5, 0], 4, 2, 128, 32, False), ([15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 129], 4, 4, 64, 16, True),
    ([1000, 3, 700], 32, 8, 128, 64, False), ([515], 71, 1, 64, 64, False), ([2049], 20, 4, 128, 128, True),
    ([333, 1], 24, 2, 128, 192, False), ([900], 16, 16, 64, 256, False), ([5000, 1234], 10, 2, 128, 1024, False),
]


@pytest.mark.parametrize("lens,heads,kv_heads,dim,page,bf16", DECODE)
def test_single_tokens(awq, lens, heads, kv_heads, dim, page, bf16):
    p = Problem(lens, [1] * len(lens), heads, kv_heads, dim, page, bf16, seed=sum(lens))
    p.check(awq, start=False)
    p.check(awq, window=1)
    p.check(awq, window=50)
    p.check(awq, window=100000)


MULTI = [  # (lens, new tokens), heads, kv_heads, dim, page, bf16, window
    (([9], [9]), 2, 1, 64, 16, False, 0), (([40, 3, 200], [2, 3, 5]), 8, 2, 128, 32, False, 0),
    (([70, 0, 5], [4, 0, 8]), 4, 4, 64, 16, True, 0), (([300], [7]), 16, 2, 128, 64, True, 33),
    (([130, 260], [130, 31]), 4, 1, 128, 64, False, 0), (([513, 64], [257, 64]), 6, 2, 64, 16, False, 100),
    (([400], [400]), 8, 8, 128, 128, True, 0), (([600, 31], [100, 1]), 5, 1, 128, 32, False, 17),
    (([3], [200]), 4, 2, 128, 16, False, 0), (([1100, 700, 65], [300, 129, 2]), 8, 2, 128, 64, False, 0),
    (([257], [256]), 7, 7, 64, 64, True, 1), (([0], [70]), 8, 2, 64, 16, False, 0),
    # single tokens, a few, and prompts in one call
    (([900, 500, 64, 1, 0, 200, 33], [300, 1, 5, 1, 1, 200, 13]), 8, 2, 128, 64, False, 0),
    (([700, 500, 64, 2, 200, 900], [100, 1, 40, 2, 0, 33]), 4, 2, 64, 16, True, 90),
    (([300, 77, 1000], [120, 1, 2]), 64, 1, 128, 32, False, 0), (([300, 77], [60, 1]), 12, 1, 64, 32, False, 0),
]


@pytest.mark.parametrize("shape,heads,kv_heads,dim,page,bf16,window", MULTI)
def test_several_new_tokens(awq, shape, heads, kv_heads, dim, page, bf16, window):
    p = Problem(shape[0], shape[1], heads, kv_heads, dim, page, bf16, seed=len(shape[0]) + heads)
    p.check(awq, window=window)


def test_many_sequences(awq):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 301)]
    Problem(lens, [1] * 301, 8, 4, 64, 16, seed=1).check(awq)
    Problem(lens, [int(x) for x in rng.integers(0, 4, 301)], 4, 2, 64, 32, seed=2).check(awq)


def test_more_heads_and_sequences_than_the_gpu_has_places(awq):
    Problem([150] * 40, [1] * 40, 32, 32, 64, 64, seed=5).check(awq)


def test_a_long_sequence_and_short_ones(awq):
    Problem([20000, 1, 17, 300], [1, 1, 1, 1], 8, 2, 64, 64, seed=3).check(awq)
    Problem([9000], [1], 1, 1, 128, 64, seed=4).check(awq)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("new", [1, 90])
def test_peaked_and_flat_scores(awq, bf16, new):
    Problem([700, 90], [new, new], 8, 2, 128, 64, bf16, seed=6, q_scale=60.0).check(awq)
    Problem([700, 90], [new, new], 8, 2, 128, 64, bf16, seed=7, q_scale=1e-3).check(awq)


@pytest.mark.parametrize("new", [1, 70])
def test_scales_of_very_different_size(awq, new):
    """Keys and values whose scales differ by factors of thousands from token to token."""
    Problem([800], [new], 8, 2, 128, 64, seed=8, q_scale=0.2, spread=1.6).check(awq)
    Problem([800], [new], 8, 2, 64, 16, seed=9, q_scale=0.2, spread=1.6, bf16=True).check(awq)


@pytest.mark.parametrize("new", [1, 3, 100])
def test_a_visible_nan_shows_and_a_hidden_one_does_not(awq, new):
    p = Problem([200, 150], [new, new], 4, 2, 64, 16, seed=10)
    page, token = p.table[0, 30 // 16], 30 % 16
    p.cache[page, 0, 0, 16 * 64 + 8 * token: 16 * 64 + 8 * token + 2] = np.array([np.nan], np.float16).view(np.uint8)
    out, _ = p.run(awq)
    got = out.float().cpu().numpy()
    assert np.isnan(got[:new, :2]).all() and np.isfinite(got[:new, 2:]).all() and np.isfinite(got[new:]).all()
    out, _ = p.run(awq, window=50)  # the queries look back over keys after it only
    if new < 100:
        assert np.isfinite(out.float().cpu().numpy()).all()


@pytest.mark.parametrize("heads", [2, 6])
@pytest.mark.parametrize("new", [2, 4, 120])
def test_a_nan_value_shows_only_where_it_is_seen(awq, new, heads):
    """The last token's value and the first token's key and value are NaN: all but the last query, or with a
    window the last one too, do not see them."""
    p = Problem([200], [new], heads, 2, 64, 16, seed=17)
    nan = np.array([np.nan], np.float16).view(np.uint8)
    page = p.table[0, 199 // 16]
    p.cache[page, 1, 0, 16 * 64 + 8 * (199 % 16) + 4:][:2] = nan
    out = p.run(awq)[0].float().cpu().numpy()
    half = heads // 2
    assert np.isnan(out[-1, half:]).all() and np.isfinite(out[:-1]).all() and np.isfinite(out[-1, :half]).all()
    first = p.table[0, 0]
    for at in (0, 4):
        p.cache[first, :, 0, 16 * 64 + at:][..., :2] = nan
    out = p.run(awq, window=80 - new // 2)[0].float().cpu().numpy()
    sees = np.arange(200 - new, 200) - (80 - new // 2) < 0
    assert np.isnan(out[sees]).all() and np.isfinite(out[~sees][:-1]).all()


def test_capture_takes_a_workspace_of_its_own(awq):
    """A shared workspace made during a capture would live in the graph's memory; one outgrown later stays valid."""
    p = Problem([500, 300], [1, 1], 8, 2, 128, 64, seed=22, junk=False)
    q = torch.from_numpy(p.q).cuda().half()
    cache, table, lens = (torch.from_numpy(a).cuda() for a in (p.cache, p.table, p.lens))
    out = torch.empty_like(q)
    want = awq.kv4_attention(q, cache, table, lens)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    handle = (q.device.index, stream.cuda_stream)
    kept = awq._kv4_workspaces.pop(handle, None)  # streams come from a pool: an earlier test may have used it
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="workspace"):
        with torch.cuda.graph(graph, stream=stream):
            out.zero_()
            awq.kv4_attention(q, cache, table, lens, out=out)
    assert handle not in awq._kv4_workspaces
    with torch.cuda.stream(stream):
        awq.kv4_attention(q, cache, table, lens, out=out)
        first = awq._kv4_workspaces[handle]
        awq._kv4_workspace(stream.cuda_stream, q.device, first.numel() + 1, None)
        assert awq._kv4_workspaces[handle].numel() > first.numel() and any(w is first for w in awq._kv4_outgrown)
        out.zero_()
        awq.kv4_attention(q, cache, table, lens, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del kept


@pytest.mark.parametrize("new", [1, 2, 12, 40])
@pytest.mark.parametrize("scale,q_scale", [(1e-40, 2.0), (-1e-30, 0.0), (1e-44, 1e-3), (0.0, 2.0)])
def test_scales_next_to_zero_give_the_mean(awq, new, scale, q_scale):
    """Scores that vanish: the weights are equal, and masked keys have none (the module's bound with delta = 0)."""
    p = Problem([150, 30], [new, min(new, 30)], 8, 2, 128, 64, bf16=True, seed=21, q_scale=q_scale)
    for window in (0, 33):
        out, lse = p.run(awq, window=window, scale=scale)
        want, want_lse, mag, _ = block.kv4_attention(p.q, p.cache, p.table, p.lens, p.start, scale, window)
        got = out.float().cpu().numpy()
        bound = mag * (2.0 ** -11 + 2.0 ** -17) + 2.0 ** -8 * np.abs(want) + 2.0 ** -24 * (1 + mag.max())
        seen = ~np.isneginf(want_lse)
        assert np.all(np.abs(got - want) <= bound)
        got_lse = lse.cpu().numpy()
        assert np.array_equal(~np.isneginf(got_lse), seen)
        assert np.all(np.abs(got_lse - want_lse)[seen] <= 2.0 ** -17 + 2.0 ** -22 * np.abs(want_lse)[seen])


def test_strided_queries_table_rows_and_explicit_scale(awq):
    p = Problem([90, 40], [2, 1], 4, 2, 64, 16, seed=11)
    q = torch.zeros(3, 6, 64, dtype=torch.float16, device="cuda")
    q[:, 1:5] = torch.from_numpy(p.q).cuda().half()
    table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = torch.from_numpy(p.table).cuda()
    lens, start, cache = (torch.from_numpy(a).cuda() for a in (p.lens, p.start, p.cache))
    want, _ = p.run(awq, scale=0.2)
    got = awq.kv4_attention(q[:, 1:5], cache, table[:, :p.table.shape[1]], lens, q_start=start, max_q=2, scale=0.2)
    assert torch.equal(got, want)
    ref = block.kv4_attention(p.q, p.cache, p.table, p.lens, p.start, 0.2)[0]
    assert np.abs(got.float().cpu().numpy() - ref).max() < 0.02


def test_lengths_change_under_a_captured_graph_and_on_two_streams(awq):
    p = Problem([500, 300], [1, 1], 8, 2, 128, 64, seed=12, junk=False)
    q = torch.from_numpy(p.q).cuda().half()
    cache, table, lens = (torch.from_numpy(a).cuda() for a in (p.cache, p.table, p.lens))
    need = awq.kv4_attention_workspace_bytes(2, 2, 1, 8, 2, 128)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    awq.kv4_attention(q, cache, table, lens, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.kv4_attention(q, cache, table, lens, out=out, workspace=ws)
    for new in ([500, 300], [17, 1], [0, 256], [100, 299]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, awq.kv4_attention(q, cache, table, lens))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = awq.kv4_attention(q, cache, table, lens)
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        for s in (a, b):
            with torch.cuda.stream(s):
                outs.append(awq.kv4_attention(q, cache, table, lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_a_cache_beyond_32_bit_offsets(awq):
    kv_heads, dim, page = 8, 128, 128
    pages = (5 << 30) // (kv_heads * (page // 16) * (16 * dim + 128))
    p = Problem([300], [1], 16, kv_heads, dim, page, seed=13)
    cache = torch.empty((pages, kv_heads, page // 16, 16 * dim + 128), dtype=torch.uint8, device="cuda")
    small = torch.from_numpy(p.cache).cuda()
    want, _ = p.run(awq)
    offset = pages - small.shape[0]
    cache[offset:] = small
    table = torch.from_numpy(p.table).cuda()
    table = torch.where(table >= 0, table + offset, table)
    got = awq.kv4_attention(torch.from_numpy(p.q).cuda().half(), cache, table, torch.from_numpy(p.lens).cuda())
    assert torch.equal(got, want)


def test_lengths_and_pages_out_of_range_are_memory_safe(awq):
    p = Problem([100, 60], [1, 1], 4, 2, 64, 16, seed=14, junk=False)
    p.lens = np.array([1 << 30, -5], np.int32)
    p.table[:, -1] = 1 << 30
    out, lse = p.run(awq)
    torch.cuda.synchronize()
    assert not out[1].any() and np.isneginf(lse[1].cpu().numpy()).all()
    p.start = np.array([-3, 1 << 20, 5], np.int32)
    p.run(awq)
    torch.cuda.synchronize()
    assert awq.awq_last_device_error() == 0


def test_append_then_attend(awq):
    """Tokens appended one step at a time are attended as the gathered keys and values say."""
    rng = np.random.default_rng(15)
    heads, kv_heads, dim, page = 4, 2, 64, 16
    cache = awq.kv4_cache(6, kv_heads, dim, page)
    table = torch.tensor([[4, 1, 3]], dtype=torch.int32, device="cuda")
    rope = torch.from_numpy(block.rope_table(64, dim)).cuda()
    slots = []
    for t in range(35):
        q, k, v = (torch.from_numpy(rng.normal(size=(1, h, dim)).astype(np.float32)).cuda().half() for h in (heads, kv_heads, kv_heads))
        slot = int(table[0, t // page]) * page + t % page
        slots.append(slot)
        pos = torch.tensor([t], dtype=torch.int32, device="cuda")
        q = awq.kv4_append(cache, k, v, pos, torch.tensor([slot], device="cuda"), rope, q=q)
        out = awq.kv4_attention(q, cache, table, pos + 1)
    gk, gv = awq.kv4_gather(cache, torch.tensor(slots, device="cuda"))
    gk, gv = gk.double().repeat_interleave(2, 1), gv.double().repeat_interleave(2, 1)
    score = torch.einsum("hd,jhd->hj", q[0].double(), gk) / 8
    want = torch.einsum("hj,jhd->hd", torch.softmax(score, -1), gv)
    assert (out[0].double() - want).abs().max() < 4e-3 * want.abs().max()


def test_wrong_operands_are_refused(awq):
    p = Problem([10], [1], 4, 2, 64, 16, seed=16)
    q = torch.from_numpy(p.q).cuda().half()
    cache, table, lens = (torch.from_numpy(a).cuda() for a in (p.cache, p.table, p.lens))
    for bad in (lambda: awq.kv4_attention(q.float(), cache, table, lens), lambda: awq.kv4_attention(q, cache, table.long(), lens),
                lambda: awq.kv4_attention(q, cache, table, lens.long()),
                lambda: awq.kv4_attention(q, cache, table, lens, lse=torch.zeros(1, 4, device="cuda").half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: awq.kv4_attention(q[..., :32], cache, table, lens), lambda: awq.kv4_attention(q, cache, table, lens[:0]),
                lambda: awq.kv4_attention(q, cache, table, lens, lse=torch.zeros(4, 4, device="cuda")),
                lambda: awq.kv4_attention(q, cache, table, lens, out=torch.empty(1, 8, 64, device="cuda").half()[:, ::2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.kv4_attention(q[:, :3], cache, table, lens), lambda: awq.kv4_attention(q, cache, table, lens, window=-1),
                lambda: awq.kv4_attention(q, cache, table, lens, scale=float("nan")),
                lambda: awq.kv4_attention(torch.cat((q, q)), cache, table, lens)):
        with pytest.raises(awq.AwqError):
            bad()
    assert awq.kv4_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 4, 64)
