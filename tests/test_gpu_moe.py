"""The layer with experts against the oracle's float64: router, plan, prepared weights, grouped products, combination.

Tolerance of a product.  The codes enter it as they are and their products with 16-bit x are exact in fp32, so a sum of K
of them is off by at most (8 + K / 8) roundings of 2^-23 of its terms' magnitudes `mag` (blocks of products are added
in the tensor cores, then the blocks; a group's scaled sum is one rounding more in 128 terms), plus half an ulp of its
type.  silu(g) u: |silu'| <= 1.1, so
(1.1 |u| dg + |silu(g)| du) and 2^-20 of the value for the exponential, the division and the product.
"""

import numpy as np
import pytest

import oracle
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


def dtype_of(bf16):
    return torch.bfloat16 if bf16 else torch.float16


def half_step(bf16):
    return 2.0 ** -8 if bf16 else 2.0 ** -11


def smallest(bf16):
    """Half of the smallest step, where values are subnormal."""
    return 2.0 ** -134 if bf16 else 2.0 ** -25


def dev16(a, bf16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype_of(bf16)).cuda()


def host(t):
    return t.double().cpu().numpy()


# ---- plan

@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 2, 8), (3, 5, 7), (64, 8, 512), (333, 4, 60), (1025, 1, 3),
                                   (1000, 9, 129), (4100, 8, 16), (8192, 8, 20), (8193, 8, 5), (70001, 1, 3), (16385, 1, 512),
                                   (9000, 2, 300), (40000, 8, 1)])
def test_plan(awq, T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if T > 3:
        wild = rng.random(ids.shape) < 0.05
        ids[wild] = rng.choice(np.array([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1]), wild.sum()).astype(np.int32)
        ids[rng.random(ids.shape) < 0.3] = E // 2
    plan = awq.awq_moe_plan(dev(ids), E)
    offsets, order, place = layer.plan(ids, E)
    assert plan.rows == T * k and plan.experts == E and plan.top_k == k
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.order.cpu().numpy(), order)
    assert np.array_equal(plan.place.cpu().numpy(), place)


# ---- router

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 8, 2), (7, 8, 8), (33, 33, 32), (513, 60, 4), (900, 128, 8),
                                   (100, 160, 6), (70, 512, 8), (257, 300, 10), (16, 512, 8), (32, 100, 4), (32, 8, 5), (4, 400, 32), (5, 400, 32)])
def test_route(awq, dtype, T, E, k):
    gen = torch.Generator().manual_seed(T + E)
    logits = (2.0 * torch.randn(T, E, generator=gen)).to(dtype)
    if E > 4 and T > 4:
        logits[1] = logits[1, 0]                  # all equal
        logits[2, ::2] = float("-inf")            # masked experts
        logits[3] = float("-inf")                 # all of them
        logits[4, : E // 2] = -0.0
        logits[4, E // 2 :] = 0.0
    for normalize in (True, False):
        weights, ids, plan = awq.awq_moe_route(logits.cuda(), k, normalize=normalize)
        want_w, want_ids = layer.route(logits.double().numpy(), k, normalize)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        # exp, E sums and a division in fp32
        assert np.all(np.abs(host(weights) - want_w) <= (E + 16) * 2.0 ** -24 * want_w)
        offsets, order, place = layer.plan(want_ids, E)
        assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
        assert np.array_equal(plan.order.cpu().numpy(), order) and np.array_equal(plan.place.cpu().numpy(), place)


def test_route_rows_with_nan_or_infinity_show_it(awq):
    logits = torch.randn(6, 20, generator=torch.Generator().manual_seed(1))
    logits[1, 7] = float("nan")
    logits[3, 2] = float("inf")
    logits[4] = float("nan")
    weights, ids, plan = awq.awq_moe_route(logits.cuda(), 3)
    bad = torch.tensor([False, True, False, True, True, False])
    assert torch.equal(weights.isnan().cpu(), bad[:, None].expand(6, 3))
    for row in ids.tolist():
        assert len(set(row)) == 3 and all(0 <= e < 20 for e in row)
    assert ids[1, 0] == 7 and ids[3, 0] == 2 and int(plan.offsets[-1]) == 18


def test_route_reads_strided_rows(awq):
    wide = torch.randn(50, 40, device="cuda")
    got = awq.awq_moe_route(wide[:, 3:19], 4)
    want = awq.awq_moe_route(wide[:, 3:19].contiguous(), 4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2].order, want[2].order)


# ---- prepared weights

class Experts:
    def __init__(self, E, K, N, bf16=False, symmetric=False, seed=0, gain=1.0):
        rng = np.random.default_rng(seed)
        self.E, self.K, self.N, self.bf16 = E, K, N, bf16
        self.qw = rng.integers(0, 2 ** 32, (E, K, N // 8), dtype=np.uint32).view(np.int32)
        self.qz = None if symmetric else rng.integers(0, 2 ** 32, (E, K // 128, N // 8), dtype=np.uint32).view(np.int32)
        self.sc = round16(gain * (0.5 + rng.random((E, K // 128, N))) / np.sqrt(K) / 5, bf16)
        self.sc[:, :, ::17] *= np.float32(2.0 ** -9 if not bf16 else 2.0 ** -30)  # columns next to nothing
        self.sc = round16(self.sc, bf16)

    def pack(self, awq, gated=False):
        return awq.awq_moe_prepack(dev(self.qw), None if self.qz is None else dev(self.qz), dev16(self.sc, self.bf16), gated)

    def dense(self):
        return [layer.dequantize(self.qw[e], None if self.qz is None else self.qz[e], self.sc[e]) for e in range(self.E)]


@pytest.mark.parametrize("E,K,N,gated,symmetric", [(1, 128, 32, False, False), (2, 128, 64, True, True), (3, 256, 544, False, False),
                                                   (2, 384, 320, True, False), (1, 128, 512, True, False)])
def test_prepack_layout_and_back(awq, E, K, N, gated, symmetric):
    p = Experts(E, K, N, symmetric=symmetric, seed=N)
    bits = p.sc.astype(np.float16).view(np.uint16)
    w = p.pack(awq, gated)
    want = layer.prepack(p.qw, p.qz, bits, gated)
    assert np.array_equal(w.data.cpu().numpy(), want.reshape(-1))
    qw, qz, sc = awq.awq_moe_unprepack(w)
    assert np.array_equal(qw.cpu().numpy(), p.qw) and np.array_equal(sc.cpu().numpy().view(np.uint16), bits)
    if symmetric:
        assert (qz.cpu().numpy().view(np.uint32) == 0x88888888).all()
    else:
        assert np.array_equal(qz.cpu().numpy(), p.qz)
    assert awq.awq_moe_unprepack(w, with_zeros=False)[1] is None


# ---- grouped products

def counts_to_plan(awq, counts, top_k=1, seed=0):
    """A plan of these rows for each expert, positions in any order."""
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(seed).shuffle(ids)
    return awq.awq_moe_plan(dev(ids.reshape(-1, top_k)), len(counts))


def check_gemm(awq, counts, K, N, gated=False, bf16=False, symmetric=False, gather_k=0, seed=0, x_pad=0, wide=False):
    p = Experts(len(counts), K, N, bf16, symmetric, seed)
    w = p.pack(awq, gated)
    rows = int(np.sum(counts))
    plan = counts_to_plan(awq, counts, max(1, gather_k), seed)
    rng = np.random.default_rng(seed + 1)
    n_x = rows // gather_k if gather_k else rows
    x = round16(rng.normal(size=(n_x, K)), bf16)
    xs = torch.full((n_x, K + x_pad), float("nan"), dtype=dtype_of(bf16), device="cuda")
    xs[:, :K] = dev16(x, bf16)
    y = awq.awq_moe_gemm(xs[:, :K], w, plan, gather=bool(gather_k), out_dtype=torch.float32 if wide else None)
    again = awq.awq_moe_gemm(xs[:, :K], w, plan, gather=bool(gather_k), out=torch.empty_like(y))
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    order = plan.order.cpu().numpy()
    src = order // gather_k if gather_k else np.arange(rows)
    a, mag = layer.grouped(x, p.dense(), plan.offsets.cpu().numpy(), src)
    err = (8 + K / 8) * 2.0 ** -23 * mag
    if gated:
        g, u = a[:, : N // 2], a[:, N // 2 :]
        dg, du = err[:, : N // 2], err[:, N // 2 :]
        s = layer.silu(g)
        want = s * u
        err = 1.1 * np.abs(u) * dg + (np.abs(s) + 1.1 * dg) * du + 2.0 ** -20 * np.abs(want)
    else:
        want = a
    tol = err + (2.0 ** -24 if wide else half_step(bf16)) * (np.abs(want) + err) + (2.0 ** -150 if wide else smallest(bf16))
    got = host(y)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    assert awq.awq_last_device_error() == 0


SMALL = [[1], [0, 1], [2, 0, 1], [5, 16, 17], [8, 0, 64, 33], [1] * 9, [3, 0, 0, 130], [65, 200, 1, 15]]


@pytest.mark.parametrize("counts", SMALL, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_gemm_rows_of_experts(awq, counts, gated):
    check_gemm(awq, counts, 256, 320, gated=gated, seed=len(counts))


@pytest.mark.parametrize("K,N", [(128, 32), (128, 256), (1280, 64), (384, 288), (640, 1088), (2048, 512), (4096, 160)])
@pytest.mark.parametrize("gated", [False, True])
def test_gemm_sizes(awq, K, N, gated):
    if gated and N % 64:
        N += 32
    check_gemm(awq, [3, 21, 0, 40], K, N, gated=gated, seed=K + N)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("rows", [2, 40, 700])
def test_gemm_types(awq, bf16, symmetric, rows):
    check_gemm(awq, [rows, rows // 2, 0, 7], 512, 384, gated=True, bf16=bf16, symmetric=symmetric, seed=rows)
    check_gemm(awq, [rows, rows // 2, 0, 7], 512, 384, bf16=bf16, symmetric=symmetric, seed=rows)
    check_gemm(awq, [rows, rows // 2, 0, 7], 512, 384, bf16=bf16, symmetric=symmetric, seed=rows, wide=True)
    check_gemm(awq, [rows, 1], 512, 384, gated=True, bf16=bf16, symmetric=symmetric, seed=rows, wide=True)


@pytest.mark.parametrize("counts,k", [([2, 4], 2), ([6, 0, 30], 4), ([100, 51, 29], 3), ([640, 10], 5)])
@pytest.mark.parametrize("bf16", [False, True])
def test_gemm_gathers_tokens(awq, counts, k, bf16):
    check_gemm(awq, counts, 384, 256, gated=True, bf16=bf16, gather_k=k, seed=k, x_pad=8)


def test_gemm_many_experts_and_rows(awq):
    rng = np.random.default_rng(3)
    check_gemm(awq, rng.integers(0, 9, 160).tolist(), 256, 128, gated=True, seed=5)
    check_gemm(awq, [0] * 511 + [5], 128, 64, seed=6)
    check_gemm(awq, [1000, 3, 900, 0, 193, 192, 191], 256, 512, seed=7)
    check_gemm(awq, [385, 1, 97], 1024, 768, gated=True, bf16=True, seed=8)


def test_gemm_long_sums_split_over_ctas(awq):
    """Few tiles with a long axis: every tile is shared by several CTAs."""
    check_gemm(awq, [3], 8192, 64, seed=9)
    check_gemm(awq, [3, 9], 14336, 128, gated=True, seed=10)
    check_gemm(awq, [40], 4096, 256, seed=11)
    check_gemm(awq, [300], 4096, 256, bf16=True, seed=12)


def test_gemm_leaves_rows_of_no_expert(awq):
    """Choices without an expert have no row: rows behind the last expert's stay as they were."""
    p = Experts(3, 128, 64, seed=1)
    ids = np.array([[0, 7], [2, 1], [-1, 2]], np.int32)
    plan = awq.awq_moe_plan(dev(ids), 3)
    x = round16(np.random.default_rng(2).normal(size=(3, 128)), False)
    out = torch.full((6, 64), 7.0, dtype=torch.float16, device="cuda")
    awq.awq_moe_gemm(dev16(x, False), p.pack(awq), plan, gather=True, out=out)
    want, mag = layer.grouped(x, p.dense(), [0, 1, 2, 4], [0, 1, 1, 2])
    got = host(out)
    assert np.all(np.abs(got[:4] - want) <= 24 * 2.0 ** -23 * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -24)
    assert np.all(got[4:] == 7.0)


def test_gemm_with_offsets_that_make_no_sense_stays_in_bounds(awq):
    p = Experts(4, 128, 256, seed=1)
    w = p.pack(awq)
    x = torch.randn(20, 128, device="cuda").half()
    out = torch.full((20 + 64, 256), 7.0, dtype=torch.float16, device="cuda")
    for offsets in ([-5, 30, 3, 90, 8], [0, 0, 0, 0, 0], [19, 2, 1, 0, 50], [2 ** 31 - 1] * 5, [-2 ** 31] * 5):
        plan = awq.MoePlan(dev(np.array(offsets, np.int32)), torch.arange(20, dtype=torch.int32, device="cuda"),
                           torch.arange(20, dtype=torch.int32, device="cuda"), 1)
        awq.awq_moe_gemm(x, w, plan, out=out[:20])
        order = dev(np.array([2 ** 31 - 1, -1, -2 ** 31, 20] * 5, np.int32))  # and none of the rows exists
        bad = awq.MoePlan(plan.offsets, order, plan.place, 1)
        awq.awq_moe_gemm(x, w, bad, gather=True, out=out[:20])
        torch.cuda.synchronize()
        assert (out[20:] == 7.0).all() and awq.awq_last_device_error() == 0


def test_gemm_and_combine_beyond_32_bits(awq):
    """More than 2^31 elements of y: the last rows are those of a call of their own."""
    E, K, N, rows = 2, 128, 8192, 270000
    w = Experts(E, K, N, seed=1).pack(awq)
    x = torch.randn(rows, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()

    def plan_of(*counts):
        offsets = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
        order = torch.arange(sum(counts), dtype=torch.int32, device="cuda")
        return awq.MoePlan(offsets, order, order, 1)

    y = awq.awq_moe_gemm(x, w, plan_of(1000, rows - 1000), out_dtype=torch.float32)
    last = awq.awq_moe_gemm(x[-300:].contiguous(), w, plan_of(0, 300), out_dtype=torch.float32)
    assert y.numel() > 2 ** 31 and torch.equal(y[-300:], last)
    ones = torch.ones(rows, 1, device="cuda")
    out = awq.awq_moe_combine(y, plan_of(1000, rows - 1000), ones, dtype=torch.float16)
    assert torch.equal(out[-300:], last.half())


def test_choices_of_one_expert_twice(awq):
    """A router of one's own may choose an expert twice for a token: two rows, added up."""
    p = Experts(3, 128, 64, seed=1)
    ids = dev(np.array([[2, 2], [0, 2]], np.int32))
    plan = awq.awq_moe_plan(ids, 3)
    x = dev16(np.random.default_rng(1).normal(size=(2, 128)), False)
    y = awq.awq_moe_gemm(x, p.pack(awq), plan, gather=True)
    assert torch.equal(y[1], y[2])
    out = awq.awq_moe_combine(y, plan, torch.full((2, 2), 0.5, device="cuda"))
    assert torch.equal(out[0], y[1])


# ---- combination

@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (3, 2, 64), (70, 8, 520), (33, 5, 4096), (5, 32, 16)])
@pytest.mark.parametrize("bf16", [False, True])
def test_combine(awq, T, k, H, bf16):
    rng = np.random.default_rng(T + k)
    ids = rng.integers(-1, 5, (T, k)).astype(np.int32)  # -1: no row
    plan = awq.awq_moe_plan(dev(ids), 5)
    y = round16(rng.normal(size=(T * k, H)), bf16)
    y[int(plan.offsets[-1]):] = np.nan  # what lies behind the rows is not read
    w = rng.random((T, k)).astype(np.float32)
    res = round16(rng.normal(size=(T, H)), bf16)
    _, _, place = layer.plan(ids, 5)
    place = place.reshape(T, k)
    for residual in (None, res):
        want = np.zeros((T, H)) if residual is None else residual.astype(np.float64)
        mag = np.abs(want)
        for t in range(T):
            for j in range(k):
                if place[t, j] >= 0:
                    term = w[t, j].astype(np.float64) * y[place[t, j]].astype(np.float64)
                    want[t] += term
                    mag[t] += np.abs(term)
        wide = None
        if residual is not None:
            wide = torch.zeros((T, H + 8), dtype=dtype_of(bf16), device="cuda")
            wide[:, :H] = dev16(residual, bf16)
        res_in = None if wide is None else wide[:, :H]
        got = awq.awq_moe_combine(dev16(y, bf16), plan, dev(w), residual=res_in)
        assert torch.equal(got, awq.awq_moe_combine(dev(y), plan, dev(w), residual=res_in, dtype=dtype_of(bf16)))  # fp32 y
        err = (k + 1) * 2.0 ** -24 * mag
        assert np.all(np.abs(host(got) - want) <= err + half_step(bf16) * (np.abs(want) + err) + smallest(bf16))
    same = dev16(res, bf16)
    assert torch.equal(awq.awq_moe_combine(dev16(y, bf16), plan, dev(w), residual=same, out=same), got)


# ---- the layer

def reference_layer(p_up, p_down, x, ids, weights, bf16):
    """float64 layer and its error bound: the product's, and h's rounding, carried through down."""
    up, down = p_up.dense(), p_down.dense()
    T, k = ids.shape
    K, inner, H = p_up.K, p_up.N // 2, p_down.N
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            row = x[t].astype(np.float64)
            a, mag = row @ up[e].astype(np.float64), np.abs(row) @ np.abs(up[e].astype(np.float64))
            da = (8 + K / 8) * 2.0 ** -23 * mag
            g, u, dg, du = a[:inner], a[inner:], da[:inner], da[inner:]
            s = layer.silu(g)
            h = s * u
            dh = 1.1 * np.abs(u) * dg + (np.abs(s) + 1.1 * dg) * du + 2.0 ** -20 * np.abs(h)
            dh = dh + half_step(bf16) * (np.abs(h) + dh) + smallest(bf16)
            wd = np.abs(down[e].astype(np.float64))
            y = h @ down[e].astype(np.float64)
            dy = dh @ wd + (8 + inner / 8) * 2.0 ** -23 * (np.abs(h) @ wd)
            out[t] += weights[t, j] * y
            err[t] += abs(weights[t, j]) * dy + 2.0 ** -20 * np.abs(weights[t, j] * y)
    return out, err + half_step(bf16) * (np.abs(out) + err) + smallest(bf16)


@pytest.mark.parametrize("T,E,k,K,inner,bf16", [(1, 8, 2, 256, 384, False), (13, 16, 6, 256, 128, True), (90, 4, 2, 512, 256, False),
                                                (150, 40, 8, 128, 128, True)])
def test_layer(awq, T, E, k, K, inner, bf16):
    up, down = Experts(E, K, 2 * inner, bf16, seed=1), Experts(E, inner, K, bf16, symmetric=True, seed=2)
    w_up, w_down = up.pack(awq, True), down.pack(awq)
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=gen).to(dtype_of(bf16))
    logits = torch.randn(T, E, generator=gen)
    logits[:, E // 2] = -50.0
    weights, ids, plan = awq.awq_moe_route(logits.cuda(), k)
    out = awq.awq_moe(x.cuda(), w_up, w_down, weights, plan)
    want, tol = reference_layer(up, down, x.float().numpy(), ids.cpu().numpy(), host(weights), bf16)
    assert np.all(np.abs(host(out) - want) <= tol), np.max(np.abs(host(out) - want) / tol)
    assert torch.equal(out, awq.awq_moe(x.cuda(), w_up, w_down, weights, plan))
    # the three calls that it is made of
    h = awq.awq_moe_gemm(x.cuda(), w_up, plan, gather=True)
    y = awq.awq_moe_gemm(h, w_down, plan, out_dtype=torch.float32)
    assert torch.equal(out, awq.awq_moe_combine(y, plan, weights, dtype=x.dtype))


def test_layer_in_a_graph_follows_the_routing(awq):
    T, E, k, K, inner = 20, 8, 2, 256, 256
    up, down = Experts(E, K, 2 * inner, seed=1).pack(awq, True), Experts(E, inner, K, seed=2).pack(awq)
    x, logits = torch.zeros(T, K, device="cuda").half(), torch.zeros(T, E, device="cuda")

    def pass_(workspace=None):
        weights, _, plan = awq.awq_moe_route(logits, k)
        return awq.awq_moe(x, up, down, weights, plan, workspace=workspace)

    ws = torch.zeros(awq.awq_moe_workspace_bytes(T, k, up, down), dtype=torch.uint8, device="cuda")
    pass_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pass_(ws)
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=gen, device="cuda"))
        logits.copy_(torch.randn(T, E, generator=gen, device="cuda"))
        logits[:, seed] += 9.0 * (seed % 2)
        graph.replay()
        want = pass_()
        assert torch.equal(out, want)
    with pytest.raises(RuntimeError, match="workspace of its own"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            pass_()
    torch.cuda.synchronize()
    assert awq.awq_last_device_error() == 0


def test_two_graphs_of_the_layer_at_once(awq):
    """Captured calls have workspaces of their own: their graphs may run side by side."""
    T, E, k, K, inner = 24, 8, 2, 512, 256
    up, down = Experts(E, K, 2 * inner, seed=1).pack(awq, True), Experts(E, inner, K, seed=2).pack(awq)
    xs = [torch.randn(T, K, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").half() for i in range(2)]
    logits = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    weights, _, plan = awq.awq_moe_route(logits, k)
    want = [awq.awq_moe(x, up, down, weights, plan) for x in xs]
    graphs, outs, spaces = [], [], []
    for x in xs:
        spaces.append(torch.zeros(awq.awq_moe_workspace_bytes(T, k, up, down), dtype=torch.uint8, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(awq.awq_moe(x, up, down, weights, plan, workspace=spaces[-1]))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        awq.awq_moe(xs[0], up, down, weights, plan)  # and the shared workspace's call beside them
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert awq.awq_last_device_error() == 0


def test_layer_on_two_streams_at_once(awq):
    T, E, k, K, inner = 30, 8, 2, 512, 256
    up, down = Experts(E, K, 2 * inner, seed=1).pack(awq, True), Experts(E, inner, K, seed=2).pack(awq)
    xs = [torch.randn(T, K, device="cuda").half() for _ in range(2)]
    weights, _, plan = awq.awq_moe_route(torch.randn(T, E, device="cuda"), k)
    want = [awq.awq_moe(x, up, down, weights, plan) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(awq.awq_moe(x, up, down, weights, plan))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert awq.awq_last_device_error() == 0


def test_empty_batch(awq):
    up, down = Experts(2, 128, 256, seed=1).pack(awq, True), Experts(2, 128, 128, seed=2).pack(awq)
    weights, ids, plan = awq.awq_moe_route(torch.zeros(0, 2, device="cuda"), 2)
    assert weights.shape == ids.shape == (0, 2) and plan.offsets.tolist() == [0, 0, 0]
    assert awq.awq_moe(torch.zeros(0, 128, device="cuda").half(), up, down, weights, plan).shape == (0, 128)


def test_binding_refusals(awq):
    up, down = Experts(2, 128, 256, seed=1).pack(awq, True), Experts(2, 128, 128, seed=2).pack(awq)
    x = torch.zeros(4, 128, device="cuda").half()
    weights, _, plan = awq.awq_moe_route(torch.zeros(4, 2, device="cuda"), 1)
    for bad in (lambda: awq.awq_moe(x, down, down, weights, plan), lambda: awq.awq_moe(x, up, up, weights, plan),
                lambda: awq.awq_moe_gemm(x[:3], up, plan), lambda: awq.awq_moe_gemm(x[:, :64], up, plan),
                lambda: awq.awq_moe_combine(x[:3], plan, weights), lambda: awq.awq_moe_combine(x, plan, weights[:2]),
                lambda: awq.awq_moe_gemm(x, up, awq.awq_moe_plan(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 3)),
                lambda: awq.awq_moe_gemm(x, up, plan, out=torch.zeros(4, 256, device="cuda").half()),
                lambda: awq.awq_moe_plan(torch.zeros(4, dtype=torch.int32, device="cuda"), 3)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.awq_moe_gemm(x.bfloat16(), up, plan), lambda: awq.awq_moe_gemm(x.float(), up, plan),
                lambda: awq.awq_moe_plan(torch.zeros(4, 1, dtype=torch.int64, device="cuda"), 3),
                lambda: awq.awq_moe_route(torch.zeros(4, 2, device="cuda").double(), 1),
                lambda: awq.awq_moe_combine(x, plan, weights.double()), lambda: awq.awq_moe_combine(x.float(), plan, weights),
                lambda: awq.awq_moe_combine(x, plan, weights, residual=x.bfloat16()),
                lambda: awq.awq_moe_gemm(x, up, plan, out_dtype=torch.bfloat16), lambda: awq.awq_moe_gemm(x.cpu(), up, plan)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: awq.awq_moe_route(torch.zeros(4, 2, device="cuda"), 3),
                lambda: awq.awq_moe_route(torch.zeros(4, 513, device="cuda"), 3),
                lambda: awq.awq_moe_plan(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 600)):
        with pytest.raises(awq.AwqError):
            bad()
