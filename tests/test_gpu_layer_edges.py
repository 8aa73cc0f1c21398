"""Calls of the layers with experts and the e4m3 layers in company: of other threads, streams, buffers and lengths.

Results that are compared bit for bit come from the same call made by itself, whose own bounds other tests hold.
"""

import threading

import numpy as np
import pytest

from oracle import layer as oracle_layer
from oracle.block_oracle import round16
from tests.test_gpu_fp8 import Problem, dev16
from tests.test_gpu_moe import Experts, awq  # noqa: F401  (awq is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, dtype=torch.float16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


class Layers:
    """A layer with experts and an e4m3 layer, both of K = 512 channels, and their calls on inputs of a number."""

    def __init__(self, awq, tokens, E=8, k=2, K=512, inner=256):
        self.awq, self.tokens = awq, tokens
        self.up, self.down = Experts(E, K, 2 * inner, seed=1).pack(awq, True), Experts(E, inner, K, seed=2).pack(awq)
        _, _, self.wq, self.s_w = Problem(1, K, K, seed=3).on_gpu()
        self.weights, _, self.plan = awq.awq_moe_route(normal(tokens, E, seed=9, dtype=torch.float32), k)

    def x(self, i):
        return normal(self.tokens, 512, seed=100 + i)

    def experts(self, x, **kw):
        return self.awq.awq_moe(x, self.up, self.down, self.weights, self.plan, **kw)

    def fp8(self, x, **kw):
        return self.awq.awq_fp8_linear(x, self.wq, self.s_w, **kw)


@pytest.mark.parametrize("tokens", [3, 40])
def test_threads_on_one_stream(awq, tokens):  # noqa: F811
    """Two threads' calls pass their rows and codes through the stream's one workspace."""
    layers = Layers(awq, tokens)
    calls = (layers.experts, layers.fp8)
    xs = [layers.x(i) for i in range(4)]
    want = [[call(x) for x in xs] for call in calls]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(me):
        try:
            start.wait()
            for turn in range(100):
                i = (turn + 2 * me) % 4
                got = [call(xs[i]) for call in calls]
                if turn % 10 == 9:
                    wrong.extend((me, turn, c) for c in range(2) if not torch.equal(got[c], want[c][i]))
        except BaseException as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:4]
    assert awq.awq_last_device_error() == 0


def test_stale_flags_do_not_outlive_the_report_of_an_expired_wait(awq):  # noqa: F811
    """A wait that expired may leave any flags behind.  Here nothing runs while all of a stream's shared workspaces are
    filled with ones, and an unrelated wait expires; calls whose tiles several CTAs share come after the report."""
    layers = Layers(awq, 6)
    _, _, wq, s_w = Problem(1, 14336, 512, seed=4).on_gpu()
    deep = normal(20, 14336, seed=5)
    calls = [lambda: layers.experts(layers.x(0)), lambda: layers.fp8(layers.x(0)), lambda: awq.awq_fp8_linear(deep, wq, s_w)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    spaces = list(awq._layer_workspaces.values())
    assert spaces
    for ws in spaces:
        ws.fill_(1)
    torch.cuda.synchronize()
    awq.awq_selftest_wait_timeout(1_000_000)
    assert awq.awq_last_device_error() != 0
    for _ in range(3):
        assert all(torch.equal(call(), w) for call, w in zip(calls, want))
    assert awq.awq_last_device_error() == 0


def tensors(result):
    if result is None or torch.is_tensor(result):
        return [] if result is None else [result]
    if isinstance(result, tuple):
        return [t for r in result for t in tensors(r)]
    return [v for v in vars(result).values() if torch.is_tensor(v)]  # plans, prepared weights


def prepared_calls(awq, name):  # noqa: F811
    """Two calls of an operator, whose operands exist."""
    layers = Layers(awq, 40)
    weights, plan, w_up = layers.weights, layers.plan, layers.up
    e = Experts(1, 512, 256, seed=7)
    dense = [torch.from_numpy(a).cuda() for a in (e.qw[0], e.qz[0])]
    words = torch.randint(-2 ** 31, 2 ** 31, (2, 256, 16), dtype=torch.int32, device="cuda")
    ones = torch.ones(4, 40, device="cuda")
    operands = {
        "awq_moe_plan": lambda x: ((x[:, :2] > 0).int(), 8),
        "awq_moe_route": lambda x: (x[:, :8].float(), 2),
        "awq_moe_prepack": lambda x: (words, None, x[:4, :128].reshape(2, 2, 128).contiguous()),
        "awq_moe_unprepack": lambda x: (w_up,),
        "awq_moe_gemm": lambda x: (x, w_up, plan, True),
        "awq_moe_combine": lambda x: (x.repeat(2, 1), plan, weights),
        "awq_moe": lambda x: (x, layers.up, layers.down, weights, plan),
        "awq_fp8_quant_act": lambda x: (x,),
        "awq_fp8_gemm": lambda x: (x.to(torch.float8_e4m3fn), ones, layers.wq, layers.s_w),
        "awq_fp8_linear": lambda x: (x, layers.wq, layers.s_w),
        "awq_gemm": lambda x: (x, *dense, x[:4, :256].contiguous()),
        "awq_rmsnorm": lambda x: (x, x[0]),
        "w4a8_quant_act": lambda x: (x,),
    }[name]
    fn = getattr(awq, name)
    return [lambda stream=None, args=operands(normal(40, 512, seed=seed)): fn(*args, stream=stream) for seed in (1, 2)]


NAMES = ("awq_moe_plan", "awq_moe_route", "awq_moe_prepack", "awq_moe_unprepack", "awq_moe_gemm", "awq_moe_combine", "awq_moe",
         "awq_fp8_quant_act", "awq_fp8_gemm", "awq_fp8_linear", "awq_gemm", "awq_rmsnorm", "w4a8_quant_act")


def as_bytes(result):
    return [t.view(torch.uint8).flatten() for t in tensors(result)]


@pytest.mark.parametrize("name", NAMES)
def test_results_for_another_stream(awq, name):  # noqa: F811
    """A result's memory is neither what the current stream has yet to read nor given away while it has the result to read."""
    first, second = prepared_calls(awq, name)
    side = torch.cuda.Stream()
    want = [t.clone() for t in as_bytes(first())]
    for call in (first, second):  # the side's workspace, the kernels
        call(side)
    seen, old = [torch.zeros_like(w) for w in want], [torch.full_like(w, 7) for w in want]
    torch.cuda.synchronize()

    torch.cuda._sleep(40_000_000)  # about 20 ms
    for s in seen:
        s.copy_(old.pop(0))  # freed here, read later
    got = first(side)
    torch.cuda.synchronize()
    assert all((s == 7).all() for s in seen)
    assert all(torch.equal(g, w) for g, w in zip(as_bytes(got), want))

    torch.cuda._sleep(40_000_000)
    for s, t in zip(seen, as_bytes(got)):
        s.copy_(t)
    del got, t
    got = second(side)  # may not take the memory yet
    torch.cuda.synchronize()
    assert all(torch.equal(s, w) for s, w in zip(seen, want))
    assert awq.awq_last_device_error() == 0


@pytest.mark.parametrize("tokens,K", [(1, 24576), (2, 24576), (1, 4096), (2, 1024), (3, 4096), (40, 1024), (300, 1024)])
@pytest.mark.parametrize("bf16", [False, True])
def test_fp8_layer_in_place(awq, tokens, K, bf16):  # noqa: F811
    """out=x.  192 tiles of 24576 channels over fewer SMs: results are written while other CTAs still have channels to read."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    wq = torch.randn(K, K, generator=gen, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s_w = torch.rand(-(-K // 128), -(-K // 128), generator=gen, device="cuda") * 1e-4
    wide = normal(tokens + 2, K + 16, seed=tokens, dtype=torch.bfloat16 if bf16 else torch.float16)
    x = wide[1:-1, :K]
    want = awq.awq_fp8_linear(x, wq, s_w)
    dense = x.clone(memory_format=torch.contiguous_format)
    assert awq.awq_fp8_linear(dense, wq, s_w, out=dense) is dense and torch.equal(dense, want)
    # rows that cross: out begins where the first row of x does, or ends where the last one ends
    for first in (wide.flatten()[K + 16:], wide.flatten()[(tokens + 1) * (K + 16) - 16 - tokens * K:]):
        keep = wide.clone()
        out = first[: tokens * K].view(tokens, K)
        awq.awq_fp8_linear(x, wq, s_w, out=out)
        assert torch.equal(out, want)
        wide.copy_(keep)
    assert awq.awq_last_device_error() == 0


@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_layer_with_experts_in_place(awq, tokens):  # noqa: F811
    """out=x, and out=x with x the residual too."""
    layers = Layers(awq, tokens)
    x = layers.x(1)
    want, added = layers.experts(x), layers.experts(x, residual=x)
    for residual, result in ((False, want), (True, added)):
        own = x.clone()
        assert layers.experts(own, residual=own if residual else None, out=own) is own and torch.equal(own, result)


def test_results_over_operands_are_refused(awq):  # noqa: F811
    layers = Layers(awq, 40)
    rows = normal(80, 256, seed=1)
    wide = normal(40, 520, seed=2)
    square = Experts(8, 256, 256, seed=5).pack(awq)
    for bad in (lambda: awq.awq_moe_gemm(rows, square, layers.plan, out=rows),
                lambda: awq.awq_moe_combine(rows, layers.plan, layers.weights, out=rows[:40]),
                lambda: layers.experts(layers.x(0), residual=wide[:, :512], out=wide.flatten()[: 40 * 512].view(40, 512))):
        with pytest.raises(awq.AwqError):
            bad()


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows", [5, 200, 700])
def test_silu_over_its_range(awq, rows, bf16, wide):  # noqa: F811
    """Gates and ups that are exact in fp32 (one channel, scales that are powers of two), from -104 to 104 and 0.

    e = exp(-|g|) is off by 2 units of 2^-23 (expf) or 2 + 1.173 |g| (the approximate one), which counts once in g e and at most
    half in 1 + e; the products, the sum and the division add 4 roundings of 2^-24 (the approximate division 2 units): 2.5 2^-22 in
    fp32, (7 + 1.8 |g|) 2^-23 for 16 bits.  Where e is subnormal its error is at most 2^-148, times |g u|."""
    I = 64
    qw, qz = np.zeros((1, 128, 2 * I), np.uint8), np.zeros((1, 1, 2 * I // 8), np.int32)
    qw[0, 0, :I], qw[0, 0, I:] = 1 + np.arange(I) % 13, 1 + np.arange(I) % 7
    words = awq.awq_pack(torch.from_numpy(qw.reshape(128, 2 * I)).cuda()).view(1, 128, 2 * I // 8)
    scales = np.ones((1, 1, 2 * I), np.float32)
    scales[0, 0, :I] = 2.0 ** -(np.arange(I) % 4)
    scales[0, 0, I:] = 2.0 ** (np.arange(I) % 5 - 2)
    x = np.zeros((rows, 128), np.float32)
    x[:, 0] = round16(np.random.default_rng(rows).uniform(-8, 8, rows).astype(np.float32), bf16)
    x[:3, 0] = 0, 7.375, -7.375
    dtype = torch.bfloat16 if bf16 else torch.float16
    w = awq.awq_moe_prepack(words, torch.from_numpy(qz).cuda(), torch.from_numpy(scales).to(dtype).cuda(), gated=True)
    order = torch.arange(rows, dtype=torch.int32, device="cuda")
    plan = awq.MoePlan(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), order, order, 1)
    y = awq.awq_moe_gemm(torch.from_numpy(x).to(dtype).cuda(), w, plan, out_dtype=torch.float32 if wide else None)
    a = x[:, :1].astype(np.float64) * (qw[0, 0] * scales[0, 0]).astype(np.float64)
    g, u = a[:, :I], a[:, I:]
    want = oracle_layer.silu(g) * u
    tol = 2.0 ** -148 * np.abs(g * u)
    if wide:
        tol += 2.5 * 2.0 ** -22 * np.abs(want) + 2.0 ** -149
    else:
        half, least = (2.0 ** -8, 2.0 ** -134) if bf16 else (2.0 ** -11, 2.0 ** -25)
        tol += (7 + 1.8 * np.abs(g)) * 2.0 ** -23 * np.abs(want)
        tol += half * (np.abs(want) + tol) + least
    err = np.abs(y.double().cpu().numpy() - want)
    assert g.min() < -88 and np.all(err <= tol), np.max(err / np.maximum(tol, 2.0 ** -1000))


def test_growing_workspaces_while_calls_are_queued(awq):  # noqa: F811
    """Outgrown memory goes back to its stream: what is queued there before still has it."""
    small, large = Layers(awq, 20), Layers(awq, 3000)
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            xs, xl = small.x(0), large.x(1)
            want = small.experts(xs), large.experts(xl), small.fp8(xs)
            torch.cuda.synchronize()
            awq._layer_workspaces.clear()
            torch.cuda._sleep(20_000_000)
            first = small.experts(xs)
            got = first, large.experts(xl), small.fp8(xs)
            junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
            torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        del junk
    assert awq.awq_last_device_error() == 0


@pytest.mark.parametrize("tokens", [4, 60, 900])
def test_rows_between_up_and_down_beyond_fp16_show_in_their_token_alone(awq, tokens):  # noqa: F811
    layers = Layers(awq, tokens)
    x = layers.x(3)
    want = layers.experts(x)
    x[2] = torch.where(x[2] < 0, -30000.0, 30000.0)
    got = layers.experts(x)
    assert not got[2].isfinite().any()
    others = torch.arange(tokens, device="cuda") != 2
    assert got[others].isfinite().all() and torch.equal(got[others], want[others])


@pytest.mark.parametrize("tokens", [1, 2, 40, 60, 300, 900])
def test_graphs_of_every_form(awq, tokens):  # noqa: F811
    """Captured with a workspace of its own and replayed on other inputs: rows four at a time and in order, tiles of all heights,
    codes inside the product and before it."""
    layers = Layers(awq, tokens)
    x, out = layers.x(0), torch.empty(tokens, 512, dtype=torch.float16, device="cuda")
    spaces = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in
              (awq.awq_moe_workspace_bytes(tokens, 2, layers.up, layers.down), awq.awq_fp8_linear_workspace_bytes(tokens, 512, 512))]
    layers.fp8(layers.experts(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers.fp8(layers.experts(x, workspace=spaces[0]), workspace=spaces[1], out=out)
    for i in range(1, 4):
        x.copy_(layers.x(i))
        graph.replay()
        assert torch.equal(out, layers.fp8(layers.experts(layers.x(i))))
    assert awq.awq_last_device_error() == 0


def fp8_reference(awq, x, wq, s_w):  # noqa: F811
    """float64 product of the codes that x quantizes to, and its magnitudes."""
    xq, s_x = awq.awq_fp8_quant_act(x)
    (m, k), n = x.shape, wq.shape[0]
    a = xq.double() * s_x.double().t().repeat_interleave(128, 1)[:, :k]
    w = wq.double() * s_w.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return a @ w.t(), a.abs() @ w.abs().t()


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (2, 16, 8), (3, 16, 8), (1, 2 ** 20, 8), (2, 2 ** 20, 8), (70, 2 ** 20, 8), (1, 16, 2 ** 20),
                                   (20, 16, 2 ** 20), (200, 16, 2 ** 20), (2 ** 22 + 5, 16, 8)])
def test_e4m3_layer_at_the_ends_of_its_sizes(awq, M, K, N):  # noqa: F811
    """The bound of the operator's own test: (27 + K / 128) 2^-23 of the magnitudes and half a step."""
    gen = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = torch.randn(M, K, generator=gen, device="cuda").half()
    wq = torch.randn(N, K, generator=gen, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s_w = (0.5 + torch.rand(-(-N // 128), -(-K // 128), generator=gen, device="cuda")) * 1e-3 / K ** 0.5
    y = awq.awq_fp8_linear(x, wq, s_w)
    rows = torch.arange(M, device="cuda") if M < 1000 else torch.tensor([0, 1, M // 2, 2 ** 22 - 1, 2 ** 22, M - 1], device="cuda")
    want, mag = fp8_reference(awq, x[rows], wq, s_w)
    err = (27 + K / 128) * 2.0 ** -23 * mag
    tol = err + 2.0 ** -11 * (want.abs() + err) + 2.0 ** -25
    off = (y[rows].double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert awq.awq_last_device_error() == 0


@pytest.mark.parametrize("rows,K,N", [(1, 2 ** 20, 32), (20, 2 ** 20, 64), (90, 2 ** 20, 32), (1, 128, 2 ** 20), (40, 128, 2 ** 20),
                                      (200, 128, 2 ** 20)])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_product_at_the_ends_of_its_sizes(awq, rows, K, N, gated):  # noqa: F811
    """(8 + K / 8) 2^-23 of the magnitudes, silu's share and half a step, as in the operator's own test."""
    if gated and N % 64:
        N = 64
    gen = torch.Generator(device="cuda").manual_seed(rows + N)
    words = torch.randint(-2 ** 31, 2 ** 31, (1, K, N // 8), generator=gen, device="cuda", dtype=torch.int32)
    scales = (0.2 / K ** 0.5 * (0.5 + torch.rand(1, K // 128, N, generator=gen, device="cuda"))).half()
    w = awq.awq_moe_prepack(words, None, scales, gated=gated)
    x = torch.randn(rows, K, generator=gen, device="cuda").half()
    order = torch.arange(rows, dtype=torch.int32, device="cuda")
    y = awq.awq_moe_gemm(x, w, awq.MoePlan(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), order, order, 1))
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device="cuda")
    a, mag = (torch.zeros(rows, N, dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, 2 ** 26 // N // 128) * 128
    for k in range(0, K, step):
        q = (((words[0, k : k + step, :, None] >> shift) & 15).flatten(-2) - 8).double()
        q *= scales[0, k // 128 : (k + step) // 128].double().repeat_interleave(128, 0)[: q.shape[0]]
        part = x[:, k : k + step].double()
        a += part @ q
        mag += part.abs() @ q.abs()
    err = (8 + K / 8) * 2.0 ** -23 * mag
    if gated:
        (g, u), (dg, du) = a.chunk(2, dim=1), err.chunk(2, dim=1)
        s = g * torch.sigmoid(g)
        a = s * u
        err = 1.1 * u.abs() * dg + (s.abs() + 1.1 * dg) * du + 2.0 ** -20 * a.abs()
    tol = err + 2.0 ** -11 * (a.abs() + err) + 2.0 ** -25
    off = (y.double() - a).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert awq.awq_last_device_error() == 0


def test_plan_of_many_rows(awq):  # noqa: F811
    R, E = 2 ** 26 + 77, 200
    ids = torch.randint(-1, E + 1, (R, 1), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    plan = awq.awq_moe_plan(ids, E)
    flat = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
    order = torch.sort(flat, stable=True).indices.int()
    n = int((flat < E).sum())
    count = torch.bincount(flat, minlength=E + 1)
    assert torch.equal(plan.offsets.long(), torch.cat((count.new_zeros(1), count[:E].cumsum(0))))
    assert torch.equal(plan.order[:n], order[:n]) and (plan.order[n:] == -1).all()
    place = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    place[order[:n].long()] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(plan.place, place)
