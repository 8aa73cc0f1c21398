"""Calls of the layers with experts and the e4m3 layers in company: of other threads, streams, buffers and lengths.

Results that are compared bit for bit come from the same call made by itself, whose own bounds other tests hold.
"""

import threading

import numpy as np
import pytest

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
