"""Host-side behaviour of the Python binding that no GPU is needed for: workspaces that calls share, streams of results.

The library is replaced by a stand-in and the checks of devices are taken out, so that tensors may be the host's.
"""

import contextlib
import threading
import time
import types
import weakref

import pytest

from bit_weight_only_awq_gb300 import build as awq_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def awq():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq as mod
    return mod


class Library:
    """Calls that take a while, as several launches do, and the workspaces that are in use at once."""

    def __init__(self):
        self.lock, self.inside, self.shared, self.calls = threading.Lock(), [], [], 0

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *shape: 256

        def call(*args):
            workspace, stream = args[-3], args[-1]
            with self.lock:
                self.calls += 1
                if workspace in self.inside:
                    self.shared.append((name, stream))
                self.inside.append(workspace)
            time.sleep(0.01)
            with self.lock:
                self.inside.remove(workspace)
            return 0

        return call


@pytest.fixture
def on_host(awq, monkeypatch):
    """The binding with the stand-in and two streams' workspaces in host memory; the stream of a thread is its own choice."""
    library, stream, fp8_out = Library(), threading.local(), awq._fp8_out
    spaces = {handle: torch.zeros(256, dtype=torch.uint8) for handle in (7, 8, 9)}
    monkeypatch.setattr(awq, "lib", library)
    for check in ("_need", "_on_current_gpu"):
        monkeypatch.setattr(awq, check, lambda *a: None)
    monkeypatch.setattr(awq, "_dtype16", lambda *a: 0)
    monkeypatch.setattr(awq, "_fp8_out", lambda name, out, M, N, *rest: torch.zeros(M, N))
    monkeypatch.setattr(awq, "_raw_stream", lambda s, device: stream.handle)
    monkeypatch.setattr(awq, "_stream", lambda s: stream.handle)
    monkeypatch.setattr(awq, "_layer_workspace", lambda name, handle, device, nbytes, s: spaces[handle])
    monkeypatch.setattr(awq, "_kv4_workspace", lambda handle, device, nbytes, s: spaces[handle])
    monkeypatch.setattr(awq, "device_workspace", lambda nbytes, device: spaces[7])
    monkeypatch.setattr(awq, "_kv4_shape", lambda name, cache: (4, 2, 64, 16))
    return types.SimpleNamespace(library=library, stream=stream, spaces=spaces, fp8_out=fp8_out)


def layers(awq):
    x, ids = torch.zeros(4, 128), torch.zeros(4, dtype=torch.int32)
    plan = awq.MoePlan._of(torch.zeros(3, dtype=torch.int32), ids, ids, 1)
    up, down = (types.SimpleNamespace(data=x, experts=2, K=128, N=n, gated=g, dtype=x.dtype, outputs=128)
                for n, g in ((256, True), (128, False)))
    table = types.SimpleNamespace(shape=(4, 1), stride=lambda: (1, 1), dtype=torch.int32, is_cuda=True, data_ptr=lambda: 0)
    wq, s_w, s_x = torch.zeros(128, 128), torch.zeros(1, 1), torch.zeros(1, 4)
    return {
        "awq_fp8_linear": lambda **kw: awq.awq_fp8_linear(x, wq, s_w, **kw),
        "awq_fp8_gemm": lambda **kw: awq.awq_fp8_gemm(x, s_x, wq, s_w, **kw),
        "awq_moe_gemm": lambda **kw: awq.awq_moe_gemm(x, down, plan, **kw),
        "awq_moe": lambda **kw: awq.awq_moe(x, up, down, torch.zeros(4, 1), plan, **kw),
        "kv4_attention": lambda **kw: awq.kv4_attention(torch.zeros(4, 2, 64), x, table, ids, **kw),
        "w4a8_linear": lambda **kw: awq.w4a8_linear(x, torch.zeros(128, 16), None, **kw),
    }


NAMES = ("awq_fp8_linear", "awq_fp8_gemm", "awq_moe_gemm", "awq_moe", "kv4_attention", "w4a8_linear")


def run_threads(work):
    failed = []

    def guarded(i):
        try:
            work(i)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("name", NAMES)
def test_threads_of_one_stream_use_its_workspace_one_after_another(awq, on_host, name):
    call = layers(awq)[name]

    def work(i):
        on_host.stream.handle = 7
        for _ in range(5):
            call()

    run_threads(work)
    assert on_host.library.calls == 10 and on_host.library.shared == []


def test_different_operators_of_one_stream_do_not_mix(awq, on_host):
    calls = layers(awq)

    def work(i):
        on_host.stream.handle = 7
        for _ in range(5):
            calls[("awq_moe", "awq_fp8_linear")[i]]()

    run_threads(work)
    assert on_host.library.calls == 10 and on_host.library.shared == []


def test_other_streams_and_given_workspaces_do_not_wait(awq, on_host):
    """A lock is one stream's: another's calls go on while it is held, and so do calls with a workspace of their own."""
    call, entered, leave = layers(awq)["awq_fp8_linear"], threading.Event(), threading.Event()
    real = on_host.library

    def slow(*args):
        if args[-1] == 7 and args[-3] == on_host.spaces[7].data_ptr():
            entered.set()
            assert leave.wait(30)
        return 0

    awq.lib = types.SimpleNamespace(awq_fp8_linear=slow, awq_fp8_linear_workspace_bytes=real.awq_fp8_linear_workspace_bytes)

    def work(i):
        if i == 0:
            on_host.stream.handle = 7
            call()
            return
        try:
            assert entered.wait(30)
            on_host.stream.handle = 8
            call()
            on_host.stream.handle = 7
            call(workspace=torch.zeros(256, dtype=torch.uint8))
        finally:
            leave.set()

    run_threads(work)


def test_each_threads_default_stream_is_another(awq):
    """Handle 2 names the stream of whichever thread asks; that of one that has ended may still be busy."""
    device, keys = torch.device("cuda", 0), []

    def work(i):
        keys.append((awq._stream_key(device, 2), awq._stream_key(device, 5)))
        assert awq._stream_key(device, 2) == keys[-1][0]

    for i in range(20):  # one after another: the system gives a thread's ident out again
        t = threading.Thread(target=work, args=(i,))
        t.start()
        t.join()
    assert len(keys) == len({own for own, _ in keys}) == 20 and all(other == (0, 5) for _, other in keys)


def test_a_call_from_within_the_taking_of_a_workspace_goes_first(awq, on_host, monkeypatch):
    """As a signal handler or a finalizer makes it, on the thread that holds the lock."""
    call, taking, inner = layers(awq)["awq_fp8_linear"], awq._layer_workspace, []

    def interrupted(*args):
        if not inner:
            inner.append(on_host.library.calls)
            call()
            inner.append(on_host.library.calls)
        return taking(*args)

    monkeypatch.setattr(awq, "_layer_workspace", interrupted)
    done = threading.Thread(target=lambda: (setattr(on_host.stream, "handle", 9), call()), daemon=True)
    done.start()
    done.join(20)
    assert not done.is_alive() and inner == [0, 1] and on_host.library.calls == 2


def test_workspaces_are_made_anew_after_an_expired_wait(awq, monkeypatch):
    """What the wait's call left in its flags must not reach the next one; other devices' and other errors' do not matter."""
    code = [0]

    def last_error(p):
        p._obj.value = code[0]
        return -5 if code[0] else 0

    def dirty():
        return torch.ones(8, dtype=torch.uint8)

    waited = []
    monkeypatch.setattr(awq, "lib", types.SimpleNamespace(awq_last_device_error=last_error))
    monkeypatch.setattr(awq, "_current_device", lambda: 0)
    monkeypatch.setattr(awq.torch.cuda, "current_stream",
                        lambda device: types.SimpleNamespace(synchronize=lambda: waited.append(device)))
    pools = {"_kv4_workspaces": {(0, 5): dirty(), (1, 5): dirty()},
             "_layer_workspaces": {(0, 5): dirty(), (0, 2, 99): dirty(), (1, 5): dirty()},
             "_workspaces": {0: dirty(), 1: dirty()}}
    for name, pool in pools.items():
        monkeypatch.setattr(awq, name, pool)
    graphs = pools["_workspaces"][0]  # a captured graph of the dense layers keeps this address
    assert awq.awq_last_device_error() == 0 and len(pools["_layer_workspaces"]) == 3 and graphs.all()
    code[0] = 703
    assert awq.awq_last_device_error() == 703
    assert list(pools["_kv4_workspaces"]) == [(1, 5)] and list(pools["_layer_workspaces"]) == [(1, 5)]
    assert pools["_workspaces"][0] is graphs and not graphs.any() and pools["_workspaces"][1].all() and waited == [0]


@pytest.mark.parametrize("name", ["awq_fp8_linear", "awq_fp8_gemm", "awq_moe_gemm", "awq_moe", "w4a8_linear"])
def test_results_for_a_given_stream_are_that_streams(awq, on_host, monkeypatch, name):
    """Memory of another stream may have readers there still; the current stream, which gets the result, is noted."""
    side, entered, made, noted = object(), [], [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *_):
            entered.pop()

    class Result(torch.Tensor):
        def record_stream(self, stream):
            noted.append(stream)

    real = torch.empty

    def empty(*a, **kw):
        made.append(list(entered))
        return real(*a, **kw).as_subclass(Result)

    on_host.stream.handle = 7
    call = layers(awq)[name]
    monkeypatch.setattr(awq, "_fp8_out", on_host.fp8_out)
    monkeypatch.setattr(awq.torch, "empty", empty)
    monkeypatch.setattr(awq.torch.cuda, "stream", On)
    monkeypatch.setattr(awq.torch.cuda, "current_stream", lambda device=None: "current")
    call(stream=side)
    assert made and all(streams == [side] for streams in made) and noted == ["current"] * len(made)


def test_an_outgrown_workspace_of_the_layers_is_given_back(awq, monkeypatch):
    """Each length of prompt would keep one of its own otherwise."""
    monkeypatch.setattr(awq, "_layer_workspaces", {})
    monkeypatch.setattr(awq.torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(awq.torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(awq.torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    host, made = torch.device("cpu"), []
    for nbytes in (1 << 20, 100, 5 << 20, 6 << 20, 7 << 20, 40 << 20):  # 6 MB make it 7.5
        ws = awq._layer_workspace("awq_moe", 7, host, nbytes, None)
        assert ws.numel() >= nbytes and not ws.any()
        if not made or made[-1]() is not ws:
            made.append(weakref.ref(ws))
        del ws
    assert [ref() is None for ref in made] == [True, True, True, False]
