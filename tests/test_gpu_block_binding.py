"""What the Python binding of the block operators makes of its arguments: layouts, defaults, workspaces."""

import numpy as np
import pytest

from oracle import block
from tests.test_gpu_kv4_attention import Problem, awq  # noqa: F401  (awq is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def operands(p):
    return (torch.from_numpy(p.q).cuda().half(), *(torch.from_numpy(a).cuda() for a in (p.cache, p.table, p.lens)))


def test_tables_whose_rows_overlap_are_refused(awq):  # noqa: F811
    """Read with another stride, they would name what lies behind them as pages."""
    p = Problem([150], [1], 4, 2, 64, 16, seed=51)
    q, cache, table, lens = operands(p)
    want = awq.kv4_attention(q, cache, table, lens)
    q3, lens3, width = q.expand(3, -1, -1).contiguous(), lens.expand(3).contiguous(), table.shape[1]
    for bad in (table.expand(3, -1), table.flatten().as_strided((3, width - 2), (1, 1))):
        with pytest.raises(ValueError, match="block_table"):
            awq.kv4_attention(q3, cache, bad, lens3)
    got = awq.kv4_attention(q3, cache, table.expand(3, -1).contiguous(), lens3)
    assert torch.equal(got, want.expand(3, -1, -1))
    # the stride of a single row has no meaning
    assert torch.equal(awq.kv4_attention(q, cache, table.flatten().as_strided((1, width), (0, 1)), lens), want)
    assert torch.equal(awq.kv4_attention(q, cache, table[:, :width - 1], lens), want)


def test_without_max_q_every_query_is_answered(awq):  # noqa: F811
    p = Problem([200, 60, 9], [70, 3, 1], 4, 2, 64, 16, seed=34)
    q, cache, table, lens = operands(p)
    start = torch.from_numpy(p.start).cuda()
    out = torch.full_like(q, 7.0)
    awq.kv4_attention(q, cache, table, lens, q_start=start, out=out)
    want = block.kv4_attention(p.q, p.cache, p.table, p.lens, p.start, p.scale)[0]
    assert np.abs(out.float().cpu().numpy() - want).max() < 0.02
    assert torch.equal(awq.kv4_attention(q, cache, table, lens, q_start=start, max_q=70), out)
    one = awq.kv4_attention(q[:3], cache, table, lens)  # without q_start one query a sequence
    assert torch.equal(one, awq.kv4_attention(q[:3], cache, table, lens, max_q=1))


@pytest.mark.parametrize("given", [False, True])
def test_a_capture_never_shares_a_workspace(awq, given):  # noqa: F811
    """A graph that held the stream's workspace could run beside eager calls of that stream, or beside another graph."""
    p = Problem([500, 300], [1, 1], 8, 2, 128, 64, seed=35, junk=False)
    q, cache, table, lens = operands(p)
    out = torch.empty_like(q)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = awq.kv4_attention(q, cache, table, lens)  # the stream has a workspace now
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="workspace"):
        with torch.cuda.graph(graph, stream=stream):
            out.zero_()
            awq.kv4_attention(q, cache, table, lens, out=out, stream=stream if given else None)
    ws = torch.zeros(awq.kv4_attention_workspace_bytes(2, 2, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        awq.kv4_attention(q, cache, table, lens, out=out, workspace=ws, stream=stream if given else None)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_every_entry_point_takes_tensors_of_the_current_gpu_alone(awq, monkeypatch):  # noqa: F811
    p = Problem([30], [1], 4, 2, 64, 16, seed=36)
    q, cache, table, lens = operands(p)
    k, slots, x = q[:, :2].contiguous(), torch.tensor([5]).cuda(), q.view(1, -1)
    rope = torch.from_numpy(block.rope_table(8, 64)).cuda()
    calls = {
        "w4a8_rmsnorm_quant": lambda: awq.w4a8_rmsnorm_quant(x, x[0]), "awq_rmsnorm": lambda: awq.awq_rmsnorm(x, x[0]),
        "kv4_append": lambda: awq.kv4_append(cache, k, k, slots.int(), slots, rope, q=q),
        "kv4_gather": lambda: awq.kv4_gather(cache, slots), "kv4_attention": lambda: awq.kv4_attention(q, cache, table, lens)}
    for call in calls.values():
        call()
    with pytest.raises(ValueError, match="current GPU"):  # the library would take the host's address for the device's
        awq.kv4_attention(q, cache, table, lens, workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    monkeypatch.setattr(awq, "_current_device", lambda: 1)
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"{name}: every tensor is on the current GPU"):
            call()
