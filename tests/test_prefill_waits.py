"""The prompt attention kernel's barriers, on the CPU: no wait may meet a phase that has already gone round twice.

An mbarrier shows a waiting thread only the parity of its phase, so a thread that waits for completion n must look before
completion n + 1 has happened; afterwards it waits for a completion that may need the thread itself.  Here the kernel's
roles (copies, operands, products, softmax warps) are sequences of waits and arrivals on counted barriers, with the
ring sizes and the barrier that guards the scales read from the source.  Each schedule holds one role up before one of its
steps and lets the others run as far as they can.
"""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_awq_gb300", "csrc",
                      "kv4_prefill.cu")


def from_source():
    """(ring sizes, barrier array that the softmax warps watch for the scales, its size's name)."""
    with open(SOURCE) as fh:
        text = fh.read()
    sizes = {name: int(re.search(rf"constexpr int {name} = (\d+);", text).group(1)) for name in ("kBufs", "kMetas", "kRaw")}
    softmax = text[text.index("softmax: a thread has a row"):text.index("products: a warp for each row tile")]
    guard = re.search(r"bars\.(\w+)\[step % (k\w+)\]", softmax)
    return sizes, guard.group(1), sizes[guard.group(2)]


class Barrier:
    def __init__(self, arrivals):
        self.need, self.have, self.done = arrivals, 0, 0

    def arrive(self):
        self.have += 1
        if self.have == self.need:
            self.have, self.done = 0, self.done + 1


SOFTMAX_WARPS = 2  # of a row tile: one may run ahead of the other


def roles(steps, mine, sizes, guard, guard_size):
    """name -> list of ("wait", barrier, completion) and ("arrive", barrier), for row tiles of mine[m] steps."""
    bufs, raw, metas = sizes["kBufs"], sizes["kRaw"], sizes["kMetas"]
    bars = {}

    def bar(name, *index):
        arrivals = {"k_empty": 2, "v_empty": 2, "p_full": SOFTMAX_WARPS}.get(name, 1)
        return bars.setdefault((name, *index), Barrier(arrivals))

    copies, operands, out = [], [], {}
    for k in range(steps):
        if k >= raw:
            copies.append(("wait", bar("raw_empty", k % raw), k // raw - 1))
        copies.append(("arrive", bar("raw_full", k % raw)))
        operands.append(("wait", bar("raw_full", k % raw), k // raw))
        if k >= bufs:
            operands.append(("wait", bar("k_empty", k % bufs), k // bufs - 1))
        operands.append(("write scales", k % metas, k))
        if guard != "k_full":
            operands.append(("arrive", bar(guard, k % guard_size)))
        operands.append(("arrive", bar("k_full", k % bufs)))
        if k >= bufs:
            operands.append(("wait", bar("v_empty", k % bufs), k // bufs - 1))
        operands += [("arrive", bar("v_full", k % bufs)), ("arrive", bar("raw_empty", k % raw))]
    out["copies"], out["operands"] = copies, operands
    for m in range(2):
        prog = []

        def scores(step):
            prog.append(("wait", bar("k_full", step % bufs), step // bufs))
            if step < mine[m]:
                prog.append(("arrive", bar("s_full", m, step % 2)))
            prog.append(("arrive", bar("k_empty", step % bufs)))

        for step in range(min(2, steps)):
            scores(step)
        for step in range(steps):
            prog.append(("wait", bar("v_full", step % bufs), step // bufs))
            if step < mine[m]:
                prog.append(("wait", bar("p_full", m, step % 2), step // 2))
                prog.append(("arrive", bar("o_done", m, step % 2)))
            prog.append(("arrive", bar("v_empty", step % bufs)))
            if step + 2 < steps:
                scores(step + 2)
        out[f"products {m}"] = prog
        for w in range(SOFTMAX_WARPS):
            prog = []
            for step in range(mine[m]):
                prog += [("wait", bar("s_full", m, step % 2), step // 2),
                         ("wait", bar(guard, step % guard_size), step // guard_size), ("read scales", step % metas, step)]
                if step:
                    prog.append(("wait", bar("o_done", m, (step - 1) % 2), (step - 1) // 2))
                prog.append(("arrive", bar("p_full", m, step % 2)))
            out[f"softmax {m} {w}"] = prog
    return out


class Lapped(Exception):
    pass


def run(programs, held=None, at=None):
    """Runs all roles; the role `held` does not pass its instruction `at` until nothing else can."""
    place = {name: 0 for name in programs}
    scales = {}

    def advance(name):
        moved = False
        while place[name] < len(programs[name]) and not (name == held and place[name] == at and not released):
            op = programs[name][place[name]]
            if op[0] == "wait":
                if op[1].done <= op[2]:
                    break
                if op[1].done != op[2] + 1:
                    raise Lapped(f"{name} waits for completion {op[2]} of a barrier that has had {op[1].done}")
            elif op[0] == "arrive":
                op[1].arrive()
            elif op[0] == "write scales":
                scales[op[1]] = op[2]
            elif scales[op[1]] != op[2]:
                raise Lapped(f"{name} reads the scales of step {scales[op[1]]} for those of {op[2]}")
            place[name] += 1
            moved = True
        return moved

    released = held is None
    while True:
        if any([advance(name) for name in programs]):
            continue
        if released:
            break
        released = True
    assert all(place[name] == len(programs[name]) for name in programs), "a role never ends"


def every_schedule(steps, mine, sizes, guard, guard_size):
    make = lambda: roles(steps, mine, sizes, guard, guard_size)  # noqa: E731
    run(make())
    for name, program in make().items():
        for at in range(len(program)):
            run(make(), name, at)


@pytest.mark.parametrize("steps,mine", [(2, (2, 2)), (14, (14, 14)), (18, (14, 18)), (14, (14, 0)), (16, (4, 16))])
def test_no_wait_is_lapped(steps, mine):
    sizes, guard, guard_size = from_source()
    every_schedule(steps, mine, sizes, guard, guard_size)


def test_the_model_finds_a_barrier_that_its_readers_do_not_hold():
    """Scales guarded by the keys' barrier, which the products alone give back, and a ring one buffer too short."""
    sizes, _, _ = from_source()
    with pytest.raises(Lapped):
        every_schedule(14, (14, 14), sizes, "k_full", sizes["kBufs"])
    with pytest.raises(Lapped):
        every_schedule(14, (14, 14), {**sizes, "kMetas": 4}, "meta_full", 4)
