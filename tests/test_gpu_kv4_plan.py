"""Batch plans on the GPU against the plain 64-bit implementation: steps after a
shortage of pages, entries of -1 in tables and lists of free pages."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import say
from test_gpu_kv4 import run_plan

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def check(args):
    got, want = run_plan(*args), R.plan(*args)
    for k in want:
        assert np.array_equal(got[k], np.asarray(want[k])), (k, got[k], want[k])
    return want


def test_plan_steps_through_a_shortage():
    """Steps that go on with held_out and the table of a step whose pages ran
    out: entries of -1 below held count as lost.  With held lowered to the
    pages that are there and the lost tokens brought again, they get places."""
    table = np.full((2, 6), -1)
    first = check(([0, 3], [40, 20], [0, 0], [5], 16, table, 6, 80))
    assert first["info"] == [1, 44] and first["held_out"] == [3, 2]
    second = check(([40, 23], [8, 4], first["held_out"], [6, 7], 16, first["table"], 6, 80))
    assert second["info"] == [0, 12]
    there = (np.asarray(first["table"]) >= 0).sum(1)
    again = check(([16, 0], [24, 23], there, [6, 7, 8, 9], 16, first["table"], 6, 80))
    assert again["info"] == [4, 0]
    check(([10], [30], [1], [], 16, [[3, -1, -1, -1]], 4, 50))
    assert check(([40], [4], [3], [], 16, [[3, -1, -1, -1]], 4, 50))["info"] == [0, 4]


@pytest.mark.parametrize("n,long", [(1, 3000), (3, 5000), (70, 900), (1025, 60), (4000, 20)])
@pytest.mark.parametrize("page", [16, 256])
def test_plan_holes(n, long, page):
    """Entries of -1 among the held ones and in the list of free pages, pages
    held far ahead, lists that end early, narrow tables, few tokens."""
    for turn in range(4):
        g = np.random.default_rng([n, page, turn])
        ctx, new = g.integers(0, 700, n), g.integers(0, 9, n)
        many = g.random(n) < 0.2
        many[0] = True
        new = np.where(many, g.integers(0, long, n), new)
        need = -(-(ctx + new) // page)
        held = np.where(g.random(n) < 0.5, -(-ctx // page), need + g.integers(-2, 6, n)).clip(0)
        width = int(max(1, need.max() + 4 - 5 * (turn & 1)))
        table = np.where(g.random((n, width)) < 0.9, g.integers(0, 10 ** 6, (n, width)), -1)
        free = g.permutation(max(1, int(np.maximum(0, need - held).sum()) + 3))
        if turn & 1:
            free = np.where(g.random(len(free)) < 0.9, free, -1)
        if turn & 2:
            free = free[:len(free) // 2]
        tokens = max(1, int(new.sum()) - (30 if turn == 3 else -30))
        say("plan holes n=%d page=%d turn=%d tokens=%d free=%d" % (n, page, turn, tokens, len(free)))
        check((ctx, new, held, free, page, table, width, tokens))


def test_plan_arrays_side_by_side():
    """All of a plan's arrays next to each other in one buffer: none is refused, none runs into another."""
    ctx, new, held, free, page, width, tokens = [40, 0, 7], [5, 20, 0], [3, 0, 1], [9, 8, 7], 16, 4, 30
    table = [[5, 4, 3, -1], [-1] * 4, [2, -1, -1, -1]]
    want = R.plan(ctx, new, held, free, page, table, width, tokens)
    parts = [("slots", [0] * 2 * tokens), ("ctx", ctx), ("new", new), ("held", held), ("free", free),
             ("table", sum(table, [])), ("held_out", [0] * 3), ("q_start", [0] * 4), ("kv_len", [0] * 3),
             ("positions", [0] * tokens), ("info", [0] * 2)]
    flat = torch.tensor(sum((v for _, v in parts), []), dtype=torch.int32, device="cuda")
    at, n = {}, 0
    for name, v in parts:
        at[name] = flat[n:n + len(v)]
        n += len(v)
    B.pn_kv4_plan(at["ctx"], at["new"], at["held"], 3, at["free"], 3, page, at["table"], width, width, at["held_out"],
                  at["q_start"], at["kv_len"], at["positions"], at["slots"], tokens, at["info"])
    torch.cuda.synchronize()
    for name in want:
        got = at[name].view(torch.int64) if name == "slots" else at[name]
        assert got.tolist() == np.asarray(want[name]).reshape(-1).tolist(), name
    for name, v in parts[1:5]:
        assert at[name].tolist() == v
