"""Block tables and slot maps from request lengths against a loop over tokens: exact."""
import random

import pytest
import torch

from dense_ref import extend_loop
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    return lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(seed, lens, new, width=None, spare=None, wrap=True, slots_extra=3):
    rng = random.Random(seed)
    have = [-(-max(0, c) // 64) for c in lens]
    want = [-(-(max(0, c) + max(0, n)) // 64) for c, n in zip(lens, new)]
    need = sum(w - h for w, h in zip(want, have))
    spare = need + 5 if spare is None else spare
    width = max(1, *want) if width is None else width
    ids = list(range(sum(have) + spare))
    rng.shuffle(ids)
    table, at = [], 0
    for h in have:
        row = ids[at:at + h] + [-1] * width
        table.append(row[:width])
        at += h
    free = ids[at:]
    head = 10 ** 12 + (spare // 2 if wrap else 0)
    return dict(ctx=lens, new=new, table=table, free=free, state=[head, head + len(free), 77],
                blocks=len(ids), slots=sum(max(0, n) for n in new) + slots_extra)


def run(m, c, **kw):
    table = i32(c["table"])
    got = m.mla_block_table_extend(i32(c["ctx"]), i32(c["new"]), table, i32(c["free"]),
                                   torch.tensor(c["state"], dtype=torch.int64, device=DEV), c["blocks"], c["slots"],
                                   **kw)
    torch.cuda.synchronize()
    return [t.tolist() for t in got] + [table.tolist()]


def check(m, c):
    want = extend_loop(c["ctx"], c["new"], c["table"], c["free"], c["state"], c["blocks"], c["slots"])
    got = run(m, c)
    for name, g, w in zip(("slots", "positions", "query_start", "context", "state", "table"), got, want):
        assert g == list(w), name


@pytest.mark.parametrize("lens,new", [
    ([0], [1]),
    ([0], [0]),
    ([63, 64, 65, 0, 128], [1, 1, 1, 1, 1]),
    ([63, 64, 65, 0, 128], [2, 64, 0, 65, 129]),
    ([1000] * 7, [0] * 7),
    ([10, 20, 30], [0, 5000, 0]),           # one request's tokens over several CTAs
    ([5] * 600, [1] * 600),                 # more requests than one pass takes
    ([i % 200 for i in range(1300)], [(i * 7) % 90 for i in range(1300)]),
    ([64 * i for i in range(520)], [0] * 511 + [700] * 9),
    ([-5, 3], [4, -9]),                     # negative lengths count as 0
])
def test_extend(m, lens, new):
    check(m, make(len(lens), lens, new))


def test_empty_batch_and_no_slots(m):
    table = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    got = m.mla_block_table_extend(i32([]), i32([]), table, i32([1, 2]),
                                   torch.tensor([0, 2, 0], dtype=torch.int64, device=DEV), 3, 5)
    torch.cuda.synchronize()
    assert [t.tolist() for t in got] == [[-1] * 5, [-1] * 5, [0], [], [0, 2, 0]]
    c = make(3, [10, 64], [0, 0], slots_extra=0)
    assert c["slots"] == 0
    check(m, c)


@pytest.mark.parametrize("spare", [0, 1, 3])
def test_ring_runs_short(m, spare):
    """What is left goes to the first requests; the rest gets -1 and is counted."""
    check(m, make(5, [60, 64, 10, 640], [10, 130, 2, 64], spare=spare))


def test_empty_ring_of_no_capacity(m):
    c = make(5, [60, 1], [3, 2], spare=0)
    c["free"], c["state"] = [], [0, 0, 0]
    check(m, c)


def test_table_too_narrow(m):
    check(m, make(6, [60, 100, 128], [200, 29, 70], width=3))


def test_too_few_slots(m):
    c = make(7, [60, 100, 128], [20, 30, 70])
    for n in (0, 1, 20, 33, 119):
        c["slots"] = n
        check(m, c)


def test_bad_ids_give_no_slot(m):
    """A block of the table outside the pool, and a ring that holds one."""
    c = make(8, [70, 70], [60, 60])
    c["table"][0][1] = c["blocks"] + 3
    c["free"][0] = -4
    c["free"][1] = 2 ** 31 - 1
    check(m, c)


def test_backward_state(m):
    c = make(9, [64], [3])
    c["state"] = [10, 4, 0]  # tail before head: nothing can be taken
    check(m, c)


@pytest.mark.parametrize("new", [[1] * 50, [3000, 0, 2500] + [1] * 47])
def test_in_place_replayed(m, new):
    """Lengths and ring state updated in place by a captured call, replayed: the same as as many loops."""
    lens = [(i * 37) % 150 for i in range(50)]
    c = make(10, lens, [5 * n for n in new])
    c["new"], c["slots"] = new, sum(new) + 2
    ctx, grow, table, free = i32(c["ctx"]), i32(new), i32(c["table"]), i32(c["free"])
    state = torch.tensor(c["state"], dtype=torch.int64, device=DEV)
    outs = [torch.empty(c["slots"], dtype=torch.int64, device=DEV), torch.empty(c["slots"], dtype=torch.int32, device=DEV),
            torch.empty(51, dtype=torch.int32, device=DEV)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mla_block_table_extend(ctx, grow, table, free, state, c["blocks"], c["slots"], 64, *outs,
                                 context_lens_out=ctx, free_state_out=state)
    lens, tab, st = c["ctx"], c["table"], c["state"]
    for _ in range(4):
        slots, pos, start, lens, st, tab = extend_loop(lens, new, tab, c["free"], st, c["blocks"], c["slots"])
        graph.replay()
        torch.cuda.synchronize()
        assert outs[0].tolist() == slots and outs[1].tolist() == pos and outs[2].tolist() == start
        assert ctx.tolist() == lens and state.tolist() == st and table.tolist() == tab


def test_refusals(m):
    ok = dict(context_lens=i32([1]), new_lens=i32([1]), block_table=i32([[0, -1]]), free_blocks=i32([1]),
              free_state=torch.tensor([0, 1, 0], dtype=torch.int64, device=DEV), num_blocks=2, num_slots=4)
    for bad, error in ((dict(num_blocks=-1), m.MlaError), (dict(block_size=16), m.MlaError),
                       (dict(new_lens=i32([1, 2])), ValueError), (dict(block_table=i32([0, -1])), ValueError),
                       (dict(context_lens=torch.tensor([1], device=DEV)), TypeError),
                       (dict(free_state=torch.tensor([0, 1], dtype=torch.int64, device=DEV)), ValueError),
                       (dict(slot_mapping=torch.empty(3, dtype=torch.int64, device=DEV)), ValueError),
                       (dict(context_lens=torch.tensor([1], dtype=torch.int32)), ValueError)):
        with pytest.raises(error):
            m.mla_block_table_extend(**{**ok, **bad})
