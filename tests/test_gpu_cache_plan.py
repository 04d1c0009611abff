"""cache_plan on the GPU against the plain definition: whole numbers, all equal."""
import random

import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import step as os_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def state(B, per, page, fill, seed, spare=0):
    """Lengths, table, stack, its count and the number of pages, every page held once."""
    r = random.Random(seed)
    pages = B * per + spare
    lengths = [r.randrange(0, int(per * page * fill) + 1) for _ in range(B)]
    order = r.sample(range(pages), pages)
    table = [[order.pop() if e * page < n else -1 for e in range(per)] for n in lengths]
    return lengths, table, order + [-9] * (pages - len(order)), len(order), pages


def check(lengths, change, table, stack, count, pages, page, T, stride=0, per=None):
    B, per = len(lengths), len(table[0]) if table else per
    want = os_.cache_plan(lengths, change, table, stack, count, page, T, pages)
    wide = torch.full((B, per + stride), 77, dtype=torch.int32, device=DEV)
    if B and per:
        wide[:, :per] = i32(table)
    n, c, st, ct = i32(lengths), i32(change), i32(stack), i32([count])
    missing = i32([5])
    starts, slots, positions = tcm.cache_plan(n, c, wide[:, :per], st, ct, page, T, pages=pages, missing=missing)
    assert n.tolist() == want[0] and wide[:, :per].tolist() == want[1] and (wide[:, per:] == 77).all()
    assert st.tolist() == want[2] and ct.tolist() == [want[3]]
    assert starts.tolist() == want[4] and slots.tolist() == want[5] and positions.tolist() == want[6]
    assert missing.tolist() == [want[7]] and c.tolist() == list(change)
    return want


@pytest.mark.parametrize("page", [1, 2, 7, 16, 24, 64])
@pytest.mark.parametrize("B", [1, 2, 5, 63, 64, 65, 300])
def test_grow_and_shrink(B, page):
    per = 9
    lengths, table, stack, count, pages = state(B, per, page, 0.6, B + page)
    r = random.Random(B)
    change = [r.choice([0, 1, -1, r.randrange(-2 * page, 3 * page + 1), -n]) for n in lengths]
    check(lengths, change, table, stack, count, pages, page, sum(max(0, c) for c in change) + 5, stride=B % 3)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 2500])
def test_more_sequences_than_lanes(B):
    lengths, table, stack, count, pages = state(B, 3, 4, 0.7, B)
    r = random.Random(B)
    check(lengths, [r.randrange(-12, 13) for _ in lengths], table, stack, count, pages, 4, 12 * B)


@pytest.mark.parametrize("T", [0, 1, 8191, 8192, 8193, 30000, 70000])
def test_room_for_tokens(T):
    """Less room than tokens, as much, and more; on both sides of where the slots get a kernel of their own."""
    lengths, table, stack, count, pages = state(40, 60, 16, 0.2, T)
    change = [700 + 3 * b for b in range(40)]
    change[7] = change[39] = 0
    change[20] = -3
    check(lengths, change, table, stack, count, pages, 16, T)


def test_missing_pages():
    lengths, table, stack, count, pages = state(6, 10, 4, 0.3, 1)
    for left in (0, 1, 7):
        check(lengths, [13, -5, 9, 0, 30, 1], table, stack, left, pages, 4, 100)
    check(lengths, [13] * 6, table, [], 0, pages, 4, 100)
    check(lengths, [13, -20, 9, -20, 30, 1], table, stack[:2], 2, pages, 4, 100)  # returned pages past the stack's room


def test_numbers_outside_their_ranges():
    """Lengths below zero and past the table's room, changes of any size, a count past the stack, holes in
    what is returned."""
    lengths, table, stack, count, pages = state(8, 5, 8, 0.8, 2)
    table[0][0] = table[1][0] = pages
    table[2] = [-1] * 5
    big = 2**31 - 1
    lengths[3], lengths[4], lengths[5] = -7, 1000, big
    for change in ([-40, -40, -40, 9, 3, -9, 2, 1], [big] * 8, [-big - 1] * 8, [0] * 8):
        check(lengths, change, table, stack, count, pages, 8, 400)
        check(lengths, change, table, stack, big, pages, 8, 3)
        check(lengths, change, table, stack, -4, pages, 8, 3)


def test_no_sequences_and_no_table():
    check([], [], [], [3, 1], 2, 4, 16, 7, per=4)
    check([0, 5], [4, -2], [[], []], [3, 1], 2, 4, 16, 7)


@pytest.mark.parametrize("page", [1, 16])
def test_undone(page):
    lengths, table, stack, count, pages = state(50, 12, page, 0.7, 3)
    r = random.Random(4)
    change = [r.randrange(-n, 12 * page - n + 1) for n in lengths]
    n, t, st, ct = i32(lengths), i32(table), i32(stack), i32([count])
    for c in (change, [-x for x in change]):
        tcm.cache_plan(n, i32(c), t, st, ct, page, 1000)
    assert n.tolist() == lengths and t.tolist() == table and ct.tolist() == [count]
    assert st.tolist()[:count] == stack[:count]


def test_in_a_graph():
    """One captured step, replayed with other changes."""
    page, B, per = 8, 30, 20
    lengths, table, stack, count, pages = state(B, per, page, 0.5, 5)
    n, t, st, ct, c = i32(lengths), i32(table), i32(stack), i32([count]), i32([0] * B)
    starts, slots, positions = (torch.empty(k, dtype=torch.int32, device=DEV) for k in (B + 1, 100, 100))
    tcm.cache_plan(n, c, t, st, ct, page, starts=starts, slots=slots, positions=positions)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tcm.cache_plan(n, c, t, st, ct, page, starts=starts, slots=slots, positions=positions)
    r = random.Random(6)
    want = (lengths, table, stack, count)
    for _ in range(6):
        change = [r.randrange(-5, 7) for _ in range(B)]
        c.copy_(i32(change))
        graph.replay()
        want = os_.cache_plan(*want[:1], change, *want[1:4], page, 100, pages)
        assert (n.tolist(), t.tolist(), st.tolist(), ct.item(), starts.tolist(), slots.tolist(), positions.tolist()) == want[:7]
