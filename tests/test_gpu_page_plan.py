"""mla_page_plan against a plain Python allocator, value for value."""
import random

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def reference(cached, new, table, free, nf, max_new, num_pages):
    """The allocator, one request at a time; None where the call refuses."""
    max_pages = len(table[0]) if table else 0
    if any(c < 0 or n < -1 or c + max(n, 0) > 64 * max_pages for c, n in zip(cached, new)):
        return None
    stack = free[:nf]
    for r, (c, n) in enumerate(zip(cached, new)):
        if n < 0:
            stack += table[r][:-(-c // 64)]
    if not 0 <= nf <= num_pages or len(stack) > num_pages:
        return None
    if sum(max(n, 0) for n in new) > max_new or sum(-(-(c + n) // 64) - -(-c // 64)
                                                     for c, n in zip(cached, new) if n >= 0) > len(stack):
        return None
    out_free = stack + free[len(stack):]
    table = [list(t) for t in table]
    lens, cu, slots, pos = [], [0], [], []
    for r, (c, n) in enumerate(zip(cached, new)):
        n = max(n, 0)
        for k in range(-(-c // 64), -(-(c + n) // 64)):
            table[r][k] = stack.pop()
        lens.append(0 if new[r] < 0 else c + n)
        for i in range(n):
            page = table[r][(c + i) // 64]
            slots.append(page * 64 + (c + i) % 64 if 0 <= page < num_pages else -1)
            pos.append(c + i)
        cu.append(cu[-1] + n)
    pad = max_new - len(slots)
    return lens, len(stack), cu, slots + [-1] * pad, pos + [0] * pad, table, out_free


def run(cached, new, table, free, nf, max_new, in_place=False, stream=None):
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    b, width = len(cached), (len(table[0]) if table else 1)
    c, f, n = t(cached), t(free), t([nf])
    tab = t(table) if table else torch.zeros(0, 1, dtype=torch.int32, device=DEV)
    lens, nfo = (c, n) if in_place else (torch.full((b,), -9, dtype=torch.int32, device=DEV), t([-9]))
    cu, slots, pos = t([-9] * (b + 1)), t([-9] * max_new), t([-9] * max_new)
    err = t([0])
    torch.cuda.synchronize()
    mla.page_plan(c, t(new), tab.view(b, width), f, n, lens, nfo, cu, slots, pos, error=err, stream=stream)
    torch.cuda.synchronize()
    return (lens.tolist(), int(nfo), cu.tolist(), slots.tolist(), pos.tolist(), tab.tolist(), f.tolist()), int(err)


def make(seed, b, max_pages, new_of, spare=40, cached_of=None):
    rng = random.Random(seed)
    cached = [(cached_of or (lambda: rng.choice([0, 1, 63, 64, 65, rng.randrange(0, 32 * max_pages)])))() for _ in range(b)]
    new = [min(new_of(rng), 64 * max_pages - c) for c in cached]
    held = [-(-c // 64) for c in cached]
    need = sum(-(-(c + n) // 64) - h for c, n, h in zip(cached, new, held) if n >= 0)
    num_pages = sum(held) + need + spare
    ids = rng.sample(range(num_pages), num_pages)
    table = []
    for h in held:
        table.append([ids.pop() for _ in range(h)] + [-1] * (max_pages - h))
    nf = len(ids)
    return cached, new, table, ids + [7777777] * (num_pages - nf), nf, num_pages


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,max_pages,kind", [
    (1, 4, "one"), (1, 40, "long"), (2, 3, "mixed"), (31, 9, "decode"), (64, 20, "mixed"), (257, 6, "mixed"),
    (1023, 5, "decode"), (1025, 4, "mixed"), (3000, 3, "decode"), (8192, 2, "decode"), (5, 300, "long")])
def test_matches_the_reference_allocator(b, max_pages, kind, in_place):
    new_of = {"one": lambda r: 1, "decode": lambda r: r.choice([1, 1, 1, 0, -1]),
              "mixed": lambda r: r.choice([-1, 0, 1, 2, 63, 64, 65, 130]),
              "long": lambda r: r.randrange(500, 20000)}[kind]
    cached, new, table, free, nf, num_pages = make(b, b, max_pages, new_of,
                                                   cached_of=(lambda: 64) if b == 8192 else None)
    total = sum(max(n, 0) for n in new)
    for max_new in {total, total + 5, total + 4099}:
        got, err = run(cached, new, table, list(free), nf, max_new, in_place)
        assert err == 0
        want = reference(cached, new, table, list(free), nf, max_new, num_pages)
        for name, g, w in zip(("lens", "num_free", "cu", "slots", "positions", "table", "free"), got, want):
            assert g == w, name


def test_no_requests_and_nothing_new():
    got, err = run([], [], [], [3, 1, 2], 3, 6)
    assert err == 0 and got[1] == 3 and got[2] == [0] and got[3] == [-1] * 6 and got[4] == [0] * 6
    got, err = run([10, 0], [0, 0], [[2, -1], [-1, -1]], [3, 1, 0], 2, 4)
    assert err == 0 and got[0] == [10, 0] and got[1] == 2 and got[2] == [0, 0, 0] and got[3] == [-1] * 4
    got, err = run([130], [-1], [[4, 5, 6]], [0, 1, 0, 0, 0, 0, 0], 2, 0)      # no slots at all: releases only
    assert err == 0 and got[0] == [0] and got[1] == 5 and got[6][:5] == [0, 1, 4, 5, 6]


def test_pages_given_back_are_taken_in_the_same_call():
    # One free page and two given back cover three requests that need one each.
    got, err = run([128, 0, 0, 64], [-1, 1, 1, 1], [[5, 6], [-1, -1], [-1, -1], [4, -1]], [3, 0, 0, 0, 0, 0, 0], 1, 3)
    assert err == 0
    assert got[1] == 0 and got[5] == [[5, 6], [6, -1], [5, -1], [4, 3]]
    assert got[3] == [6 * 64, 5 * 64, 3 * 64] and got[4] == [0, 0, 64] and got[0] == [0, 1, 1, 65]


@pytest.mark.parametrize("case,bit", [
    ("negative", mla.DEVERR_BAD_LENGTH), ("below -1", mla.DEVERR_BAD_LENGTH), ("past the row", mla.DEVERR_BAD_LENGTH),
    ("huge", mla.DEVERR_BAD_LENGTH), ("pages", mla.DEVERR_NO_ROOM), ("slots", mla.DEVERR_NO_ROOM),
    ("stack", mla.DEVERR_BAD_METADATA), ("stack below", mla.DEVERR_BAD_METADATA), ("double", mla.DEVERR_BAD_METADATA)])
@pytest.mark.parametrize("in_place", [False, True])
def test_refuses_as_a_whole(case, bit, in_place):
    cached, new, table, free, nf, max_new = [10, 100, 64], [1, 20, 1], [[0, -1], [1, 2], [3, -1]], [4, 5, 6, 0, 0, 0, 0], 3, 70
    if case == "negative":
        cached[1] = -1
    elif case == "below -1":
        new[2] = -2
    elif case == "past the row":
        new[1] = 29
    elif case == "huge":
        cached[0], new[0] = 2 ** 31 - 1, 2 ** 31 - 1
    elif case == "pages":
        nf = 0
    elif case == "slots":
        max_new = 21
    elif case == "stack":
        nf = 8
    elif case == "stack below":
        nf = -1
    elif case == "double":
        new[1], free = -1, [4, 5, 6, 0]      # three free and two more make five of four
    # The last call asks for one page more than there is; the first ones fail for their own reason.
    new = list(new)
    if case in ("slots", "pages"):
        assert reference(cached, new, table, free, nf, max_new, len(free)) is None
    got, err = run(cached, new, table, list(free), nf, max_new, in_place)
    assert err == bit
    assert got == (cached, nf, [0, 0, 0, 0], [-1] * max_new, [0] * max_new, table, free)


@pytest.mark.parametrize("cached,new", [(-100, -1), (2 ** 31 - 1, -1), (-2 ** 31, 0)])
def test_a_bad_length_is_flagged_as_that_alone(cached, new):
    """Sums over bad lengths say nothing about the stack."""
    got, err = run([cached, 10], [new, 1], [[0, -1], [1, -1]], [2, 3, 0, 0], 2, 3)
    assert err == mla.DEVERR_BAD_LENGTH
    assert got == ([cached, 10], 2, [0, 0, 0], [-1] * 3, [0] * 3, [[0, -1], [1, -1]], [2, 3, 0, 0])


def test_bad_page_ids_are_skipped_and_flagged():
    got, err = run([64, 10], [1, 2], [[0, -1], [9, -1]], [100, 0, 0, 0, 0], 1, 4)
    assert err == mla.DEVERR_BAD_INDEX
    assert got[3] == [-1, -1, -1, -1] and got[4] == [64, 10, 11, 0] and got[0] == [65, 12]


@pytest.mark.parametrize("b", [3, 300])               # a warp to a request, a thread to a page
def test_bad_page_ids_given_back_are_flagged(b):
    """An ended request's row with ids outside the pool: they return to the stack, which keeps its count, and the call
    says so."""
    cached, new = [200] + [64] * (b - 1), [-1] + [0] * (b - 1)
    pages = b + 10
    for bad in (-3, pages, 2 ** 31 - 1):
        table = [[0, bad, 2, 3]] + [[4 + r, -1, -1, -1] for r in range(b - 1)]
        got, err = run(cached, new, table, [7] * pages, 1, 5)
        assert err == mla.DEVERR_BAD_INDEX
        assert got[0] == [0] + [64] * (b - 1) and got[1] == 5 and got[6][:5] == [7, 0, bad, 2, 3] and got[3] == [-1] * 5
    # What lies past the held pages is not looked at.
    got, err = run([64] + cached[1:], new, [[0, -3, -3, -3]] + table[1:], [7] * pages, 1, 5)
    assert err == 0 and got[1] == 2


def test_replayed_graph_advances_the_state_in_place():
    """Captured once, replayed: lengths, stack and tables go on from step to step."""
    cached, new, table, free, nf, num_pages = make(5, 33, 4, lambda r: 1, spare=200, cached_of=lambda: 40)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    c, n, tab, f, k = t(cached), t(new), t(table), t(free), t([nf])
    cu, slots, pos, err = t([0] * 34), t([0] * 40), t([0] * 40), t([0])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        mla.page_plan(c, n, tab, f, k, c, k, cu, slots, pos, error=err)
    s.synchronize()
    want = reference(cached, new, table, list(free), nf, 40, num_pages)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mla.page_plan(c, n, tab, f, k, c, k, cu, slots, pos, error=err)
    for _ in range(50):
        g.replay()
        want = reference(want[0], new, want[5], want[6], want[1], 40, num_pages)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert (c.tolist(), int(k), cu.tolist(), slots.tolist(), pos.tolist(), tab.tolist()) == want[:6]


def test_replayed_graph_with_a_long_map():
    """The map's own kernel, captured behind the plan: requests of 5000 tokens grow from replay to replay, then end."""
    cached, new, table, free, nf, num_pages = make(6, 24, 320, lambda r: 5000, spare=7000, cached_of=lambda: 70)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    room = 24 * 5000 + 3
    c, n, tab, f, k = t(cached), t(new), t(table), t(free), t([nf])
    cu, slots, pos, err = t([0] * 25), torch.zeros(room, dtype=torch.int32, device=DEV), t([0] * room), t([0])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        mla.page_plan(c, n, tab, f, k, c, k, cu, slots, pos, error=err)
    want = (cached, nf, None, None, None, table, list(free))
    for step in ([5000] * 24, [5000, 0] * 12, [-1, 5000] * 12, [4999] * 24):
        n.copy_(t(step))
        g.replay()
        torch.cuda.synchronize()
        want = reference(want[0], step, want[5], want[6], want[1], room, num_pages)
        assert want is not None and int(err) == 0
        assert (c.tolist(), int(k), cu.tolist(), slots.tolist(), pos.tolist(), tab.tolist()) == want[:6]


def test_slots_at_odd_addresses():
    cached, new, table, free, nf, num_pages = make(9, 7, 5, lambda r: 33, spare=10)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    total = sum(new)
    big = torch.full((2, total + 11), -9, dtype=torch.int32, device=DEV)
    slots, pos = big[0, 1:total + 4], big[1, 3:total + 6]
    lens, nfo, cu = t([0] * 7), t([0]), t([0] * 8)
    mla.page_plan(t(cached), t(new), t(table), t(free), t([nf]), lens, nfo, cu, slots, pos)
    want = reference(cached, new, table, list(free), nf, total + 3, num_pages)
    assert slots.tolist() == want[3] and pos.tolist() == want[4]
    assert big[0, 0] == -9 and torch.all(big[0, total + 4:] == -9) and torch.all(big[1, :3] == -9)


@pytest.mark.parametrize("in_place", [False, True])
def test_long_maps(in_place):
    """Maps long enough for a kernel of their own: whole, refused, and with a bad page in the stack."""
    cached, new, table, free, nf, num_pages = make(20, 40, 300, lambda r: r.choice([-1, 0, 1, 9000, 16000]),
                                                   cached_of=lambda: 70)
    total = sum(max(n, 0) for n in new)
    assert total > 98304
    for max_new in (total, total + 7):
        got, err = run(cached, new, table, list(free), nf, max_new, in_place)
        assert err == 0 and list(got) == list(reference(cached, new, table, list(free), nf, max_new, num_pages))
    got, err = run(cached, new, table, list(free), nf, total - 1, in_place)
    assert err == mla.DEVERR_NO_ROOM and got[2] == [0] * 41 and got[5] == table and got[6] == free
    assert got[0] == cached and got[1] == nf and got[3] == [-1] * (total - 1) and got[4] == [0] * (total - 1)
    free[nf - 5] = num_pages
    got, err = run(cached, new, table, list(free), nf, total, in_place)
    want = reference(cached, new, table, list(free), nf, total, num_pages)
    assert err == mla.DEVERR_BAD_INDEX and got[3] == want[3] and got[4] == want[4] and -1 in got[3]
