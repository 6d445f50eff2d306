"""Page plans against the same plan made of lists, pages given back, and refusals."""
import ctypes
import random

import pytest
import torch

from tests import cache_ref as ref

gpu = pytest.mark.gpu
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def make(n, page, past, new, width=None, short=0, seed=0):
    r = random.Random(seed)
    kv = [r.randrange(past + 1) for _ in range(n)]
    q = [r.randrange(new + 1) for _ in range(n)]
    have = [-(-x // page) for x in kv]
    width = width or max(1, max(-(-(x + y) // page) for x, y in zip(kv, q)))
    have = [min(h, width) for h in have]
    need = sum(-(-(x + y) // page) - -(-x // page) for x, y in zip(kv, q))
    pages = list(range(sum(have) + need + 3))
    r.shuffle(pages)
    table, at = [], 0
    for h in have:
        table.append(pages[at:at + h] + [-1] * (width - h))
        at += h
    free = pages[at:]
    return table, [min(x, width * page) for x in kv], q, free, max(0, len(free) - short)


def run(table, kv, q, free, count, page, rows, **kw):
    from gated_delta_rule_03_gb300 import page_plan
    t = ints(table)
    p = page_plan(t, ints(kv), ints(free), ints([count]), page, q_lens=None if q is None else ints(q), rows=rows, **kw)
    got = {n: getattr(p, n).tolist() for n in p._fields}
    got["table"] = t.tolist()
    return got


CASES = [  # requests, page, longest past, most new tokens, width, pages that are missing, rows behind
    (1, 16, 0, 1, None, 0, 0), (3, 64, 500, 90, None, 0, 5), (256, 16, 8000, 1, None, 0, 0),
    (256, 16, 300, 1, None, 9, 3), (40, 32, 1000, 400, None, 60, 0), (7, 128, 2000, 3000, None, 0, 100),
    (9, 64, 900, 1500, 12, 0, 0), (1500, 16, 200, 40, None, 300, 17), (2500, 128, 5, 1, None, 0, 0), (5, 16, 60, 0, None, 0, 4),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_plan_against_lists(case):
    n, page, past, new, width, short, behind = case
    for seed in range(3):
        table, kv, q, free, count = make(n, page, past, new, width, short, seed)
        rows = sum(q) + behind
        got = run(table, kv, q, free, count, page, rows)
        want = ref.plan([list(r) for r in table], kv, free, count, page, q, rows)
        for name, w in want.items():
            assert got[name] == w, name


@gpu
def test_refused_requests():
    """Behind the rows, behind the table, no pages, a negative length; those after them are served."""
    page, q, kv = 16, [20, 16, 33, 5, -3, 40], [0, 16, 0, -1, 8, 3]
    table = [[-1] * 3, [0, -1, -1], [-1] * 3, [-1] * 3, [1, -1, -1], [2, -1, -1]]
    free = [9, 8, 7, 6, 5, 4]
    for count, rows in ((6, 114), (2, 114), (0, 114), (3, 113), (6, 20), (6, 0)):
        got = run(table, kv, q, free, count, page, rows)
        want = ref.plan([list(r) for r in table], kv, free, count, page, q, rows)
        for name, w in want.items():
            assert got[name] == w, (name, count, rows)


@gpu
def test_single_tokens_in_place_and_from_a_graph():
    from gated_delta_rule_03_gb300 import page_plan
    page, n, steps = 16, 5, 40
    table, kv, free, count = torch.full((n, 8), -1, dtype=I32, device="cuda"), ints([0, 3, 15, 16, 31]), ints(list(range(40))), ints([40])
    for i, pages in enumerate((0, 1, 1, 1, 2)):
        for j in range(pages):
            table[i, j] = 40 + 2 * i + j
    lists = [table.tolist(), kv.tolist(), 40]
    out = page_plan(table.clone(), kv.clone(), free, count.clone(), page)  # memory of the right sizes
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        page_plan(table, kv, free, count, page, kv_lens_out=kv, free_count_out=count, cu_q=out.cu_q, start=out.start,
                  positions=out.positions, slots=out.slots)
    for _ in range(steps):
        graph.replay()
        want = ref.plan(lists[0], lists[1], free.tolist(), lists[2], page, [1] * n, n)
        lists = [want["table"], want["kv_lens"], want["free_count"][0]]
        assert table.tolist() == want["table"] and kv.tolist() == want["kv_lens"] and count.tolist() == want["free_count"]
        assert out.positions.tolist() == want["positions"] and out.slots.tolist() == want["slots"]
        assert out.start.tolist() == want["start"] and out.cu_q.tolist() == want["cu_q"]


@gpu
@pytest.mark.parametrize("n,page", [(6, 16), (1300, 32)])
@pytest.mark.parametrize("room", [0, 2, 10 ** 6])
def test_release(n, page, room):
    from gated_delta_rule_03_gb300 import page_release
    table, kv, _, free, _ = make(n, page, 400, 0, seed=3)
    r = random.Random(1)
    done = [r.random() < 0.5 for _ in range(n)]
    held = sum(-(-kv[i] // page) for i in range(n) if done[i])
    size = len(free) + min(room, held)
    t, k, f, c = ints(table), ints(kv), ints(free + [-7] * (size - len(free))), ints([len(free)])
    page_release(t, k, torch.tensor(done, device="cuda"), f, c, page)
    full = False
    for i in range(n):
        m = -(-kv[i] // page)
        if not done[i] or full:
            continue
        if len(free) + m > size:
            full = True
            continue
        free = free + table[i][:m]
        table[i][:m] = [-1] * m
        kv[i] = 0
    got = k.tolist()
    assert c.tolist() == [len(free)] and f.tolist()[:len(free)] == free and t.tolist() == table
    assert got == kv


def test_refusals_on_the_host():
    from gated_delta_rule_03_gb300 import ops
    from gated_delta_rule_03_gb300.cache import PageShape
    lib = ops._load()
    A = [0x10000000 * (i + 1) for i in range(11)]
    base = dict(num_seqs=4, width=8, rows=100, num_pages=50, page=16)

    def plan(i=None, to=None, **kw):
        args = list(A)
        if i is not None:
            args[i] = to
        return lib.gdr_page_plan(ctypes.byref(PageShape(**dict(base, **kw))), *args, None)

    def release(i=None, to=None, **kw):
        args = A[:5]
        if i is not None:
            args[i] = to
        return lib.gdr_page_release(ctypes.byref(PageShape(**dict(base, **kw))), *args, None)

    for f in (plan, release):
        for kw in (dict(num_seqs=0), dict(width=0), dict(rows=-1), dict(num_pages=-1), dict(num_pages=2 ** 28)):
            assert f(**kw) == -1, kw
        for kw in (dict(page=8), dict(page=48), dict(page=256)):
            assert f(**kw) == -2, kw
        assert f(1, None) == -1 and f(1, A[1] + 2) == -3
    for i in (2, 3, 4, 5, 6, 7, 8, 9, 10):
        assert plan(i, None) == -1
    assert plan(4, A[1]) == -1 and plan(5, A[4]) == -1 and plan(10, A[9]) == -1 and plan(7, A[0]) == -1
    for i in (0, 2, 3, 4):
        assert release(i, None) == -1
    assert release(2, A[1]) == -1 and release(3, A[0]) == -1
    assert lib.gdr_page_plan(None, *A, None) == -1 and lib.gdr_page_release(None, *A[:5], None) == -1


@gpu
def test_entries_that_can_be_no_page_give_no_slot():
    """The next tokens of four requests whose last page is half full, by a table that holds no page there."""
    from gated_delta_rule_03_gb300 import page_plan
    page = 16
    table = torch.tensor([[0, 3], [-7, -1], [2 ** 27, 0], [2 ** 28, 0], [2 ** 31 - 1, 0], [2 ** 27 - 1, 0]], dtype=I32, device="cuda")
    plan = page_plan(table, ints([8] * 6), ints([5]), ints([1]), page)
    assert plan.slots.tolist() == [8, -1, -1, -1, -1, 2 ** 31 - 8] and plan.positions.tolist() == [8] * 6 and plan.free_count.tolist() == [1]
