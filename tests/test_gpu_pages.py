"""References to pages (kvx_pages_*, kvx_cache8_copy) against a model that goes row by
row: everything is integers and copied bytes, and has to be equal."""
import random

import numpy as np
import pytest
import torch

import continuation_reference as cref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def dev(t):
    return torch.tensor(np.asarray(t, dtype=np.int32), device="cuda")


def caches_of(layers, blocks, heads, bs, d, seed):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(layers):
        codes = torch.randint(0, 256, (2, blocks, heads, bs, d), generator=g, dtype=torch.uint8).cuda()
        scale = torch.rand((2, blocks, heads), generator=g).cuda()
        out.append(kvx.Cache8(codes[0], codes[1], scale[0], scale[1]))
    return out


def parts(caches):
    return [t.cpu() for c in caches for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]


def same_contents(caches, model):
    for got, want in zip(parts(caches), model.contents):
        assert torch.equal(got, torch.stack(want))


def reserve(pages, t, l, *args, **kw):
    copies = torch.full((t.shape[0], 2), 77, dtype=torch.int32, device="cuda")
    pages.reserve(t, l, *args, copies=copies, **kw)
    return copies


def program(rng, blocks, bs, width, rows):
    """A random table and the references of it: rows share pages as forks leave them."""
    free = list(range(blocks))
    rng.shuffle(free)
    table, lens = [], []
    refs = [0] * blocks
    for r in range(rows):
        if table and rng.random() < 0.6:
            p = rng.randrange(len(table))
            n = lens[p] if rng.random() < 0.7 else rng.randint(0, lens[p])
            held = -(-n // bs)
            row = table[p][:held]
        else:
            n = rng.randint(0, width * bs)
            held = min(-(-n // bs), len(free))
            n = min(n, held * bs)
            row = [free.pop() for _ in range(held)]
        for page in row:
            refs[page] += 1
        table.append(row + [-1] * (width - len(row)))
        lens.append(n)
    return table, lens, refs


@pytest.mark.parametrize("blocks,bs,width,rows,layers,heads,d", [
    (1, 16, 1, 1, 1, 1, 16), (40, 4, 5, 6, 1, 2, 16), (300, 16, 7, 33, 3, 3, 48), (1000, 1, 40, 70, 2, 1, 64),
    (20000, 8, 9, 90, 1, 1, 16), (70000, 16, 300, 40, 1, 1, 16), (5000, 32, 3, 1500, 1, 2, 16),
    (200, 16, 5, 9, 35, 1, 16)])
def test_a_random_program(blocks, bs, width, rows, layers, heads, d):
    rng = random.Random(blocks + rows)
    table, lens, refs = program(rng, blocks, bs, width, rows)
    caches = caches_of(layers, blocks, heads, bs, d, 3)
    model = cref.Pages(refs, bs, [list(t) for t in parts(caches)])
    pages = kvx.Pages(dev(refs), bs)
    ws, status = pages.workspace(), torch.zeros(1, dtype=torch.int32, device="cuda")
    t, l = dev(table), dev(lens)
    for turn in range(4):
        N = rng.choice([1, len(lens), max(1, len(lens) // 2), len(lens) + 3])
        parents = [rng.randrange(-1 if rng.random() < 0.2 else 0, len(lens)) for _ in range(N)]
        t, l = pages.fork(t, l, dev(parents), status=status)
        table, lens = model.fork(table, lens, parents)
        assert t.tolist() == table and l.tolist() == lens and pages.refs.tolist() == model.refs
        add = [rng.choice([0, 1, 1, 2, bs, 3 * bs + 1]) for _ in lens]
        add = [min(a, width * bs - n) for a, n in zip(add, lens)]
        status.zero_()
        if turn % 2:
            add = [min(1, width * bs - max(lens))] * len(lens)
            got = reserve(pages, t, l, add[0], caches=caches, workspace=ws, status=status)
        else:
            got = reserve(pages, t, l, dev(add), caches=caches, workspace=ws, status=status)
        want = model.reserve(table, lens, add)
        if want is None:
            assert int(status.item()) == kvx.KVX_FLAG_NO_PAGES
            want = [(-1, -1)] * len(lens)
        else:
            assert int(status.item()) == 0
            lens = [a + n for a, n in zip(add, lens)]
            l = dev(lens)
        assert got.tolist() == [list(x) for x in want]
        assert t.tolist() == table and pages.refs.tolist() == model.refs
        same_contents(caches, model)
        if turn == 2:
            used, moved = pages.compact([t], caches, workspace=ws, status=status)
            u, m = model.compact([table])
            assert int(used.item()) == u and moved.tolist() == m
            assert t.tolist() == table and pages.refs.tolist() == model.refs
            same_contents(caches, model)
        status.zero_()
    pages.free(t, status=status)
    model.free(table)
    assert t.tolist() == table and pages.refs.tolist() == model.refs == [0] * blocks
    assert int(status.item()) == 0


@pytest.mark.parametrize("blocks", [4000, 40000])
def test_prompts_are_reserved_from_nothing(blocks):
    """Rows of many pages each, some of none, until the pool is full."""
    bs, width = 16, 700
    pages = kvx.Pages.empty(blocks, bs)
    model = cref.Pages([0] * blocks, bs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    add = [0, 1, 16, 17, 9000, 333, 0, 11200, 700 * 16]
    table = [[-1] * width for _ in add]
    t = dev(table)
    got = reserve(pages, t, dev([0] * len(add)), dev(add), max_new=width * bs, status=status)
    model.reserve(table, [0] * len(add), add)
    assert (got == -1).all() and t.tolist() == table and pages.refs.tolist() == model.refs
    assert int(status.item()) == 0
    # more than is left: nothing changes
    left = model.refs.count(0)
    more = dev([[-1] * (left + 1)])
    pages.reserve(more, dev([0]), (left + 1) * bs, status=status)
    assert int(status.item()) == kvx.KVX_FLAG_NO_PAGES and (more == -1).all()
    assert pages.refs.tolist() == model.refs
    # exactly what is left
    status.zero_()
    pages.reserve(more, dev([0]), left * bs, status=status)
    assert int(status.item()) == 0 and (pages.refs == 1).all()
    assert more.tolist() == [[b for b, n in enumerate(model.refs) if n == 0] + [-1]]


def test_too_few_pages_leave_shared_rows_as_they_were():
    bs = 4
    pages = kvx.Pages(dev([3, 1, 0]), bs)
    t, l = dev([[0, -1], [0, -1], [0, -1], [1, -1]]), dev([2, 2, 2, 4])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = t.clone()
    copies = reserve(pages, t, l, status=status)     # two copies and a new page
    assert int(status.item()) == kvx.KVX_FLAG_NO_PAGES and (copies == -1).all()
    assert torch.equal(t, before) and pages.refs.tolist() == [3, 1, 0]


def test_a_page_held_outside_the_call_stays():
    """Two rows of three that hold a page: both get copies."""
    pages = kvx.Pages(dev([3, 0, 0, 0]), 4)
    t = dev([[0], [0], [0]])
    caches = caches_of(1, 4, 2, 4, 16, 5)
    copies = reserve(pages, t[:2], dev([3, 1]), caches=caches)
    assert copies.tolist() == [[0, 1], [0, 2]] and t.tolist() == [[1], [2], [0]]
    assert pages.refs.tolist() == [1, 1, 1, 0]
    for x in parts(caches):
        assert torch.equal(x[1], x[0]) and torch.equal(x[2], x[0])
    # a shared page without slots of the row is replaced, not copied
    pages = kvx.Pages(dev([2, 0, 0]), 4)
    t = dev([[0], [0]])
    assert reserve(pages, t, dev([0, 0])).tolist() == [[-1, -1], [-1, -1]]
    assert t.tolist() == [[1], [0]] and pages.refs.tolist() == [1, 1, 0]


def test_bad_rows_and_entries_are_flagged_and_skipped():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flags():
        x = int(status.item())
        status.zero_()
        return x
    # fork: a parent that is no row, a length beyond the width, entries that are no pages
    pages = kvx.Pages(dev([1, 1, 0, 0]), 4)
    t, l = pages.fork(dev([[0, -1], [1, -1]]), dev([4, 4]), dev([0, 7, -2, 1]), status=status)
    assert flags() == kvx.KVX_FLAG_BAD_ROW and l.tolist() == [4, 0, 0, 4]
    assert t.tolist() == [[0, -1], [-1, -1], [-1, -1], [1, -1]] and pages.refs.tolist() == [1, 1, 0, 0]
    t, l = pages.fork(t[:1], dev([9]), dev([0]), status=status)
    assert flags() == kvx.KVX_FLAG_BAD_LENGTH and t.tolist() == [[-1, -1]] and l.tolist() == [0]
    assert pages.refs.tolist() == [0, 1, 0, 0]
    t, l = pages.fork(dev([[1, 99]]), dev([8]), dev([0, 0]), status=status)
    assert flags() == kvx.KVX_FLAG_BAD_BLOCK and t.tolist() == [[1, -1], [1, -1]]
    assert pages.refs.tolist() == [0, 2, 0, 0]
    # free
    t = dev([[1, 50], [-3, 1]])
    pages.free(t, status=status)
    assert flags() == kvx.KVX_FLAG_BAD_BLOCK and (t == -1).all() and pages.refs.tolist() == [0] * 4
    # reserve: rows whose slots do not fit, or that ask for more than the bound
    t = dev([[-1, -1]] * 4)
    got = reserve(pages, t, dev([8, -1, 0, 2]), dev([1, 1, 3, 1]), max_new=2, status=status)
    assert flags() == kvx.KVX_FLAG_BAD_LENGTH and (got == -1).all()
    assert t.tolist() == [[-1, -1]] * 3 + [[0, -1]] and pages.refs.tolist() == [1, 0, 0, 0]
    t = dev([[70, -5]])
    pages.reserve(t, dev([0]), 8, status=status)
    assert flags() == kvx.KVX_FLAG_BAD_BLOCK and t.tolist() == [[1, 2]]
    # compact: entries that are no pages stay, those of a free page go
    pages = kvx.Pages(dev([0, 0, 1, 1]), 4)
    t = dev([[3, 0, 9, -1, -4, 2]])
    used, moved = pages.compact([t], status=status)
    assert flags() == kvx.KVX_FLAG_BAD_BLOCK and t.tolist() == [[1, -1, 9, -1, -4, 0]]
    assert int(used.item()) == 2 and moved.tolist() == [-1, -1, 0, 1]


def test_copies():
    caches = caches_of(3, 50, 3, 5, 16, 7) + caches_of(1, 50, 8, 64, 128, 8)
    want = [t.clone() for t in parts(caches)]
    pairs = [[3, 4], [-1, 5], [6, -1], [49, 0], [3, 7], [9, 8]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvx.copy_pages(caches, dev(pairs), status=status)
    for x in want:
        for a, b in pairs:
            if min(a, b) >= 0:
                x[b] = x[a]
    assert all(torch.equal(a, b) for a, b in zip(parts(caches), want)) and int(status.item()) == 0
    # a count, and pages outside the pool
    kvx.copy_pages(caches, dev([[10, 11], [12, 13]]), dev([1]), status=status)
    for x in want:
        x[11] = x[10]
    assert all(torch.equal(a, b) for a, b in zip(parts(caches), want)) and int(status.item()) == 0
    kvx.copy_pages(caches, dev([[50, 1], [2, 50]]), status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK
    status.zero_()
    for n in (-1, 3):
        kvx.copy_pages(caches, dev([[10, 1], [12, 1]]), dev([n]), status=status)
        assert int(status.item()) == kvx.KVX_FLAG_BAD_LENGTH
        status.zero_()
    assert all(torch.equal(a, b) for a, b in zip(parts(caches), want))
    kvx.copy_pages(caches, dev(np.zeros((0, 2))))
    kvx.copy_pages([], dev(pairs))


@pytest.mark.parametrize("held", [0, 1, 2, 30])
@pytest.mark.parametrize("blocks", [1, 2, 63, 64, 33000])
def test_compaction_at_the_ends(blocks, held):
    rng = random.Random(blocks + held)
    where = rng.sample(range(blocks), min(held, blocks))
    refs = [0] * blocks
    for i, b in enumerate(where):
        refs[b] = 1 + i % 3
    caches = caches_of(1, blocks, 1, 2, 16, 9)
    model = cref.Pages(refs, 2, [list(t) for t in parts(caches)])
    pages = kvx.Pages(dev(refs), 2)
    tables = [[[b, -1]] for b in where[:7]]
    got = [dev(x) for x in tables]
    used, moved = pages.compact(got, caches)
    u, m = model.compact(tables)
    assert int(used.item()) == u and moved.tolist() == m and pages.refs.tolist() == model.refs
    assert [x.tolist() for x in got] == tables
    same_contents(caches, model)
