"""The care of pages on the GPU against plain lists (latent_ref.Pages): whole numbers, equal."""
import random

import pytest
import torch

import moe_decode_quantized_gb300 as moe

import latent_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool and table on the GPU, and as lists."""

    def __init__(self, n_pages, page, rows, table_pages, strided=False):
        self.plain = ref.Pages(n_pages, page, rows, table_pages)
        self.pool = moe.PagePool(torch.zeros(n_pages, dtype=torch.int32, device="cuda"), page)
        wide = torch.full((rows, table_pages + (3 if strided else 0)), -1, dtype=torch.int32, device="cuda")
        self.table = wide[:, :table_pages]
        self.status = i32([0])

    def same(self, status=0):
        assert self.pool.refs.tolist() == self.plain.refs
        assert self.table.tolist() == self.plain.table
        assert self.status.item() == status


@pytest.mark.parametrize("n_pages,page,rows,table_pages,strided", [(50, 16, 6, 9, False), (5000, 64, 40, 120, True),
                                                                   (9001, 16, 200, 40, False), (3, 16, 2, 4, True)])
def test_a_serving_loop(n_pages, page, rows, table_pages, strided):
    """Rows that grow, are forked, freed and compacted at random, the pages' contents with them."""
    rng = random.Random(n_pages)
    b = Both(n_pages, page, rows, table_pages, strided)
    lens = [0] * rows
    contents = torch.zeros((2, n_pages, 32), dtype=torch.uint8, device="cuda")
    what = [0] * n_pages  # each page's contents
    made = 0
    for step in range(30):
        act = rng.choice(["grow", "grow", "fork", "free", "compact"])
        if act == "grow":
            room = page * table_pages
            new = [min(room, n + rng.choice([0, 1, page, 3 * page + 1])) if n or rng.random() < 0.6 else 0 for n in lens]
            free = sum(r == 0 for r in b.plain.refs)
            need = sum(-(-n // page) for n in new) - sum(p >= 0 for row in b.plain.table for p in row)
            if need > free:
                continue
            before = list(b.plain.refs)
            b.plain.grow(new)
            moe.pages_grow(b.pool, b.table, i32(new), b.status)
            lens = new
            for p, (x, y) in enumerate(zip(before, b.plain.refs)):
                if x == 0 and y:
                    made += 1
                    what[p] = made % 251
                    contents[:, p] = made % 251
        elif act == "fork":
            held = [r for r in range(rows) if lens[r]]
            empty = [r for r in range(rows) if not lens[r]]
            rng.shuffle(empty)
            pairs = [(rng.choice(held), t) for t in empty[:rng.randint(1, 8)]] if held else []
            if not pairs or sum(r == 0 for r in b.plain.refs) < len(pairs):
                continue
            copies = torch.empty((len(pairs), 2), dtype=torch.int32, device="cuda")
            want = b.plain.fork(lens, pairs)
            moe.pages_fork(b.pool, b.table, i32(lens), i32([s for s, _ in pairs]), i32([t for _, t in pairs]), copies, b.status)
            assert copies.tolist() == [list(x) for x in want]
            moe.pages_copy(contents, copies, status=b.status)
            for s, d in want:
                if d >= 0:
                    what[d] = what[s]
            for s, t in pairs:
                lens[t] = lens[s]
        elif act == "free":
            gone = rng.sample(range(rows), rng.randint(1, max(1, rows // 3)))
            b.plain.free(gone)
            moe.pages_free(b.pool, b.table, i32(gone + gone[:1]), b.status)
            for r in gone:
                lens[r] = 0
        else:
            place = rng.random() < 0.5
            copies = torch.empty((n_pages // 2 + rng.randint(0, 3), 2), dtype=torch.int32, device="cuda")
            count = i32([-1])
            refs_out = b.pool.refs if place else torch.empty_like(b.pool.refs)
            table_out = b.table if place else torch.full_like(b.table.contiguous(), 5) if not strided else \
                torch.full((rows, table_pages + 3), 5, dtype=torch.int32, device="cuda")[:, :table_pages]
            want = b.plain.compact()
            moe.pages_compact(b.pool, b.table, refs_out, table_out, copies, count, b.status)
            assert count.item() == len(want)
            assert copies.tolist() == [list(x) for x in want] + [[-1, -1]] * (copies.shape[0] - len(want))
            moe.pages_copy(contents, copies, count, status=b.status)
            b.pool = moe.PagePool(refs_out, page)
            b.table = table_out
            for s, d in want:
                what[d] = what[s]
        b.same()
        for p, r in enumerate(b.plain.refs):
            if r and p % 7 == 0:
                assert (contents[:, p] == what[p]).all()
    assert made


def test_no_page_left():
    b = Both(5, 16, 3, 4)
    moe.pages_grow(b.pool, b.table, i32([33, 16, 40]), b.status)
    b.plain.grow([33, 16, 40])
    b.same(moe.MOE_WS_PAGES)
    assert b.plain.table[2] == [4, -1, -1, -1]
    b.status.zero_()
    moe.pages_grow(b.pool, b.table, i32([33, 16, 16]), b.status)  # what is held is enough
    b.same()
    moe.pages_free(b.pool, b.table, i32([2]), b.status)
    b.plain.free([2])
    b.same()
    copies = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    bb = Both(5, 16, 5, 4)
    moe.pages_grow(bb.pool, bb.table, i32([33, 16, 0, 0, 0]), bb.status)
    bb.plain.grow([33, 16, 0, 0, 0])
    moe.pages_fork(bb.pool, bb.table, i32([33, 16, 0, 0, 0]), i32([0, 0]), i32([3, 4]), copies, bb.status)
    assert bb.plain.fork([33, 16, 0, 0, 0], [(0, 3), (0, 4)]) == [(2, 4), (-1, -1)]
    assert copies.tolist() == [[2, 4], [-1, -1]]
    bb.same(moe.MOE_WS_PAGES)


def test_what_lies_outside_is_passed_over():
    b = Both(20, 16, 6, 3)
    lens = [40, 16, 0, 0, 0, 0]
    b.plain.grow(lens)
    moe.pages_grow(b.pool, b.table, i32([40, 16, -1, 49, 2 ** 31 - 1, 0]), b.status)  # rows 2, 3, 4: no such lengths
    b.same(moe.MOE_WS_INDEX)
    for source, target in (([0, 6], [2, 3]), ([0, -1], [2, 3]), ([0, 1], [2, 6]), ([0, 1], [2, 2]), ([0, 2], [2, 3]),
                           ([0, 3], [2, 3])):
        b.status.zero_()
        copies = torch.full((2, 2), 7, dtype=torch.int32, device="cuda")
        moe.pages_fork(b.pool, b.table, i32(lens), i32(source), i32(target), copies, b.status)
        want = b.plain.fork(lens, [(0, 2)])
        assert copies.tolist() == [list(want[0]), [-1, -1]]
        b.same(moe.MOE_WS_INDEX)
        b.status.zero_()
        moe.pages_free(b.pool, b.table, i32([2, 6, -1]), b.status)
        b.plain.free([2])
        b.same(moe.MOE_WS_INDEX)
    b.status.zero_()
    pages = torch.arange(3 * 20 * 4, dtype=torch.int32, device="cuda").view(3, 20, 4)
    want = pages.clone()
    want[:, 5] = want[:, 3]
    moe.pages_copy(pages, i32([[3, 5], [4, 20], [20, 4], [-1, 6], [6, -1], [2 ** 31 - 1, 1]]), status=b.status)
    assert torch.equal(pages, want) and b.status.item() == moe.MOE_WS_INDEX


def test_many_rows_and_pages():
    rows, n_pages = 1024, 40000
    b = Both(n_pages, 16, rows, 60)
    rng = random.Random(5)
    lens = [rng.randint(0, 500) for _ in range(rows)]
    moe.pages_grow(b.pool, b.table, i32(lens), b.status)
    at = 0
    table = b.table.tolist()
    for row, n in zip(table, lens):  # from an empty pool: pages in order
        k = -(-n // 16)
        assert row == list(range(at, at + k)) + [-1] * (60 - k)
        at += k
    moe.pages_free(b.pool, b.table, i32([r for r in range(rows) if r % 3]), b.status)
    refs = b.pool.refs.tolist()
    held = [p for r in range(0, rows, 3) for p in table[r] if p >= 0]
    assert sum(refs) == len(held) and all(refs[p] == 1 for p in held)
    copies, count = torch.empty((n_pages // 2, 2), dtype=torch.int32, device="cuda"), i32([0])
    moe.pages_compact(b.pool, b.table, b.pool.refs, b.table, copies, count, b.status)
    assert b.pool.refs.tolist() == [1] * len(held) + [0] * (n_pages - len(held))
    assert sorted(p for row in b.table.tolist() for p in row if p >= 0) == list(range(len(held)))
    assert b.status.item() == 0


def test_copies_past_4_gigabytes():
    """Two layers of 5 GB; pages of an odd number of pieces."""
    n, per = 70000, 16 * 4501
    pages = torch.empty((2, n, per), dtype=torch.uint8, device="cuda")
    src = torch.randint(0, 256, (2, per), dtype=torch.uint8, device="cuda")
    pages[:, 3] = src
    pages[:, n - 2] = 0
    moe.pages_copy(pages, i32([[3, n - 1], [-1, -1]]))
    assert torch.equal(pages[:, n - 1], src) and (pages[:, n - 2] == 0).all() and torch.equal(pages[:, 3], src)


def test_in_a_graph():
    """Free, fork, grow and copy captured together and replayed: the same pages each time."""
    b = Both(64, 16, 6, 8)
    lens = [50, 33, 0, 0, 0, 0]
    moe.pages_grow(b.pool, b.table, i32(lens), b.status)
    pages = torch.randint(0, 256, (1, 64, 16), dtype=torch.uint8, device="cuda")
    kids, source, new = i32([2, 3, 4]), i32([0, 1, 0]), i32([50, 33, 60, 60, 60, 0])
    kv = i32(lens)
    copies = torch.empty((3, 2), dtype=torch.int32, device="cuda")

    def step():
        moe.pages_free(b.pool, b.table, kids, b.status)
        moe.pages_fork(b.pool, b.table, kv, source, kids, copies, b.status)
        moe.pages_grow(b.pool, b.table, new, b.status)
        moe.pages_copy(pages, copies, status=b.status)

    step()
    b.plain.grow(lens)
    want = b.plain.fork(lens, [(0, 2), (1, 3), (0, 4)])
    b.plain.grow(new.tolist())
    b.same()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        b.same()
        assert copies.tolist() == [list(x) for x in want]
        for s, d in want:
            if d >= 0:
                assert torch.equal(pages[0, s], pages[0, d])
