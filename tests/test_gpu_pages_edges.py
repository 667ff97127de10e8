"""GPU tests of the page pool's calls at their edges, in the form of one block and the form of many: pools
without arrays against the oracle (whole numbers, all equal), source rows that lack pages."""
import numpy as np
import pytest

from oracle import kv8 as O

import _kv8 as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K = pytest.importorskip("kv_cache_compression_rotation_b200")

i32 = lambda x: torch.tensor(list(x), dtype=torch.int32, device="cuda")
dev = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()


@pytest.mark.parametrize("rows,mp,page,pages", [(6, 5, 16, 23), (40, 9, 16, 300), (60, 300, 16, 16384), (80, 300, 16, 20011)])
def test_pool_without_arrays(rows, mp, page, pages):
    """Counts, entries, map and number of live pages are those of a pool with arrays."""
    r = H.rng(rows + pages)
    table, refs, lens = np.full((rows, mp), -1), np.zeros(pages, int), [0] * rows
    d_table, d_refs = dev(table), dev(refs)
    pool = K.PagePool(d_table, d_refs, page)

    def check():
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_refs.cpu().numpy(), refs)

    for step in range(6):
        grow = [i for i in range(rows) if lens[i] == 0 and r.random() < 0.7]
        new = [int(r.integers(1, mp * page + 1)) for _ in grow]
        if grow:
            want = O.pool_reserve(table, refs, grow, [0] * len(grow), new, page)
            assert K.pages_reserve(pool, i32(grow), i32([0] * len(grow)), i32(new)).item() == want
            if want == 0:
                for i, n in zip(grow, new):
                    lens[i] = n
            check()
        held = [i for i in range(rows) if lens[i]]
        dst = [i for i in range(rows) if not lens[i]][:5]
        if held and dst:
            src = [held[int(r.integers(len(held)))] for _ in dst]
            ln = [lens[i] for i in src]
            want = O.pool_fork(table, refs, [], src, dst, ln, page)
            assert K.pages_fork(pool, i32(src), i32(dst), i32(ln)).item() == want
            if want == 0:
                for i, n in zip(dst, ln):
                    lens[i] = n
            check()
        gone = [i for i in range(rows) if lens[i] and r.random() < 0.5]
        if gone:
            ln = [lens[i] for i in gone]
            O.pool_free(table, refs, gone, ln, page)
            K.pages_free(pool, i32(gone), i32(ln))
            for i in gone:
                lens[i] = 0
        page_map, n = O.pool_compact(table, refs, [])
        live = i32([0])
        got = K.pages_compact(pool, live=live)
        assert np.array_equal(got.cpu().numpy(), page_map) and live.item() == n
        check()
    assert K.get_status() == 0


@pytest.mark.parametrize("rows,mp,pages", [(6, 8, 40), (6, 8, 17000), (300, 400, 6000)],
                         ids=["one_block", "many_pages", "many_entries"])
def test_fork_of_a_row_that_lacks_pages_changes_nothing(rows, mp, pages):
    """Entries that were never given, that name a free page or none of the pool, in the whole pages or
    in the tail: the call is refused whole, whatever its other requests are."""
    page, n = 16, 5 * 16 + 7
    table = torch.full((rows, mp), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    data = torch.arange(pages * 4, dtype=torch.int32, device="cuda")
    pool = K.PagePool(table, refs, page, [data])
    assert K.pages_reserve(pool, i32([0, 1]), i32([0, 0]), i32([n, n])).item() == 0
    good = table.clone()
    many = rows - 2 if rows > 100 else 4
    dst = list(range(2, 2 + many))
    for col, entry, length in ((5, -1, n), (2, -1, n), (0, pages - 1, n), (5, pages, n), (3, 1 << 30, n), (0, -5, 1), (6, -1, 16 * 7),
                               (6, -1, 16 * 6 + 1)):
        for where in (0, many - 1):
            table.copy_(good)
            if col < 6:
                table[1, col] = entry
            state = [t.clone() for t in (table, refs, data)]
            src, lens = [0] * many, [n] * many
            src[where], lens[where] = 1, length
            assert K.pages_fork(pool, i32(src), i32(dst), i32(lens)).item() == -1 and K.get_status() == 1
            for t, x in zip((table, refs, data), state):
                assert torch.equal(t, x)
    table.copy_(good)
    assert K.pages_fork(pool, i32([0, 1]), i32([2, 3]), i32([n, n])).item() == 0 and K.get_status() == 0
    assert torch.equal(table[2:4, :5], table[:2, :5]) and refs.sum().item() == 12 + 10 + 2


@pytest.mark.parametrize("pages", [64, 20000])
@pytest.mark.parametrize("rows", [2, 3, 4, 5])
def test_more_pages_wanted_than_32_bits_count(rows, pages):
    """rows x 2^30 pages are wanted (a table of up to 21 GB, of which nothing is touched): refused for want of
    pages, whatever the sum is modulo 2^32."""
    mp = 1 << 30
    table = torch.empty((rows, mp), dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[7] = 1
    pool = K.PagePool(table, refs, 1)
    edge = table[:, :8].clone()
    short = K.pages_reserve(pool, i32(range(rows)), i32([0] * rows), i32([mp] * rows)).item()
    assert short == 2 ** 31 - 1 - (pages - 1) and K.get_status() == 0
    assert refs.sum().item() == 1 and torch.equal(table[:, :8], edge)
