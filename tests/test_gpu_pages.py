"""GPU parity of the page pool's operations with the oracle: whole numbers and bytes, all equal."""
import numpy as np
import pytest

from oracle import kv8 as O

import _kv8 as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K = pytest.importorskip("kv_cache_compression_rotation_b200")

i32 = lambda x: torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Both:
    """A pool on the device and in the oracle."""

    def __init__(self, r, rows, mp, page, pages, widths=((8, torch.int32), (3, torch.float32))):
        self.page, self.lens = page, [0] * rows
        self.table, self.refs = np.full((rows, mp), -1), np.zeros(pages, int)
        # arrays of whole 16 bytes a page, and of odd multiples of 4
        self.arrays = [r.integers(0, 1 << 30, (pages, w)).astype(np.int32 if dt is torch.int32 else np.float32)
                       for w, dt in widths]
        self.d_arrays = [torch.from_numpy(a.copy()).cuda() for a in self.arrays]
        self.d_table = torch.from_numpy(self.table.astype(np.int32)).cuda()
        self.d_refs = torch.from_numpy(self.refs.astype(np.int32)).cuda()
        self.pool = K.PagePool(self.d_table, self.d_refs, page, self.d_arrays)

    def check(self):
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        for a, b in zip(self.arrays, self.d_arrays):
            assert np.array_equal(a, b.cpu().numpy())

    def reserve(self, rows, new):
        old = [self.lens[i] for i in rows]
        want = O.pool_reserve(self.table, self.refs, rows, old, new, self.page)
        got = K.pages_reserve(self.pool, i32(rows), i32(old), i32(new)).item()
        assert got == want
        if want == 0:
            for i, n in zip(rows, new):
                self.lens[i] = max(n, self.lens[i])

    def fork(self, src, dst):
        lens = [self.lens[i] for i in src]
        want = O.pool_fork(self.table, self.refs, self.arrays, src, dst, lens, self.page)
        assert K.pages_fork(self.pool, i32(src), i32(dst), i32(lens)).item() == want
        if want == 0:
            for d, n in zip(dst, lens):
                self.lens[d] = n

    def free(self, rows):
        lens = [self.lens[i] for i in rows]
        O.pool_free(self.table, self.refs, rows, lens, self.page)
        K.pages_free(self.pool, i32(rows), i32(lens))
        for i in rows:
            self.lens[i] = 0

    def compact(self):
        page_map, n = O.pool_compact(self.table, self.refs, self.arrays)
        live = i32([0])
        got = K.pages_compact(self.pool, live=live)
        assert np.array_equal(got.cpu().numpy(), page_map) and live.item() == n


@pytest.mark.parametrize("rows,mp,page,pages,widths", [
    (6, 5, 16, 23, ((4, torch.int32),)),
    (40, 9, 16, 300, ((8, torch.int32), (3, torch.float32), (1, torch.int32))),
    (64, 70, 48, 4096, ((64, torch.int32), (5, torch.int32))),
    (100, 90, 32, 9001, ((16, torch.int32), (2, torch.float32))),
    (3, 2, 256, 7, ((9000, torch.int32), (4101, torch.int32))),         # pages of several slices
])
def test_random_steps_equal_the_oracle(rows, mp, page, pages, widths):
    r = H.rng(rows * 7 + mp)
    p = Both(r, rows, mp, page, pages, widths)
    counts = [0] * 4
    for _ in range(40):
        kind = int(r.integers(4))
        pick = [int(x) for x in r.permutation(rows)[:int(r.integers(1, rows + 1))]]
        if kind == 0:
            p.reserve(pick, [int(r.integers(0, mp * page + 1)) for _ in pick])
        elif kind == 1:
            p.free(pick[:max(1, len(pick) // 2)])
        elif kind == 2:
            dst = [i for i in pick if p.lens[i] == 0][:rows // 2]
            src = [i for i in range(rows) if p.lens[i] and i not in dst]
            if not dst or not src:
                continue
            p.fork([src[int(r.integers(len(src)))] for _ in dst], dst)
        else:
            p.compact()
        counts[kind] += 1
        p.check()
    assert K.get_status() == 0 and min(counts) > 0


def test_shortfall_changes_nothing():
    r = H.rng(1)
    p = Both(r, 6, 8, 16, 10)
    p.reserve([0, 1], [100, 40])              # 7 + 3 pages: all
    p.check()
    p.reserve([2, 3], [1, 17])                # 3 lacking
    p.check()
    p.fork([0, 1], [4, 5])                    # two tails lacking
    p.check()
    p.free([1])
    p.fork([0, 0], [4, 5])
    p.check()
    assert K.get_status() == 0


def test_bad_requests_are_refused_whole():
    r = H.rng(2)
    p = Both(r, 5, 4, 16, 30)
    p.reserve([0, 1], [40, 64])
    pool = p.pool
    for rows, old, new in (([0, 0], [40, 40], [50, 50]), ([5], [0], [1]), ([-1], [0], [1]), ([2], [0], [65]), ([2], [-1], [9]),
                           ([2, 1], [0, 64], [10, -3])):
        assert K.pages_reserve(pool, i32(rows), i32(old), i32(new)).item() == -1 and K.get_status() == 1
        p.check()
    for src, dst, lens in (([0], [0], [40]), ([0, 1], [2, 2], [40, 64]), ([0, 2], [2, 3], [40, 16]), ([7], [2], [4]), ([0], [9], [4]),
                           ([0], [2], [65])):
        assert K.pages_fork(pool, i32(src), i32(dst), i32(lens)).item() == -1 and K.get_status() == 1
        p.check()
    K.pages_free(pool, i32([9, 0, 0]), i32([16, 40, 40]))       # a bad row is skipped, a repeated one freed once
    assert K.get_status() == 1
    p_len, p.lens[0] = p.lens[0], 0
    O.pool_free(p.table, p.refs, [0], [p_len], 16)
    p.check()
    K.pages_free(pool, i32([0]), i32([40]))                     # no pages: nothing to do
    assert K.get_status() == 0
    p.check()


def test_copy_pages():
    r = H.rng(3)
    p = Both(r, 2, 2, 16, 50, ((12, torch.int32), (5, torch.float32), (5000, torch.int32)))
    src, dst = [3, 3, 7, 11, 0], [4, 49, 8, 11, 1]
    for a in p.arrays:
        a[dst] = a[src]
    K.pages_copy(p.pool, i32(src), i32(dst))
    assert K.get_status() == 0
    p.check()
    K.pages_copy(p.pool, i32([50, 3, 2]), i32([1, -1, 9]))
    assert K.get_status() == 1
    for a in p.arrays:
        a[9] = a[2]
    p.check()
    assert K.tq.lib().tq_pages_copy(p.pool.pa, 3, 50, None, None, 0, None) == 0


def test_packed_records_share_and_move_with_their_pool():
    """Packed TurboQuant records: a fork and a compaction leave each row's attention as it was."""
    import tq_inputs as ti
    D, Hkv, page, pages = 128, 2, 16, 24
    q = K.Quantizer.mse(ti.haar_rotation(D, 1003), 4)
    pools = [q.alloc(pages * Hkv * page) for _ in range(2)]
    table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    pool = K.PagePool(table, refs, page, [t for pk in pools for t in (pk.codes, pk.norms)])
    assert K.pages_reserve(pool, i32([2, 0]), i32([0, 0]), i32([90, 77])).item() == 0
    n = 77
    for pk, seed in zip(pools, (11, 12)):
        x = ti.normal_torch((Hkv * n, D), seed, "cuda", torch.bfloat16)
        rec = K.quantize(q, x)
        t = torch.arange(n, device="cuda")
        at = torch.cat([(table[0].long()[t // page] * Hkv + h) * page + t % page for h in range(Hkv)])
        pk.codes[at], pk.norms[at] = rec.codes, rec.norms
    qv = ti.normal_torch((1, 4, D), 13, "cuda", torch.bfloat16)
    run = lambda row: K.decode_attn_paged(q, q, qv, i32([n]), K.Pages(table[row:row + 1].clone(), page, pages), *pools, Hkv)
    want = run(0)
    assert K.pages_fork(pool, i32([0]), i32([1]), i32([n])).item() == 0
    K.pages_free(pool, i32([2]), i32([90]))
    K.pages_compact(pool)
    assert refs.sum().item() == 2 * 5 and torch.equal(run(0), want) and torch.equal(run(1), want)
    K.pages_free(pool, i32([0]), i32([n]))
    assert torch.equal(run(1), want) and refs.max().item() == 1 and K.get_status() == 0


@pytest.mark.parametrize("rows,mp,page,pages,widths", [
    (80, 300, 16, 20011, ((8, torch.int32),)),                          # more pages than one block takes
    (16400, 2, 32, 9000, ((4, torch.int32),)),                          # more rows
])
def test_large_pools_equal_the_oracle(rows, mp, page, pages, widths):
    r = H.rng(rows + pages)
    p = Both(r, rows, mp, page, pages, widths)
    for step in range(4):
        pick = [int(x) for x in r.permutation(rows)[:min(rows // 2, 1500 if step else 2500)]]
        p.reserve([i for i in pick if p.lens[i] == 0] or pick[:1], [int(r.integers(0, mp * page + 1)) for i in pick if p.lens[i] == 0]
                  or [mp * page])
        p.check()
        dst = [i for i in range(rows) if p.lens[i] == 0][:40]
        src = [i for i in range(rows) if p.lens[i]]
        if dst and src:
            p.fork([src[int(r.integers(len(src)))] for _ in dst], dst)
            p.check()
        p.free([i for i in range(rows) if p.lens[i]][::2])
        p.compact()
        p.check()
    assert K.get_status() == 0
