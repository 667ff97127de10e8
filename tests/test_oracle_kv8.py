"""The 8-bit cache's oracle pinned by definitions that it does not use itself."""
import math

import numpy as np
import pytest

from oracle import kv8 as O

import _kv8 as H

torch = pytest.importorskip("torch")


def test_e4m3_values_and_codes_match_the_format():
    b = torch.arange(256, dtype=torch.uint8)
    v = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.VALUES[~np.isnan(v)], v[~np.isnan(v)]) and np.isnan(O.VALUES[[127, 255]]).all()
    r = H.rng(1)
    x = np.concatenate([r.standard_normal(20000) * 2.0 ** r.integers(-12, 9, 20000), O.VALUES[:127],
                        (O.VALUES[:126] + O.VALUES[1:127]) / 2]).clip(-448, 448)
    x = np.concatenate([x, -x]).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_code(x), t)


@pytest.mark.parametrize("amax", [0.0, 1e-45, 2.0 ** -126, 1.0, 1.75, 1.7500001, 447.99, 448.0, 448.00003, 3e38])
def test_scale_is_the_smallest_power_that_covers(amax):
    a = float(np.float32(amax))
    s = O.scale_of(a)
    assert math.frexp(s)[0] == 0.5 and a <= 448 * s
    assert s == 2.0 ** -126 or a > 448 * s / 2


def test_append_in_pieces_covers_every_token():
    """Tokens appended one by one, in runs or at once: each value is off by at most a rounding of
    the block's final scale (2^-4 of the value, or half the smallest step 2^-10 s), twice."""
    r = H.rng(2)
    d, n = 64, 75
    x = r.standard_normal((n, d)) * np.exp(r.standard_normal((n, 1)))
    for cuts in ([n], [1] * n, [3, 13, 16, 1, 31, 11]):
        codes, scales = np.zeros((80, d), np.uint8), np.zeros(5, np.float32)
        at = 0
        for k in cuts:
            O.append(codes, scales, np.arange(80), x[at:at + k], at)
            at += k
        got = H.values(codes, scales)[:n]
        s = np.repeat(scales.astype(np.float64), 16)[:n, None]
        assert np.all(np.abs(got - x) <= 2 * (2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s))
        if cuts == [n]:
            assert np.all(np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


def test_attention_matches_a_direct_softmax():
    r = H.rng(3)
    q, k, v = r.standard_normal(16), r.standard_normal((40, 16)), r.standard_normal((40, 16))
    o, lse, ob, lb = O.attention(q, k, v, 30, 5, 31, 0.25, cap=2.0, slope=0.1)
    s = 2 * np.tanh(k @ q * 0.25 / 2) - 0.1 * np.abs(30 - np.arange(40))
    e = np.where((np.arange(40) >= 5) & (np.arange(40) < 31), np.exp(s), 0)
    assert np.allclose(o, e @ v / e.sum(), rtol=1e-12) and math.isclose(lse, math.log(e.sum()), rel_tol=1e-12)
    assert np.all(ob > 0) and lb > 0
    o, lse, *_ = O.attention(q, k, v, 30, 7, 7, 0.25)
    assert not o.any() and lse == -math.inf


def test_visible_sets():
    assert O.visible(9, 20) == (0, 10) and O.visible(9, 5) == (0, 5) and O.visible(-1, 5, prefix=3) == (0, 0)
    assert O.visible(9, 20, window=4) == (6, 10) and O.visible(3, 20, prefix=8) == (0, 8)
    assert O.visible(9, 20, first=9) == (9, 10) and O.visible(9, 20, first=12) == (12, 12)


def test_pool_steps_keep_counts():
    """After any steps a page's count is the number of table entries that name it, and content
    follows the rows."""
    r = H.rng(4)
    rows, mp, page, pages = 8, 6, 4, 40
    table, refs = np.full((rows, mp), -1), np.zeros(pages, int)
    data = r.integers(0, 1 << 30, (pages, 3))
    lens = [0] * rows
    seen = {}
    for step in range(60):
        kind = r.integers(4)
        i = int(r.integers(rows))
        if kind == 0:
            new = int(r.integers(0, mp * page + 1))
            if new > lens[i] and O.pool_reserve(table, refs, [i], [lens[i]], [new], page) == 0:
                lens[i] = new
        elif kind == 1:
            O.pool_free(table, refs, [i], [lens[i]], page)
            lens[i] = 0
        elif kind == 2:
            j = int(r.integers(rows))
            if i != j and lens[i] == 0 and lens[j] and O.pool_fork(table, refs, [data], [j], [i], [lens[j]], page) == 0:
                lens[i] = lens[j]
                c = O.pages_of(lens[i], page) - 1
                assert np.array_equal(data[table[i, c]], data[table[j, c]])
        else:
            before = {(a, b): data[table[a, b]].copy() for a in range(rows) for b in range(mp) if table[a, b] >= 0}
            page_map, n = O.pool_compact(table, refs, [data])
            assert n == (refs > 0).sum() and (refs[:n] > 0).all()
            for (a, b), x in before.items():
                assert np.array_equal(data[table[a, b]], x)
        assert np.array_equal(np.bincount(table[table >= 0], minlength=pages), refs)
        seen[kind] = seen.get(kind, 0) + 1
    assert len(seen) == 4
