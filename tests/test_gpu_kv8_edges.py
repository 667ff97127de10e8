"""GPU tests of the 8-bit attention at the edges of what its calls accept, against the float64 oracle's
formulas in matrix form.

Bounds (nats), before the output's own rounding: a score 2^-19 scale sum|q k| + 2^-20 |s|, a capped one
2^-19 |s| more (three roundings of its factors, a series cut at 2^-20 of the result or an exponential and a
division, each within 2^-22 of 1, where tanh is above 0.46), 2^-20 (1 + distance from the largest) for the
exponential; the output P_EPS + the score's error + their mean + n 2^-27, each times sum p |v|."""
import math

import numpy as np
import pytest

from oracle import kv8 as O

import _kv8 as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K = pytest.importorskip("kv_cache_compression_rotation_b200")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
P_EPS = {"bf16": 2.0 ** -11, "f16": 2.0 ** -11, "f32": 2.0 ** -21}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def side(codes, scales):
    return K.Kv8(dev(codes), dev(scales))


def attend(q, pos, lens, kc, vc, Hkv, cap_tokens, **kw):
    """The decode call for one query a sequence, else the call for blocks of queries."""
    if q.shape[2] == 1:
        o, l = K.kv8_decode_attn(q[:, :, 0], lens, kc, vc, Hkv, Nmax=cap_tokens, return_lse=True, **kw)
        return o[:, :, None], l[:, :, None]
    return K.kv8_prefill_attn(q, pos, lens, kc, vc, Hkv, Nmax=cap_tokens, return_lse=True, **kw)


def setup(seed, T, d, dtype, n=300, Hq=4, Hkv=2, q_spread=1.0):
    """One sequence of n tokens whose last T are the queries."""
    r = H.rng(seed)
    lay = H.Layout(r, 1, Hkv, n, 0)
    data = [H.random_side(r, lay.records, d) for _ in range(2)]
    qt = torch.from_numpy(r.standard_normal((1, Hq, T, d)).astype(np.float32) * np.float32(q_spread)).to(DT[dtype])
    pos = np.arange(n - T, n, dtype=np.int32)[None]
    return lay, data, qt, pos, dev(np.array([n], np.int32))


@pytest.mark.parametrize("cap", [0.5, 6.0, 50.0, 1e3, 1e6, 1e30])
@pytest.mark.parametrize("T,d,dtype", [(1, 128, "bf16"), (1, 64, "f32"), (3, 64, "f16"), (60, 128, "f16"), (60, 64, "bf16"), (40, 128, "f32")])
def test_caps_of_any_size(T, d, dtype, cap):
    lay, data, qt, pos, lens = setup(100 + T + d, T, d, dtype, q_spread=2.0)
    kc, vc = (side(c, s) for c, s in data)
    out, lse = attend(qt.cuda(), dev(pos), lens, kc, vc, 2, lay.cap, scoring=K.Scoring(softcap=cap))
    assert K.get_status() == 0
    out, lse, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), qt.double().numpy()
    values, n, scale = [H.values(c, s) for c, s in data], 300, d ** -0.5
    see = np.arange(n) <= pos[0][:, None]
    for hq in range(4):
        rec = lay.rec(0, hq // 2, n)
        k, v = (x[rec] for x in values)
        s = cap * np.tanh(scale * (q64[0, hq] @ k.T) / cap)
        mag = scale * (np.abs(q64[0, hq]) @ np.abs(k).T)
        s = np.where(see, s, -np.inf)
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        w = e / e.sum(1, keepdims=True)
        fin = np.where(see, s, m)
        err = np.where(see, 2.0 ** -19 * mag + (2.0 ** -20 + 2.0 ** -19) * np.abs(fin) + 2.0 ** -20 * (1 + (m - fin).clip(0, 200)), 0)
        mean = (w * err).sum(1, keepdims=True)
        ob = (w * (P_EPS[dtype] + err + mean + n * 2.0 ** -27)) @ np.abs(v)
        want = w @ v
        tol = ob + HALF_STEP[dtype] * (np.abs(want) + ob) + TINY[dtype]
        assert np.all(np.abs(out[0, hq] - want) <= tol), float(np.max(np.abs(out[0, hq] - want) / tol))
        l = m[:, 0] + np.log(e.sum(1))
        assert np.all(np.abs(lse[0, hq] - l) <= mean[:, 0] + 2.0 ** -20 + 2.0 ** -23 * np.abs(l))


@pytest.mark.parametrize("cap", [0.01, 4.0, 1e4])
@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (3, "f32"), (30, "f16"), (100, "bf16"), (30, "f32")])
def test_nan_under_a_cap_stays_nan(T, dtype, cap):
    """A NaN in a query gives NaN in its row and nowhere else, whether its neighbours' scores are small or
    large against the cap; a NaN key gives NaN to the rows that see it."""
    lay, data, qt, pos, lens = setup(200 + T, T, 128, dtype)
    kc, vc = (side(c, s) for c, s in data)
    run = lambda x, k=kc: attend(x, dev(pos), lens, k, vc, 2, lay.cap, scoring=K.Scoring(softcap=cap))
    q = qt.cuda()
    want = run(q)
    bad = q.clone()
    bad[0, 2, T // 2, 17] = float("nan")
    out, lse = run(bad)
    assert out[0, 2, T // 2].isnan().all() and lse[0, 2, T // 2].isnan()
    keep = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    keep[0, 2, T // 2] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    codes = data[0][0].copy()
    codes[lay.rec(0, 1, 300)[299]] = 0x7f                 # the last token of key head 1: the last query sees it
    out, lse = run(q, side(codes, data[0][1]))
    assert out[0, 2:, T - 1].isnan().all() and lse[0, 2:, T - 1].isnan().all()
    assert not out[0, :2].isnan().any() and not out[0, :, :T - 1].isnan().any()
    assert K.get_status() == 0


@pytest.mark.parametrize("T,d", [(1, 128), (3, 64), (40, 128), (100, 64)])
def test_capped_bits_do_not_depend_on_others(T, d):
    """Under a cap, stale codes behind the length and a neighbouring row's large scores leave a row's bits
    as they are."""
    lay, data, qt, pos, _ = setup(300 + T, T, d, "f16", n=300)
    lens = dev(np.array([299], np.int32))                 # 299 .. 303 stand in the last block
    pos = dev(np.minimum(pos, 298))
    (kcodes, kscales), v = data
    vc = side(*v)
    run = lambda q, codes: attend(q, pos, lens, side(codes, kscales), vc, 2, lay.cap, scoring=K.Scoring(softcap=64.0))
    clean = kcodes.copy()
    big = np.where(qt[0, 1, 0].numpy() > 0, 0x7e, 0xfe).astype(np.uint8)      # far above half the cap
    for h in range(2):
        clean[lay.rec(0, h, lay.cap)[299:]] = 0
    dirty = clean.copy()
    for h in range(2):
        dirty[lay.rec(0, h, lay.cap)[299:]] = big
    q = qt.cuda()
    want = run(q, clean)
    got = run(q, dirty)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    loud = q.clone()
    loud[0, 1, 0] *= 64
    got = run(loud, clean)
    keep = torch.ones(want[1].shape, dtype=torch.bool, device="cuda")
    keep[0, 1, 0] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    assert K.get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_with_append_and_places_not_in_use(dtype):
    """A padded batch: sequences of no tokens bring none, keep their pages as they are and get zeros; nothing
    is reported, and the others get what a batch of their own gives them."""
    r = H.rng(400)
    B, Hq, Hkv, d = 5, 4, 2, 128
    lay = H.Layout(r, B, Hkv, 64, 16)
    data = [H.random_side(r, lay.records, d) for _ in range(2)]
    lens = np.array([0, 33, 0, 1, 0], np.int32)
    used = [1, 3]
    q, kn, vn = (torch.from_numpy(r.standard_normal((B, h, d)).astype(np.float32)).to(DT[dtype]).cuda() for h in (Hq, Hkv, Hkv))
    table = lay.table.copy()
    table[lens == 0] = -1                                 # they need no pages
    sides = [[side(c, s) for c, s in data] for _ in range(2)]
    out, lse = K.kv8_decode_attn(q, dev(lens), *sides[0], Hkv, pages=K.Pages(dev(table), 16, lay.num_pages), k_new=kn, v_new=vn,
                                 return_lse=True)
    assert K.get_status() == 0
    want = K.kv8_decode_attn(q[used], dev(lens[used]), *sides[1], Hkv, pages=K.Pages(dev(table[used]), 16, lay.num_pages),
                             k_new=kn[used], v_new=vn[used], return_lse=True)
    assert K.get_status() == 0
    assert torch.equal(out[used], want[0]) and torch.equal(lse[used], want[1])
    empty = [0, 2, 4]
    assert not out[empty].any() and (lse[empty] == -math.inf).all()
    for a, b in zip(*sides):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_workspaces_that_are_not_contiguous_are_refused():
    """Nothing is launched for a workspace whose elements share memory."""
    lay, data, qt, pos, lens = setup(500, 40, 64, "bf16")
    kc, vc = (side(c, s) for c, s in data)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 26)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pool = K.PagePool(torch.full((4, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda"), 16)
    for call in (lambda: attend(qt.cuda(), dev(pos), lens, kc, vc, 2, lay.cap, workspace=one),
                 lambda: attend(qt.cuda()[:, :, :1], None, lens, kc, vc, 2, lay.cap, workspace=one),
                 lambda: K.pages_reserve(pool, i32(0), i32(0), i32(9), workspace=one),
                 lambda: K.pages_fork(pool, i32(0), i32(1), i32(9), workspace=one),
                 lambda: K.pages_compact(pool, workspace=one)):
        with pytest.raises(ValueError):
            call()
    assert K.get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinities_and_nans_that_are_appended(dtype):
    """An infinity takes the largest code (its block's scale is 2^120, so finite neighbours become 0), a NaN
    the NaN code and no part in the scale; other blocks are as without them."""
    r = H.rng(600)
    x = r.standard_normal((1, 1, 48, 64)).astype(np.float32)
    x[0, 0, 3, 5], x[0, 0, 9, 60], x[0, 0, 20, 7] = np.inf, -np.inf, np.nan
    t = torch.from_numpy(x).to(DT[dtype])
    kc, vc = (K.kv8_alloc(48, 64) for _ in range(2))
    K.kv8_append(kc, vc, t.cuda(), t.cuda(), dev(np.array([48], np.int32)), Nmax=48)
    assert K.get_status() == 0
    want, scales = np.zeros((48, 64), np.uint8), np.zeros(3, np.float32)
    O.append(want, scales, np.arange(48), np.nan_to_num(t.double().numpy()[0, 0], nan=0.0, posinf=0.0, neginf=0.0), 0)
    for c in (kc, vc):
        codes, sc = c.codes.cpu().numpy(), c.scales.cpu().numpy()
        assert sc[0] == 2.0 ** 120 and np.array_equal(sc[1:], scales[1:])
        assert codes[3, 5] == 0x7e and codes[9, 60] == 0xfe and (codes[20, 7] & 0x7f) == 0x7f
        rest = codes[:16].copy()
        rest[3, 5] = rest[9, 60] = 0
        assert not (rest & 0x7f).any()
        later = codes[16:].copy()
        later[4, 7] = want[20, 7]
        assert np.array_equal(later, want[16:])
