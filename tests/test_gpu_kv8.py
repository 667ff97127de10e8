"""GPU parity of the 8-bit block-scaled cache with the float64 oracle.

Append is exact arithmetic up to one rounding: codes and scales must be equal.  Attention is held
to the bound that the oracle derives for each row (probabilities rounded to halves, or to pairs of
halves for fp32 queries; fp32 scores and sums) plus half a step of the output's type.
"""
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
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}     # half the smallest step
P_EPS = {"bf16": 2.0 ** -11, "f16": 2.0 ** -11, "f32": 2.0 ** -21}


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dt is None else t.to(dt)


def pages_of(lay):
    return None if lay.table is None else K.Pages(dev(lay.table), lay.page, lay.num_pages)


def side(codes, scales):
    return K.Kv8(dev(codes), dev(scales))


def typed(r, shape, dtype, spread=1.0):
    """Random values in `dtype`: the CUDA tensor and its values in float64."""
    t = torch.from_numpy(r.standard_normal(shape).astype(np.float32) * np.float32(spread)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


# ------------------------------------------------------------------------------------- append
APPEND = [
    # B, Hkv, T, d, page, lens (with the new), new
    (1, 1, 1, 128, 0, [1], [1]),
    (3, 2, 1, 128, 16, [16, 17, 33], [1, 1, 1]),
    (2, 3, 1, 64, 48, [5, 96], [1, 1]),
    (4, 2, 40, 128, 16, [40, 41, 55, 100], [40, 40, 39, 1]),
    (4, 1, 40, 64, 64, [40, 16, 77, 3], [40, 0, 33, 3]),
    (2, 2, 77, 128, 0, [77, 130], [77, 61]),
    (1, 8, 1000, 128, 256, [1500], [1000]),
    (3, 1, 17, 64, 32, [17, 31, 48], [17, 16, 17]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_equals_the_oracle(case, dtype):
    B, Hkv, T, d, page, lens, new = APPEND[case]
    r = H.rng(100 + case)
    lay = H.Layout(r, B, Hkv, max(lens) + 20, page)
    init = [H.random_side(r, lay.records, d, exp_range=4) for _ in range(2)]
    # rows of widely unlike size, zeros and subnormals among them
    x = []
    for _ in range(2):
        v = r.standard_normal((B, T, Hkv, d)) * 2.0 ** r.integers(-10, 6, (B, T, Hkv, 1))
        v[:, T // 2] = 0 if case % 2 else v[:, T // 2]
        t = torch.from_numpy(v.astype(np.float32)).to(DT[dtype])
        x.append((t.cuda().transpose(1, 2), t.double().numpy().transpose(0, 2, 1, 3)))
    kc, vc = (side(c, s) for c, s in init)
    K.kv8_append(kc, vc, x[0][0], x[1][0], dev(np.array(lens, np.int32)), new_lens=dev(np.array(new, np.int32)),
                 Nmax=0 if page else lay.cap, pages=pages_of(lay))
    assert K.get_status() == 0
    for (codes, scales), (_, v), got in zip(init, x, (kc, vc)):
        for b in range(B):
            for h in range(Hkv):
                rec = lay.rec(b, h, lens[b])
                O.append(codes, scales, rec, v[b, h, :new[b]], lens[b] - new[b])
        assert np.array_equal(got.scales.cpu().numpy(), scales)
        assert np.array_equal(got.codes.cpu().numpy(), codes)


def test_append_token_by_token_and_bad_lengths():
    """60 single appends equal the oracle's; sequences with impossible lengths are left alone and
    reported, the others of the call are written."""
    r = H.rng(7)
    lay = H.Layout(r, 2, 2, 64, 16)
    codes, scales = H.random_side(r, lay.records, 128)
    kc, vc = side(codes, scales), side(codes, scales)
    for n in range(1, 61):
        t, v = typed(r, (2, 2, 1, 128), "bf16", 2.0 ** (n % 7 - 3))
        K.kv8_append(kc, vc, t, t, dev(np.array([n, n], np.int32)), pages=pages_of(lay))
        for b in range(2):
            for h in range(2):
                O.append(codes, scales, lay.rec(b, h, n), v[b, h], n - 1)
    assert K.get_status() == 0
    for c in (kc, vc):
        assert np.array_equal(c.codes.cpu().numpy(), codes) and np.array_equal(c.scales.cpu().numpy(), scales)
    t, v = typed(r, (2, 2, 3, 128), "bf16")
    for lens, new in (([2, 64], [3, 1]), ([65, 64], [1, 1]), ([9, 64], [4, 1]), ([9, 64], [-1, 1])):
        K.kv8_append(kc, vc, t, t, dev(np.array(lens, np.int32)), new_lens=dev(np.array(new, np.int32)), pages=pages_of(lay))
        assert K.get_status() == 1
        for h in range(2):
            O.append(codes, scales, lay.rec(1, h, 64), v[1, h, :1], 63)
        assert np.array_equal(kc.codes.cpu().numpy(), codes) and np.array_equal(vc.scales.cpu().numpy(), scales)


# ------------------------------------------------------------------------------------- attention
def check_rows(out, lse, q64, kv, lay, lens, pos, G, scale, dtype, cap=0.0, slopes=None, window=0, first=None, prefix=None):
    """out [B, Hq, T, d], lse [B, Hq, T] against the oracle, row by row."""
    B, Hq, T, d = q64.shape
    worst = 0.0
    for b in range(B):
        for h in range(Hq // G):
            rec = lay.rec(b, h, lens[b])
            k, v = kv[0][rec], kv[1][rec]
            for g in range(G):
                hq = h * G + g
                for i in range(T):
                    lo, hi = O.visible(int(pos[b][i]), lens[b], window, None if first is None else int(first[b][i]),
                                       None if prefix is None else int(prefix[b]))
                    o, l, ob, lb = O.attention(q64[b, hq, i], k, v, int(pos[b][i]), lo, hi, scale, cap,
                                               0.0 if slopes is None else float(slopes[hq]), P_EPS[dtype])
                    tol = ob + HALF_STEP[dtype] * (np.abs(o) + ob) + TINY[dtype]
                    err = np.abs(out[b, hq, i] - o)
                    assert np.all(err <= tol), (b, hq, i, float(np.max(err / tol)))
                    if hi <= lo:
                        assert lse[b, hq, i] == -math.inf
                    else:
                        assert abs(lse[b, hq, i] - l) <= lb + 2.0 ** -23 * abs(l), (b, hq, i, lse[b, hq, i], l)
                        worst = max(worst, float(np.max(err / tol)))
    return worst


def attention_case(seed, B, Hq, Hkv, d, lens, page, dtype, T=0, cap=0.0, alibi=False, window=0, docs=False, prefix=0,
                   exp_range=2, scale=None, append=False, pos=None, q_spread=1.0):
    r = H.rng(seed)
    lay = H.Layout(r, B, Hkv, max(max(lens), 1) + 5, page)
    init = [H.random_side(r, lay.records, d, exp_range=exp_range) for _ in range(2)]
    kc, vc = (side(c, s) for c, s in init)
    G, steps = Hq // Hkv, max(T, 1)
    qt = torch.from_numpy(r.standard_normal((B, steps, Hq, d)).astype(np.float32) * np.float32(q_spread)).to(DT[dtype])
    q = qt.cuda().transpose(1, 2)
    q64 = qt.double().numpy().transpose(0, 2, 1, 3)
    if pos is None:
        pos = [[n - steps + i for i in range(steps)] for n in lens]
    first = [[max(0, p - int(r.integers(0, 2 * max(lens) // 3 + 1))) for p in row] for row in pos] if docs else None
    pre = [prefix + b for b in range(B)] if prefix else None
    slopes = (2.0 ** -(1 + np.arange(Hq) % 8)).astype(np.float32) if alibi else None
    sc = K.Scoring(scale=scale, softcap=cap, slopes=None if slopes is None else dev(slopes), window=window,
                   first=None if first is None else dev(np.array(first, np.int32)),
                   prefix=None if pre is None else dev(np.array(pre, np.int32)))
    kw = dict(Nmax=0 if page else lay.cap, pages=pages_of(lay), scoring=sc, return_lse=True)
    lt = dev(np.array(lens, np.int32))
    if T:
        out, lse = K.kv8_prefill_attn(q, dev(np.array(pos, np.int32)), lt, kc, vc, Hkv, **kw)
    else:
        if append:
            new = [typed(r, (B, Hkv, d), dtype) for _ in range(2)]
            kw.update(k_new=new[0][0], v_new=new[1][0])
            for (codes, scales), (_, x) in zip(init, new):
                for b in range(B):
                    for h in range(Hkv):
                        O.append(codes, scales, lay.rec(b, h, lens[b]), x[b, h][None], lens[b] - 1)
        out, lse = K.kv8_decode_attn(q[:, :, 0], lt, kc, vc, Hkv, **kw)
        out, lse = out[:, :, None], lse[:, :, None]
        if append:
            assert np.array_equal(kc.codes.cpu().numpy(), init[0][0]) and np.array_equal(vc.codes.cpu().numpy(), init[1][0])
    assert K.get_status() == 0
    kv = [H.values(c, s) for c, s in init]
    check_rows(out.double().cpu().numpy(), lse.double().cpu().numpy(), q64, kv, lay, lens, pos, G,
               1 / math.sqrt(d) if scale is None else scale, dtype, cap, slopes, window, first, pre)


DECODE = [
    # B, Hq, Hkv, d, lens, page, options
    dict(B=1, Hq=1, Hkv=1, d=128, lens=[1], page=0),
    dict(B=1, Hq=8, Hkv=1, d=128, lens=[33], page=16),
    dict(B=4, Hq=8, Hkv=2, d=128, lens=[0, 1, 16, 700], page=0),
    dict(B=3, Hq=12, Hkv=2, d=64, lens=[31, 32, 257], page=48),
    dict(B=2, Hq=32, Hkv=2, d=128, lens=[515, 96], page=64),          # 16 query heads a key head
    dict(B=2, Hq=40, Hkv=2, d=64, lens=[129, 300], page=16),          # 20: two row groups
    dict(B=5, Hq=7, Hkv=1, d=64, lens=[1000, 3, 999, 17, 480], page=16, append=True),
    dict(B=2, Hq=6, Hkv=2, d=128, lens=[1, 400], page=32, append=True, cap=5.0),
    dict(B=2, Hq=8, Hkv=4, d=128, lens=[300, 301], page=0, cap=30.0, alibi=True, window=37),
    dict(B=2, Hq=4, Hkv=1, d=64, lens=[600, 599], page=16, window=1, alibi=True),
    dict(B=2, Hq=4, Hkv=2, d=128, lens=[300, 100], page=16, docs=True),
    dict(B=1, Hq=4, Hkv=1, d=128, lens=[4000], page=256, exp_range=24),    # value blocks of unlike scales
    dict(B=1, Hq=2, Hkv=1, d=64, lens=[900], page=0, scale=-0.3, q_spread=3.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_attention(case, dtype):
    attention_case(200 + case, dtype=dtype, **DECODE[case])


PREFILL = [
    dict(B=1, Hq=2, Hkv=2, d=128, lens=[5], page=0, T=5),
    dict(B=2, Hq=4, Hkv=2, d=128, lens=[40, 300], page=16, T=3),
    dict(B=2, Hq=4, Hkv=1, d=64, lens=[130, 200], page=48, T=67),
    dict(B=1, Hq=5, Hkv=1, d=128, lens=[150], page=0, T=150),
    dict(B=2, Hq=8, Hkv=2, d=128, lens=[333, 140], page=64, T=131, cap=8.0),
    dict(B=2, Hq=6, Hkv=2, d=64, lens=[257, 256], page=16, T=100, alibi=True, docs=True, prefix=9, cap=20.0),
    dict(B=1, Hq=16, Hkv=1, d=128, lens=[500], page=16, T=33, window=50),
    dict(B=1, Hq=3, Hkv=3, d=64, lens=[300], page=0, T=300, prefix=128),
    dict(B=1, Hq=2, Hkv=1, d=128, lens=[700], page=0, T=70, exp_range=24),
    dict(B=1, Hq=2, Hkv=1, d=128, lens=[260], page=0, T=70, scale=-0.2),
    # positions out of order, repeated, past the length and padding rows
    dict(B=2, Hq=4, Hkv=2, d=128, lens=[90, 0], page=0, T=8, pos=[[5, 5, -1, 89, 300, 0, -7, 44], [0, 1, 2, 3, -1, 5, 6, 7]],
         prefix=3),
    dict(B=1, Hq=4, Hkv=1, d=64, lens=[500], page=16, T=40, pos=[[(37 * i) % 500 if i % 5 else -1 for i in range(40)]],
         docs=True, window=90),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill_attention(case, dtype):
    attention_case(300 + case, dtype=dtype, **PREFILL[case])


@pytest.mark.parametrize("T", [1, 24])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_masked_places_changes_nothing(T, d):
    """NaN codes and scales in records that no query sees (behind the length, before the window,
    unused pages), and NaN value codes that only some see: rows that do not see them are bitwise as
    without; pages outside the visible tokens need not exist."""
    r = H.rng(400 + d + T)
    B, Hq, Hkv, page, n, win = 1, 4, 1, 16, 200, 60
    lay = H.Layout(r, B, Hkv, 320, page)
    sides = [H.random_side(r, lay.records, d) for _ in range(2)]
    q, _ = typed(r, (B, Hq, T, d), "bf16")
    pos = np.arange(n - T, n, dtype=np.int32)[None]
    lo = n - T - win + 1                                  # first token that any query sees
    run = lambda a, pg: K.kv8_prefill_attn(q, dev(pos), dev(np.array([n], np.int32)), *a, Hkv, pages=pg,
                                           scoring=K.Scoring(window=win), return_lse=True)
    want = run([side(c, s) for c, s in sides], pages_of(lay))
    rec = lay.rec(0, 0, n)
    seen = np.zeros(lay.records, bool)
    seen[rec[lo:]] = True
    blocks = seen.reshape(-1, 16).any(1)
    dirty = []
    for c, s in sides:
        c, s = c.copy(), s.copy()
        c[~seen] = 0x7f
        s[~blocks] = np.nan
        dirty.append((c, s))
    table = lay.table.copy()
    table[0, :lo // page] = -1
    table[0, -(-n // page):] = 1 << 30
    got = run([side(c, s) for c, s in dirty], K.Pages(dev(table), page, lay.num_pages))
    assert K.get_status() == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    if T > 1:                                             # the last token is seen by the last query only
        for c, s in dirty:
            c[rec[n - 1]] = 0xff
        part = run([side(c, s) for c, s in dirty], K.Pages(dev(table), page, lay.num_pages))
        assert torch.equal(want[0][:, :, :-1], part[0][:, :, :-1]) and torch.equal(want[1][:, :, :-1], part[1][:, :, :-1])


def test_bad_page_ids_and_lengths_are_reported():
    r = H.rng(500)
    lay = H.Layout(r, 2, 1, 64, 16)
    kc, vc = (side(*H.random_side(r, lay.records, 128)) for _ in range(2))
    q, _ = typed(r, (2, 2, 128), "bf16")
    table = lay.table.copy()
    table[1, 0] = lay.num_pages
    K.kv8_decode_attn(q, dev(np.array([64, 20], np.int32)), kc, vc, 1, pages=K.Pages(dev(table), 16, lay.num_pages))
    assert K.get_status() == 1
    ok = pages_of(lay)
    full = K.kv8_decode_attn(q, dev(np.array([64, 20], np.int32)), kc, vc, 1, pages=ok)
    assert K.get_status() == 0
    got = K.kv8_decode_attn(q, dev(np.array([1000, 20], np.int32)), kc, vc, 1, pages=ok)
    assert K.get_status() == 1 and torch.equal(full, got)
    got = K.kv8_decode_attn(q, dev(np.array([-5, 20], np.int32)), kc, vc, 1, pages=ok)
    assert K.get_status() == 1 and not got[0].any() and torch.equal(full[1], got[1])


def test_long_sequences_split_over_the_device():
    """A sequence whose tiles are spread over all CTAs, beside short ones; two calls give the same
    bits, and so does a replayed graph while another call uses another workspace."""
    r = H.rng(600)
    B, Hq, Hkv, d = 3, 8, 2, 128
    lens = [40000, 1, 777]
    lay = H.Layout(r, B, Hkv, 40000, 0)
    sides = [H.random_side(r, lay.records, d) for _ in range(2)]
    kc, vc = (side(c, s) for c, s in sides)
    q, q64 = typed(r, (B, Hq, d), "bf16")
    lt = dev(np.array(lens, np.int32))
    call = lambda **kw: K.kv8_decode_attn(q, lt, kc, vc, Hkv, Nmax=lay.cap, return_lse=True, **kw)
    out, lse = call()
    again, _ = call()
    assert torch.equal(out, again)
    check_rows(out[:, :, None].double().cpu().numpy(), lse[:, :, None].double().cpu().numpy(), q64[:, :, None],
               [H.values(c, s) for c, s in sides], lay, lens, [[n - 1] for n in lens], Hq // Hkv, d ** -0.5, "bf16")
    ws = torch.empty(K.kv8_workspace_bytes(q.dtype, B, Hq, Hkv, 1, d, lay.cap), dtype=torch.uint8, device="cuda")
    g_out, g_lse = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    side_stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side_stream):
        K.kv8_decode_attn(q, lt, kc, vc, Hkv, Nmax=lay.cap, out=g_out, lse=g_lse, return_lse=True, workspace=ws)
    for _ in range(2):
        g_out.zero_()
        graph.replay()
        other, _ = call()
        torch.cuda.synchronize()
        assert torch.equal(g_out, out) and torch.equal(g_lse, lse) and torch.equal(other, out)
    assert K.get_status() == 0


def test_many_sequences_need_several_launches():
    """More sequences than one launch takes, most of them short or empty."""
    r = H.rng(700)
    B, Hq, Hkv, d = 1500, 2, 1, 64
    lens = [int(x) for x in r.integers(0, 50, B)]
    lay = H.Layout(r, B, Hkv, 50, 16)
    sides = [H.random_side(r, lay.records, d) for _ in range(2)]
    kc, vc = (side(c, s) for c, s in sides)
    q, q64 = typed(r, (B, Hq, d), "f16")
    out, lse = K.kv8_decode_attn(q, dev(np.array(lens, np.int32)), kc, vc, Hkv, pages=pages_of(lay), return_lse=True)
    assert K.get_status() == 0
    check_rows(out[:, :, None].double().cpu().numpy(), lse[:, :, None].double().cpu().numpy(), q64[:, :, None],
               [H.values(c, s) for c, s in sides], lay, lens, [[n - 1] for n in lens], 2, d ** -0.5, "f16")


def test_wait_that_runs_out_is_reported_and_recovers():
    r = H.rng(800)
    lay = H.Layout(r, 2, 2, 900, 0)
    kc, vc = (side(*H.random_side(r, lay.records, 128)) for _ in range(2))
    lt = dev(np.array([900, 500], np.int32))
    for T in (1, 100):
        q, _ = typed(r, (2, 8, T, 128), "bf16")
        pos = dev(np.stack([np.arange(n - T, n) for n in (900, 500)]).astype(np.int32))
        run = lambda: K.kv8_prefill_attn(q, pos, lt, kc, vc, 2, Nmax=lay.cap)
        want = run()
        assert K.get_status() == 0
        K.set_wait_limit(-1)
        try:
            run()
            assert K.get_status() == 6
        finally:
            K.set_wait_limit(0)
        assert torch.equal(run(), want) and K.get_status() == 0


def test_serving_steps_together():
    """A prompt is appended and read, the sequence forked, both branches decode their own tokens
    with the step's append, the pool closes up, and each branch still equals the oracle's."""
    r = H.rng(900)
    Hq, Hkv, d, page, pages, rows = 4, 2, 128, 16, 40, 4
    table = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    kc, vc = (K.kv8_alloc(pages * Hkv * page, d) for _ in range(2))
    pool = K.PagePool(table, refs, page, [kc.codes, kc.scales, vc.codes, vc.scales])
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    assert K.pages_reserve(pool, i32(3, 0), i32(0, 0), i32(70, 37)).item() == 0
    n = 37
    pt = [typed(r, (1, Hkv, n, d), "bf16") for _ in range(2)]
    view = K.Pages(table, page, pages)
    K.kv8_append(kc, vc, pt[0][0], pt[1][0], i32(n), pages=view)
    hist = [[pt[0][1][0], pt[1][1][0]]]                        # keys, values [Hkv, tokens, d] of each branch
    cuts = [[n]]
    q, q64 = typed(r, (1, Hq, n, d), "bf16")
    out, lse = K.kv8_prefill_attn(q, torch.arange(n, dtype=torch.int32, device="cuda")[None], i32(n), kc, vc, Hkv, pages=view,
                                  return_lse=True)
    assert K.pages_fork(pool, i32(0), i32(1), i32(n)).item() == 0
    hist.append([x.copy() for x in hist[0]])
    cuts.append([n])

    def values(branch):
        kv = []
        for x in hist[branch]:
            got = np.zeros((Hkv, x.shape[1], d))
            for h in range(Hkv):
                codes, scales = np.zeros((128, d), np.uint8), np.zeros(8, np.float32)
                at = 0
                for k in cuts[branch]:
                    O.append(codes, scales, np.arange(128), x[h, at:at + k], at)
                    at += k
                got[h] = H.values(codes, scales)[:at]
            kv.append(got)
        return kv

    class Flat:
        def rec(self, b, h, m):
            return h * 1000 + np.arange(m)

    def check(o, l, q64, branch, pos):
        kv = values(branch)
        flat = [np.zeros((2000, d)) for _ in kv]
        for f, x in zip(flat, kv):
            for h in range(Hkv):
                f[h * 1000:h * 1000 + x.shape[1]] = x[h]
        check_rows(o.double().cpu().numpy(), l.double().cpu().numpy(), q64, flat, Flat(), [kv[0].shape[1]], [pos], 2, d ** -0.5,
                   "bf16")

    check(out, lse, q64, 0, list(range(n)))
    lens = [n, n]
    for step in range(14):
        if lens[0] % page == 0:
            assert K.pages_reserve(pool, i32(0, 1), i32(*lens), i32(lens[0] + 1, lens[1] + 1)).item() == 0
        new = [typed(r, (2, Hkv, d), "bf16", 1.0 + step) for _ in range(2)]
        lens = [x + 1 for x in lens]
        q, q64 = typed(r, (2, Hq, d), "bf16")
        out, lse = K.kv8_decode_attn(q, i32(*lens), kc, vc, Hkv, pages=view, k_new=new[0][0], v_new=new[1][0], return_lse=True)
        for b in range(2):
            for side_i in range(2):
                hist[b][side_i] = np.concatenate([hist[b][side_i], new[side_i][1][b][:, None]], 1)
            cuts[b].append(1)
            check(out[b:b + 1, :, None], lse[b:b + 1, :, None], q64[b:b + 1, :, None], b, [lens[b] - 1])
        if step == 6:
            K.pages_free(pool, i32(3), i32(70))                 # another sequence ends, the pool closes up
            K.pages_compact(pool)
            assert int((refs > 0).sum()) == int(refs.nonzero().max()) + 1
    assert K.get_status() == 0
