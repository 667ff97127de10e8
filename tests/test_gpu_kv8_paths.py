"""GPU tests of the 8-bit attention's paths through its work: several runs a block of threads, groups of
unlike size, references that grow, pools past 32-bit byte offsets, captured graphs, streams and strides.

The reference is the float64 oracle in matrix form, with the same bounds (see oracle/kv8.py)."""
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


def check(out, lse, q64, kv, lay, lens, pos, G, scale, dtype, cap=0.0, slopes=None, window=0, first=None, prefix=None):
    """All rows of out [B, Hq, T, d] and lse [B, Hq, T], a key head at a time."""
    B, Hq, T, d = q64.shape
    for b in range(B):
        n = lens[b]
        t = np.arange(n)
        p = np.asarray(pos[b], dtype=np.int64)
        hi = np.minimum(n, np.maximum(p + 1, 0 if prefix is None else prefix[b]))
        lo = np.maximum(0, np.maximum(p - window + 1 if window else 0, 0 if first is None else np.asarray(first[b]))) + 0 * p
        see = (t[None] >= lo[:, None]) & (t[None] < np.where(p < 0, 0, hi)[:, None])
        for h in range(Hq // G):
            rec = lay.rec(b, h, n)
            k, v = kv[0][rec], kv[1][rec]
            for hq in range(h * G, h * G + G):
                q = q64[b, hq]
                s = scale * (q @ k.T)
                mag = abs(scale) * (np.abs(q) @ np.abs(k).T)
                if cap:
                    s = cap * np.tanh(s / cap)
                bias = (0.0 if slopes is None else float(slopes[hq])) * np.abs(p[:, None] - t)
                s = np.where(see, s - bias, -np.inf)
                any_ = see.any(1)
                m = np.where(any_, s.max(1, initial=-np.inf), 0.0)
                e = np.where(see, np.exp(s - m[:, None]), 0.0)
                total = e.sum(1)
                w = e / np.where(any_, total, 1.0)[:, None]
                err = np.where(see, 2.0 ** -19 * mag + 2.0 ** -20 * np.abs(np.where(see, s, 0)) + 2.0 ** -20 * (
                    1 + np.abs(np.where(see, m[:, None] - s, 0)).clip(0, 200)) + 2.0 ** -20 * cap + 2.0 ** -21 * np.abs(bias), 0.0)
                mean = (w * err).sum(1)
                seen = see.sum(1)
                ob = (w * (P_EPS[dtype] + err + mean[:, None] + seen[:, None] * 2.0 ** -27)) @ np.abs(v)
                want = w @ v
                tol = ob + HALF_STEP[dtype] * (np.abs(want) + ob) + TINY[dtype]
                bad = np.abs(out[b, hq] - want) > tol
                assert not bad.any(), (b, hq, np.argwhere(bad)[:4])
                assert np.array_equal(lse[b, hq] == -np.inf, ~any_)
                l = m[any_] + np.log(total[any_])
                assert np.all(np.abs(lse[b, hq][any_] - l) <= mean[any_] + 2.0 ** -20 + 2.0 ** -23 * np.abs(l))


def case(seed, B, Hq, Hkv, d, lens, page, dtype, T, cap=0.0, alibi=False, window=0, docs=False, prefix=0, grow=0.0, scale=None,
         pos=None):
    """T = 0: a decode step.  grow: keys and values grow by 2^grow over the sequence."""
    r = H.rng(seed)
    lay = H.Layout(r, B, Hkv, max(lens) + 5, page)
    init = []
    for _ in range(2):
        x = r.standard_normal((lay.records // 16, 16, d)) * 2.0 ** r.integers(-2, 1, (lay.records // 16, 1, 1))
        if grow:
            for b in range(B):
                for h in range(Hkv):
                    rec = lay.rec(b, h, lay.cap)
                    x.reshape(-1, d)[rec] *= 2.0 ** (grow * np.arange(lay.cap) / lay.cap)[:, None]
        s = np.array([O.scale_of(float(np.max(np.abs(b)))) for b in x])
        init.append((O.e4m3_code(x / s[:, None, None]).reshape(lay.records, d), s.astype(np.float32)))
    kc, vc = (side(c, s) for c, s in init)
    steps = max(T, 1)
    qt = torch.from_numpy(r.standard_normal((B, steps, Hq, d)).astype(np.float32)).to(DT[dtype])
    q, q64 = qt.cuda().transpose(1, 2), qt.double().numpy().transpose(0, 2, 1, 3)
    if pos is None:
        pos = [[n - steps + i for i in range(steps)] for n in lens]
    first = [[max(0, p - int(r.integers(0, max(lens) // 2 + 1))) for p in row] for row in pos] if docs else None
    pre = [prefix + b for b in range(B)] if prefix else None
    slopes = (2.0 ** -(1 + np.arange(Hq) % 8)).astype(np.float32) if alibi else None
    i32 = lambda a: None if a is None else dev(np.array(a, np.int32))
    kw = dict(Nmax=0 if page else lay.cap, pages=None if lay.table is None else K.Pages(dev(lay.table), page, lay.num_pages),
              scoring=K.Scoring(scale=scale, softcap=cap, slopes=None if slopes is None else dev(slopes), window=window,
                                first=i32(first), prefix=i32(pre)), return_lse=True)
    if T:
        out, lse = K.kv8_prefill_attn(q, i32(pos), i32(lens), kc, vc, Hkv, **kw)
    else:
        out, lse = (x[:, :, None] for x in K.kv8_decode_attn(q[:, :, 0], i32(lens), kc, vc, Hkv, **kw))
    assert K.get_status() == 0
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), q64, [H.values(c, s) for c, s in init], lay, lens, pos,
          Hq // Hkv, 1 / math.sqrt(d) if scale is None else scale, dtype, cap, slopes, window, first, pre)


def ragged(seed, B, lo, hi):
    return [int(x) for x in H.rng(seed).integers(lo, hi, B)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(B=40, Hq=16, Hkv=8, lens=ragged(1, 40, 150, 300), page=16, T=150),                 # groups of 256 and 44 rows in turn
    dict(B=60, Hq=16, Hkv=8, lens=ragged(2, 60, 20, 700), page=48, T=20, dtype="f16"),      # one row tile a run
    dict(B=30, Hq=10, Hkv=2, lens=ragged(3, 30, 60, 900), page=0, T=60, cap=3.0, window=100, docs=True),
    dict(B=7, Hq=12, Hkv=4, lens=ragged(4, 7, 500, 1200), page=64, T=333, alibi=True, prefix=40, dtype="f16"),
    dict(B=1, Hq=24, Hkv=8, lens=[1100], page=256, T=1100),
], ids=["two_sizes", "one_row_tile", "capped", "biased", "causal"])
def test_query_blocks_of_many_runs(kw, d):
    kw = {"dtype": "bf16", **kw}
    case(1000 + d, d=d, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,lens,page", [(150, 4, ragged(5, 150, 0, 900), 16), (9, 32, ragged(6, 9, 3000, 9000), 48),
                                            (300, 24, ragged(7, 300, 0, 200), 0)])
def test_decode_steps_of_many_runs(B, Hq, lens, page, d):
    case(2000 + B + d, B, Hq, 2, d, [max(1, n) if i == 0 else n for i, n in enumerate(lens)], page, "bf16", 0)


@pytest.mark.parametrize("T", [0, 40, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_and_values_that_grow_along_the_sequence(T, d, dtype):
    """Each tile raises the rows' references, and the values' largest scale, far above the last."""
    case(3000 + T + d, 2, 4, 2, d, [1500, 1431], 16, dtype, T, grow=7.0, scale=0.4)


def test_positions_far_behind_and_before_the_cache():
    """Queries whose window or document ends before the cache's end, or which see one token each."""
    T = 64
    pos = [[(97 * i) % 1000 for i in range(T)], [i for i in range(T)]]
    case(3100, 2, 4, 1, 128, [1000, 700], 16, "bf16", T, window=1, pos=pos)
    case(3101, 2, 4, 1, 64, [1000, 700], 0, "f16", T, window=130, docs=True, pos=pos)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pool_past_32_bit_byte_offsets(dtype):
    """The same sequences in a small pool and in the last pages of one of 3.3 GB a side: append, decode
    and prefill give the same bits."""
    r = H.rng(4000)
    B, Hq, Hkv, d, page, mp, T = 2, 4, 1, 128, 64, 8, 37
    lens = np.array([500, 333], np.int32)
    big = 26_000_000 // page
    tables = [r.permutation(20)[:B * mp].reshape(B, mp).astype(np.int32)]
    tables.append(tables[0] + (big - 20))
    x = [torch.from_numpy(r.standard_normal((B, 500, Hkv, d)).astype(np.float32)).to(DT[dtype]).cuda().transpose(1, 2) for _ in range(2)]
    q = torch.from_numpy(r.standard_normal((B, Hq, T, d)).astype(np.float32)).to(DT[dtype]).cuda()
    pos = dev(np.stack([np.arange(n - T, n) for n in lens]).astype(np.int32))
    got = []
    for table, num in zip(tables, (20, big)):
        sides = [K.Kv8(torch.empty((num * page, d), dtype=torch.uint8, device="cuda"),
                       torch.empty(num * page // 16, dtype=torch.float32, device="cuda")) for _ in range(2)]
        pg = K.Pages(dev(table), page, num)
        K.kv8_append(*sides, *x, dev(lens), new_lens=dev(lens), pages=pg)
        first = int(table.min())
        part = slice(first * page, (first + 1) * page)
        got.append([*K.kv8_decode_attn(q[:, :, 0], dev(lens), *sides, Hkv, pages=pg, return_lse=True),
                    *K.kv8_prefill_attn(q, pos, dev(lens), *sides, Hkv, pages=pg, return_lse=True),
                    *(s.codes[part].clone() for s in sides)])
        del sides
    assert K.get_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


def inputs(seed, B=2, Hq=8, Hkv=2, d=128, n=700, T=90, dtype="bf16"):
    r = H.rng(seed)
    lay = H.Layout(r, B, Hkv, n, 16)
    kc, vc = (side(*H.random_side(r, lay.records, d)) for _ in range(2))
    q = torch.from_numpy(r.standard_normal((B, Hq, T, d)).astype(np.float32)).to(DT[dtype]).cuda()
    lens = dev(np.array([n, n - 77][:B], np.int32))
    pos = dev(np.stack([np.arange(m - T, m) for m in (n, n - 77)[:B]]).astype(np.int32))
    return q, pos, lens, kc, vc, K.Pages(dev(lay.table), 16, lay.num_pages)


def test_graphs_that_share_a_workspace_and_other_streams():
    """Two captured calls that use one workspace, replayed in turn, and calls on other streams at the
    same time, each with its own workspace, give the bits of plain calls."""
    a, b = inputs(5000), inputs(5001, T=3, n=900)
    run = lambda x, **kw: K.kv8_prefill_attn(x[0], x[1], x[2], x[3], x[4], 2, pages=x[5], return_lse=True, **kw)
    want = [run(a), run(b)]
    ws = torch.empty(max(K.kv8_workspace_bytes(x[0].dtype, 2, 8, 2, x[0].shape[2], 128, x[5].max_pages * 16) for x in (a, b)),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x, w in zip((a, b), want):
        outs.append([torch.zeros_like(t) for t in w])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(x, out=outs[-1][0], lse=outs[-1][1], workspace=ws)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(7)
        graphs[0].replay()
        graphs[1].replay()
        beside = []
        for s, x in zip(streams, (b, a)):
            with torch.cuda.stream(s):
                beside.append(run(x))
        torch.cuda.synchronize()
        for o, w in zip([*outs, *beside], [*want, want[1], want[0]]):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    assert K.get_status() == 0


@pytest.mark.parametrize("T", [2, 90])
def test_strided_and_shared_queries(T):
    """q inside a wider buffer, in other orders, and one row for all heads (stride 0)."""
    q, pos, lens, kc, vc, pg = inputs(5100 + T, T=T)
    run = lambda x: K.kv8_prefill_attn(x, pos, lens, kc, vc, 2, pages=pg, return_lse=True)
    B, Hq, _, d = q.shape
    want = run(q)
    wide = torch.full((B, T, Hq, d + 24), float("nan"), dtype=q.dtype, device="cuda")
    wide[..., 8:d + 8] = q.transpose(1, 2)
    swap = torch.empty((T, Hq, B, d), dtype=q.dtype, device="cuda")
    swap.copy_(q.permute(2, 1, 0, 3))
    for view in (wide[..., 8:d + 8].transpose(1, 2), swap.permute(2, 1, 0, 3)):
        got = run(view)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = q[:, :1].expand(B, Hq, T, d)
    got, full = run(one), run(one.contiguous())
    assert torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])
    assert K.get_status() == 0


def test_step_with_append_equals_append_then_step():
    """The fused call's own append, at block starts and ends, on rows with strides."""
    for n in (1, 16, 17, 32, 700):
        q, _, _, kc, vc, pg = inputs(5200 + n, n=705, T=1)
        lens = dev(np.array([n, max(1, n - 5)], np.int32))
        r = H.rng(n)
        new = [torch.from_numpy(r.standard_normal((2, 5, 2, 128)).astype(np.float32)).to(q.dtype).cuda()[:, 3] for _ in range(2)]
        other = [K.Kv8(s.codes.clone(), s.scales.clone()) for s in (kc, vc)]
        got = K.kv8_decode_attn(q[:, :, 0], lens, kc, vc, 2, pages=pg, k_new=new[0], v_new=new[1], return_lse=True)
        K.kv8_append(*other, new[0][:, :, None], new[1][:, :, None], lens, pages=pg)
        want = K.kv8_decode_attn(q[:, :, 0], lens, *other, 2, pages=pg, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for a, b in zip((kc, vc), other):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert K.get_status() == 0


def test_tensors_on_another_device_are_refused():
    """Nothing is launched for a table, scales, counts or lists on the host."""
    q, pos, lens, kc, vc, pg = inputs(5300)
    host = K.Pages(pg.block_table.cpu(), 16, pg.num_pages)
    new = torch.zeros((2, 2, 1, 128), dtype=q.dtype, device="cuda")
    for call in (lambda: K.kv8_prefill_attn(q, pos, lens, kc, vc, 2, pages=host),
                 lambda: K.kv8_decode_attn(q[:, :, 0], lens, kc, vc, 2, pages=host),
                 lambda: K.kv8_append(kc, vc, new, new, lens, pages=host),
                 lambda: K.kv8_prefill_attn(q, pos.cpu(), lens, kc, vc, 2, pages=pg),
                 lambda: K.kv8_prefill_attn(q, pos, lens, kc, vc, 2, pages=pg, scoring=K.Scoring(slopes=torch.zeros(8))),
                 lambda: K.Kv8(kc.codes, kc.scales.cpu()),
                 lambda: K.PagePool(pg.block_table, torch.zeros(50, dtype=torch.int32), 16),
                 lambda: K.PagePool(pg.block_table, torch.zeros(pg.num_pages, dtype=torch.int32, device="cuda"), 16, [kc.codes.cpu()])):
        with pytest.raises(ValueError):
            call()


def test_options_that_change_between_calls_count():
    q, pos, lens, kc, vc, pg = inputs(5400)
    sc = K.Scoring(window=50)
    run = lambda s: K.kv8_prefill_attn(q, pos, lens, kc, vc, 2, pages=pg, scoring=s)
    a = run(sc)
    sc.window, sc.slopes = 0, torch.full((8,), 0.25, device="cuda")
    assert torch.equal(run(sc), run(K.Scoring(slopes=sc.slopes))) and not torch.equal(run(sc), a)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(B=1, Hq=4, Hkv=1, lens=[20000], page=64, T=25),                 # 100 rows a key head over many blocks of threads
    dict(B=3, Hq=2, Hkv=2, lens=[9001, 128, 4700], page=16, T=64, dtype="f16"),
    dict(B=2, Hq=8, Hkv=2, lens=[3000, 2999], page=0, T=32, cap=4.0, window=900, docs=True),
    dict(B=1, Hq=3, Hkv=1, lens=[130], page=16, T=40, alibi=True),
    dict(B=5, Hq=4, Hkv=1, lens=[700, 129, 257, 1025, 40], page=48, T=20),
], ids=["long", "ragged", "capped", "short", "mixed"])
def test_few_rows_over_long_sequences(kw, d):
    """One row tile a run, in many parts."""
    kw = {"dtype": "bf16", **kw}
    case(6000 + d, d=d, **kw)


@pytest.mark.parametrize("T", [1, 30, 100])
@pytest.mark.parametrize("n", [60, 6000])
def test_nan_in_a_query_stays_in_its_row(T, n):
    """A NaN query gives NaN (results joined from several parts too); the other rows keep their bits."""
    q, pos, lens, kc, vc, pg = inputs(6100 + n + T, n=n + 100, T=T)
    run = lambda x: K.kv8_prefill_attn(x, pos, lens, kc, vc, 2, pages=pg, return_lse=True)
    want = run(q)
    bad = q.clone()
    bad[1, 5, T // 2, 17] = float("nan")
    out, lse = run(bad)
    assert out[1, 5, T // 2].isnan().all() and lse[1, 5, T // 2].isnan()
    keep = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    keep[1, 5, T // 2] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert K.get_status() == 0
