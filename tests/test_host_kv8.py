"""Refusals of the 8-bit cache's and the page pool's entry points: argument errors are found on the
host before any launch, so they need no GPU."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

K = pytest.importorskip("kv_cache_compression_rotation_b200")
T = K.tq

F = 0x10000000            # addresses that are checked, never read
A = [F + i * 0x10000000 for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_rotation_b200 import build as B
    B.build()
    return T.lib()


def pages(table=F, page=16, mp=4, num=20):
    return C.byref(T.Pages_t(table, page, mp, num))


def kv8(i):
    return T.Kv8_t(A[i], A[i] + 0x8000000)


def append(lib, **kw):
    a = dict(k=A[0], v=A[1], dtype=1, ks=None, vs=None, B=2, Hkv=2, T=3, d=128, lens=A[2], new=None, pages=None, N=64, kc=kv8(3),
             vc=kv8(4))
    a.update(kw)
    return lib.tq_kv8_append(a["k"], a["v"], a["dtype"], a["ks"], a["vs"], a["B"], a["Hkv"], a["T"], a["d"], a["lens"], a["new"],
                             a["pages"], a["N"], a["kc"], a["vc"], None)


INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, WORKSPACE = 1, 2, 3, 4, 8


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(lens=None), INVALID), (dict(lens=A[2] + 4), ALIGNMENT), (dict(k=A[0] + 8), ALIGNMENT), (dict(new=A[5] + 2), ALIGNMENT),
    (dict(N=40), INVALID), (dict(N=0), INVALID), (dict(N=1 << 31), INVALID),
    (dict(kc=T.Kv8_t(None, A[3])), INVALID), (dict(vc=T.Kv8_t(A[4], None)), INVALID), (dict(kc=T.Kv8_t(A[3] + 4, A[5])), ALIGNMENT),
    (dict(vc=kv8(3)), ALIAS), (dict(k=A[3]), ALIAS), (dict(lens=A[4]), ALIAS), (dict(new=A[3]), ALIAS),
    (dict(pages=pages(page=24)), INVALID), (dict(pages=pages(table=None)), INVALID), (dict(pages=pages(table=F + 4)), ALIGNMENT),
    (dict(pages=pages(table=A[3])), ALIAS), (dict(pages=pages(num=1 << 30)), UNSUPPORTED),
    (dict(ks=C.byref(T.Strides_t(768, 384, 129))), ALIGNMENT), (dict(vs=C.byref(T.Strides_t(768, -384, 128))), INVALID),
    (dict(ks=C.byref(T.Strides_t(1 << 62, 384, 128))), INVALID),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code
    assert lib.tq_last_error()


def attn(lib, prefill, **kw):
    a = dict(q=A[0], qs=None, dtype=1, B=2, Hq=8, Hkv=2, T=40, d=128, pos=A[1], lens=A[2], sc=None, pages=None, N=64, kn=None,
             vn=None, kc=kv8(3), vc=kv8(4), out=A[5], lse=A[6], ws=A[7], wsb=1 << 27)
    a.update(kw)
    if prefill:
        return lib.tq_kv8_prefill_attn(a["q"], a["qs"], a["dtype"], a["B"], a["Hq"], a["Hkv"], a["T"], a["d"], a["pos"], a["lens"],
                                       a["sc"], a["pages"], a["N"], a["kc"], a["vc"], a["out"], a["lse"], a["ws"], a["wsb"], None)
    return lib.tq_kv8_decode_attn(a["q"], a["qs"], a["dtype"], a["B"], a["Hq"], a["Hkv"], a["d"], a["lens"], a["sc"], a["pages"],
                                  a["N"], a["kn"], a["vn"], None, None, a["kc"], a["vc"], a["out"], a["lse"], a["ws"], a["wsb"],
                                  None)


def scoring(**kw):
    a = dict(scale=0.1, softcap=0.0, slopes=None, window=0, first=None, prefix=None)
    a.update(kw)
    return C.byref(T.Scoring_t(*[a[k] for k in ("scale", "softcap", "slopes", "window", "first", "prefix")]))


COMMON = [
    (dict(Hq=7), INVALID), (dict(Hq=0), INVALID), (dict(d=80), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(lens=None), INVALID), (dict(q=A[0] + 2), ALIGNMENT), (dict(out=A[5] + 8), ALIGNMENT),
    (dict(lse=A[6] + 4), ALIGNMENT), (dict(N=65), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
    (dict(ws=A[7] + 8), ALIGNMENT), (dict(out=A[0]), ALIAS), (dict(out=A[3]), ALIAS), (dict(lse=A[5]), ALIAS),
    (dict(ws=A[4]), ALIAS), (dict(sc=scoring(scale=float("nan"))), INVALID), (dict(sc=scoring(softcap=-1.0)), INVALID),
    (dict(sc=scoring(softcap=float("inf"))), INVALID), (dict(sc=scoring(window=-1)), INVALID),
    (dict(sc=scoring(slopes=A[8] + 4)), ALIGNMENT), (dict(sc=scoring(prefix=A[5])), ALIAS), (dict(sc=scoring(first=A[6])), ALIAS),
    (dict(pages=pages(page=8)), INVALID), (dict(pages=pages(num=1 << 30)), UNSUPPORTED),
    (dict(qs=C.byref(T.Strides_t(8 * 40 * 128, 5128 + 4, 128))), ALIGNMENT),
]


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,code", COMMON)
def test_attention_refuses(lib, prefill, kw, code):
    assert attn(lib, prefill, **kw) == code


@pytest.mark.parametrize("prefill,kw,code", [
    (True, dict(pos=None), INVALID), (True, dict(T=0), INVALID), (True, dict(pos=A[1] + 4), ALIGNMENT), (True, dict(pos=A[5]), ALIAS),
    (False, dict(kn=A[9]), INVALID), (False, dict(vn=A[9]), INVALID), (False, dict(kn=A[9], vn=A[9] + 8), ALIGNMENT),
    (False, dict(kn=A[3], vn=A[9]), ALIAS), (False, dict(kn=A[5], vn=A[9]), ALIAS), (False, dict(kn=A[9], vn=A[9], q=A[4]), ALIAS),
])
def test_attention_refuses_of_its_own(lib, prefill, kw, code):
    assert attn(lib, prefill, **kw) == code


def test_workspace_queries(lib):
    n = C.c_size_t(0)
    for dtype in range(3):
        for d in (64, 128):
            assert lib.tq_kv8_attn_workspace(dtype, 2, 8, 2, 1, d, 4096, C.byref(n)) == 0 and n.value > 0
    assert lib.tq_kv8_attn_workspace(1, 2, 9, 2, 1, 128, 4096, C.byref(n)) == INVALID
    assert lib.tq_kv8_attn_workspace(1, 2, 8, 2, 1, 128, 0, C.byref(n)) == INVALID
    assert lib.tq_kv8_attn_workspace(1, 2, 8, 2, 1, 128, 64, None) == INVALID


def pool(table=A[0], refs=A[1], rows=4, mp=8, page=16, num=100):
    return C.byref(T.PagePool_t(table, refs, rows, mp, page, num))


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INVALID), (dict(refs=None), INVALID), (dict(table=A[0] + 4), ALIGNMENT), (dict(refs=A[1] + 8), ALIGNMENT),
    (dict(rows=0), INVALID), (dict(mp=0), INVALID), (dict(page=0), INVALID), (dict(num=0), INVALID), (dict(num=1 << 31), INVALID),
    (dict(mp=1 << 20, page=1 << 20), INVALID), (dict(refs=A[0] + 64), ALIAS),
])
def test_pool_descriptor_refused(lib, kw, code):
    n = C.c_size_t(0)
    p = pool(**kw)
    assert lib.tq_pages_workspace(p, 4, C.byref(n)) == code
    assert lib.tq_pages_free(p, A[2], A[3], 2, None) == code
    assert lib.tq_pages_reserve(p, A[2], A[3], A[4], 2, A[5], A[6], 1 << 20, None) == code
    assert lib.tq_pages_fork(p, None, 0, A[2], A[3], A[4], 2, A[5], A[6], 1 << 20, None) == code
    assert lib.tq_pages_compact(p, None, 0, A[2], A[3], A[6], 1 << 20, None) == code


def test_pool_arguments_refused(lib):
    n = C.c_size_t(0)
    assert lib.tq_pages_workspace(pool(), 4, C.byref(n)) == 0 and n.value > 0
    assert lib.tq_pages_workspace(pool(), -1, C.byref(n)) == INVALID
    big = 1 << 20
    assert lib.tq_pages_free(pool(), A[2], A[3], 0, None) == 0
    assert lib.tq_pages_free(pool(), A[2], A[3], -1, None) == INVALID
    assert lib.tq_pages_free(pool(), None, A[3], 2, None) == INVALID
    assert lib.tq_pages_free(pool(), A[2] + 4, A[3], 2, None) == ALIGNMENT
    assert lib.tq_pages_free(pool(), A[0], A[3], 2, None) == ALIAS
    assert lib.tq_pages_reserve(pool(), A[2], A[3], A[4], 0, A[5], A[6], big, None) == INVALID
    assert lib.tq_pages_reserve(pool(), A[2], A[3], A[4], 2, None, A[6], big, None) == INVALID
    assert lib.tq_pages_reserve(pool(), A[2], A[3], A[4], 2, A[5], None, big, None) == WORKSPACE
    assert lib.tq_pages_reserve(pool(), A[2], A[3], A[4], 2, A[5], A[6], 16, None) == WORKSPACE
    assert lib.tq_pages_reserve(pool(), A[2], A[3], A[4], 2, A[2], A[6], big, None) == ALIAS
    arr = lambda *x: (T.PoolArray_t * max(1, len(x)))(*[T.PoolArray_t(a, b) for a, b in x])
    fork = lambda a, k: lib.tq_pages_fork(pool(), a, k, A[2], A[3], A[4], 2, A[5], A[6], big, None)
    assert fork(None, 1) == INVALID and fork(arr((A[7], 16)), T.MAX_POOL_ARRAYS + 1) == INVALID
    assert fork(arr((None, 16)), 1) == INVALID and fork(arr((A[7] + 4, 16)), 1) == ALIGNMENT
    assert fork(arr((A[7], 6)), 1) == INVALID and fork(arr((A[7], 0)), 1) == INVALID
    assert fork(arr((A[7], 64), (A[7] + 640, 64)), 2) == ALIAS and fork(arr((A[1], 64)), 1) == ALIAS
    assert lib.tq_pages_compact(pool(), None, 0, None, A[3], A[6], big, None) == INVALID
    assert lib.tq_pages_compact(pool(), None, 0, A[2], A[2], A[6], big, None) == ALIAS
    copy = lambda a, k, num, s, d, m: lib.tq_pages_copy(a, k, num, s, d, m, None)
    ok = arr((A[7], 64))
    assert copy(ok, 1, 10, A[2], A[3], 0) == 0 and copy(ok, 1, 0, A[2], A[3], 1) == INVALID
    assert copy(ok, 1, 10, None, A[3], 1) == INVALID and copy(ok, 1, 10, A[7], A[3], 1) == ALIAS
    assert copy(ok, 1, 10, A[2], A[3], -1) == INVALID


def test_binding_refuses_what_the_library_cannot_see():
    c = torch.zeros((32, 128), dtype=torch.uint8)
    s = torch.zeros(2)
    with pytest.raises(ValueError):
        K.Kv8(c, torch.zeros(3))
    with pytest.raises(ValueError):
        K.Kv8(c.float(), s)
    with pytest.raises(ValueError):
        K.Kv8(c.t(), s)
    with pytest.raises(ValueError):
        K.Scoring(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        K.Scoring(first=torch.zeros((2, 3)))
    with pytest.raises(ValueError):
        K.PagePool(torch.zeros((2, 2), dtype=torch.int64), torch.zeros(4, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        K.PagePool(torch.zeros((2, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 16, [torch.zeros(7)])
    k = K.Kv8(c, s)
    x = torch.zeros((1, 1, 1, 128), dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):                      # CPU tensors
        K.kv8_append(k, k, x, x, lens, Nmax=32)
    with pytest.raises(ValueError):
        K.kv8_append(k, k, x, x.float(), lens, Nmax=32)
    with pytest.raises(ValueError):                      # more records than the cache holds
        K.kv8_decode_attn(x[:, :, 0], lens, k, k, 1, Nmax=48)
    with pytest.raises(ValueError):
        K.kv8_decode_attn(x[..., :64].contiguous()[:, :, 0], lens, k, k, 1, Nmax=32)
    with pytest.raises(ValueError):
        K.kv8_decode_attn(x[:, :, 0], lens, k, k, 1, Nmax=32, scoring=K.Scoring(slopes=torch.zeros(3)))


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(sc=scoring(softcap=1e-31)), INVALID), (dict(sc=scoring(softcap=2e30)), INVALID), (dict(sc=scoring(softcap=-1.0)), INVALID),
    # 2^30 tokens a sequence by way of pages named often, times 64 key heads
    (dict(Hq=64, Hkv=64, pages=pages(page=1 << 20, mp=1 << 10, num=16)), UNSUPPORTED),
])
def test_attention_refuses_caps_and_counts_out_of_range(lib, prefill, kw, code):
    assert attn(lib, prefill, wsb=1 << 40, **kw) == code
    assert lib.tq_last_error()
