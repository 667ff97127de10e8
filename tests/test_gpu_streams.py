"""GPU tests of calls that are given a stream other than the current one.  Their workspaces and outputs
must not be handed to anyone else while the kernels on that stream still use them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K = pytest.importorskip("kv_cache_compression_rotation_b200")

import tq_inputs as ti

BUSY = 40_000_000                             # cycles, 20 to 30 ms
D = 128
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")


def tensors(x):
    return [t for y in x for t in tensors(y)] if isinstance(x, tuple) else [x]


def late(call, sizes):
    """call(stream) on a stream that is busy; meanwhile the current stream fills buffers of the given
    numbers of bytes.  They must keep what was written to them, and the results are those of a plain call."""
    want = [t.clone() for t in tensors(call(None))]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)
    got = tensors(call(stream))
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    stream.synchronize()
    for t in held:
        assert bool((t == 7).all()), "a buffer of the current stream was written to"
    assert len(got) == len(want) > 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert K.get_status() == 0


def cache8(n, heads=2):
    g = torch.Generator(device="cuda").manual_seed(n)
    sides = []
    for _ in range(2):
        codes = torch.randint(0, 0x78, (heads * n, D), dtype=torch.uint8, device="cuda", generator=g)
        sides.append(K.Kv8(codes, torch.full((heads * n // 16,), 2.0 ** -6, device="cuda")))
    return sides


@pytest.mark.parametrize("T", [1, 100])
def test_attention_over_the_8_bit_cache(T):
    n = 4096
    kc, vc = cache8(n)
    q = ti.normal_torch((1, 8, T, D), 31, "cuda", torch.bfloat16)
    pos = torch.arange(n - T, n, dtype=torch.int32, device="cuda")[None]
    ws, lens = K.kv8_workspace_bytes(q.dtype, 1, 8, 2, T, D, n), i32(n)
    late(lambda s: K.kv8_prefill_attn(q, pos, lens, kc, vc, 2, Nmax=n, return_lse=True, stream=s), [ws])
    if T == 1:
        late(lambda s: K.kv8_decode_attn(q[:, :, 0], lens, kc, vc, 2, Nmax=n, return_lse=True, stream=s), [ws])


def pool(rows=8, mp=64, page=16, pages=600):
    table = torch.full((rows, mp), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    return K.PagePool(table, refs, page, [torch.arange(pages * 64, dtype=torch.int32, device="cuda")])


@pytest.mark.parametrize("what", ["reserve", "fork", "compact"])
@pytest.mark.parametrize("pages", [600, 20000])
def test_page_pool(what, pages):
    p = pool(pages=pages)
    assert K.pages_reserve(p, i32(0, 1), i32(0, 0), i32(500, 1000)).item() == 0
    if what == "compact":
        K.pages_free(p, i32(0), i32(500))
    mine = (p.block_table, p.refs, *p.arrays)
    state = [t.clone() for t in mine]
    rows, src, zero, lens = i32(2, 3), i32(0, 1), i32(0, 0), i32(77, 999)

    def call(s):
        for t, x in zip(mine, state):
            t.copy_(x)
        torch.cuda.current_stream().synchronize()
        if what == "reserve":
            return K.pages_reserve(p, rows, zero, lens, stream=s)
        if what == "fork":
            return K.pages_fork(p, src, rows, lens, stream=s)
        return K.pages_compact(p, stream=s)

    call(None)
    want = [t.clone() for t in mine]
    late(call, [p._work(2).numel(), p._work(0).numel()])
    for t, x in zip(mine, want):
        assert torch.equal(t, x)


def packed(n):
    q = K.Quantizer.mse(ti.haar_rotation(D, 1003), 4)
    return q, K.quantize(q, ti.normal_torch((n, D), 41, "cuda", torch.bfloat16))


@pytest.mark.parametrize("what", ["decode", "prefill", "score"])
def test_calls_over_packed_records(what):
    n, Hkv = 4096, 2
    q, rec = packed(Hkv * n)
    qv, lens = ti.normal_torch((1, 8, D), 42, "cuda", torch.bfloat16), i32(n)
    ws = ctypes.c_size_t(0)
    if what == "decode":
        size = K.decode_workspace_bytes(q, 1, 8, Hkv, n)
        late(lambda s: K.decode_attn(q, q, qv, lens, rec, rec, n, Hkv, stream=s), [size])
    elif what == "prefill":
        qp = qv[:, :, None].expand(1, 8, 3, D).contiguous()
        pos = i32(n - 3, n - 2, n - 1)[None]
        K.tq._check(K.tq.lib().tq_prefill_attn_workspace(q.ref, 1, 8, Hkv, 3, n, ctypes.byref(ws)))
        late(lambda s: K.prefill_attn(q, q, qp, pos, lens, rec, rec, Hkv, Nmax=n, stream=s), [ws.value])
    else:
        x = qv[0].float().contiguous()
        K.tq._check(K.tq.lib().tq_score_workspace(q.ref, 8, Hkv * n, 10, ctypes.byref(ws)))
        late(lambda s: K.score(q, x, rec, Hkv * n, 10, s), [max(ws.value, 16)])


def test_quantized_records_are_not_zeroed_behind_the_call():
    """The records are cleared on the stream that fills them, though the current one is behind."""
    q, want = packed(5000)
    x = ti.normal_torch((5000, D), 41, "cuda", torch.bfloat16)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = K.quantize(q, x, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.norms, want.norms)


def test_captured_with_its_stream_named():
    """A call that is captured on the stream it is given, with memory of its own, replays its bits."""
    n, T = 4096, 100
    kc, vc = cache8(n)
    q, lens = ti.normal_torch((1, 8, T, D), 51, "cuda", torch.bfloat16), i32(n)
    pos = torch.arange(n - T, n, dtype=torch.int32, device="cuda")[None]
    run = lambda s=None: K.kv8_prefill_attn(q, pos, lens, kc, vc, 2, Nmax=n, return_lse=True, stream=s)
    want, graph, stream = run(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        got = run(stream)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert K.get_status() == 0
