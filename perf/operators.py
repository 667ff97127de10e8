"""The serving operators of the 8-bit block-scaled cache and of the page pool, as timed cases.

Operators (include/tq.h): tq_kv8_append, tq_kv8_decode_attn, tq_kv8_prefill_attn and the page
pool's tq_pages_free / _fork / _reserve / _compact.  With ``own`` false ``run`` computes them in
plain torch operations, with ``own`` true through the framework's calls, on the same state.

The cache holds e4m3 codes [records][d] with one fp32 power-of-two scale for each 16 records of
a head; a record is (b * Hkv + h) * Nmax + t, or (page * Hkv + h) * page_size + t % page_size
where a block table names the page of token t.
"""
import math

import torch

own = False

BLOCK = 16
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def _attn(op, name, **kw):
    base = {"op": op, "name": name, "B": 1, "Hq": 32, "Hkv": 8, "d": 128, "T": 1, "N": 1024, "page": 0, "ragged": False,
            "dtype": "bf16", "softcap": 0.0, "alibi": False, "window": 0, "docs": 0, "prefix": 0, "append": False}
    base.update(kw)
    return base


def _pool(op, name, **kw):
    base = {"op": op, "name": name, "rows": 64, "len": 1000, "page": 16, "Hkv": 8, "d": 128, "kind": "kv8"}
    base.update(kw)
    return base


def listed():
    return [
        # one decode step's tokens of eight sequences: the smallest write
        _attn("append", "append_token", B=8, T=1, N=4096, page=64, ragged=True),
        # a padded batch of prompts of unequal length, starting at odd positions
        _attn("append", "append_prompts", B=4, T=8192, N=16384, page=64, ragged=True, dtype="f16"),
        # one short conversation: latency
        _attn("decode", "decode_short", B=1, N=1000),
        # the 128k-token decode workload of this framework's benchmark, with 8-bit records
        _attn("decode", "decode_128k", B=8, N=131072),
        # a serving step: ragged paged sequences, the step's token appended, capped scores, a
        # sliding window and 7 query heads a key head
        _attn("decode", "decode_paged_step", B=48, Hq=28, Hkv=4, d=64, N=8192, page=16, ragged=True, dtype="f16",
              softcap=30.0, window=4096, append=True),
        # a long prompt read in one causal pass
        _attn("prefill", "prefill_8k", T=8192, N=8192),
        # a chunk of a long prompt against the 32k-token cache before it (two sequences, paged)
        _attn("prefill", "prefill_chunk_32k", B=2, T=512, N=32768, page=64),
        # packed documents with distance biases, capped scores and a visible prefix; odd sizes
        _attn("prefill", "prefill_documents", B=3, Hq=20, Hkv=4, d=64, T=1777, N=2500, page=16, ragged=True, dtype="f16",
              softcap=20.0, alibi=True, docs=5, prefix=77),
        # one beam-search step: 64 children freed and forked again from 16 parents
        _pool("fork", "fork_beams", rows=64, len=1000, page=16),
        # many samples of one long prompt, over this framework's 4-bit packed records
        _pool("fork", "fork_samples", rows=192, len=30001, page=256, kind="tq4"),
        # the oldest sequences end, the pool closes up, new ones come in
        _pool("compact", "compact_small", rows=32, len=2000, page=16, d=64, Hkv=4),
        _pool("compact", "compact_large", rows=64, len=16384, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "fork", "compact"])
    if op in ("fork", "compact"):
        kind = rng.choice(["kv8", "tq4"])
        return _strip(_pool(op, "", rows=2 * _log(rng, 2, 64), len=_log(rng, 20, 12000), page=16 * rng.choice([1, 2, 3, 4, 16]),
                            Hkv=rng.choice([1, 2, 4, 8]), d=128 if kind == "tq4" else rng.choice([64, 128]), kind=kind))
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    c = _attn(op, "", Hkv=Hkv, Hq=Hkv * G, d=rng.choice([64, 128]), page=rng.choice([0, 16, 48, 64, 256]),
              dtype=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.6)
    if op == "append":
        c.update(B=rng.randint(1, 8), T=_log(rng, 1, 6000))
        c["N"] = c["T"] + _log(rng, 16, 4000)
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
    else:
        if op == "decode":
            c.update(B=_log(rng, 1, 64), append=rng.random() < 0.4)
            c["N"] = _log(rng, 17, min(131072, 4_000_000 // (c["B"] * Hkv)))
        else:
            c.update(B=rng.randint(1, 4), T=_log(rng, 2, 3000))
            c["N"] = c["T"] + _log(rng, 1, 20000)
            most = 1_200_000_000 // (c["B"] * c["Hq"] * c["T"])
            c["N"] = max(c["T"], min(c["N"], most))
            c.update(docs=rng.choice([0, 0, 3, 9]), prefix=rng.choice([0, 0, 50]))
        c.update(softcap=rng.choice([0.0, 0.0, 15.0, 50.0]), alibi=rng.random() < 0.3, window=rng.choice([0, 0, 0, 100, 1024]))
    return _strip(c)


def _strip(c):
    c.pop("name")
    return c


def _capacity(c):
    """Tokens a row can hold: whole pages, or whole blocks where the cache is not paged."""
    unit = c["page"] or BLOCK
    return -(-c["N"] // unit) * unit


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _fp8_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s (448 = 0.875 * 2^9 is the largest e4m3 value)."""
    m, e = torch.frexp(amax.float())
    e = torch.where(amax > 0, e - torch.where(m > 0.875, 8, 9), -126)
    return torch.ldexp(torch.ones_like(m), e.clamp(min=-126))


def _records(n, d, g):
    """A filled side of the cache: channels of unlike size, a few of them large, as keys have."""
    chan = torch.exp(0.5 * torch.randn(d, device=DEV, generator=g))
    codes = torch.empty((n, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty(n // BLOCK, dtype=torch.float32, device=DEV)
    step = 1 << 21
    for i in range(0, n, step):
        k = min(step, n - i)
        x = torch.randn((k, d), device=DEV, generator=g, dtype=torch.bfloat16).float() * chan
        s = _fp8_scale(x.view(-1, BLOCK * d).abs().amax(1))
        codes[i:i + k] = (x.view(-1, BLOCK * d) / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(k, d)
        scales[i // BLOCK:(i + k) // BLOCK] = s
    return codes, scales


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    return _prepare_pool(c, g) if c["op"] in ("fork", "compact") else _prepare_attn(c, g)


def _prepare_attn(c, g):
    B, Hq, Hkv, d, T, cap = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"], _capacity(c)
    dt = TYPES[c["dtype"]]
    st = {"case": c}
    if c["page"]:
        mp = cap // c["page"]
        pages = B * mp + 3
        st["table"] = torch.randperm(pages, device=DEV, generator=g)[:B * mp].view(B, mp).to(torch.int32)
        st["num_pages"] = pages
        n = pages * Hkv * c["page"]
    else:
        n = B * Hkv * cap
    st["kc"], st["ks"] = _records(n, d, g)
    st["vc"], st["vs"] = _records(n, d, g)
    spread = torch.rand(B, device=DEV, generator=g) if c["ragged"] else torch.ones(B, device=DEV)
    spread[0] = 1.0
    if c["op"] == "append":
        # lengths count the new tokens; padded rows bring fewer than T
        st["new"] = (T - (spread.neg().add(1) * (T - 1)).int()).to(torch.int32)
        free = c["N"] - T
        st["lens"] = (st["new"] + (torch.rand(B, device=DEV, generator=g) * (free + 1)).int()).to(torch.int32)
    else:
        lo = T if c["op"] == "prefill" else 1
        st["lens"] = (lo + (spread * (c["N"] - lo)).int()).to(torch.int32)
    if c["op"] == "append" or c["append"]:
        # as a projection leaves them: [B][T][Hkv][d], read through their strides
        st["k_new"], st["v_new"] = (torch.randn((B, T, Hkv, d), device=DEV, generator=g).mul_(1.5).to(dt).transpose(1, 2)
                                    for _ in range(2))
    if c["op"] != "append":
        q = torch.randn((B, T, Hq, d), device=DEV, generator=g).to(dt).transpose(1, 2)
        st["q"] = q[:, :, 0] if c["op"] == "decode" else q
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if c["alibi"] else None
        if c["op"] == "prefill":
            # the block's tokens are the last T of each sequence
            st["pos"] = (st["lens"][:, None] - T + torch.arange(T, device=DEV)).to(torch.int32)
            st["first"] = None
            if c["docs"]:
                # starts of the documents that a sequence packs: each query sees its own only
                cuts = torch.sort((torch.rand((B, c["docs"]), device=DEV, generator=g) * c["N"]).int(), 1).values
                cuts = torch.cat([torch.zeros((B, 1), device=DEV, dtype=torch.int32), cuts], 1)
                k = (cuts[:, None, :] <= st["pos"][:, :, None]).sum(2) - 1
                st["first"] = cuts.gather(1, k).to(torch.int32)
            st["prefix"] = torch.full((B,), c["prefix"], device=DEV, dtype=torch.int32) if c["prefix"] else None
    return st


def _prepare_pool(c, g):
    rows, page, Hkv, d = c["rows"], c["page"], c["Hkv"], c["d"]
    mp = -(-c["len"] // page) + 1
    lens = (c["len"] - (torch.rand(rows, device=DEV, generator=g) * c["len"] * 0.5).int()).to(torch.int32)
    st = {"case": c, "lens": lens}
    used = (lens + page - 1) // page
    if c["op"] == "fork":
        # the first quarter of the rows are parents (long prompts), the others children forked from them
        par = max(1, rows // 4)
        pages = par * mp + 2 * rows + 8
        st["src"] = torch.randint(0, par, (rows - par,), device=DEV, generator=g).to(torch.int32)
        st["dst"] = torch.arange(par, rows, device=DEV, dtype=torch.int32)
        st["fork_lens"] = lens[st["src"].long()].contiguous()
    else:
        par = rows
        pages = int(rows * mp * 1.25) + 8
        st["groups"] = [torch.arange(0, rows // 2, device=DEV, dtype=torch.int32),
                        torch.arange(rows // 2, rows, device=DEV, dtype=torch.int32)]
        st["turn"] = 0
        # a pool in use: pages of a sequence lie anywhere
    ids = torch.randperm(par * mp, device=DEV, generator=g).view(par, mp).to(torch.int32)
    if c["op"] == "compact":
        # first group in the lower half of the ids, second above it, as after an earlier pass
        half = (rows // 2) * mp
        ids = torch.cat([torch.randperm(half, device=DEV, generator=g), half + torch.randperm(par * mp - half, device=DEV, generator=g)])
        ids = ids.view(par, mp).to(torch.int32)
    table = torch.full((rows, mp), -1, device=DEV, dtype=torch.int32)
    live = torch.arange(mp, device=DEV)[None] < used[:par, None]
    table[:par] = torch.where(live, ids, -1)
    refs = torch.zeros(pages, device=DEV, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    st["table"], st["refs"] = table, refs
    n = pages * Hkv * page
    if c["kind"] == "kv8":
        st["arrays"] = [torch.randint(0, 120, (n, d), device=DEV, generator=g, dtype=torch.uint8),
                        torch.rand(n // BLOCK, device=DEV, generator=g),
                        torch.randint(0, 120, (n, d), device=DEV, generator=g, dtype=torch.uint8),
                        torch.rand(n // BLOCK, device=DEV, generator=g)]
    else:
        st["arrays"] = [torch.randint(0, 1 << 30, (n, d // 8), device=DEV, generator=g, dtype=torch.int32),
                        torch.rand(n, device=DEV, generator=g)]
    if c["op"] == "fork":
        _plain_fork(st, st["src"], st["dst"], st["fork_lens"])
    return st


# ------------------------------------------------------------------------------------- plain forms
def _plain_records(st, t):
    """Record of tokens t [B, n] (or [n]) for every head: int64 [B, Hkv, n]."""
    c, B = st["case"], st["lens"].numel()
    t = t.expand(B, -1).long()
    h = torch.arange(c["Hkv"], device=DEV)[None, :, None]
    if not c["page"]:
        return (torch.arange(B, device=DEV)[:, None, None] * c["Hkv"] + h) * _capacity(c) + t[:, None]
    page = st["table"].long().gather(1, t // c["page"])
    return (page[:, None] * c["Hkv"] + h) * c["page"] + t[:, None] % c["page"]


def _plain_append_side(st, codes, scales, x):
    """Writes x [B, Hkv, T, d] behind the tokens that the cache holds: the blocks of 16 records
    that get new ones take a scale that covers old and new, and the old are rounded again to it."""
    c, d, T = st["case"], st["case"]["d"], x.shape[2]
    lens = st["lens"].long()
    new = st["new"].long() if "new" in st else torch.ones_like(lens)
    p0 = lens - new
    nb = (T + BLOCK - 1) // BLOCK + 1
    t = (p0 // BLOCK * BLOCK)[:, None] + torch.arange(nb * BLOCK, device=DEV)      # tokens of the touched blocks
    i = t - p0[:, None]
    is_new = (i >= 0) & (i < new[:, None])
    is_old = i < 0
    rec = _plain_records(st, torch.minimum(t, torch.tensor(_capacity(c) - 1, device=DEV)))
    shape = (*rec.shape, d)
    blk = rec.view(*rec.shape[:2], nb, BLOCK)[..., 0] // BLOCK
    s_old = scales[blk]
    old = codes[rec].view(torch.float8_e4m3fn).float() * s_old.repeat_interleave(BLOCK, 2)[..., None]
    fresh = x.float().gather(2, i.clamp(0, T - 1)[:, None, :, None].expand(shape))
    val = torch.where(is_new[:, None, :, None], fresh, torch.where(is_old[:, None, :, None], old, 0.0))
    amax = torch.where(is_new[:, None, :, None], fresh, 0.0).abs().view(*blk.shape, BLOCK * d).amax(-1)
    any_old = is_old.view(-1, 1, nb, BLOCK).any(-1)
    any_new = is_new.view(-1, 1, nb, BLOCK).any(-1).expand(blk.shape)
    s = torch.where(any_old, torch.maximum(s_old, _fp8_scale(amax)), _fp8_scale(amax))
    q = (val / s.repeat_interleave(BLOCK, 2)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (any_new[..., None].expand(*blk.shape, BLOCK) & (is_new | is_old).view(-1, 1, nb, BLOCK)).reshape(rec.shape)
    codes[rec[keep]] = q[keep]
    scales[blk[any_new]] = s[any_new]


def _plain_append(st):
    _plain_append_side(st, st["kc"], st["ks"], st["k_new"])
    _plain_append_side(st, st["vc"], st["vs"], st["v_new"])


def _plain_attn(st):
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G, n = Hq // Hkv, c["N"]
    t = torch.arange(n, device=DEV)
    lens = st["lens"].long()
    q = st["q"] if c["op"] == "prefill" else st["q"][:, :, None]
    pos = st["pos"].long() if c["op"] == "prefill" else (lens - 1)[:, None]
    inside = t[None] < lens[:, None]
    rec = _plain_records(st, torch.where(inside, t[None], 0))
    k = st["kc"][rec].view(torch.float8_e4m3fn).float() * st["ks"][rec // BLOCK][..., None]
    s = torch.matmul(q.float().reshape(B, Hkv, G * T, d), k.transpose(2, 3)).view(B, Hkv, G, T, n)
    del k
    s *= 1.0 / math.sqrt(d)
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    far = (pos[:, :, None] - t).abs()
    if c["alibi"]:
        s -= st["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None].float()
    see = t <= pos[:, :, None]
    if c["prefix"]:
        see |= t < st["prefix"][:, None, None]
    if c["docs"]:
        see &= t >= st["first"][:, :, None]
    if c["window"]:
        see &= t > pos[:, :, None] - c["window"]
    see = (see & inside[:, None])[:, None, None]
    s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s -= m
    s.exp_()
    total = s.sum(-1)
    v = st["vc"][rec].view(torch.float8_e4m3fn).float() * st["vs"][rec // BLOCK][..., None]
    o = torch.matmul(s.view(B, Hkv, G * T, n), v).view(B, Hkv, G, T, d)
    o = (o / torch.where(total > 0, total, 1.0)[..., None]).view(B, Hq, T, d).to(st["q"].dtype)
    lse = (m[..., 0] + total.log()).view(B, Hq, T)
    return (o, lse) if c["op"] == "prefill" else (o[:, :, 0], lse[:, :, 0])


def _plain_copy(st, src, dst):
    c = st["case"]
    for a in st["arrays"]:
        pages = a.view(st["refs"].numel(), -1)
        pages[dst] = pages[src]


def _used_cols(st, lens):
    page, mp = st["case"]["page"], st["table"].shape[1]
    return torch.arange(mp, device=DEV)[None] < ((lens.long() + page - 1) // page)[:, None]


def _plain_free(st, rows, lens):
    rows = rows.long()
    gone = _used_cols(st, lens) & (st["table"][rows] >= 0)
    ids = st["table"][rows][gone].long()
    st["refs"].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    st["table"][rows] = torch.where(gone, -1, st["table"][rows])


def _plain_take(st, count):
    """The `count` free pages of the lowest ids."""
    return torch.nonzero(st["refs"] == 0)[:count, 0]


def _plain_fork(st, src, dst, lens):
    page = st["case"]["page"]
    src, dst, lens = src.long(), dst.long(), lens.long()
    whole = torch.arange(st["table"].shape[1], device=DEV)[None] < (lens // page)[:, None]
    st["table"][dst] = torch.where(whole, st["table"][src], st["table"][dst])
    ids = st["table"][src][whole].long()
    st["refs"].index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    part = lens % page > 0
    src, dst, at = src[part], dst[part], (lens // page)[part]
    new = _plain_take(st, at.numel())
    _plain_copy(st, st["table"][src, at].long(), new)
    st["table"][dst, at] = new.to(torch.int32)
    st["refs"][new] = 1


def _plain_reserve(st, rows, old, new):
    rows = rows.long()
    want = _used_cols(st, new) & ~_used_cols(st, old)
    r, col = torch.nonzero(want, as_tuple=True)
    ids = _plain_take(st, r.numel())
    st["table"][rows[r], col] = ids.to(torch.int32)
    st["refs"][ids] = 1


def _plain_compact(st):
    refs = st["refs"]
    live = torch.nonzero(refs > 0)[:, 0]
    n = live.numel()
    src = live[live >= n]
    dst = torch.nonzero(refs[:n] == 0)[:, 0]
    move = torch.full((refs.numel(),), -1, device=DEV, dtype=torch.int32)
    move[live] = live.to(torch.int32)
    move[src] = dst.to(torch.int32)
    _plain_copy(st, src, dst)
    refs[dst] = refs[src]
    refs[src] = 0
    t = st["table"]
    st["table"].copy_(torch.where(t >= 0, move[t.clamp(min=0).long()], t))
    return move


# ------------------------------------------------------------------------------------- one pass
def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st, c)
    if c["op"] == "append":
        _plain_append(st)
        return _cache(st)
    if c["op"] in ("decode", "prefill"):
        if c["append"]:
            _plain_append(st)
        o, lse = _plain_attn(st)
        return {"out": o, "lse": lse, **(_cache(st) if c["append"] else {})}
    if c["op"] == "fork":
        # the children of the step before end, the next ones are forked
        _plain_free(st, st["dst"], st["fork_lens"])
        _plain_fork(st, st["src"], st["dst"], st["fork_lens"])
        return {"table": st["table"], "refs": st["refs"], "arrays": st["arrays"]}
    ended = st["groups"][st["turn"]]
    st["turn"] ^= 1
    lens = st["lens"][ended.long()]
    _plain_free(st, ended, lens)
    move = _plain_compact(st)
    _plain_reserve(st, ended, torch.zeros_like(lens), lens)
    return {"table": st["table"], "refs": st["refs"], "map": move, "arrays": st["arrays"]}


def _cache(st):
    """The cache as the values its bytes stand for, with the blocks' scales."""
    f8 = torch.float8_e4m3fn
    return {"kc": st["kc"].view(f8), "ks": st["ks"], "vc": st["vc"].view(f8), "vs": st["vs"]}


def _run_own(st, c):
    import kv_cache_compression_rotation_b200 as K
    h = st.get("handles")
    if h is None:                      # what a server keeps beside its cache
        if c["op"] in ("fork", "compact"):
            h = {"pool": K.PagePool(st["table"], st["refs"], c["page"], st["arrays"])}
        else:
            h = {"k": K.Kv8(st["kc"], st["ks"]), "v": K.Kv8(st["vc"], st["vs"]), "Nmax": 0 if c["page"] else _capacity(c),
                 "pages": K.Pages(st["table"], c["page"], st["num_pages"]) if c["page"] else None}
            if c["op"] != "append":
                h["scoring"] = K.Scoring(softcap=c["softcap"], slopes=st["slopes"], window=c["window"],
                                         first=st.get("first"), prefix=st.get("prefix"))
        st["handles"] = h
    if c["op"] == "append":
        K.kv8_append(h["k"], h["v"], st["k_new"], st["v_new"], st["lens"], new_lens=st["new"], Nmax=h["Nmax"], pages=h["pages"])
        return _cache(st)
    if c["op"] == "decode":
        o, lse = K.kv8_decode_attn(st["q"], st["lens"], h["k"], h["v"], c["Hkv"], Nmax=h["Nmax"], pages=h["pages"],
                                   k_new=st["k_new"][:, :, 0] if c["append"] else None,
                                   v_new=st["v_new"][:, :, 0] if c["append"] else None, scoring=h["scoring"], return_lse=True)
        return {"out": o, "lse": lse, **(_cache(st) if c["append"] else {})}
    if c["op"] == "prefill":
        o, lse = K.kv8_prefill_attn(st["q"], st["pos"], st["lens"], h["k"], h["v"], c["Hkv"], Nmax=h["Nmax"], pages=h["pages"],
                                    scoring=h["scoring"], return_lse=True)
        return {"out": o, "lse": lse}
    pool = h["pool"]
    if c["op"] == "fork":
        K.pages_free(pool, st["dst"], st["fork_lens"])
        K.pages_fork(pool, st["src"], st["dst"], st["fork_lens"])
        return {"table": st["table"], "refs": st["refs"], "arrays": st["arrays"]}
    ended = st["groups"][st["turn"]]
    st["turn"] ^= 1
    lens = st["lens"][ended.long()]
    K.pages_free(pool, ended, lens)
    move = K.pages_compact(pool)
    K.pages_reserve(pool, ended, torch.zeros_like(lens), lens)
    return {"table": st["table"], "refs": st["refs"], "map": move, "arrays": st["arrays"]}


# ------------------------------------------------------------------------------------- work
def work(case):
    """Bytes in once and out once, and multiply-adds of the products, for lengths at their mean."""
    c = case
    if c["op"] in ("fork", "compact"):
        rec = c["Hkv"] * (2 * c["d"] + 2 * 4 / BLOCK if c["kind"] == "kv8" else c["d"] / 2 + 4)   # bytes a token
        page = c["page"] * rec
        mp = 0.75 * c["len"] / c["page"] + 0.5
        if c["op"] == "fork":
            kids = c["rows"] - max(1, c["rows"] // 4)
            return {"bytes": 2 * kids * page + 6 * 4 * kids * mp, "flops": 0}
        return {"bytes": 2 * (c["rows"] // 2) * mp * page + 8 * 4 * c["rows"] * mp, "flops": 0}
    e = 4 if c["dtype"] == "f32" else 2
    mean = 0.55 if c["ragged"] and c["B"] > 2 else 1.0
    if c["op"] == "append":
        n = c["B"] * c["Hkv"] * max(1.0, mean * c["T"])
        return {"bytes": 2 * n * (c["d"] * (e + 1) + 4 / BLOCK), "flops": 0}
    T, N = c["T"], c["N"]
    if c["op"] == "decode":
        seen = mean * N
        if c["window"]:
            seen = min(seen, c["window"])
        bytes_ = 2 * c["B"] * c["Hkv"] * seen * (c["d"] + 4 / BLOCK) + 2 * c["B"] * c["Hq"] * c["d"] * e
        return {"bytes": bytes_, "flops": 4 * c["B"] * c["Hq"] * seen * c["d"]}
    before = max(0.0, mean * (N - T))
    seen = before + T / 2
    if c["docs"]:
        seen = min(seen, N / (c["docs"] + 1) / 1.5 + c["prefix"] / 4)
    if c["window"]:
        seen = min(seen, c["window"])
    bytes_ = 2 * c["B"] * c["Hkv"] * (before + T) * (c["d"] + 4 / BLOCK) + 2 * c["B"] * c["Hq"] * T * c["d"] * e
    return {"bytes": bytes_, "flops": 4 * c["B"] * c["Hq"] * T * seen * c["d"]}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = dict(case)
    if c["op"] in ("fork", "compact"):
        return None                    # whole numbers and moved bytes: nothing is computed
    st = prepare(c, seed)
    out = {}
    if c["op"] == "append" or c["append"]:
        for side, x in (("k", st["k_new"]), ("v", st["v_new"])):
            _exact_append(st, st[side + "c"], st[side + "s"], x)
        out = {"kc": _e4m3_values(st["kc"]), "ks": st["ks"].double(), "vc": _e4m3_values(st["vc"]), "vs": st["vs"].double()}
    if c["op"] == "append":
        return out
    o, lse = _exact_attn(st)
    return {"out": o, "lse": lse, **out}


def _e4m3_table():
    """The 256 values of e4m3 from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = torch.arange(256, dtype=torch.float64, device=DEV)
    sign = torch.where(b >= 128, -1.0, 1.0).double()
    e, m = torch.floor((b % 128) / 8), b % 8
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    v[127] = v[255] = math.nan
    return sign * v


def _e4m3_values(codes):
    return _e4m3_table()[codes.long()] if codes.numel() <= 1 << 28 else None


def _e4m3_code(y):
    """Nearest e4m3 code of y (float64), ties to the even mantissa, by the definition's steps."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    step = torch.where(a / step >= 16, step * 2, torch.where(a / step < 8, torch.where(step > 2.0 ** -9, step / 2, step), step))
    a = torch.round(a / step) * step
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)) + 1e-12)
    code = torch.where(a < 2.0 ** -6, a * 512, (e + 7) * 8 + a / torch.exp2(e) * 8 - 8)
    return (code.to(torch.int64) + torch.where(torch.signbit(y), 128, 0)).to(torch.uint8)


def _exact_append(st, codes, scales, x):
    c = st["case"]
    T, table, lens = x.shape[2], _e4m3_table(), st["lens"].tolist()
    new = st["new"].tolist() if "new" in st else [1] * len(lens)
    heads = torch.arange(c["Hkv"], device=DEV)
    for b, (n, k) in enumerate(zip(lens, new)):
        t0 = (n - k) // BLOCK * BLOCK
        t = torch.arange(t0, n, device=DEV)
        if c["page"]:
            rec = (st["table"][b].long()[t // c["page"]] * c["Hkv"] + heads[:, None]) * c["page"] + t % c["page"]
        else:
            rec = (b * c["Hkv"] + heads[:, None]) * _capacity(c) + t
        pad = -len(t) % BLOCK
        held = n - k - t0                                    # tokens of the first block that were there
        first = rec[:, ::BLOCK] // BLOCK
        fresh = torch.nn.functional.pad(x[b, :, :k].double(), (0, 0, held, pad)).view(c["Hkv"], -1, BLOCK, c["d"])
        big = fresh.abs().amax((2, 3))
        s = torch.exp2(torch.ceil(torch.log2(big / 448)).clamp(min=-126))
        s = torch.where(448 * s < big, s * 2, torch.where((448 * s / 2 >= big) & (s > 2.0 ** -126), s / 2, s))
        if held:
            s[:, 0] = torch.maximum(s[:, 0], scales[first[:, 0]].double())
            fresh[:, 0, :held] = table[codes[rec[:, :held]].long()] * scales[first[:, 0]].double()[:, None, None]
        got = _e4m3_code(fresh / s[..., None, None]).view(c["Hkv"], -1, c["d"])[:, :len(t)]
        codes[rec] = got
        scales[first] = s.float()


def _exact_attn(st):
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G, table = Hq // Hkv, _e4m3_table()
    q = st["q"] if c["op"] == "prefill" else st["q"][:, :, None]
    out = torch.zeros((B, Hq, T, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"].tolist()):
        pos = st["pos"][b].double() if c["op"] == "prefill" else torch.tensor([n - 1.0], dtype=torch.float64, device=DEV)
        t = torch.arange(n, device=DEV, dtype=torch.float64)
        hi = pos + 1
        if c["prefix"]:
            hi = torch.clamp(hi, min=float(c["prefix"]))
        lo = torch.zeros_like(pos)
        if c["docs"]:
            lo = torch.maximum(lo, st["first"][b].double())
        if c["window"]:
            lo = torch.maximum(lo, pos - c["window"] + 1)
        hidden = (t < lo[:, None]) | (t >= hi[:, None])
        ti = t.long()
        for h in range(Hkv):
            if c["page"]:
                rec = (st["table"][b].long()[ti // c["page"]] * Hkv + h) * c["page"] + ti % c["page"]
            else:
                rec = (b * Hkv + h) * _capacity(c) + ti
            k = table[st["kc"][rec].long()] * st["ks"].double()[rec // BLOCK, None]
            v = table[st["vc"][rec].long()] * st["vs"].double()[rec // BLOCK, None]
            for g in range(h * G, h * G + G):
                s = q[b, g].double() @ k.T / math.sqrt(d)
                if c["softcap"]:
                    s = c["softcap"] * torch.tanh(s / c["softcap"])
                if c["alibi"]:
                    s = s - st["slopes"][g].double() * (pos[:, None] - t).abs()
                s = s.masked_fill(hidden, -math.inf)
                lse[b, g] = torch.logsumexp(s, 1)
                out[b, g] = torch.nan_to_num(torch.exp(s - lse[b, g][:, None])) @ v
    return (out, lse) if c["op"] == "prefill" else (out[:, :, 0], lse[:, :, 0])
