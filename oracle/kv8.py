"""8-bit block-scaled cache and page pool, restated in float64 / plain Python.

Block of 16 tokens of a head: s = min{2^e >= 2^-126 : max|x| <= 448 * 2^e}, codes rn_e4m3(x / s).
Tokens that join a block which holds some: s' = max(s_old, s(new)), the held codes become
rn_e4m3(code * s_old / s').  Scores s = scale <q, k>, capped cap * tanh(s / cap), minus
slope * |pos - t|; visible tokens [lo, hi); out = softmax(s) v, lse = ln sum e^s.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = np.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


VALUES = e4m3_values()
_POS = VALUES[:127]                       # 0 .. 448 ascending


def e4m3_code(x) -> np.ndarray:
    """Nearest code, ties to the even one, magnitudes above 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(take_hi, hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_of(amax: float) -> float:
    if amax == 0:
        return 2.0 ** -126
    e = max(-126, math.ceil(math.log2(amax / 448)) - 1)
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scales, records, x, p0):
    """Writes rows x [n, d] as tokens p0 .. p0 + n - 1 of one (sequence, head); records[t] is token
    t's record.  codes uint8 [R, d] and scales [R / 16] are changed in place."""
    n = len(x)
    for t0 in range(p0 // BLOCK * BLOCK, p0 + n, BLOCK):
        a, z = max(p0, t0), min(p0 + n, t0 + BLOCK)
        if a >= z:
            continue
        blk = records[t0] // BLOCK
        s = scale_of(float(np.max(np.abs(x[a - p0:z - p0]))))
        if a > t0:
            held = np.asarray(records[t0:a])
            old = float(scales[blk])
            s = max(s, old)
            codes[held] = e4m3_code(VALUES[codes[held]] * old / s)
        codes[np.asarray(records[a:z])] = e4m3_code(np.asarray(x[a - p0:z - p0], dtype=np.float64) / s)
        scales[blk] = s


def visible(pos, n, window=0, first=None, prefix=None):
    """Tokens [lo, hi) that a query at pos sees in a sequence of n."""
    if pos < 0:
        return 0, 0
    hi = min(n, max(pos + 1, prefix or 0))
    lo = max(0, first if first is not None else 0, pos - window + 1 if window else 0)
    return lo, max(lo, hi)


def attention(q, k, v, pos, lo, hi, scale, cap=0.0, slope=0.0, p_eps=2.0 ** -11):
    """One query over its visible tokens: (out, lse, out_bound, lse_bound).

    The bounds are what a computation may be off (before its output's own rounding) that keeps
    scores, sums and outputs in fp32 and rounds each probability by at most p_eps:
      score t: 2^-19 scale sum|q k| (sequential fp32 sums, truncating, of 8 to 9 steps), 2^-20 |s| and
      2^-20 for exp2 and its argument, 2^-20 cap for tanh's absolute error, 2^-21 of the bias;
      output: p_eps + score errors (own and, through the sum, their mean) + n 2^-27 for the sums,
      each times sum p |v|."""
    if hi <= lo:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1]), 0.0
    k, v = k[lo:hi], v[lo:hi]
    t = np.arange(lo, hi)
    s = scale * (k @ q)
    mag = abs(scale) * (np.abs(k) @ np.abs(q))
    if cap:
        s = cap * np.tanh(s / cap)
    bias = slope * np.abs(pos - t)
    s = s - bias
    m = s.max()
    e = np.exp(s - m)
    p = e / e.sum()
    err = 2.0 ** -19 * mag + 2.0 ** -20 * np.abs(s) + 2.0 ** -20 * (1 + abs(m - s).clip(0, 200)) + \
        2.0 ** -20 * cap + 2.0 ** -21 * np.abs(bias)
    mean = float(p @ err)
    n = hi - lo
    out_bound = (p * (p_eps + err + mean + n * 2.0 ** -27)) @ np.abs(v)
    return p @ v, m + math.log(e.sum()), out_bound, mean + 2.0 ** -20


# ------------------------------------------------------------------ page pool
def pages_of(n, page):
    return -(-n // page)


def pool_free(table, refs, rows, lens, page):
    for r, n in zip(rows, lens):
        for c in range(pages_of(n, page)):
            if table[r, c] >= 0:
                refs[table[r, c]] -= 1
                table[r, c] = -1


def pool_reserve(table, refs, rows, old, new, page):
    """Pages lacking (0 = done); nothing changes unless all are there."""
    want = [(r, c) for r, o, n in zip(rows, old, new) for c in range(pages_of(o, page), pages_of(n, page))]
    free = [i for i in range(len(refs)) if refs[i] == 0]
    if len(free) < len(want):
        return len(want) - len(free)
    for (r, c), i in zip(want, free):
        table[r, c], refs[i] = i, 1
    return 0


def pool_fork(table, refs, arrays, src, dst, lens, page):
    """arrays: [num_pages, ...] arrays whose pages are copied."""
    tails = [i for i, n in enumerate(lens) if n % page]
    free = [i for i in range(len(refs)) if refs[i] == 0]
    if len(free) < len(tails):
        return len(tails) - len(free)
    for i, id_ in zip(tails, free):
        full = lens[i] // page
        for a in arrays:
            a[id_] = a[table[src[i], full]]
        table[dst[i], full], refs[id_] = id_, 1
    for s, d, n in zip(src, dst, lens):
        for c in range(n // page):
            table[d, c] = table[s, c]
            refs[table[s, c]] += 1
    return 0


def pool_compact(table, refs, arrays):
    live = [i for i in range(len(refs)) if refs[i] > 0]
    n = len(live)
    holes = [i for i in range(n) if refs[i] == 0]
    page_map = np.full(len(refs), -1, dtype=np.int64)
    page_map[live] = live
    for a, b in zip([i for i in live if i >= n], holes):
        page_map[a] = b
        for x in arrays:
            x[b] = x[a]
        refs[b], refs[a] = refs[a], 0
    t = table >= 0
    table[t] = page_map[table[t]]
    return page_map, n
