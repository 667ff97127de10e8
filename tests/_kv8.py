"""Inputs of the 8-bit cache's tests: caches filled by the oracle's own rounding, in float64."""
import numpy as np

from oracle import kv8 as O

torch_types = ("bf16", "f16", "f32")


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def values(codes, scales):
    """Float64 values of codes [R, d] with scales [R / 16]."""
    return O.VALUES[codes] * np.repeat(np.asarray(scales, dtype=np.float64), O.BLOCK)[:, None]


def random_side(r, records, d, spread=3.0, exp_range=0):
    """Codes and scales of `records` records; exp_range > 0 spreads the blocks' scales over that
    many powers of two."""
    x = r.standard_normal((records // O.BLOCK, O.BLOCK, d)) * spread
    if exp_range:
        x *= 2.0 ** r.integers(-exp_range, 1, (x.shape[0], 1, 1))
    scales = np.array([O.scale_of(float(np.max(np.abs(b)))) for b in x])
    codes = O.e4m3_code(x / scales[:, None, None]).reshape(records, d)
    return codes, scales.astype(np.float32)


class Layout:
    """Records of a contiguous or paged cache; table is None or int32 [B, max_pages]."""

    def __init__(self, r, B, Hkv, cap, page):
        self.B, self.Hkv, self.page, self.table = B, Hkv, page, None
        if page:
            mp = -(-cap // page)
            self.cap, self.num_pages = mp * page, B * mp + 3
            self.table = r.permutation(self.num_pages)[:B * mp].reshape(B, mp).astype(np.int32)
            self.records = self.num_pages * Hkv * page
        else:
            self.cap = -(-cap // O.BLOCK) * O.BLOCK
            self.records = B * Hkv * self.cap

    def rec(self, b, h, n):
        t = np.arange(n)
        if self.table is None:
            return (b * self.Hkv + h) * self.cap + t
        return (self.table[b, t // self.page].astype(np.int64) * self.Hkv + h) * self.page + t % self.page
