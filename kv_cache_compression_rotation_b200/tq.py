"""ctypes binding of libtq (include/tq.h): argument marshalling only.

Every computation runs in the CUDA library; PyTorch supplies device memory and the
current stream.  With ``stream=`` a call runs on that stream, which also owns what the call
allocates; its inputs must be ready there and live until it is done with them.  If ``libtq.so`` is missing the first call raises -- there is no CPU
fallback.  Build it with ``python -m kv_cache_compression_rotation_b200.build``.
"""
from __future__ import annotations

import ctypes as C
import functools
import inspect
import math
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_OK = 0
STATUS_NAMES = {0: "TQ_OK", 1: "TQ_ERR_INVALID_ARG", 2: "TQ_ERR_UNSUPPORTED", 3: "TQ_ERR_ALIGNMENT",
                4: "TQ_ERR_ALIAS", 5: "TQ_ERR_CUDA", 6: "TQ_ERR_TIMEOUT", 7: "TQ_ERR_NOT_CONVERGED",
                8: "TQ_ERR_WORKSPACE"}
DIST = {"beta": 0, "gaussian": 1}
KIND_MSE, KIND_PROD, KIND_SPECTRAL = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
MAX_TOP = 8

EXPORTS = [
    "tq_version", "tq_last_error", "tq_codebook_build", "tq_waterfill", "tq_spectral_calibrate",
    "tq_spectral_unit_codebooks", "tq_record_layout", "tq_quantize_mse", "tq_quantize_prod",
    "tq_quantize_spectral", "tq_dequantize", "tq_score_workspace", "tq_score",
    "tq_decode_attn_workspace", "tq_decode_attn", "tq_get_status", "tq_set_wait_limit", "tq_lut_scale",
    "tq_decode_attn_fixed_ws", "tq_quantize_split", "tq_score_split_workspace", "tq_score_split",
    "tq_decode_attn_split_workspace", "tq_decode_attn_split", "tq_spectral_descriptor", "tq_spectral_prepare",
    "tq_decode_attn_paged", "tq_prefill_attn_workspace", "tq_prefill_attn", "tq_quantize_workspace",
    "tq_quantize_ws", "tq_kv8_append", "tq_kv8_attn_workspace", "tq_kv8_decode_attn", "tq_kv8_prefill_attn",
    "tq_pages_workspace", "tq_pages_free", "tq_pages_reserve", "tq_pages_fork", "tq_pages_compact", "tq_pages_copy",
]


class TqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Quantizer_t(C.Structure):
    _fields_ = [
        ("kind", C.c_int32), ("d", C.c_int32), ("bits", C.c_int32), ("m", C.c_int32),
        ("rot", C.c_void_p), ("S", C.c_void_p), ("centroids", C.c_void_p), ("boundaries", C.c_void_p),
        ("k_top", C.c_int32), ("tail_bits", C.c_int32), ("qjl", C.c_int32),
        ("top_bits", C.c_int32 * MAX_TOP),
        ("dim_sigma", C.c_void_p), ("unit_centroids", C.c_void_p), ("unit_boundaries", C.c_void_p),
        ("lut_scale", C.c_float), ("rot_pm1", C.c_int32),
    ]


class Packed_t(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("signs", C.c_void_p), ("norms", C.c_void_p), ("rnorms", C.c_void_p)]


MAX_GROUPS = 4


class Split_t(C.Structure):
    _fields_ = [("n_groups", C.c_int32), ("d", C.c_int32),
                ("groups", C.POINTER(Quantizer_t) * MAX_GROUPS), ("cols", C.c_void_p * MAX_GROUPS)]


class Pages_t(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("page_size", C.c_int32), ("max_pages", C.c_int32),
                ("num_pages", C.c_int64)]


class Kv8_t(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p)]


class Strides_t(C.Structure):
    _fields_ = [("b", C.c_int64), ("h", C.c_int64), ("t", C.c_int64)]


class Scoring_t(C.Structure):
    _fields_ = [("scale", C.c_float), ("softcap", C.c_float), ("slopes", C.c_void_p), ("window", C.c_int32),
                ("first", C.c_void_p), ("prefix", C.c_void_p)]


class PagePool_t(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("refs", C.c_void_p), ("rows", C.c_int32), ("max_pages", C.c_int32),
                ("page_size", C.c_int32), ("num_pages", C.c_int64)]


class PoolArray_t(C.Structure):
    _fields_ = [("data", C.c_void_p), ("page_bytes", C.c_int64)]


KV8_BLOCK = 16
MAX_POOL_ARRAYS = 16


class Layout_t(C.Structure):
    _fields_ = [("code_words", C.c_int32), ("sign_words", C.c_int32), ("has_norms", C.c_int32),
                ("has_rnorms", C.c_int32)]


_lib_handle = None


def lib():
    """Load libtq.so (raises if it was not built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtq.so not found at {LIB_PATH}; build it with "
                               "`python -m kv_cache_compression_rotation_b200.build`")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, f64p = C.c_void_p, C.c_int32, C.c_int64, C.POINTER(C.c_double)
        qp = C.POINTER(Quantizer_t)
        sig = {
            "tq_version": ([], C.c_char_p),
            "tq_last_error": ([], C.c_char_p),
            "tq_codebook_build": ([i32, i32, i32, C.c_double, f64p, f64p, C.POINTER(i32)], C.c_int),
            "tq_waterfill": ([f64p, i32, i32, i32, C.POINTER(i32)], C.c_int),
            "tq_spectral_calibrate": ([vp, i64, i32, f64p, f64p], C.c_int),
            "tq_spectral_unit_codebooks": ([f64p, f64p], C.c_int),
            "tq_record_layout": ([qp, C.POINTER(Layout_t)], C.c_int),
            "tq_quantize_mse": ([qp, vp, i32, i64, Packed_t, vp], C.c_int),
            "tq_quantize_prod": ([qp, vp, i32, i64, Packed_t, vp], C.c_int),
            "tq_quantize_spectral": ([qp, vp, i32, i64, Packed_t, vp], C.c_int),
            "tq_quantize_workspace": ([qp, i32, i64, C.POINTER(C.c_size_t)], C.c_int),
            "tq_quantize_ws": ([qp, vp, i32, i64, Packed_t, vp, C.c_size_t, vp], C.c_int),
            "tq_dequantize": ([qp, Packed_t, i64, vp, vp], C.c_int),
            "tq_score_workspace": ([qp, i64, i64, i32, C.POINTER(C.c_size_t)], C.c_int),
            "tq_score": ([qp, vp, i32, i64, Packed_t, i64, i32, vp, vp, vp, C.c_size_t, vp], C.c_int),
            "tq_decode_attn_workspace": ([qp, i32, i32, i32, i64, C.POINTER(C.c_size_t)], C.c_int),
            "tq_decode_attn": ([qp, qp, vp, i32, i32, i32, i32, i64, vp, Packed_t, Packed_t, C.c_float,
                                vp, vp, C.c_size_t, vp], C.c_int),
            "tq_decode_attn_fixed_ws": ([qp, qp, vp, i32, i32, i32, i32, i64, vp, Packed_t, Packed_t,
                                         C.c_float, vp, vp], C.c_int),
            "tq_get_status": ([vp], C.c_int),
            "tq_set_wait_limit": ([i64], C.c_int),
            "tq_lut_scale": ([f64p, i32, C.POINTER(C.c_float)], C.c_int),
            "tq_spectral_descriptor": ([f64p, f64p, i32, i32, i32, i32, i32, vp, vp, vp, vp, C.POINTER(i32),
                                        C.POINTER(C.c_float)], C.c_int),
            "tq_spectral_prepare": ([vp, i64, i32, i32, i32, i32, i32, vp, vp, vp, vp, C.POINTER(i32),
                                     C.POINTER(C.c_float), f64p], C.c_int),
            "tq_decode_attn_paged": ([qp, qp, vp, vp, vp, i32, i32, i32, i32, vp, C.POINTER(Pages_t), Packed_t,
                                      Packed_t, C.c_float, vp, vp, C.c_size_t, vp], C.c_int),
            "tq_prefill_attn_workspace": ([qp, i32, i32, i32, i32, i64, C.POINTER(C.c_size_t)], C.c_int),
            "tq_prefill_attn": ([qp, qp, vp, i32, i32, i32, i32, i32, vp, vp, C.POINTER(Pages_t), i64, Packed_t,
                                 Packed_t, C.c_float, vp, vp, C.c_size_t, vp], C.c_int),
            "tq_quantize_split": ([C.POINTER(Split_t), vp, i32, i64, C.POINTER(Packed_t), vp], C.c_int),
            "tq_score_split_workspace": ([C.POINTER(Split_t), i64, i64, i32, C.POINTER(C.c_size_t)], C.c_int),
            "tq_score_split": ([C.POINTER(Split_t), vp, i32, i64, C.POINTER(Packed_t), i64, i32, vp, vp, vp,
                                C.c_size_t, vp], C.c_int),
            "tq_decode_attn_split_workspace": ([C.POINTER(Split_t), C.POINTER(Split_t), i32, i32, i32, i64,
                                                C.POINTER(C.c_size_t)], C.c_int),
            "tq_decode_attn_split": ([C.POINTER(Split_t), C.POINTER(Split_t), vp, i32, i32, i32, i32, i64, vp,
                                      C.POINTER(Packed_t), C.POINTER(Packed_t), C.c_float, vp, vp, C.c_size_t,
                                      vp], C.c_int),
            "tq_kv8_append": ([vp, vp, i32, C.POINTER(Strides_t), C.POINTER(Strides_t), i32, i32, i32, i32, vp, vp,
                               C.POINTER(Pages_t), i64, Kv8_t, Kv8_t, vp], C.c_int),
            "tq_kv8_attn_workspace": ([i32, i32, i32, i32, i32, i32, i64, C.POINTER(C.c_size_t)], C.c_int),
            "tq_kv8_decode_attn": ([vp, C.POINTER(Strides_t), i32, i32, i32, i32, i32, vp, C.POINTER(Scoring_t),
                                    C.POINTER(Pages_t), i64, vp, vp, C.POINTER(Strides_t), C.POINTER(Strides_t), Kv8_t,
                                    Kv8_t, vp, vp, vp, C.c_size_t, vp], C.c_int),
            "tq_kv8_prefill_attn": ([vp, C.POINTER(Strides_t), i32, i32, i32, i32, i32, i32, vp, vp,
                                     C.POINTER(Scoring_t), C.POINTER(Pages_t), i64, Kv8_t, Kv8_t, vp, vp, vp,
                                     C.c_size_t, vp], C.c_int),
            "tq_pages_workspace": ([C.POINTER(PagePool_t), i32, C.POINTER(C.c_size_t)], C.c_int),
            "tq_pages_free": ([C.POINTER(PagePool_t), vp, vp, i32, vp], C.c_int),
            "tq_pages_reserve": ([C.POINTER(PagePool_t), vp, vp, vp, i32, vp, vp, C.c_size_t, vp], C.c_int),
            "tq_pages_fork": ([C.POINTER(PagePool_t), C.POINTER(PoolArray_t), i32, vp, vp, vp, i32, vp, vp, C.c_size_t,
                               vp], C.c_int),
            "tq_pages_compact": ([C.POINTER(PagePool_t), C.POINTER(PoolArray_t), i32, vp, vp, vp, C.c_size_t, vp],
                                 C.c_int),
            "tq_pages_copy": ([C.POINTER(PoolArray_t), i32, i64, vp, vp, i32, vp], C.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib_handle = L
    return _lib_handle


def _check(status: int) -> None:
    if status != TQ_OK:
        raise TqError(status, lib().tq_last_error().decode())


def _dptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    if stream is not None:
        return stream.cuda_stream
    if not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _tensors(x):
    """The tensors of what a call returns."""
    if isinstance(x, (tuple, list)):
        return [t for y in x for t in _tensors(y)]
    if isinstance(x, Packed):
        return [t for t in (x.codes, x.signs, x.norms, x.rnorms) if t is not None]
    return [x] if hasattr(x, "record_stream") else []


def _allocated(stream, f, *args):
    """f(*args), which allocates, with `stream` as the current one, so that the memory belongs to it: a
    workspace that is dropped at return goes to nobody else while the kernels use it, and an output's
    memory to nobody while the caller's stream reads it."""
    import torch
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        result = f(*args)
    if here != stream:
        for t in _tensors(result):
            t.record_stream(here)
    return result


def _on_stream(f):
    """For calls that allocate: with stream= the whole call runs as if that were the current stream."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        return f(*args, **kw) if stream is None else _allocated(stream, functools.partial(f, **kw), *args)

    return call


@functools.lru_cache(maxsize=None)
def _dtype_codes() -> dict:
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _dtype_code(t) -> int:
    return _dtype_codes()[t.dtype]


def version() -> str:
    return lib().tq_version().decode()


# ------------------------------------------------------------------ host math
def codebook_build(bits: int, dist: str = "beta", d: int = 0, sigma: float = 0.0):
    """Lloyd-Max codebook: (centroids [2^b], boundaries [2^b-1], iterations) as float64."""
    k = 1 << bits
    c = np.zeros(k, dtype=np.float64)
    t = np.zeros(k - 1, dtype=np.float64)
    it = C.c_int32(0)
    _check(lib().tq_codebook_build(d, bits, DIST[dist], float(sigma),
                                   c.ctypes.data_as(C.POINTER(C.c_double)),
                                   t.ctypes.data_as(C.POINTER(C.c_double)), C.byref(it)))
    return c, t, it.value


def waterfill(lam, budget: int, max_bits: int = 8) -> np.ndarray:
    lam = np.ascontiguousarray(lam, dtype=np.float64)
    out = np.zeros(lam.shape[0], dtype=np.int32)
    _check(lib().tq_waterfill(lam.ctypes.data_as(C.POINTER(C.c_double)), lam.shape[0], budget, max_bits,
                              out.ctypes.data_as(C.POINTER(C.c_int32))))
    return out


def spectral_calibrate(X: np.ndarray):
    X = np.ascontiguousarray(X, dtype=np.float32)
    n, d = X.shape
    vecs = np.zeros((d, d), dtype=np.float64)
    vals = np.zeros(d, dtype=np.float64)
    _check(lib().tq_spectral_calibrate(X.ctypes.data, n, d, vecs.ctypes.data_as(C.POINTER(C.c_double)),
                                       vals.ctypes.data_as(C.POINTER(C.c_double))))
    return vecs, vals


def lut_scale(values) -> float:
    """Shared scale s for a half-precision table of `values` (entries v / s)."""
    v = np.ascontiguousarray(values, dtype=np.float64)
    out = C.c_float(0.0)
    _check(lib().tq_lut_scale(v.ctypes.data_as(C.POINTER(C.c_double)), v.shape[0], C.byref(out)))
    return float(out.value)


def spectral_unit_codebooks():
    c = np.zeros(510, dtype=np.float64)
    t = np.zeros(502, dtype=np.float64)
    _check(lib().tq_spectral_unit_codebooks(c.ctypes.data_as(C.POINTER(C.c_double)),
                                            t.ctypes.data_as(C.POINTER(C.c_double))))
    return c, t


# ------------------------------------------------------------------ descriptors
@dataclass
class Packed:
    """Packed records (structure of arrays) on the device."""
    codes: object
    signs: object = None
    norms: object = None
    rnorms: object = None

    def as_c(self) -> Packed_t:
        return Packed_t(_dptr(self.codes) if self.codes is not None and self.codes.numel() else None,
                        _dptr(self.signs), _dptr(self.norms), _dptr(self.rnorms))


class Quantizer:
    """Device-resident quantizer descriptor (owns the tensors the C struct points at)."""

    def __init__(self, kind: int, d: int, rot, *, bits=0, m=0, S=None, centroids=None, boundaries=None,
                 k_top=0, tail_bits=0, qjl=0, top_bits=(), dim_sigma=None, unit_c=None, unit_t=None,
                 lut_scale=0.0, rot_pm1=None):
        self.kind, self.d, self.bits, self.m = kind, d, bits, m
        self._keep = [rot, S, centroids, boundaries, dim_sigma, unit_c, unit_t]
        self.rot, self.S, self.centroids, self.boundaries = rot, S, centroids, boundaries
        self.dim_sigma, self.unit_c, self.unit_t = dim_sigma, unit_c, unit_t
        self.k_top, self.tail_bits, self.qjl, self.top_bits = k_top, tail_bits, qjl, tuple(top_bits)
        tb = (C.c_int32 * MAX_TOP)(*(list(top_bits) + [0] * (MAX_TOP - len(top_bits))))
        self.c = Quantizer_t(kind, d, bits, m, _dptr(rot), _dptr(S), _dptr(centroids), _dptr(boundaries),
                             k_top, tail_bits, qjl, tb, _dptr(dim_sigma), _dptr(unit_c), _dptr(unit_t),
                             float(lut_scale), int(bool(rot_pm1)))

    @property
    def ref(self):
        return C.byref(self.c)

    @staticmethod
    def _dev(a, device):
        import torch
        return torch.as_tensor(np.ascontiguousarray(a, dtype=np.float32), device=device).contiguous()

    @staticmethod
    def _is_pm1(rot) -> bool:
        """True when every entry of rot is +-1/sqrt(d) in fp32 (Hadamard-type rotation)."""
        r = np.asarray(rot, dtype=np.float32)
        return bool(np.all(np.abs(r) == np.float32(1.0 / math.sqrt(r.shape[0]))))

    @classmethod
    def mse(cls, rot, bits: int, dist: str = "beta", sigma: float = 0.0, device="cuda"):
        d = rot.shape[0]
        c, t, _ = codebook_build(bits, dist, d=d, sigma=sigma)
        return cls(KIND_MSE, d, cls._dev(rot, device), bits=bits,
                   centroids=cls._dev(c, device), boundaries=cls._dev(t, device), lut_scale=lut_scale(c),
                   rot_pm1=cls._is_pm1(rot))

    @classmethod
    def prod(cls, rot, S, bits: int, dist: str = "beta", sigma: float = 0.0, device="cuda"):
        d = rot.shape[0]
        m = S.shape[0]
        cen = bnd = None
        sc = 0.0
        if bits > 1:
            c, t, _ = codebook_build(bits - 1, dist, d=d, sigma=sigma)
            cen, bnd = cls._dev(c, device), cls._dev(t, device)
            sc = lut_scale(c)
        return cls(KIND_PROD, d, cls._dev(rot, device), bits=bits, m=m, S=cls._dev(S, device),
                   centroids=cen, boundaries=bnd, lut_scale=sc)

    @classmethod
    def _spectral_from_host(cls, d, k_top, tail_bits, qjl, S_top, device, host):
        rot, sig, uc, ut, top, lut = host
        return cls(KIND_SPECTRAL, d, cls._dev(rot, device), S=None if S_top is None else cls._dev(S_top, device),
                   k_top=k_top, tail_bits=tail_bits, qjl=1 if qjl else 0, top_bits=list(top[:k_top]),
                   dim_sigma=cls._dev(sig, device), unit_c=cls._dev(uc, device), unit_t=cls._dev(ut, device),
                   lut_scale=lut)

    @staticmethod
    def _spectral_outputs(d):
        return (np.zeros((d, d), dtype=np.float32), np.zeros(d, dtype=np.float32), np.zeros(510, dtype=np.float32),
                np.zeros(502, dtype=np.float32), np.zeros(MAX_TOP, dtype=np.int32))

    @classmethod
    def spectral(cls, eigvecs, eigvals, k_top: int, budget_bits: int, tail_bits: int, qjl: bool, S_top=None,
                 max_bits: int = 8, device="cuda"):
        """SPECTRAL descriptor from a given eigen-decomposition (rows of eigvecs, descending
        eigvals): tq_spectral_descriptor water-fills the top bits and builds the scales and
        codebooks; this wrapper only copies its outputs to the device."""
        d = eigvecs.shape[0]
        vecs = np.ascontiguousarray(eigvecs, dtype=np.float64)
        vals = np.ascontiguousarray(eigvals, dtype=np.float64)
        rot, sig, uc, ut, top = cls._spectral_outputs(d)
        lut = C.c_float(0.0)
        _check(lib().tq_spectral_descriptor(vecs.ctypes.data_as(C.POINTER(C.c_double)),
                                            vals.ctypes.data_as(C.POINTER(C.c_double)), d, k_top, budget_bits,
                                            tail_bits, max_bits, rot.ctypes.data, sig.ctypes.data, uc.ctypes.data,
                                            ut.ctypes.data, top.ctypes.data_as(C.POINTER(C.c_int32)), C.byref(lut)))
        return cls._spectral_from_host(d, k_top, tail_bits, qjl, S_top, device,
                                       (rot, sig, uc, ut, top, float(lut.value)))

    @classmethod
    def spectral_calibrated(cls, X, k_top: int, budget_bits: int, tail_bits: int, qjl: bool, S_top=None,
                            max_bits: int = 8, device="cuda"):
        """SPECTRAL descriptor straight from calibration rows X [n, d] (tq_spectral_prepare:
        calibration, water-filling, scales and codebooks in the library).  Returns
        (quantizer, eigenvalues)."""
        X = np.ascontiguousarray(X, dtype=np.float32)
        n, d = X.shape
        rot, sig, uc, ut, top = cls._spectral_outputs(d)
        vals = np.zeros(d, dtype=np.float64)
        lut = C.c_float(0.0)
        _check(lib().tq_spectral_prepare(X.ctypes.data, n, d, k_top, budget_bits, tail_bits, max_bits,
                                         rot.ctypes.data, sig.ctypes.data, uc.ctypes.data, ut.ctypes.data,
                                         top.ctypes.data_as(C.POINTER(C.c_int32)), C.byref(lut),
                                         vals.ctypes.data_as(C.POINTER(C.c_double))))
        q = cls._spectral_from_host(d, k_top, tail_bits, qjl, S_top, device, (rot, sig, uc, ut, top, float(lut.value)))
        return q, vals

    def layout(self) -> Layout_t:
        L = Layout_t()
        _check(lib().tq_record_layout(self.ref, C.byref(L)))
        return L

    def alloc(self, n: int, device="cuda") -> Packed:
        """Zeroed packed arrays for n records."""
        import torch
        L = self.layout()
        codes = torch.zeros((n, L.code_words), dtype=torch.int32, device=device)
        signs = torch.zeros((n, L.sign_words), dtype=torch.int32, device=device) if L.sign_words else None
        norms = torch.zeros(n, dtype=torch.float32, device=device) if L.has_norms else None
        rnorms = torch.zeros(n, dtype=torch.float32, device=device) if L.has_rnorms else None
        return Packed(codes, signs, norms, rnorms)


# ------------------------------------------------------------------ device calls
@_on_stream
def quantize(q: Quantizer, x, out: Optional[Packed] = None, stream=None) -> Packed:
    """tq_quantize_{mse,prod,spectral} of x [n, d] (fp32 / bf16 / fp16 CUDA tensor)."""
    assert x.is_cuda and x.is_contiguous() and x.shape[-1] == q.d
    n = x.numel() // q.d
    out = q.alloc(n, x.device) if out is None else out
    fn = {KIND_MSE: lib().tq_quantize_mse, KIND_PROD: lib().tq_quantize_prod,
          KIND_SPECTRAL: lib().tq_quantize_spectral}[q.kind]
    _check(fn(q.ref, x.data_ptr(), _dtype_code(x), n, out.as_c(), _stream(stream)))
    return out


def tq_quantize_workspace_bytes(q: Quantizer, x) -> int:
    ws = C.c_size_t(0)
    _check(lib().tq_quantize_workspace(q.ref, _dtype_code(x), x.numel() // q.d, C.byref(ws)))
    return ws.value


@_on_stream
def quantize_ws(q: Quantizer, x, out: Optional[Packed] = None, workspace=None, stream=None) -> Packed:
    """tq_quantize_ws: the same records as quantize(), with device scratch (wide fp32 vectors
    take the tensor-core split-precision path)."""
    import torch
    assert x.is_cuda and x.is_contiguous() and x.shape[-1] == q.d
    n = x.numel() // q.d
    out = q.alloc(n, x.device) if out is None else out
    ws = C.c_size_t(0)
    _check(lib().tq_quantize_workspace(q.ref, _dtype_code(x), n, C.byref(ws)))
    if workspace is None or workspace.numel() < ws.value:
        workspace = torch.empty(max(ws.value, 16), dtype=torch.uint8, device=x.device)
    _check(lib().tq_quantize_ws(q.ref, x.data_ptr(), _dtype_code(x), n, out.as_c(), workspace.data_ptr(),
                                workspace.numel(), _stream(stream)))
    return out


@_on_stream
def dequantize(q: Quantizer, packed: Packed, n: int, stream=None):
    import torch
    out = torch.empty((n, q.d), dtype=torch.float32, device=packed.codes.device)
    _check(lib().tq_dequantize(q.ref, packed.as_c(), n, out.data_ptr(), _stream(stream)))
    return out


@_on_stream
def score(q: Quantizer, qv, packed: Packed, n: int, topk: int = 0, stream=None):
    """Dense estimates [nq, n], or (scores [nq, topk], ids [nq, topk]) when topk > 0."""
    import torch
    nq = qv.numel() // q.d
    ws = C.c_size_t(0)
    _check(lib().tq_score_workspace(q.ref, nq, n, topk, C.byref(ws)))
    work = torch.empty(max(ws.value, 16), dtype=torch.uint8, device=qv.device)
    if topk == 0:
        scores = torch.empty((nq, n), dtype=torch.float32, device=qv.device)
        ids = None
    else:
        scores = torch.empty((nq, topk), dtype=torch.float32, device=qv.device)
        ids = torch.empty((nq, topk), dtype=torch.int32, device=qv.device)
    _check(lib().tq_score(q.ref, qv.data_ptr(), _dtype_code(qv), nq, packed.as_c(), n, topk, scores.data_ptr(),
                          _dptr(ids), work.data_ptr(), ws.value, _stream(stream)))
    return scores if topk == 0 else (scores, ids)


class Split:
    """Outlier-channel split: group g is the quantizer ``groups[g]`` over the channels
    ``cols[g]`` (int32 CUDA tensor) of d-wide vectors."""

    def __init__(self, d: int, groups, cols):
        assert 1 <= len(groups) == len(cols) <= MAX_GROUPS
        self.d, self.groups, self.cols = d, list(groups), list(cols)
        gp = (C.POINTER(Quantizer_t) * MAX_GROUPS)(*[C.pointer(q.c) for q in self.groups])
        cp = (C.c_void_p * MAX_GROUPS)(*[_dptr(c) for c in self.cols])
        self.c = Split_t(len(self.groups), d, gp, cp)

    @property
    def ref(self):
        return C.byref(self.c)

    def alloc(self, n: int, device="cuda"):
        return [q.alloc(n, device) for q in self.groups]


def _packed_array(packs):
    return (Packed_t * len(packs))(*[p.as_c() for p in packs])


@_on_stream
def quantize_split(sp: Split, x, out=None, stream=None):
    """tq_quantize_split of x [n, d]: one list entry of packed records per group."""
    assert x.is_cuda and x.is_contiguous() and x.shape[-1] == sp.d
    n = x.numel() // sp.d
    out = sp.alloc(n, x.device) if out is None else out
    _check(lib().tq_quantize_split(sp.ref, x.data_ptr(), _dtype_code(x), n, _packed_array(out), _stream(stream)))
    return out


@_on_stream
def score_split(sp: Split, qv, packs, n: int, topk: int = 0, stream=None):
    """Summed split estimates [nq, n], or (scores, ids) of the top-k when topk > 0."""
    import torch
    nq = qv.numel() // sp.d
    ws = C.c_size_t(0)
    _check(lib().tq_score_split_workspace(sp.ref, nq, n, topk, C.byref(ws)))
    work = torch.empty(max(ws.value, 16), dtype=torch.uint8, device=qv.device)
    if topk == 0:
        scores = torch.empty((nq, n), dtype=torch.float32, device=qv.device)
        ids = None
    else:
        scores = torch.empty((nq, topk), dtype=torch.float32, device=qv.device)
        ids = torch.empty((nq, topk), dtype=torch.int32, device=qv.device)
    _check(lib().tq_score_split(sp.ref, qv.data_ptr(), _dtype_code(qv), nq, _packed_array(packs), n, topk,
                                scores.data_ptr(), _dptr(ids), work.data_ptr(), ws.value, _stream(stream)))
    return scores if topk == 0 else (scores, ids)


@_on_stream
def decode_attn_split(ks: Split, vs: Split, q, seq_lens, kpacks, vpacks, Nmax: int, Hkv: int, scale=None,
                      out=None, stream=None):
    """tq_decode_attn_split for q [B, Hq, d] over split caches (one packed list per split)."""
    import torch
    B, Hq, d = q.shape
    assert d == ks.d == vs.d and q.is_contiguous()
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws = C.c_size_t(0)
    _check(lib().tq_decode_attn_split_workspace(ks.ref, vs.ref, B, Hq, Hkv, Nmax, C.byref(ws)))
    work = torch.empty(max(ws.value, 16), dtype=torch.uint8, device=q.device)
    out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device) if out is None else out
    _check(lib().tq_decode_attn_split(ks.ref, vs.ref, q.data_ptr(), _dtype_code(q), B, Hq, Hkv, Nmax,
                                      seq_lens.data_ptr(), _packed_array(kpacks), _packed_array(vpacks),
                                      float(scale), out.data_ptr(), work.data_ptr(), ws.value, _stream(stream)))
    return out


def decode_workspace_bytes(kq: Quantizer, B: int, Hq: int, Hkv: int, Nmax: int) -> int:
    ws = C.c_size_t(0)
    _check(lib().tq_decode_attn_workspace(kq.ref, B, Hq, Hkv, Nmax, C.byref(ws)))
    return ws.value


@_on_stream
def decode_attn(kq: Quantizer, vq: Quantizer, q, seq_lens, kcache: Packed, vcache: Packed, Nmax: int,
                Hkv: int, scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """One decode-attention step; q [B, Hq, d], seq_lens int32 [B] on the device."""
    import torch
    B, Hq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = decode_workspace_bytes(kq, B, Hq, Hkv, Nmax)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device) if out is None else out
    _check(lib().tq_decode_attn(kq.ref, vq.ref, q.data_ptr(), _dtype_code(q), B, Hq, Hkv, Nmax,
                                seq_lens.data_ptr(), kcache.as_c(), vcache.as_c(), float(scale), out.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


class Pages:
    """Paged record pool: block_table int32 [B, max_pages] CUDA tensor of page ids, page_size
    tokens per page (a multiple of 16), num_pages pages; token t of (b, kv-head h) is record
    (block_table[b, t // page_size] * Hkv + h) * page_size + t % page_size of every array."""

    def __init__(self, block_table, page_size: int, num_pages: int):
        assert block_table.dtype.is_floating_point is False and block_table.is_contiguous()
        self.block_table, self.page_size, self.num_pages = block_table, page_size, num_pages
        self.max_pages = block_table.shape[1]
        self.c = Pages_t(block_table.data_ptr(), page_size, self.max_pages, num_pages)

    @property
    def ref(self):
        return C.byref(self.c)

    def records(self, Hkv: int) -> int:
        return self.num_pages * Hkv * self.page_size


@_on_stream
def decode_attn_paged(kq: Quantizer, vq: Quantizer, q, seq_lens, pages: Pages, kpool: Packed, vpool: Packed,
                      Hkv: int, k_new=None, v_new=None, scale: Optional[float] = None, out=None, workspace=None,
                      stream=None):
    """tq_decode_attn_paged: append k_new / v_new [B*Hkv, d] (optional) as token seq_lens[b]-1,
    then one decode step over the pool; q [B, Hq, d]."""
    import torch
    B, Hq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = decode_workspace_bytes(kq, B, Hq, Hkv, pages.max_pages * pages.page_size)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device) if out is None else out
    _check(lib().tq_decode_attn_paged(kq.ref, vq.ref, q.data_ptr(), _dptr(k_new), _dptr(v_new), _dtype_code(q), B, Hq,
                                      Hkv, seq_lens.data_ptr(), pages.ref, kpool.as_c(), vpool.as_c(), float(scale),
                                      out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


@_on_stream
def prefill_attn(kq: Quantizer, vq: Quantizer, q, q_pos, kv_lens, kcache: Packed, vcache: Packed, Hkv: int,
                 Nmax: int = 0, pages: Optional[Pages] = None, scale: Optional[float] = None, out=None,
                 workspace=None, stream=None):
    """tq_prefill_attn: causal attention of q [B, Hq, T, d] at positions q_pos [B, T] over the
    packed cache ([B, Hkv, Nmax] records, or a paged pool)."""
    import torch
    B, Hq, T, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    n = pages.max_pages * pages.page_size if pages is not None else Nmax
    ws = C.c_size_t(0)
    _check(lib().tq_prefill_attn_workspace(kq.ref, B, Hq, Hkv, T, n, C.byref(ws)))
    if workspace is None or workspace.numel() < ws.value:
        workspace = torch.empty(max(ws.value, 16), dtype=torch.uint8, device=q.device)
    out = torch.empty((B, Hq, T, d), dtype=torch.float32, device=q.device) if out is None else out
    _check(lib().tq_prefill_attn(kq.ref, vq.ref, q.data_ptr(), _dtype_code(q), B, Hq, Hkv, T, q_pos.data_ptr(),
                                 kv_lens.data_ptr(), pages.ref if pages is not None else None, Nmax, kcache.as_c(),
                                 vcache.as_c(), float(scale), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                 _stream(stream)))
    return out


# ------------------------------------------------------------------ 8-bit block-scaled cache
class Kv8:
    """One side of an 8-bit cache: codes uint8 [records, d] (e4m3 bytes) and scales fp32
    [records / 16] (CUDA tensors)."""

    def __init__(self, codes, scales):
        import torch
        if codes.dtype not in (torch.uint8, torch.float8_e4m3fn) or scales.dtype is not torch.float32:
            raise ValueError("codes must be uint8 or float8_e4m3fn and scales float32")
        if codes.dim() != 2 or not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes [records, d] and scales must be contiguous")
        if codes.device != scales.device:
            raise ValueError(f"codes on {codes.device} and scales on {scales.device}")
        if scales.numel() * KV8_BLOCK != codes.shape[0]:
            raise ValueError(f"scales must hold one value for each {KV8_BLOCK} of the {codes.shape[0]} records")
        self.codes, self.scales, self.d, self.records = codes, scales, codes.shape[1], codes.shape[0]
        self.device = codes.device
        self.c = Kv8_t(codes.data_ptr(), scales.data_ptr())


def kv8_alloc(records: int, d: int, device="cuda") -> Kv8:
    """A zeroed side of `records` records (a multiple of 16)."""
    import torch
    return Kv8(torch.zeros((records, d), dtype=torch.uint8, device=device),
               torch.zeros(records // KV8_BLOCK, dtype=torch.float32, device=device))


class Scoring:
    """Options of the 8-bit attention's scores (tq_scoring): scale (default 1/sqrt(d)), softcap,
    slopes fp32 [Hq], window, first int32 [B, T] (document starts), prefix int32 [B]."""

    def __init__(self, scale: Optional[float] = None, softcap: float = 0.0, slopes=None, window: int = 0, first=None,
                 prefix=None):
        import torch
        for name, t, dt in (("slopes", slopes, torch.float32), ("first", first, torch.int32),
                            ("prefix", prefix, torch.int32)):
            if t is not None and (t.dtype is not dt or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dt} tensor")
        self.scale, self.slopes, self.first, self.prefix = scale, slopes, first, prefix
        self.softcap, self.window = float(softcap), int(window)

    def as_c(self, d: int):
        return Scoring_t(1.0 / math.sqrt(d) if self.scale is None else float(self.scale), self.softcap,
                         _dptr(self.slopes), self.window, _dptr(self.first), _dptr(self.prefix))

    def check(self, B: int, Hq: int, T: int) -> None:
        for name, t, n in (("slopes", self.slopes, Hq), ("first", self.first, B * T), ("prefix", self.prefix, B)):
            if t is not None and t.numel() != n:
                raise ValueError(f"{name} must hold {n} values (got {t.numel()})")


def _ints(t, n: int, name: str):
    import torch
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} values")
    return t.data_ptr()


def _scratch(t):
    """A caller's workspace: numel() stands for its bytes, which must be there one after the other."""
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t


def _rows(t, name: str, d: int):
    if t.stride(-1) != 1 or t.shape[-1] != d:
        raise ValueError(f"{name}: the last dimension must be {d} contiguous elements")
    return t.data_ptr()


def _same_device(device, *ts):
    import torch
    if device.type != "cuda" or device.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current CUDA device (got {device})")
    index = device.index
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {device} and {t.device} in one call")


def _kv8_cache(kcache: Kv8, vcache: Kv8, B: int, Hkv: int, Nmax: int, pages):
    """Checks that the sides hold what the layout addresses; returns the capacity in tokens."""
    if kcache.d != vcache.d or kcache.records != vcache.records:
        raise ValueError("kcache and vcache differ in shape")
    need = pages.records(Hkv) if pages is not None else B * Hkv * Nmax
    if need > kcache.records:
        raise ValueError(f"the cache holds {kcache.records} records, the layout addresses {need}")
    if pages is not None:
        if pages.block_table.shape[0] < B or pages.block_table.element_size() != 4:
            raise ValueError(f"block_table must be int32 with a row for each of {B} sequences")
        if pages.block_table.device != kcache.device:
            raise ValueError(f"block_table on {pages.block_table.device}, the cache on {kcache.device}")
        return pages.max_pages * pages.page_size
    return Nmax


def kv8_append(kcache: Kv8, vcache: Kv8, k_new, v_new, kv_lens, new_lens=None, Nmax: int = 0,
               pages: Optional[Pages] = None, stream=None) -> None:
    """tq_kv8_append: k_new / v_new [B, Hkv, T, d] (any strides, d contiguous) become the last tokens
    of each sequence; kv_lens int32 [B] counts them, new_lens int32 [B] says how many of the T."""
    B, Hkv, T, d = k_new.shape
    if v_new.shape != k_new.shape or v_new.dtype is not k_new.dtype or kcache.d != d:
        raise ValueError("k_new, v_new and the cache differ in shape or dtype")
    _same_device(k_new.device, v_new, kv_lens, new_lens, kcache.codes, vcache.codes)
    _kv8_cache(kcache, vcache, B, Hkv, Nmax, pages)
    ks, vs = k_new.stride(), v_new.stride()
    _check(lib().tq_kv8_append(_rows(k_new, "k_new", d), _rows(v_new, "v_new", d), _dtype_code(k_new),
                               C.byref(Strides_t(ks[0], ks[1], ks[2])), C.byref(Strides_t(vs[0], vs[1], vs[2])), B, Hkv,
                               T, d, _ints(kv_lens, B, "kv_lens"),
                               None if new_lens is None else _ints(new_lens, B, "new_lens"),
                               None if pages is None else pages.ref, Nmax, kcache.c, vcache.c, _stream(stream)))


def kv8_workspace_bytes(dtype, B: int, Hq: int, Hkv: int, T: int, d: int, Nmax: int) -> int:
    """Workspace of the 8-bit attention calls (T = 1: decode); dtype as a torch dtype."""
    import torch
    code = _dtype_codes()[dtype]
    return _kv8_ws_bytes(torch.cuda.current_device() if torch.cuda.is_initialized() else -1, code, B, Hq, Hkv, T, d, Nmax)


@functools.lru_cache(maxsize=1024)
def _kv8_ws_bytes(device: int, code: int, *shape) -> int:
    ws = C.c_size_t(0)
    _check(lib().tq_kv8_attn_workspace(code, *shape, C.byref(ws)))
    return ws.value


_PLAIN_SCORING = Scoring()


def _kv8_attn_checks(B, Hq, T, d, kcache, vcache, Hkv, Nmax, pages, scoring):
    cap = _kv8_cache(kcache, vcache, B, Hkv, Nmax, pages)
    if kcache.d != d:
        raise ValueError(f"q has d = {d}, the cache {kcache.d}")
    scoring = _PLAIN_SCORING if scoring is None else scoring
    scoring.check(B, Hq, T)
    return cap, scoring


def kv8_decode_attn(q, kv_lens, kcache: Kv8, vcache: Kv8, Hkv: int, Nmax: int = 0, pages: Optional[Pages] = None,
                    k_new=None, v_new=None, scoring: Optional[Scoring] = None, out=None, lse=None,
                    return_lse: bool = False, workspace=None, stream=None):
    """tq_kv8_decode_attn: one step for q [B, Hq, d], output of q's dtype (with lse fp32 [B, Hq] when
    return_lse); k_new / v_new [B, Hkv, d] are appended as token kv_lens[b] - 1 first (none where
    kv_lens[b] is 0)."""
    B, Hq, d = q.shape
    cap, scoring = _kv8_attn_checks(B, Hq, 1, d, kcache, vcache, Hkv, Nmax, pages, scoring)
    _same_device(q.device, kv_lens, kcache.codes, vcache.codes, k_new, v_new, out, lse, workspace, scoring.slopes,
                 scoring.first, scoring.prefix)
    kst = vst = None
    if k_new is not None:
        if v_new is None or k_new.shape != (B, Hkv, d) or v_new.shape != (B, Hkv, d) or \
                k_new.dtype is not q.dtype or v_new.dtype is not q.dtype:
            raise ValueError(f"k_new and v_new must be [{B}, {Hkv}, {d}] of q's dtype")
        kst, vst = (C.byref(Strides_t(t.stride(0), t.stride(1), 0)) for t in (k_new, v_new))
    out, lse, ws = _kv8_outputs(q, kcache, (B, Hq, d), out, lse, return_lse, workspace, stream, B, Hq, Hkv, 1, d, cap)
    _check(lib().tq_kv8_decode_attn(_rows(q, "q", d), C.byref(Strides_t(q.stride(0), q.stride(1), 0)), _dtype_code(q), B,
                                    Hq, Hkv, d, _ints(kv_lens, B, "kv_lens"), C.byref(scoring.as_c(d)),
                                    None if pages is None else pages.ref, Nmax,
                                    None if k_new is None else _rows(k_new, "k_new", d),
                                    None if v_new is None else _rows(v_new, "v_new", d), kst, vst, kcache.c, vcache.c,
                                    out.data_ptr(), _dptr(lse), ws.data_ptr(), ws.numel(), _stream(stream)))
    return (out, lse) if return_lse else out


def _kv8_outputs(q, kcache, shape, out, lse, return_lse, workspace, stream, *call):
    import torch
    if stream is not None:
        return _allocated(stream, _kv8_outputs, q, kcache, shape, out, lse, return_lse, workspace, None, *call)
    if out is None:                            # (new_empty costs the host a third less than empty)
        out = q.new_empty(shape)
    elif out.shape != shape or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} tensor {tuple(shape)}")
    if lse is None:
        lse = kcache.scales.new_empty(shape[:-1]) if return_lse else None
    elif lse.shape != shape[:-1] or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor {tuple(shape[:-1])}")
    if workspace is not None:
        _scratch(workspace)
    else:
        workspace = torch.empty(kv8_workspace_bytes(q.dtype, *call), dtype=torch.uint8, device=q.device)
    return out, lse, workspace


def kv8_prefill_attn(q, q_pos, kv_lens, kcache: Kv8, vcache: Kv8, Hkv: int, Nmax: int = 0,
                     pages: Optional[Pages] = None, scoring: Optional[Scoring] = None, out=None, lse=None,
                     return_lse: bool = False, workspace=None, stream=None):
    """tq_kv8_prefill_attn: q [B, Hq, T, d] (any strides, d contiguous) at positions q_pos int32 [B, T]
    over the 8-bit cache; output [B, Hq, T, d] of q's dtype (with lse fp32 [B, Hq, T] when return_lse)."""
    B, Hq, T, d = q.shape
    cap, scoring = _kv8_attn_checks(B, Hq, T, d, kcache, vcache, Hkv, Nmax, pages, scoring)
    _same_device(q.device, q_pos, kv_lens, kcache.codes, vcache.codes, out, lse, workspace, scoring.slopes,
                 scoring.first, scoring.prefix)
    out, lse, ws = _kv8_outputs(q, kcache, (B, Hq, T, d), out, lse, return_lse, workspace, stream, B, Hq, Hkv, T, d, cap)
    st = q.stride()
    _check(lib().tq_kv8_prefill_attn(_rows(q, "q", d), C.byref(Strides_t(st[0], st[1], st[2])), _dtype_code(q), B, Hq, Hkv,
                                     T, d, _ints(q_pos, B * T, "q_pos"), _ints(kv_lens, B, "kv_lens"),
                                     C.byref(scoring.as_c(d)), None if pages is None else pages.ref, Nmax, kcache.c,
                                     vcache.c, out.data_ptr(), _dptr(lse), ws.data_ptr(), ws.numel(), _stream(stream)))
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ page pool
class PagePool:
    """Which pages each row (sequence) of a paged cache holds: block_table int32 [rows, max_pages],
    refs int32 [num_pages] (counts, 0 = free), and the record arrays whose pages move together
    (Packed or Kv8 arrays: [num_pages * Hkv * page_size, ...] tensors)."""

    def __init__(self, block_table, refs, page_size: int, arrays=()):
        import torch
        for name, t in (("block_table", block_table), ("refs", refs)):
            if t.dtype is not torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor")
        self.block_table, self.refs, self.page_size, self.arrays = block_table, refs, page_size, list(arrays)
        if refs.device != block_table.device:
            raise ValueError(f"block_table on {block_table.device} and refs on {refs.device}")
        self.rows, self.max_pages = block_table.shape
        self.num_pages = refs.numel()
        self.device = block_table.device
        if len(self.arrays) > MAX_POOL_ARRAYS:
            raise ValueError(f"at most {MAX_POOL_ARRAYS} arrays")
        pa = (PoolArray_t * max(1, len(self.arrays)))()
        for i, a in enumerate(self.arrays):
            nbytes = a.numel() * a.element_size()
            if not a.is_contiguous() or nbytes % self.num_pages or a.device != self.device:
                raise ValueError(f"array {i} must be contiguous, on {self.device}, and a whole number of bytes a page")
            pa[i] = PoolArray_t(a.data_ptr(), nbytes // self.num_pages)
        self.pa = pa
        self.ws_bytes = {}                     # by number of requests
        self.c = PagePool_t(block_table.data_ptr(), refs.data_ptr(), self.rows, self.max_pages, page_size,
                            self.num_pages)

    def pages(self) -> Pages:
        """The pool's block table as the paged calls take it (row b = sequence b)."""
        return Pages(self.block_table, self.page_size, self.num_pages)

    def _work(self, n: int):
        import torch
        size = self.ws_bytes.get(n)
        if size is None:
            ws = C.c_size_t(0)
            _check(lib().tq_pages_workspace(C.byref(self.c), n, C.byref(ws)))
            size = self.ws_bytes[n] = ws.value
        return torch.empty(size, dtype=torch.uint8, device=self.device)


def _pool_outputs(pool: PagePool, n: int, out, size: int, workspace, stream):
    """An int32 output of `size` values and the workspace of n requests, where they are not given."""
    if stream is not None:
        return _allocated(stream, _pool_outputs, pool, n, out, size, workspace, None)
    return (pool.refs.new_empty(size) if out is None else out), (pool._work(n) if workspace is None else _scratch(workspace))


def pages_free(pool: PagePool, rows, lens, stream=None) -> None:
    """tq_pages_free: rows int32 [n] give back the pages of their first lens int32 [n] tokens."""
    n = rows.numel()
    _same_device(pool.device, rows, lens)
    _check(lib().tq_pages_free(C.byref(pool.c), _ints(rows, n, "rows"), _ints(lens, n, "lens"), n, _stream(stream)))


def pages_reserve(pool: PagePool, rows, old_lens, new_lens, shortfall=None, workspace=None, stream=None):
    """tq_pages_reserve: rows int32 [n] grow from old_lens to new_lens tokens.  Returns the device
    int32 [1] shortfall (0 = done)."""
    n = rows.numel()
    _same_device(pool.device, rows, old_lens, new_lens, shortfall, workspace)
    shortfall, ws = _pool_outputs(pool, n, shortfall, 1, workspace, stream)
    _check(lib().tq_pages_reserve(C.byref(pool.c), _ints(rows, n, "rows"), _ints(old_lens, n, "old_lens"),
                                  _ints(new_lens, n, "new_lens"), n, _ints(shortfall, 1, "shortfall"), ws.data_ptr(),
                                  ws.numel(), _stream(stream)))
    return shortfall


def pages_fork(pool: PagePool, src, dst, lens, shortfall=None, workspace=None, stream=None):
    """tq_pages_fork: row dst[i] continues from the first lens[i] tokens of row src[i] (int32 [n]
    each).  Returns the device int32 [1] shortfall (0 = done)."""
    n = src.numel()
    _same_device(pool.device, src, dst, lens, shortfall, workspace)
    shortfall, ws = _pool_outputs(pool, n, shortfall, 1, workspace, stream)
    _check(lib().tq_pages_fork(C.byref(pool.c), pool.pa, len(pool.arrays), _ints(src, n, "src"), _ints(dst, n, "dst"),
                               _ints(lens, n, "lens"), n, _ints(shortfall, 1, "shortfall"), ws.data_ptr(), ws.numel(),
                               _stream(stream)))
    return shortfall


def pages_compact(pool: PagePool, page_map=None, live=None, workspace=None, stream=None):
    """tq_pages_compact: live pages move to the lowest ids.  Returns page_map int32 [num_pages] (new
    id of each page, -1: free); live int32 [1], where given, receives their number."""
    _same_device(pool.device, page_map, live, workspace)
    page_map, ws = _pool_outputs(pool, 0, page_map, pool.num_pages, workspace, stream)
    if live is None:
        live = pool.refs.new_empty(1) if stream is None else _allocated(stream, pool.refs.new_empty, 1)
    _check(lib().tq_pages_compact(C.byref(pool.c), pool.pa, len(pool.arrays), _ints(page_map, pool.num_pages, "page_map"),
                                  _ints(live, 1, "live"), ws.data_ptr(), ws.numel(), _stream(stream)))
    return page_map


def pages_copy(pool: PagePool, src, dst, stream=None) -> None:
    """tq_pages_copy: page src[i] to page dst[i] (int32 [n]) in every array of the pool."""
    n = src.numel()
    _same_device(pool.device, src, dst)
    _check(lib().tq_pages_copy(pool.pa, len(pool.arrays), pool.num_pages, _ints(src, n, "src"), _ints(dst, n, "dst"), n,
                               _stream(stream)))


def get_status(stream=None) -> int:
    """Synchronize and return the device status code (0 = OK, 6 = a bounded wait timed out)."""
    return lib().tq_get_status(_stream(stream))


def set_wait_limit(polls: int) -> None:
    _check(lib().tq_set_wait_limit(polls))
