"""ctypes binding of ``liblla.so`` (the C ABI declared in ``include/lla.h``).

Argument marshalling only: torch tensors become device pointers and the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no fallback: a missing library raises at import time, and a non-zero
status raises ``LLAError`` with the library's message.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from functools import cached_property

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblla.so")

MODE_PER_HEAD = 0
MODE_2D = 1
STATUS_POSITION_RANGE = 1
STATUS_CTX_RANGE = 2
STATUS_SLOT_RANGE = 4
STATUS_TIMEOUT = 8
STATUS_PAGE_RANGE = 16
STATUS_PAGES_SHORT = 32
STATUS_NONFINITE = 64
STATUS_ROPE_TABLE = 128

ROPE_SCALES = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_TOO_SMALL, ERR_CUDA = 0, -1, -2, -3, -4


class LLAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"lla error {code}: {msg}")
        self.code = code


class CCfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("d_head", ctypes.c_int32),
                ("r_k", ctypes.c_int32), ("r_v", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("rope_base", ctypes.c_float), ("sm_scale", ctypes.c_float),
                ("d_rope", ctypes.c_int32)]


@dataclass(frozen=True)
class Cfg:
    T: int
    H: int
    d_head: int
    r_k: int
    r_v: int
    mode: int = MODE_PER_HEAD
    rope_base: float = 10000.0
    sm_scale: float = 0.0
    d_rope: int = 0          # decoupled RoPE: rotary dims (0 = the whole head)

    def c(self) -> CCfg:
        return CCfg(self.T, self.H, self.d_head, self.r_k, self.r_v, self.mode, self.rope_base,
                    self.sm_scale, self.d_rope)

    @cached_property
    def ref(self):
        """ctypes reference to the configuration's C struct (made once; the fields are frozen)."""
        return ctypes.byref(self.c())

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "ref"}


class CRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("orig_len", ctypes.c_int32),
                ("factor", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double)]


@dataclass(frozen=True)
class RopeScaling:
    """Frequencies of a stretched context (``lla_rope_scaling``)."""
    kind: str = "none"       # "none", "linear", "ntk" or "yarn"
    factor: float = 1.0
    orig_len: int = 1        # yarn: trained context
    beta_fast: float = 0.0   # yarn; 0 selects 32
    beta_slow: float = 0.0   # yarn; 0 selects 1

    def c(self) -> CRopeScaling:
        if self.kind not in ROPE_SCALES:
            raise ValueError(f"rope scaling kind {self.kind!r} not in {sorted(ROPE_SCALES)}")
        return CRopeScaling(ROPE_SCALES[self.kind], self.orig_len, self.factor, self.beta_fast,
                            self.beta_slow)


class CQ8Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page", ctypes.c_int32)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                      "g.build()\"` (nvcc, sm_100a). There is no CPU fallback.")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_CFG = ctypes.POINTER(CCfg)
_Q8 = ctypes.POINTER(CQ8Cache)
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t

SIGNATURES = {
    "lla_last_error": (ctypes.c_char_p, []),
    "lla_version": (ctypes.c_char_p, []),
    "lla_ratio": (ctypes.c_int, [_CFG, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "lla_cache_bytes": (ctypes.c_int, [_CFG, _I64, _I64, ctypes.c_int, ctypes.POINTER(_I64)]),
    "lla_codec_packed_bytes": (_SZ, [_CFG]),
    "lla_codec_pack": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "lla_rope_table_bytes": (_SZ, [_CFG, _I32]),
    "lla_rope_table": (ctypes.c_int, [_CFG, _I32, _P, _SZ, _P]),
    "lla_encode": (ctypes.c_int, [_CFG, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P]),
    "lla_decode_workspace_bytes": (_SZ, [_CFG, _I32, _I32]),
    "lla_decode_attn": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _P, _P, _SZ, _P]),
    "lla_decode_launches": (ctypes.c_int, [_CFG, _I32, _I32]),
    "lla_decode_attn_noalloc": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P,
                                               _P, _P, _P, _P, _P, _P, _P, _P]),
    "lla_evict_slot": (_I64, [_I32, _I32, _I64]),
    "lla_evict_append": (ctypes.c_int, [_I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "lla_full_kv_bytes": (_SZ, [_CFG, _I32, _I32]),
    "lla_full_rebuild": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                        _I64, _P, _P, _P, _P]),
    "lla_full_decode_workspace_bytes": (_SZ, [_CFG, _I32, _I32]),
    "lla_full_decode_launches": (ctypes.c_int, [_CFG, _I32, _I32]),
    "lla_full_decode_attn": (ctypes.c_int, [_CFG, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                            _P, _P, _P, _SZ, _P]),
    "lla_rope_table_scaled": (ctypes.c_int, [_CFG, ctypes.POINTER(CRopeScaling), _I32, _P, _SZ, _P]),
    "lla_rope_apply": (ctypes.c_int, [_CFG, _P, _I32, _I32, _I32, _I32, _I64, _I32, _P, _P, _I64,
                                      _P, _I64, _P, _P]),
    "lla_page_map": (ctypes.c_int, [_I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I64, _P, _P, _P,
                                    _P, _P]),
    "lla_q8_cache_bytes": (_SZ, [_CFG, _I32, _I32]),
    "lla_q8_append": (ctypes.c_int, [_CFG, _Q8, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32, _P,
                                     _P, _P, _I64, _P, _I64, _P, _P]),
    "lla_q8_append_rows": (ctypes.c_int, [_CFG, _Q8, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32,
                                          _P, _P, _P, _P, _I64, _P, _I64, _P, _P]),
    "lla_q8_read": (ctypes.c_int, [_CFG, _Q8, _I64, _P, _P, _P, _P, _P]),
    "lla_q8_decode_workspace_bytes": (_SZ, [_CFG, _I32, _I32]),
    "lla_q8_decode_launches": (ctypes.c_int, [_CFG, _I32, _I32]),
    "lla_q8_decode_attn": (ctypes.c_int, [_CFG, _Q8, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P,
                                          _P, _P, _P, _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def last_error() -> str:
    return lib.lla_last_error().decode()


def check(code: int) -> None:
    if code != OK:
        raise LLAError(code, last_error())
