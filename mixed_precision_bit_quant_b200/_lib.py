"""ctypes binding of libthrift (include/thrift.h): argument marshalling only.

Every step of the path runs in the library's CUDA kernels; this module only
allocates output tensors with PyTorch, passes device pointers and the
current stream, and turns status codes into exceptions.  There is no CPU
fallback: if the library is missing, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libthrift.so")

THRIFT_OK, THRIFT_ERR_INVALID, THRIFT_ERR_UNSUPPORTED, THRIFT_ERR_CUDA, THRIFT_ERR_TIMEOUT = range(5)
OP_QUANTIZE, OP_SELECT, OP_ATTN, OP_SELECT_VERTICAL, OP_QUANTIZE_MX = range(5)
FORMATS = ("nvfp4", "mxfp4")
QUANT_FIELDS = ["q_fp4", "q_sf", "q_sf_mma", "q_gs", "k_fp4", "k_sf", "k_sf_mma", "k_gs",
                "v_fp8t", "v_st", "v_exp"]
_FIELD_DTYPES = {"q_gs": torch.float32, "k_gs": torch.float32, "v_st": torch.bfloat16,
                 "v_exp": torch.int8}


class ThriftError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class QuantStruct(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in QUANT_FIELDS]


DECODE_FIELDS = ["kc", "ksc", "vc", "vsc"]


class DecodeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("L", ctypes.c_int32), ("d", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]


class DecodeCacheStruct(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in DECODE_FIELDS]


class Kv8Shape(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "Hq", "Hkv", "d", "page", "table_cols", "n", "max_q", "max_len",
                                              "dtype")]


class Kv8CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class Kv8Mask(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libthrift.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libthrift.so not found at {LIB_PATH}; build it with "
                               "`python -m mixed_precision_bit_quant_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, I32, U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_uint64
        SP = ctypes.POINTER(Shape)
        QP = ctypes.POINTER(QuantStruct)
        L.thrift_quant_bytes.argtypes = [SP, ctypes.c_int]
        L.thrift_quant_bytes.restype = S
        L.thrift_workspace_bytes.argtypes = [SP, ctypes.c_int]
        L.thrift_workspace_bytes.restype = S
        L.thrift_quantize.argtypes = [SP, P, P, P, QP, P, S, P]
        L.thrift_quantize.restype = ctypes.c_int
        L.thrift_select.argtypes = [SP, P, P, I32, I32, P, P, P, S, P]
        L.thrift_select.restype = ctypes.c_int
        L.thrift_quantize_mx.argtypes = [SP, P, P, P, QP, P, S, P]
        L.thrift_quantize_mx.restype = ctypes.c_int
        L.thrift_attn_fwd_mx.argtypes = [SP, QP, P, P, P, P, P, P]
        L.thrift_attn_fwd_mx.restype = ctypes.c_int
        L.thrift_select_vertical.argtypes = [SP, P, P, I32, I32, P, P, P, S, P]
        L.thrift_select_vertical.restype = ctypes.c_int
        L.thrift_attn_fwd.argtypes = [SP, QP, P, P, P, P, P, P, S, P]
        L.thrift_attn_fwd.restype = ctypes.c_int
        L.thrift_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        L.thrift_device_status.restype = ctypes.c_int
        L.thrift_status_string.argtypes = [ctypes.c_int]
        L.thrift_status_string.restype = ctypes.c_char_p
        L.thrift_debug_withhold_v_load.argtypes = [I32]
        L.thrift_debug_withhold_v_load.restype = ctypes.c_int
        DSP = ctypes.POINTER(DecodeShape)
        DCP = ctypes.POINTER(DecodeCacheStruct)
        L.thrift_decode_cache_bytes.argtypes = [DSP, ctypes.c_int]
        L.thrift_decode_cache_bytes.restype = S
        L.thrift_decode_workspace_bytes.argtypes = [DSP]
        L.thrift_decode_workspace_bytes.restype = S
        L.thrift_decode_quantize_cache.argtypes = [DSP, P, P, DCP, I32, I32, P]
        L.thrift_decode_quantize_cache.restype = ctypes.c_int
        L.thrift_decode_step.argtypes = [DSP, P, P, P, DCP, P, P, P, S, P]
        L.thrift_decode_step.restype = ctypes.c_int
        I64, KSP, KCP = ctypes.c_int64, ctypes.POINTER(Kv8Shape), ctypes.POINTER(Kv8CacheStruct)
        KMP = ctypes.POINTER(Kv8Mask)
        L.thrift_kv8_cache_bytes.argtypes = [I32, I32, I32, I32, ctypes.c_int]
        L.thrift_kv8_cache_bytes.restype = S
        L.thrift_kv8_append.argtypes = [KSP, KCP, P, I64, P, I64, P, P, P, P]
        L.thrift_kv8_append.restype = ctypes.c_int
        L.thrift_kv8_attn_workspace_bytes.argtypes = [KSP, KMP, ctypes.c_int]
        L.thrift_kv8_attn_workspace_bytes.restype = S
        L.thrift_kv8_attn.argtypes = [KSP, KMP, KCP, P, I64, P, P, P, P, P, P, I64, P, S, P]
        L.thrift_kv8_attn.restype = ctypes.c_int
        L.thrift_kv8_evict.argtypes = [KSP, KCP, P, P, P, I64, I32, I32, I32, KCP, P, I32, P, P, I64, P, P]
        L.thrift_kv8_evict.restype = ctypes.c_int
        L.thrift_probe_mma.argtypes = [I32, I32, I32, I32, ctypes.POINTER(ctypes.c_float), P, P]
        L.thrift_probe_mma.restype = ctypes.c_int
        L.thrift_launch_count.argtypes = []
        L.thrift_launch_count.restype = U64
        L.thrift_version.argtypes = []
        L.thrift_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().thrift_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != THRIFT_OK:
        raise ThriftError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The C ABI takes plain pointers and reads every buffer as dense and of the size
# its shape implies, so a strided view, another dtype, a host tensor or a buffer
# sized for another problem would be read or written out of bounds.  These checks
# run before any call into the library.
def _want(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    _on_device(t, name, device)


def _on_device(t: torch.Tensor, name: str, device=None) -> None:
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _check_qkv(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor] = None) -> None:
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q: expected a [B, Hq, N, d] tensor")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k: expected a [B, Hkv, N, d] tensor")
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    _want(q, "q", torch.bfloat16)
    _want(k, "k", torch.bfloat16, (B, Hkv, N, d), q.device)
    if v is not None:
        _want(v, "v", torch.bfloat16, (B, Hkv, N, d), q.device)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def make_shape(B, Hq, Hkv, N, d, causal, softmax_scale: float = 0.0) -> Shape:
    return Shape(int(B), int(Hq), int(Hkv), int(N), int(d), int(bool(causal)), float(softmax_scale))


def shape_of(q: torch.Tensor, k: torch.Tensor, causal: bool, softmax_scale: float = 0.0) -> Shape:
    B, Hq, N, d = q.shape
    return make_shape(B, Hq, k.shape[1], N, d, causal, softmax_scale)


def quant_bytes(shape: Shape, field: int) -> int:
    return int(lib().thrift_quant_bytes(ctypes.byref(shape), field))


def workspace_bytes(shape: Shape, op: int) -> int:
    return int(lib().thrift_workspace_bytes(ctypes.byref(shape), op))


@dataclasses.dataclass
class Quantized:
    """The quantised operands (device tensors), in thrift_quant field order, and their FP4 format."""
    tensors: dict
    fmt: str = "nvfp4"

    def struct(self) -> QuantStruct:
        return QuantStruct(*[self.tensors[f].data_ptr() for f in QUANT_FIELDS])

    def __getitem__(self, k):
        return self.tensors[k]


def _check_quantized(quant: "Quantized", shape: Shape, device) -> None:
    for idx, f in enumerate(QUANT_FIELDS):
        t = quant.tensors.get(f)
        if t is None:
            raise ValueError(f"quantized operands: missing {f}")
        _want(t, f, _FIELD_DTYPES.get(f, torch.uint8), device=device)
        if t.numel() * t.element_size() < quant_bytes(shape, idx):
            raise ValueError(f"{f}: {t.numel() * t.element_size()} bytes, the shape needs {quant_bytes(shape, idx)}")


def alloc_quantized(shape: Shape, device) -> Quantized:
    out = {}
    for idx, f in enumerate(QUANT_FIELDS):
        nbytes = quant_bytes(shape, idx)
        if nbytes == 0:
            raise ThriftError(THRIFT_ERR_INVALID, "thrift_quant_bytes")
        dt = _FIELD_DTYPES.get(f, torch.uint8)
        out[f] = torch.empty(nbytes // torch.empty((), dtype=dt).element_size(), dtype=dt, device=device)
    return Quantized(out)


def _workspace(shape: Shape, op: int, device) -> Optional[torch.Tensor]:
    n = workspace_bytes(shape, op)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device) if n > 0 else None


def _want_fmt(fmt: str) -> None:
    if fmt not in FORMATS:
        raise ValueError(f"fmt: {fmt!r}, expected one of {FORMATS}")


def quantize(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
             out: Optional[Quantized] = None, ws: Optional[torch.Tensor] = None, fmt: str = "nvfp4") -> Quantized:
    """thrift_quantize (fmt "nvfp4") or thrift_quantize_mx (fmt "mxfp4"): FP4 Q, K and FP8 V
    (all device tensors)."""
    _want_fmt(fmt)
    _check_qkv(q, k, v)
    shape = shape_of(q, k, causal)
    if out is None:
        out = alloc_quantized(shape, q.device)
    else:
        _check_quantized(out, shape, q.device)
    op = OP_QUANTIZE if fmt == "nvfp4" else OP_QUANTIZE_MX
    if ws is not None:
        _want(ws, "ws", torch.uint8, device=q.device)
        if ws.numel() < workspace_bytes(shape, op):
            raise ValueError(f"ws: {ws.numel()} bytes, the shape needs {workspace_bytes(shape, op)}")
    ws = ws if ws is not None else _workspace(shape, op, q.device)
    st = out.struct()
    fn = lib().thrift_quantize if fmt == "nvfp4" else lib().thrift_quantize_mx
    _check(fn(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(st), _ptr(ws),
              0 if ws is None else ws.numel(), _stream()),
           "thrift_quantize" if fmt == "nvfp4" else "thrift_quantize_mx")
    out.fmt = fmt
    return out


def select(q: torch.Tensor, k: torch.Tensor, causal: bool, budget_bp: int = 500, budget_tiles: int = 0,
           mask: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = None, mode: str = "score"):
    """thrift_select (mode "score") or thrift_select_vertical (mode "vertical"):
    returns (mask[B,Hq,T,W] int32 view of the uint32 words, counts[B,Hq,T])."""
    if mode not in ("score", "vertical"):
        raise ValueError(f"mode: {mode!r}, expected 'score' or 'vertical'")
    _check_qkv(q, k)
    shape = shape_of(q, k, causal)
    B, Hq, N, _ = q.shape
    T = (N + 127) // 128
    W = (T + 31) // 32
    if mask is None:
        mask = torch.empty((B, Hq, T, W), dtype=torch.int32, device=q.device)
    else:
        _want(mask, "mask", torch.int32, (B, Hq, T, W), q.device)
    if counts is None:
        counts = torch.empty((B, Hq, T), dtype=torch.int32, device=q.device)
    else:
        _want(counts, "counts", torch.int32, (B, Hq, T), q.device)
    op = OP_SELECT if mode == "score" else OP_SELECT_VERTICAL
    if ws is not None:
        _want(ws, "ws", torch.uint8, device=q.device)
    ws = ws if ws is not None else _workspace(shape, op, q.device)
    fn = lib().thrift_select if mode == "score" else lib().thrift_select_vertical
    _check(fn(ctypes.byref(shape), _ptr(q), _ptr(k), int(budget_bp), int(budget_tiles), _ptr(mask), _ptr(counts),
              _ptr(ws), 0 if ws is None else ws.numel(), _stream()),
           "thrift_select" if mode == "score" else "thrift_select_vertical")
    return mask, counts


def attn_fwd(q: torch.Tensor, k: torch.Tensor, quant: Quantized, mask: torch.Tensor, causal: bool,
             softmax_scale: float = 0.0, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             want_lse: bool = False):
    """thrift_attn_fwd (NVFP4 operands) or thrift_attn_fwd_mx (MXFP4 operands, by quant.fmt):
    returns (o[B,Hq,N,d] bf16, lse[B,Hq,N] fp32 or None)."""
    _want_fmt(quant.fmt)
    _check_qkv(q, k)
    shape = shape_of(q, k, causal, softmax_scale)
    B, Hq, N, _ = q.shape
    T = (N + 127) // 128
    _check_quantized(quant, shape, q.device)
    _want(mask, "mask", torch.int32, (B, Hq, T, (T + 31) // 32), q.device)
    if o is None:
        o = torch.empty_like(q)
    else:
        _want(o, "o", torch.bfloat16, tuple(q.shape), q.device)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    elif lse is not None:
        _want(lse, "lse", torch.float32, tuple(q.shape[:3]), q.device)
    st = quant.struct()
    if quant.fmt == "nvfp4":
        _check(lib().thrift_attn_fwd(ctypes.byref(shape), ctypes.byref(st), _ptr(q), _ptr(k), _ptr(mask),
                                     _ptr(o), _ptr(lse), None, 0, _stream()), "thrift_attn_fwd")
    else:
        _check(lib().thrift_attn_fwd_mx(ctypes.byref(shape), ctypes.byref(st), _ptr(q), _ptr(k), _ptr(mask),
                                        _ptr(o), _ptr(lse), _stream()), "thrift_attn_fwd_mx")
    return o, lse


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool, budget_bp: int = 500,
              budget_tiles: int = 0, softmax_scale: float = 0.0, want_lse: bool = False, mode: str = "score",
              fmt: str = "nvfp4"):
    """The whole forward pass: quantize (NVFP4 or MXFP4) -> select (score or vertical mode) ->
    fused mixed attention."""
    quant = quantize(q, k, v, causal, fmt=fmt)
    mask, _ = select(q, k, causal, budget_bp, budget_tiles, mode=mode)
    return attn_fwd(q, k, quant, mask, causal, softmax_scale, want_lse=want_lse)


def decode_shape(q: torch.Tensor, k: torch.Tensor, softmax_scale: float = 0.0) -> DecodeShape:
    B, Hq, d = q.shape
    return DecodeShape(int(B), int(Hq), int(k.shape[1]), int(k.shape[2]), int(d), float(softmax_scale))


def _check_decode_kv(k: torch.Tensor, v: torch.Tensor) -> None:
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k: expected a [B, Hkv, L, d] tensor")
    _want(k, "k", torch.bfloat16)
    _want(v, "v", torch.bfloat16, tuple(k.shape), k.device)


def decode_quantize_cache(k: torch.Tensor, v: torch.Tensor, cache: Optional[dict] = None, t_begin: int = 0,
                          t_end: Optional[int] = None) -> dict:
    """thrift_decode_quantize_cache: per-token MXFP4 K / MXFP8 V of cache rows [t_begin, t_end).
    Returns the cache dict (kc, ksc, vc, vsc uint8 device tensors), allocated when not given."""
    _check_decode_kv(k, v)
    B, Hkv, L, d = k.shape
    shape = DecodeShape(int(B), int(Hkv), int(Hkv), int(L), int(d), 0.0)
    if cache is None:
        cache = {}
        for idx, f in enumerate(DECODE_FIELDS):
            n = int(lib().thrift_decode_cache_bytes(ctypes.byref(shape), idx))
            if n == 0:
                raise ThriftError(THRIFT_ERR_INVALID, "thrift_decode_cache_bytes")
            cache[f] = torch.empty(n, dtype=torch.uint8, device=k.device)
    else:
        for idx, f in enumerate(DECODE_FIELDS):
            _want(cache[f], f, torch.uint8, device=k.device)
            if cache[f].numel() < int(lib().thrift_decode_cache_bytes(ctypes.byref(shape), idx)):
                raise ValueError(f"{f}: buffer too small for the cache shape")
    st = DecodeCacheStruct(*[cache[f].data_ptr() for f in DECODE_FIELDS])
    t_end = L if t_end is None else t_end
    _check(lib().thrift_decode_quantize_cache(ctypes.byref(shape), _ptr(k), _ptr(v), ctypes.byref(st),
                                              int(t_begin), int(t_end), _stream()), "thrift_decode_quantize_cache")
    return cache


def decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: dict, softmax_scale: float = 0.0,
                o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, want_lse: bool = False,
                ws: Optional[torch.Tensor] = None):
    """thrift_decode_step: q[B,Hq,d] against the cache -> (o[B,Hq,d] bf16, lse[B,Hq] fp32 or None)."""
    _check_decode_kv(k, v)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a [B, Hq, d] tensor")
    _want(q, "q", torch.bfloat16, device=k.device)
    B, Hkv, L, d = k.shape
    if q.shape[0] != B or q.shape[2] != d:
        raise ValueError(f"q: shape {tuple(q.shape)} does not match the cache {tuple(k.shape)}")
    shape = decode_shape(q, k, softmax_scale)
    for idx, f in enumerate(DECODE_FIELDS):
        _want(cache[f], f, torch.uint8, device=k.device)
        if cache[f].numel() < int(lib().thrift_decode_cache_bytes(ctypes.byref(shape), idx)):
            raise ValueError(f"{f}: buffer too small for the cache shape")
    if o is None:
        o = torch.empty_like(q)
    else:
        _want(o, "o", torch.bfloat16, tuple(q.shape), k.device)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=k.device)
    elif lse is not None:
        _want(lse, "lse", torch.float32, tuple(q.shape[:2]), k.device)
    need = int(lib().thrift_decode_workspace_bytes(ctypes.byref(shape)))
    if need == 0:
        raise ThriftError(THRIFT_ERR_UNSUPPORTED, "thrift_decode_workspace_bytes")
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=k.device)
    else:
        _want(ws, "ws", torch.uint8, device=k.device)
    st = DecodeCacheStruct(*[cache[f].data_ptr() for f in DECODE_FIELDS])
    _check(lib().thrift_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(st), _ptr(o),
                                    _ptr(lse), _ptr(ws), ws.numel(), _stream()), "thrift_decode_step")
    return o, lse


# ---------------------------------------------------------------------------
# The paged 8-bit cache.  These calls run once per layer and token, so their checks
# touch each tensor once; they follow the tensors' device, not the current one.
# ---------------------------------------------------------------------------
_KV8_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class Kv8Cache:
    """A pool of 8-bit pages: k, v uint8 [num_pages, Hkv, page, d] (e4m3 codes), ks, vs uint8
    [num_pages, Hkv] (the exponent of a page and kv head, plus 127)."""

    __slots__ = ("k", "v", "ks", "vs", "num_pages", "Hkv", "page", "d", "device", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, ks: torch.Tensor, vs: torch.Tensor):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k: expected a [num_pages, Hkv, page, d] tensor")
        _want(k, "k", torch.uint8)
        _want(v, "v", torch.uint8, tuple(k.shape), k.device)
        _want(ks, "ks", torch.uint8, tuple(k.shape[:2]), k.device)
        _want(vs, "vs", torch.uint8, tuple(k.shape[:2]), k.device)
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.num_pages, self.Hkv, self.page, self.d = (int(x) for x in k.shape)
        if int(lib().thrift_kv8_cache_bytes(self.num_pages, self.Hkv, self.page, self.d, 0)) == 0:
            raise ThriftError(THRIFT_ERR_UNSUPPORTED, "thrift_kv8_cache_bytes")
        self.device = k.device
        self._ref = ctypes.byref(Kv8CacheStruct(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                                                self.num_pages))


def kv8_alloc(num_pages: int, Hkv: int, page: int, d: int, device) -> Kv8Cache:
    """An empty pool of pages."""
    k = torch.empty((num_pages, Hkv, page, d), dtype=torch.uint8, device=device)
    ks = torch.empty((num_pages, Hkv), dtype=torch.uint8, device=device)
    return Kv8Cache(k, torch.empty_like(k), ks, torch.empty_like(ks))


def _want_kv8(cache, name: str) -> None:
    if not isinstance(cache, Kv8Cache):
        raise TypeError(f"{name}: expected a Kv8Cache")


def _kv8_tokens(x: torch.Tensor, name: str, heads: int, d: int, device) -> int:
    """Checks packed rows [n, heads, d] whose tokens may be strided; returns the token stride."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name}: expected a [n, heads, d] tensor")
    if x.dtype not in _KV8_DTYPES:
        raise ValueError(f"{name}: dtype {x.dtype}, expected torch.bfloat16 or torch.float16")
    n, h, w = x.shape
    if w != d or (heads and h != heads):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected (n, {heads or 'Hq'}, {d})")
    if x.device != device or device.type != "cuda":
        _on_device(x, name, device)
    if x.is_contiguous():
        return h * d
    st, sh, sd = x.stride()
    if sd != 1 or (sh != d and h != 1) or (st % 8 and n != 1):
        raise ValueError(f"{name}: heads and channels must be contiguous and the token stride a multiple of 8")
    return h * d if n == 1 else st


def _kv8_ints(t: torch.Tensor, name: str, shape, device) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous torch.int32 tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.device != device or device.type != "cuda":
        _on_device(t, name, device)
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _kv8_args(B, Hq, Hkv, d, page, cols, n, max_q, max_len, dtype, window=0, sinks=0, softmax_scale=0.0, with_w=None):
    """The structs of a call with these numbers, as they are passed, and (for attention) the bytes of workspace.
    They depend on nothing else, so a serving loop makes them once."""
    numbers = (B, Hq, Hkv, d, page, cols, n, max_q, max_len, dtype)
    for x in numbers + (window, sinks):
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{x}: does not fit 32 bits")
    shape, mask = ctypes.byref(Kv8Shape(*numbers)), ctypes.byref(Kv8Mask(window, sinks, softmax_scale))
    need = 0 if with_w is None else int(lib().thrift_kv8_attn_workspace_bytes(shape, mask, with_w))
    return shape, mask, need


def _kv8_rows(cache: Kv8Cache, table, lens, cu, n, max_q, max_len):
    """B, the columns of table, the bounds, and the pointers of table, lens and cu."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table: expected a [B, pages] tensor")
    B, cols = table.shape
    dev = cache.device
    tp = _kv8_ints(table, "table", (B, cols), dev)
    lp = _kv8_ints(lens, "lens", (B,), dev)
    cp = None if cu is None else _kv8_ints(cu, "cu", (B + 1,), dev)
    if cu is None and n != B:
        raise ValueError(f"{n} rows for {B} sequences: without cu each sequence has one new token")
    max_q = (1 if cu is None else n) if max_q is None else int(max_q)
    return B, cols, max_q, cols * cache.page if max_len is None else int(max_len), tp, lp, cp


# The current stream's handle without a Stream object around it, which costs 3 us a call --
# as much as the launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _kv8_call(fn, what: str, device, *args) -> None:
    """The call on the device's current stream, with the device current while it launches."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != THRIFT_OK:
        raise ThriftError(status, what)


def kv8_append(cache: Kv8Cache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
               cu: Optional[torch.Tensor] = None, max_q: Optional[int] = None) -> None:
    """thrift_kv8_append: quantise the new tokens k, v [n, Hkv, d] (bf16 or fp16, tokens may be strided) into
    the pages of their sequences.  table int32 [B, pages]; lens int32 [B], the new tokens included; cu int32
    [B + 1], sequence b's rows being cu[b] .. cu[b + 1] (None: one token each); max_q bounds a sequence's new
    tokens (default n, or 1 without cu)."""
    _want_kv8(cache, "cache")
    ks = _kv8_tokens(k, "k", cache.Hkv, cache.d, cache.device)
    vs = _kv8_tokens(v, "v", cache.Hkv, cache.d, cache.device)
    if v.dtype is not k.dtype or v.shape != k.shape:
        raise ValueError("v: expected the dtype and shape of k")
    n = k.shape[0]
    B, cols, max_q, max_len, tp, lp, cp = _kv8_rows(cache, table, lens, cu, n, max_q, None)
    shape, _, _ = _kv8_args(B, cache.Hkv, cache.Hkv, cache.d, cache.page, cols, n, max_q, max_len, _KV8_DTYPES[k.dtype])
    _kv8_call(lib().thrift_kv8_append, "thrift_kv8_append", cache.device, shape, cache._ref, k.data_ptr(), ks,
              v.data_ptr(), vs, tp, lp, cp)


def _kv8_weights(w: torch.Tensor, name: str, B: int, Hkv: int, device) -> int:
    if not isinstance(w, torch.Tensor) or w.dim() != 3 or w.shape[0] != B or w.shape[1] != Hkv:
        raise ValueError(f"{name}: expected a [B, Hkv, columns] tensor for B = {B}, Hkv = {Hkv}")
    if w.dtype is not torch.float32 or not w.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous torch.float32 tensor")
    if w.device != device or device.type != "cuda":
        _on_device(w, name, device)
    return w.shape[2]


def kv8_attention(q: torch.Tensor, cache: Kv8Cache, table: torch.Tensor, lens: torch.Tensor,
                  cu: Optional[torch.Tensor] = None, max_q: Optional[int] = None, max_len: Optional[int] = None,
                  window: int = 0, sinks: int = 0, softmax_scale: float = 0.0,
                  weights: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, want_lse: bool = False, ws: Optional[torch.Tensor] = None):
    """thrift_kv8_attn: attention of the new tokens' queries q [n, Hq, d] (bf16 or fp16, tokens may be strided)
    over the cache that already holds those tokens -> (o [n, Hq, d], lse fp32 [n, Hq] or None).  Causal; with
    window > 0 a query at position p sees t > p - window and the first `sinks` tokens.  table, lens, cu, max_q as
    for kv8_append, and max_q picks the kernel: a batch of single tokens that has a cu should pass 1.  max_len bounds
    lens (default: what the table holds).  weights: fp32 [B, Hkv, >= max_len], to which each token's attention
    weights are added."""
    _want_kv8(cache, "cache")
    qs = _kv8_tokens(q, "q", 0, cache.d, cache.device)
    n, Hq, d = q.shape
    B, cols, max_q, max_len, tp, lp, cp = _kv8_rows(cache, table, lens, cu, n, max_q, max_len)
    dev = cache.device
    w_cols, wp = 0, None
    if weights is not None:
        w_cols, wp = _kv8_weights(weights, "weights", B, cache.Hkv, dev), weights.data_ptr()
    shape, mask, need = _kv8_args(B, Hq, cache.Hkv, d, cache.page, cols, n, max_q, max_len, _KV8_DTYPES[q.dtype],
                                  window, sinks, softmax_scale, wp is not None)
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _want(o, "o", q.dtype, (n, Hq, d), dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, (n, Hq), dev)
    elif want_lse:
        lse = q.new_empty((n, Hq), dtype=torch.float32)
    if ws is not None:
        _want(ws, "ws", torch.uint8, device=dev)
        if ws.numel() < need:
            raise ValueError(f"ws: {ws.numel()} bytes, the call needs {need}")
    elif need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _kv8_call(lib().thrift_kv8_attn, "thrift_kv8_attn", dev, shape, mask, cache._ref, q.data_ptr(), qs, tp, lp, cp,
              o.data_ptr(), None if lse is None else lse.data_ptr(), wp, w_cols, None if ws is None else ws.data_ptr(),
              need)
    return o, lse


def kv8_attention_workspace(q: torch.Tensor, cache: Kv8Cache, table: torch.Tensor, lens: torch.Tensor,
                            cu: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                            max_len: Optional[int] = None, window: int = 0, sinks: int = 0,
                            weights: Optional[torch.Tensor] = None) -> int:
    """thrift_kv8_attn_workspace_bytes of a kv8_attention call with these arguments."""
    _want_kv8(cache, "cache")
    _kv8_tokens(q, "q", 0, cache.d, cache.device)
    B, cols, max_q, max_len, _, _, _ = _kv8_rows(cache, table, lens, cu, q.shape[0], max_q, max_len)
    return _kv8_args(B, q.shape[1], cache.Hkv, cache.d, cache.page, cols, q.shape[0], max_q, max_len,
                     _KV8_DTYPES[q.dtype], window, sinks, 0.0, weights is not None)[2]


def kv8_evict(cache: Kv8Cache, table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor, dst: Kv8Cache,
              dst_table: torch.Tensor, dst_weights: torch.Tensor, keep: int, sinks: int = 0, recent: int = 0,
              max_len: Optional[int] = None, dst_lens: Optional[torch.Tensor] = None,
              kept: Optional[torch.Tensor] = None):
    """thrift_kv8_evict: copy every sequence's and kv head's `keep` tokens with the largest weights (the first
    `sinks` and the last `recent` always among them) to the pages dst_table of dst -> (dst_lens int32 [B], kept
    int32 [B, Hkv, keep], the old positions, -1 past the last).  dst may be `cache` if its pages dst_table are
    none that the call reads; dst_weights must not overlap weights, nor dst_lens lens."""
    _want_kv8(cache, "cache")
    _want_kv8(dst, "dst")
    dev, Hkv = cache.device, cache.Hkv
    n = table.shape[0] if isinstance(table, torch.Tensor) else 0
    B, cols, max_q, max_len, tp, lp, _ = _kv8_rows(cache, table, lens, None, n, 1, max_len)
    shape, _, _ = _kv8_args(B, Hkv, Hkv, cache.d, cache.page, cols, B, max_q, max_len, 0)
    if (dst.Hkv, dst.page, dst.d, dst.device) != (Hkv, cache.page, cache.d, dev):
        raise ValueError("dst: expected a Kv8Cache with the heads, page, d and device of cache")
    if not isinstance(dst_table, torch.Tensor) or dst_table.dim() != 2:
        raise ValueError("dst_table: expected a [B, pages] tensor")
    dtp = _kv8_ints(dst_table, "dst_table", (B, dst_table.shape[1]), dev)
    w_cols = _kv8_weights(weights, "weights", B, Hkv, dev)
    dw_cols = _kv8_weights(dst_weights, "dst_weights", B, Hkv, dev)
    a, b = weights.data_ptr(), dst_weights.data_ptr()
    if a < b + 4 * dst_weights.numel() and b < a + 4 * weights.numel():
        raise ValueError("dst_weights: must not overlap weights")
    keep, sinks, recent = int(keep), int(sinks), int(recent)
    if not (-2 ** 31 <= keep < 2 ** 31 and -2 ** 31 <= sinks < 2 ** 31 and -2 ** 31 <= recent < 2 ** 31):
        raise ValueError("keep, sinks, recent: must fit 32 bits")
    if dst_lens is None:
        dst_lens = torch.empty_like(lens)
        lens_ptr = dst_lens.data_ptr()
    else:
        lens_ptr = _kv8_ints(dst_lens, "dst_lens", (B,), dev)
        if -4 * B < lens_ptr - lp < 4 * B:
            raise ValueError("dst_lens: must not overlap lens")
    if kept is None:
        kept = torch.empty((B, Hkv, max(keep, 0)), dtype=torch.int32, device=dev)
        kept_ptr = kept.data_ptr()
    else:
        kept_ptr = _kv8_ints(kept, "kept", (B, Hkv, keep), dev)
    _kv8_call(lib().thrift_kv8_evict, "thrift_kv8_evict", dev, shape, cache._ref, tp, lp, a, w_cols, keep, sinks,
              recent, dst._ref, dtp, dst_table.shape[1], lens_ptr, b, dw_cols, kept_ptr)
    return dst_lens, kept


def device_status() -> tuple:
    """Synchronise the current stream and read (status, raw word) of the device watchdog."""
    w = ctypes.c_uint32(0)
    s = lib().thrift_device_status(_stream(), ctypes.byref(w))
    return int(s), int(w.value)


def debug_withhold_v_load(tile: int) -> None:
    """Watchdog test hook: later attention launches skip key tile `tile`'s V load (-1: off)."""
    _check(lib().thrift_debug_withhold_v_load(int(tile)), "thrift_debug_withhold_v_load")


def probe_mma(kind: int, n: int = 128, iters: int = 20000, ctas: Optional[int] = None) -> dict:
    """thrift_probe_mma: dense tensor-core rate of one MMA form (kind 0 NVFP4, 1 e4m3 with A in
    tensor memory, 2 BF16), one CTA per SM by default.  Returns TFLOP/s and cycle figures."""
    if ctas is None:
        ctas = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    cyc = torch.zeros(ctas, dtype=torch.int64, device="cuda")
    ms = ctypes.c_float(0.0)
    _check(lib().thrift_probe_mma(int(kind), int(n), int(iters), int(ctas), ctypes.byref(ms), cyc.data_ptr(),
                                  _stream()), "thrift_probe_mma")
    flops = 2.0 * 128 * n * 128 * iters * ctas
    c = cyc.cpu().double()
    return {"tflops": flops / (ms.value * 1e-3) / 1e12, "ms": float(ms.value),
            "flop_per_clk_per_sm": 2.0 * 128 * n * 128 * iters / float(c.max()),
            "cycles_max": float(c.max()), "ctas": ctas, "iters": iters}


def launch_count() -> int:
    return int(lib().thrift_launch_count())


def version() -> str:
    return lib().thrift_version().decode()
