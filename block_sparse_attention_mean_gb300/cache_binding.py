"""ctypes binding of attention over packed sequences and paged caches (include/bsa_cache.h): one Python function per
entry point with the same name (argument marshalling only), plus helpers that take tensors, check that they go
together and allocate outputs and workspaces with torch.

As in ``binding`` there is no fallback, and the helpers read the device error word after the call unless ``check`` is
false: a loop of calls, or one captured into a graph, passes check=False and a workspace, and looks at it with
``cache_check`` when it likes. As in ``block_binding`` they run on the tensors' device and on ``stream`` (that device's
current stream by default), record nothing for autograd, and refuse a tensor that requires a gradient while gradients
are recorded, or carries a tangent.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad as _forward_ad

from . import binding
from .binding import BF16, ERR_DTYPE, ERR_INVALID_ARG, ERR_SHAPE, BsaError, _check, _ptr, _stream
from .block_binding import _current_stream as _block_current_stream
from .block_binding import _cuda_device, _elsewhere, _no_tangents, _view

CACHE_BF16 = 0
CACHE_E4M3 = 1
PAGE_SIZES = (16, 32, 64, 128, 256)
ROWS_WORKSPACE = 8192  # BSA_CACHE_ROWS_WORKSPACE

# every symbol declared in include/bsa_cache.h
EXPORTS = ("bsa_cache_write", "bsa_cache_read", "bsa_cache_attention", "bsa_prompt_attention",
           "bsa_cache_workspace_size")

_I64 = ctypes.c_int64


class KvCacheStruct(ctypes.Structure):
    """Mirror of bsa_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("kind", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
                ("d", ctypes.c_int)]


class PageTable(ctypes.Structure):
    """Mirror of bsa_page_table."""
    _fields_ = [("pages", ctypes.c_void_p), ("stride", _I64), ("B", ctypes.c_int), ("width", ctypes.c_int)]


class Packed(ctypes.Structure):
    """Mirror of bsa_packed."""
    _fields_ = [("ptr", ctypes.c_void_p), ("token", _I64), ("head", _I64)]


_lib = None


def load():
    """Load libbsa.so (raises OSError if it was not built) with this header's signatures."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.bsa_cache_write.argtypes = [P, P, P, I, I, P, P, P, P, SZ, P]
    lib.bsa_cache_read.argtypes = [P, P, P, P, P, I, I, P, SZ, P]
    lib.bsa_cache_attention.argtypes = [P, P, I, I, P, P, F, P, P, P, SZ, P]
    lib.bsa_prompt_attention.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, I, F, P, P, P, SZ, P]
    lib.bsa_cache_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(SZ)]
    for name in EXPORTS:
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _ref(s):
    return ctypes.byref(s) if s is not None else None


# ------------------------------------------------------------------ C ABI mirror


def bsa_cache_write(cache: Optional[KvCacheStruct], k: Optional[Packed], v: Optional[Packed], dt: int, T: int,
                    table: Optional[PageTable], kv_lens, cu, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_cache_write(_ref(cache), _ref(k), _ref(v), dt, T, _ref(table), _ptr(kv_lens), _ptr(cu),
                                  _ptr(workspace), workspace_bytes, _stream(stream)), "bsa_cache_write")


def bsa_cache_read(cache: Optional[KvCacheStruct], table: Optional[PageTable], cu, k: Optional[Packed],
                   v: Optional[Packed], dt: int, T: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_cache_read(_ref(cache), _ref(table), _ptr(cu), _ref(k), _ref(v), dt, T, _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "bsa_cache_read")


def bsa_cache_attention(cache: Optional[KvCacheStruct], q: Optional[Packed], dt: int, H: int,
                        table: Optional[PageTable], kv_lens, scale: float, O: Optional[Packed], LSE, workspace,
                        workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_cache_attention(_ref(cache), _ref(q), dt, H, _ref(table), _ptr(kv_lens), scale, _ref(O),
                                      _ptr(LSE), _ptr(workspace), workspace_bytes, _stream(stream)),
           "bsa_cache_attention")


def bsa_prompt_attention(q: Optional[Packed], k: Optional[Packed], v: Optional[Packed], dt: int, T_q: int, T_k: int,
                         B: int, H: int, Hk: int, d: int, cu_q, cu_k, causal: int, scale: float, O: Optional[Packed],
                         LSE, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_prompt_attention(_ref(q), _ref(k), _ref(v), dt, T_q, T_k, B, H, Hk, d, _ptr(cu_q), _ptr(cu_k),
                                       causal, scale, _ref(O), _ptr(LSE), _ptr(workspace), workspace_bytes,
                                       _stream(stream)), "bsa_prompt_attention")


def bsa_cache_workspace_size(T: int, B: int, H: int, Hk: int, d: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().bsa_cache_workspace_size(T, B, H, Hk, d, ctypes.byref(out)), "bsa_cache_workspace_size")
    return out.value


# ------------------------------------------------------------------ helpers
#
# As in block_binding, descriptors go as bytes in the structures' layout, and messages wait for a failure: a tensor is
# looked at in as few calls as tell that it is right, and _view says what is wrong with it if it is not.

_CACHE = struct.Struct("4P5i4x")
_TABLE = struct.Struct("Pq2i")
_PACKED = struct.Struct("Pqq")
_BF16, _E4M3, _INT, _FP32, _UINT8 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.uint8
_grad_enabled = torch.is_grad_enabled
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _block_current_stream
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class KvCache(NamedTuple):
    """Pages of keys and values: k, v [pages, key heads, page size, d], bf16, or float8_e4m3fn with the bytes k_exp, v_exp
    [pages, key heads, page size] of their exponents: a row is data * 2 ** (exp - 127)."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: Optional[torch.Tensor] = None
    v_exp: Optional[torch.Tensor] = None


def kv_cache(n_pages: int, page_size: int, kv_heads: int, d: int, kind: str = "bf16", device="cuda") -> KvCache:
    """A cache of zeros. kind: "bf16", or "e4m3" for 8 bits a channel and one exponent a row."""
    if kind not in ("bf16", "e4m3"):
        raise BsaError(ERR_INVALID_ARG, f"kv_cache: kind {kind!r}")
    shape = (n_pages, kv_heads, page_size)
    dtype = _BF16 if kind == "bf16" else torch.float8_e4m3fn
    k, v = (torch.zeros(*shape, d, dtype=dtype, device=device) for _ in range(2))
    if kind == "bf16":
        return KvCache(k, v)
    return KvCache(k, v, *(torch.full(shape, 27, dtype=torch.uint8, device=device) for _ in range(2)))


def cache_workspace(tokens: int, sequences: int, heads: int, kv_heads: int, d: int, device="cuda") -> torch.Tensor:
    """Device workspace of the four calls, for at most so many query tokens of so many sequences a call; the part that has
    to be zero in a new one is."""
    ws = torch.empty(bsa_cache_workspace_size(tokens, sequences, heads, kv_heads, d), dtype=torch.uint8, device=device)
    ws[:ROWS_WORKSPACE].zero_()
    return ws


def _rows_workspace(device) -> torch.Tensor:
    return torch.zeros(ROWS_WORKSPACE, dtype=torch.uint8, device=device)


def cache_check(ws: torch.Tensor, stream=None) -> None:
    """Raises what the calls that used this workspace met on the device (and clears it). Waits for the stream."""
    device = _cuda_device(ws, "cache_check")
    with torch.cuda.device(device):
        _check(binding.bsa_check_device_error(ws, stream), "cache (device)")


def _contiguous(t: torch.Tensor, shape, dtype, device, what: str, name: str) -> int:
    """Address of a contiguous tensor of this shape, dtype and device."""
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device and
            (dtype is _INT or not (t.requires_grad and _grad_enabled()))):
        _view(t, shape, dtype, device, what, name)
        raise BsaError(ERR_INVALID_ARG, f"{what}: {name} must be contiguous")
    return t.data_ptr()


def _packed(t: torch.Tensor, shape, device, what: str, name: str) -> bytes:
    """bsa_packed of a bf16 tensor of this shape and device, channels contiguous."""
    s = t.stride()
    if t.dtype is _BF16 and t.shape == shape and s[2] == 1 and t.device == device and not (t.requires_grad and _grad_enabled()):
        return _PACKED.pack(t.data_ptr(), s[0], s[1])
    at, s = _view(t, shape, _BF16, device, what, name)
    return _PACKED.pack(at, s[0], s[1])


def _cache_args(cache: KvCache, what: str):
    """(descriptor, device, key heads, d)"""
    k, v, k_exp, v_exp = cache
    device = _cuda_device(k, what)
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4:
        raise BsaError(ERR_SHAPE, f"{what}: a cache of {len(shape)} dimensions, expected 4")
    if dtype is _BF16:
        kind, ke, ve = CACHE_BF16, 0, 0
        if k_exp is not None or v_exp is not None:
            raise BsaError(ERR_INVALID_ARG, f"{what}: a bf16 cache has no exponents")
    elif dtype is _E4M3:
        if k_exp is None or v_exp is None:
            raise BsaError(ERR_INVALID_ARG, f"{what}: an e4m3 cache needs its exponents")
        kind, rows = CACHE_E4M3, shape[:3]
        ke = _contiguous(k_exp, rows, _UINT8, device, what, "k_exp")
        ve = _contiguous(v_exp, rows, _UINT8, device, what, "v_exp")
    else:
        raise BsaError(ERR_DTYPE, f"{what}: cache dtype {dtype}")
    at = _contiguous(k, shape, dtype, device, what, "cache k"), _contiguous(v, shape, dtype, device, what, "cache v")
    n_pages, heads, page_size, d = shape
    return _CACHE.pack(*at, ke, ve, kind, n_pages, page_size, heads, d), device, heads, d


def _table_args(table: torch.Tensor, device, what: str):
    """(descriptor, B)"""
    shape = table.shape
    if len(shape) != 2:
        raise BsaError(ERR_SHAPE, f"{what}: a page table of {len(shape)} dimensions, expected 2")
    s = table.stride()
    if not (table.dtype is _INT and s[1] == 1 and table.device == device):
        _view(table, shape, _INT, device, what, "table")
    return _TABLE.pack(table.data_ptr(), s[0], *shape), shape[0]


def _call(what: str, fn, device: torch.device, ws: torch.Tensor, check: bool, *args) -> None:
    """fn(*args, the workspace and its bytes, the device's current stream) with `device` current."""
    if not (ws.device == device and ws.is_contiguous()):
        raise BsaError(ERR_INVALID_ARG, f"{what}: the workspace must be contiguous and on {device}")
    index = device.index
    stream = _current_stream(index)
    if index == _current_device():
        code = fn(*args, ws.data_ptr(), ws.nbytes, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, ws.data_ptr(), ws.nbytes, stream)
    _check(code, what)
    if check:
        with torch.cuda.device(device):
            _check(binding.bsa_check_device_error(ws), what + " (device)")


def cache_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, kv_lens: torch.Tensor,
                cu: Optional[torch.Tensor] = None, *, ws: Optional[torch.Tensor] = None, stream=None,
                check: bool = True) -> None:
    """Run bsa_cache_write: k, v [T, key heads, d] become the last tokens of their sequences, which hold kv_lens [B]
    tokens with them. Sequence b's are cu[b] .. cu[b + 1] - 1 (None: one a sequence); table [B, width] names its pages."""
    what = "cache_write"
    if stream is not None and (there := _elsewhere(stream, k, what)):
        with there:
            return cache_write(cache, k, v, table, kv_lens, cu, ws=ws, check=check)
    if _forward_ad._current_level >= 0:
        _no_tangents(what, k, v, *cache[:2])
    desc, device, heads, d = _cache_args(cache, what)
    pages, B = _table_args(table, device, what)
    shape = (k.shape[0], heads, d)
    if ws is None:
        ws = _rows_workspace(device)
    _call("bsa_cache_write", load().bsa_cache_write, device, ws, check, desc, _packed(k, shape, device, what, "k"),
          _packed(v, shape, device, what, "v"), BF16, shape[0], pages,
          _contiguous(kv_lens, (B,), _INT, device, what, "kv_lens"),
          _contiguous(cu, (B + 1,), _INT, device, what, "cu") if cu is not None else None)


def cache_read(cache: KvCache, table: torch.Tensor, cu: torch.Tensor, tokens: Optional[int] = None, *,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None, stream=None,
               check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """Run bsa_cache_read: the first cu[b + 1] - cu[b] tokens of each sequence, packed, as bf16 k, v [T, key heads, d].
    `tokens`: T where there is no `out` (k, v). Rows of `out` that belong to no sequence are left as they were."""
    what = "cache_read"
    if stream is not None and (there := _elsewhere(stream, cache.k, what)):
        with there:
            return cache_read(cache, table, cu, tokens, out=out, ws=ws, check=check)
    if _forward_ad._current_level >= 0:
        _no_tangents(what, *cache[:2], *(out or ()))
    desc, device, heads, d = _cache_args(cache, what)
    pages, B = _table_args(table, device, what)
    if out is None:
        if tokens is None:
            raise BsaError(ERR_INVALID_ARG, f"{what}: neither tokens nor out")
        out = tuple(torch.empty((tokens, heads, d), dtype=_BF16, device=device) for _ in range(2))
    k, v = out
    shape = (k.shape[0] if tokens is None else tokens, heads, d)
    if ws is None:
        ws = _rows_workspace(device)
    _call("bsa_cache_read", load().bsa_cache_read, device, ws, check, desc, pages,
          _contiguous(cu, (B + 1,), _INT, device, what, "cu"), _packed(k, shape, device, what, "out k"),
          _packed(v, shape, device, what, "out v"), BF16, shape[0])
    return k, v


def cache_attention(q: torch.Tensor, cache: KvCache, table: torch.Tensor, kv_lens: torch.Tensor, scale: float = 0.0, *,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None, check: bool = True):
    """Run bsa_cache_attention: the new token q [B, H, d] of each sequence over its kv_lens [B] tokens in the cache (itself
    among them, written before). Returns (O like q, LSE fp32 [B, H])."""
    what = "cache_attention"
    if stream is not None and (there := _elsewhere(stream, q, what)):
        with there:
            return cache_attention(q, cache, table, kv_lens, scale, out=out, lse=lse, ws=ws, check=check)
    if _forward_ad._current_level >= 0:
        _no_tangents(what, q, *cache[:2], out, lse)
    desc, device, heads, d = _cache_args(cache, what)
    pages, B = _table_args(table, device, what)
    if q.dim() != 3:
        raise BsaError(ERR_SHAPE, f"{what}: q has {q.dim()} dimensions, expected 3")
    H = q.shape[1]
    shape = (B, H, d)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=device)
    if lse is None:
        lse = torch.empty((B, H), dtype=_FP32, device=device)
    if ws is None:
        ws = cache_workspace(1, 1, heads, heads, d, device)
    _call("bsa_cache_attention", load().bsa_cache_attention, device, ws, check, desc, _packed(q, shape, device, what, "q"), BF16,
          H, pages, _contiguous(kv_lens, (B,), _INT, device, what, "kv_lens"), scale, _packed(out, shape, device, what, "out"),
          _contiguous(lse, (B, H), _FP32, device, what, "lse"))
    return out, lse


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                     cu_k: Optional[torch.Tensor] = None, *, causal: bool = True, scale: float = 0.0,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None, check: bool = True):
    """Run bsa_prompt_attention: packed q [T, H, d] over packed k, v [T', key heads, d]; sequence b has queries cu_q[b] ..
    cu_q[b + 1] - 1 and keys cu_k[b] .. cu_k[b + 1] - 1 (cu_k None: cu_q). With fewer queries than keys the queries are
    the last tokens. Returns (O like q, LSE fp32 [H, T]); rows of no sequence are left as they were."""
    what = "prompt_attention"
    if stream is not None and (there := _elsewhere(stream, q, what)):
        with there:
            return prompt_attention(q, k, v, cu_q, cu_k, causal=causal, scale=scale, out=out, lse=lse, ws=ws, check=check)
    if _forward_ad._current_level >= 0:
        _no_tangents(what, q, k, v, out, lse)
    device = _cuda_device(q, what)
    if q.dim() != 3 or k.dim() != 3:
        raise BsaError(ERR_SHAPE, f"{what}: q and k have {q.dim()} and {k.dim()} dimensions, expected 3")
    T, H, d = shape = q.shape
    Tk, Hk, _ = k.shape
    kv_shape = (Tk, Hk, d)
    if cu_k is None:
        cu_k = cu_q
    B = cu_q.shape[0] - 1
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=device)
    if lse is None:
        lse = torch.empty((H, T), dtype=_FP32, device=device)
    if ws is None:
        ws = cache_workspace(T, B, H, Hk, d, device)
    _call("bsa_prompt_attention", load().bsa_prompt_attention, device, ws, check, _packed(q, shape, device, what, "q"),
          _packed(k, kv_shape, device, what, "k"), _packed(v, kv_shape, device, what, "v"), BF16, T, Tk, B, H, Hk, d,
          _contiguous(cu_q, (B + 1,), _INT, device, what, "cu_q"), _contiguous(cu_k, (B + 1,), _INT, device, what, "cu_k"),
          int(causal), scale, _packed(out, shape, device, what, "out"), _contiguous(lse, (H, T), _FP32, device, what, "lse"))
    return out, lse
