"""ctypes binding of the operators around the attention (include/bsa_block.h): one Python function
per entry point with the same name (argument marshalling only), plus helpers that take tensors,
check that they go together and allocate outputs and workspaces with torch.

As in ``binding`` there is no fallback: if libbsa.so cannot be loaded every call raises. The helpers
run on the tensors' device and on ``stream`` (that device's current stream by default), as under
torch.cuda.stream(stream): what they allocate, results and workspace, belongs to that stream. They record
nothing for autograd, and refuse a tensor that requires a gradient while gradients are recorded: call them
under torch.no_grad() or inside a torch.autograd.Function, whose backward calls the backward helper.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

from . import binding
from .binding import BF16, ERR_DTYPE, ERR_INVALID_ARG, ERR_SHAPE, FP32, OK, BsaError, _check, _ptr, _stream

ROTARY_MAX_AXES = 4
ROTARY_INTERLEAVED = 0
ROTARY_HALVES = 1
NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2

# every symbol declared in include/bsa_block.h
EXPORTS = ("bsa_rotary_plan_init", "bsa_rotary", "bsa_rotary_backward", "bsa_rotary_workspace_size",
           "bsa_gated_norm", "bsa_gated_norm_backward", "bsa_gated_norm_workspace_size")


class RotarySpec(ctypes.Structure):
    """Mirror of bsa_rotary_spec."""
    _fields_ = [("n_axes", ctypes.c_int), ("axis_dim", ctypes.c_int * ROTARY_MAX_AXES),
                ("theta", ctypes.c_double * ROTARY_MAX_AXES), ("scale", ctypes.c_double * ROTARY_MAX_AXES),
                ("pairing", ctypes.c_int), ("inv_freq", ctypes.c_void_p)]


class RotaryPlan(ctypes.Structure):
    """Mirror of bsa_rotary_plan."""
    _fields_ = [("magic", ctypes.c_uint32), ("d", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("pairing", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64),
                ("axis", ctypes.c_uint8 * 64)]


_I64 = ctypes.c_int64


class Heads(ctypes.Structure):
    """Mirror of bsa_heads."""
    _fields_ = [("src", ctypes.c_void_p), ("src_batch", _I64), ("src_token", _I64), ("src_head", _I64),
                ("dst", ctypes.c_void_p), ("dst_batch", _I64), ("dst_token", _I64), ("dst_head", _I64),
                ("weight", ctypes.c_void_p), ("heads", ctypes.c_int)]


class HeadsGrad(ctypes.Structure):
    """Mirror of bsa_heads_grad."""
    _fields_ = [("dy", ctypes.c_void_p), ("dy_batch", _I64), ("dy_token", _I64), ("dy_head", _I64),
                ("x", ctypes.c_void_p), ("x_batch", _I64), ("x_token", _I64), ("x_head", _I64),
                ("dx", ctypes.c_void_p), ("dx_batch", _I64), ("dx_token", _I64), ("dx_head", _I64),
                ("weight", ctypes.c_void_p), ("dweight", ctypes.c_void_p), ("heads", ctypes.c_int)]


class Norm(ctypes.Structure):
    """Mirror of bsa_norm."""
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class Rows(ctypes.Structure):
    """Mirror of bsa_rows."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", _I64), ("token", _I64)]


class Modulation(ctypes.Structure):
    """Mirror of bsa_modulation."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", _I64), ("frame", _I64)]


class GatedNormDesc(ctypes.Structure):
    """Mirror of bsa_gated_norm_desc."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int), ("F", ctypes.c_int),
                ("stream_dt", ctypes.c_int), ("branch_dt", ctypes.c_int), ("mod_dt", ctypes.c_int),
                ("alpha", ctypes.c_float), ("post", Norm), ("pre", Norm), ("gate", Modulation),
                ("scale", Modulation), ("shift", Modulation)]


class GatedNormGradArgs(ctypes.Structure):
    """Mirror of bsa_gated_norm_grads."""
    _fields_ = [("dh", Rows), ("dz", Rows), ("h", Rows), ("y", Rows), ("dx", Rows), ("dy", Rows),
                ("dgate", ctypes.c_void_p), ("dscale", ctypes.c_void_p), ("dshift", ctypes.c_void_p),
                ("dpost_weight", ctypes.c_void_p), ("dpost_bias", ctypes.c_void_p),
                ("dpre_weight", ctypes.c_void_p), ("dpre_bias", ctypes.c_void_p)]


_lib = None


def load():
    """Load libbsa.so (raises OSError if it was not built) with this header's signatures."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.bsa_rotary_plan_init.argtypes = [P, I, P]
    lib.bsa_rotary.argtypes = [P, P, P, P, I, I, I, P, _I64, I, F, P]
    lib.bsa_rotary_backward.argtypes = [P, P, P, P, I, I, I, P, _I64, I, F, P, SZ, P]
    lib.bsa_rotary_workspace_size.argtypes = [I, I, I, ctypes.POINTER(SZ)]
    lib.bsa_gated_norm.argtypes = [P, P, P, P, P, P]
    lib.bsa_gated_norm_backward.argtypes = [P, P, P, SZ, P]
    lib.bsa_gated_norm_workspace_size.argtypes = [I, I, I, ctypes.POINTER(SZ)]
    for name in EXPORTS:
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _ref(s):
    return ctypes.byref(s) if s is not None else None


# ------------------------------------------------------------------ C ABI mirror


def bsa_rotary_plan_init(spec: Optional[RotarySpec], d: int, plan: Optional[RotaryPlan]) -> None:
    _check(load().bsa_rotary_plan_init(_ref(spec), int(d), _ref(plan)), "bsa_rotary_plan_init")


def bsa_rotary(plan: Optional[RotaryPlan], q: Optional[Heads], k: Optional[Heads], v: Optional[Heads], dt: int, B: int,
               N: int, positions, pos_batch: int, norm: int, eps: float, stream=None) -> None:
    _check(load().bsa_rotary(_ref(plan), _ref(q), _ref(k), _ref(v), dt, B, N, _ptr(positions), pos_batch, norm, eps,
                             _stream(stream)), "bsa_rotary")


def bsa_rotary_backward(plan: Optional[RotaryPlan], q: Optional[HeadsGrad], k: Optional[HeadsGrad],
                        v: Optional[HeadsGrad], dt: int, B: int, N: int, positions, pos_batch: int, norm: int,
                        eps: float, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_rotary_backward(_ref(plan), _ref(q), _ref(k), _ref(v), dt, B, N, _ptr(positions), pos_batch,
                                      norm, eps, _ptr(workspace), workspace_bytes, _stream(stream)),
           "bsa_rotary_backward")


def bsa_rotary_workspace_size(B: int, N: int, d: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().bsa_rotary_workspace_size(B, N, d, ctypes.byref(out)), "bsa_rotary_workspace_size")
    return out.value


def bsa_gated_norm(desc: Optional[GatedNormDesc], x: Optional[Rows], y: Optional[Rows], h: Optional[Rows],
                   z: Optional[Rows], stream=None) -> None:
    _check(load().bsa_gated_norm(_ref(desc), _ref(x), _ref(y), _ref(h), _ref(z), _stream(stream)), "bsa_gated_norm")


def bsa_gated_norm_backward(desc: Optional[GatedNormDesc], grads: Optional[GatedNormGradArgs], workspace,
                            workspace_bytes: int, stream=None) -> None:
    _check(load().bsa_gated_norm_backward(_ref(desc), _ref(grads), _ptr(workspace), workspace_bytes,
                                          _stream(stream)), "bsa_gated_norm_backward")


def bsa_gated_norm_workspace_size(B: int, N: int, C: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().bsa_gated_norm_workspace_size(B, N, C, ctypes.byref(out)), "bsa_gated_norm_workspace_size")
    return out.value


# ------------------------------------------------------------------ helpers
#
# The helpers pass descriptors as bytes in the structures' layout (struct.pack: a tenth of the time of a ctypes
# structure), and put off every message until a check fails: what they cost counts in calls on small tensors.

_CODES = {torch.bfloat16: BF16, torch.float32: FP32}
_HEADS = struct.Struct("PqqqPqqqPi4x")
_HEADS_GRAD = struct.Struct("PqqqPqqqPqqqPPi4x")
_ROWS = struct.Struct("Pqq")
_DESC = struct.Struct("7if" + "ifPP" * 2 + "Pqq" * 3)
_GRADS = struct.Struct("Pqq" * 6 + "7P")
_NO_ROWS = (0, 0, 0)


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise BsaError(ERR_DTYPE, f"{what}: tensor dtype {t.dtype}")
    return code


def _view(t: torch.Tensor, shape, dtype: torch.dtype, device, what: str, name: str):
    """(address, strides) of a tensor that a kernel will index by this shape, dtype and device, channels contiguous."""
    s = t.stride()
    if (t.shape == shape and t.dtype == dtype and t.device == device and (s[-1] == 1 or shape[-1] <= 1) and
            not (t.requires_grad and torch.is_grad_enabled())):
        return t.data_ptr(), s
    if t.shape != shape:
        raise BsaError(ERR_SHAPE, f"{what}: {name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise BsaError(ERR_DTYPE, f"{what}: {name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise BsaError(ERR_INVALID_ARG, f"{what}: {name}: on {t.device}, expected {device}")
    if s[-1] != 1 and shape[-1] > 1:
        raise BsaError(ERR_INVALID_ARG, f"{what}: {name}: channels must be contiguous")
    raise BsaError(ERR_INVALID_ARG, f"{what}: {name}: requires a gradient, which this call does not record: call it under "
                                    "torch.no_grad() or in a torch.autograd.Function")


def _cuda_device(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise BsaError(ERR_INVALID_ARG, f"{what}: not a CUDA tensor")
    return t.device


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)  # the same without an object


def _elsewhere(stream, t: Optional[torch.Tensor], what: str):
    """A context in which `stream` is current, or None where it is already. The helpers allocate on the current
    stream, and the allocator hands a block on as soon as the work of the stream it was taken on allows: a workspace
    taken on another stream than the kernels' would go to the next tensor while they still use it."""
    if t is None:
        return None  # refused by the helper
    device = _cuda_device(t, what)
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise BsaError(ERR_INVALID_ARG, f"{what}: a stream of {stream.device}, the tensors are on {device}")
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if handle in (0, 1):  # the default stream, by either of its handles
        handle, stream = 0, torch.cuda.default_stream(device)
    if handle == _current_stream(device.index):
        return None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=device)
    return torch.cuda.stream(stream)


def _run(what: str, fn, device: torch.device, *args) -> None:
    """fn(*args, the device's current stream) with `device` current: the library launches on the current device."""
    stream = _current_stream(device.index)
    if device.index == torch.cuda.current_device():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code != OK:
        raise BsaError(code, what)


def _workspace_bytes(ws: Optional[torch.Tensor], device: torch.device, what: str) -> int:
    if ws is None:
        return 0
    if ws.device != device or not ws.is_contiguous():
        raise BsaError(ERR_INVALID_ARG, f"{what}: the workspace must be contiguous and on {device}")
    return ws.numel() * ws.element_size()


def rotary_plan(d: int, axis_dims: Sequence[int], theta: Union[float, Sequence[float]] = 10000.0,
                scale: Union[float, Sequence[float]] = 1.0, interleaved: bool = True,
                inv_freq: Optional[Sequence[float]] = None) -> RotaryPlan:
    """Frequencies of a head of d channels whose axes take `axis_dims` channels each, one after another
    (bsa_rotary_plan_init). `theta` and `scale` per axis or for all; `inv_freq` (radians per position of
    every pair) in their place. interleaved: channels (2p, 2p + 1) are a pair; else (p, p + rot / 2)."""
    dims = [int(x) for x in axis_dims]
    if not 1 <= len(dims) <= ROTARY_MAX_AXES:
        raise BsaError(ERR_INVALID_ARG, f"rotary_plan: {len(dims)} axes")

    def each(v, what):
        v = [float(v)] * len(dims) if isinstance(v, (int, float)) else [float(x) for x in v]
        if len(v) != len(dims):
            raise BsaError(ERR_INVALID_ARG, f"rotary_plan: {len(v)} values of {what} for {len(dims)} axes")
        return v

    spec = RotarySpec()
    spec.n_axes = len(dims)
    for a, (dim, th, sc) in enumerate(zip(dims, each(theta, "theta"), each(scale, "scale"))):
        spec.axis_dim[a], spec.theta[a], spec.scale[a] = dim, th, sc
    spec.pairing = ROTARY_INTERLEAVED if interleaved else ROTARY_HALVES
    keep = None
    if inv_freq is not None:
        freq = [float(x) for x in inv_freq]
        if len(freq) != sum(dims) // 2:
            raise BsaError(ERR_INVALID_ARG, f"rotary_plan: {len(freq)} frequencies for {sum(dims) // 2} pairs")
        keep = (ctypes.c_double * len(freq))(*freq)
        spec.inv_freq = ctypes.cast(keep, ctypes.c_void_p)
    plan = RotaryPlan()
    bsa_rotary_plan_init(spec, d, plan)
    return plan


def grid_positions(grid: Sequence[int], n_text: int = 0, cuboid: Optional[Sequence[int]] = None,
                   device="cuda") -> torch.Tensor:
    """int32 [n_text + prod(grid), len(grid)]: `n_text` tokens at the origin, then the grid's coordinates in
    raster order (last axis fastest). With `cuboid` (its extent per axis, dividing the grid's) in the token
    order of cuboid_spec: cuboid after cuboid in raster order, each cuboid's tokens in raster order."""
    grid = [int(g) for g in grid]
    c = torch.stack(torch.meshgrid(*[torch.arange(g, dtype=torch.int32, device=device) for g in grid],
                                   indexing="ij"), dim=-1)
    if cuboid is not None:
        cub = [int(x) for x in cuboid]
        if len(cub) != len(grid) or any(x < 1 or g % x for g, x in zip(grid, cub)):
            raise BsaError(ERR_SHAPE, f"grid_positions: cuboid {tuple(cub)} does not divide the grid {tuple(grid)}")
        n = len(grid)
        c = c.reshape(*[v for g, x in zip(grid, cub) for v in (g // x, x)], n)
        c = c.permute(*range(0, 2 * n, 2), *range(1, 2 * n, 2), 2 * n)
    c = c.reshape(-1, len(grid))
    return torch.cat((torch.zeros((n_text, len(grid)), dtype=torch.int32, device=device), c)).contiguous()


def _rotary_args(plan, first, positions, needed: bool, norm: bool, q_weight, k_weight, n_at: int, what: str):
    """What rotary and rotary_backward have in common, from the first of their tensors (tokens at dimension n_at):
    (device, dtype, dtype code, B, N, positions, pos_batch, weights)."""
    if first is None:
        raise BsaError(ERR_INVALID_ARG, f"{what}: none of q, k, v")
    device, dtype = _cuda_device(first, what), first.dtype
    if first.dim() != 4:
        raise BsaError(ERR_SHAPE, f"{what}: {first.dim()} dimensions, expected 4")
    B, N = first.shape[0], first.shape[n_at]
    pos, pos_batch = None, 0
    if needed:
        if positions is None:
            raise BsaError(ERR_INVALID_ARG, f"{what}: no positions")
        axes = plan.n_axes
        if positions.dim() == 2:
            pos, s = _view(positions, (N, axes), torch.int32, device, what, "positions")
        else:
            pos, s = _view(positions, (B, N, axes), torch.int32, device, what, "positions")
            pos_batch = s[0]
        if N > 1 and s[-2] != axes:
            raise BsaError(ERR_INVALID_ARG, f"{what}: a token's positions must follow the last token's")
    if not norm and (q_weight is not None or k_weight is not None):
        raise BsaError(ERR_INVALID_ARG, f"{what}: a weight without norm_eps, which selects the norm")
    d = plan.d
    weights = (0 if q_weight is None else _view(q_weight, (d,), torch.float32, device, what, "q_weight")[0],
               0 if k_weight is None else _view(k_weight, (d,), torch.float32, device, what, "k_weight")[0], 0)
    code = _CODES.get(dtype)
    if code is None:
        raise BsaError(ERR_DTYPE, f"{what}: tensor dtype {dtype}")
    return device, dtype, code, B, N, pos, pos_batch, weights


def rotary(plan: RotaryPlan, q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None,
           v: Optional[torch.Tensor] = None, *, positions: Optional[torch.Tensor] = None,
           norm_eps: Optional[float] = None, q_weight: Optional[torch.Tensor] = None,
           k_weight: Optional[torch.Tensor] = None,
           out: Optional[Tuple[Optional[torch.Tensor], ...]] = None, stream=None):
    """Run bsa_rotary: q, k, v [B, N, heads, d] (views of a fused projection do) to [B, heads, N, d], Q and K
    normalised per head (norm_eps not None; fp32 weights [d] optional, refused without it) and turned by `positions`
    (int32 [N, axes] or [B, N, axes]). `out`: the three results' tensors, any strides with contiguous
    channels. Returns (q, k, v), None where none was given."""
    what = "rotary"
    first = q if q is not None else k if k is not None else v
    if stream is not None and (there := _elsewhere(stream, first, what)):
        with there:
            return rotary(plan, q, k, v, positions=positions, norm_eps=norm_eps, q_weight=q_weight, k_weight=k_weight,
                          out=out)
    device, dtype, code, B, N, pos, pos_batch, weights = _rotary_args(
        plan, first, positions, q is not None or k is not None, norm_eps is not None, q_weight, k_weight, 1, what)
    d = plan.d
    res, desc = [None, None, None], [None, None, None]
    for i, t in enumerate((q, k, v)):
        if t is None:
            continue
        h = t.shape[2] if t.dim() == 4 else 0
        at, s = _view(t, (B, N, h, d), dtype, device, what, "q, k, v")
        o = out[i] if out is not None else None
        if o is None:
            o = t.new_empty((B, h, N, d))
        o_at, r = _view(o, (B, h, N, d), dtype, device, what, "out")
        desc[i] = _HEADS.pack(at, s[0], s[1], s[2], o_at, r[0], r[2], r[1], weights[i], h)
        res[i] = o
    norm = norm_eps is not None
    _run("bsa_rotary", load().bsa_rotary, device, ctypes.byref(plan), *desc, code, B, N, pos, pos_batch, norm,
         norm_eps if norm else 0.0)
    return tuple(res)


def rotary_workspace(B: int, N: int, d: int, device="cuda") -> torch.Tensor:
    """Device workspace of rotary_backward."""
    return torch.empty(bsa_rotary_workspace_size(B, N, d), dtype=torch.uint8, device=device)


def rotary_backward(plan: RotaryPlan, dq: Optional[torch.Tensor], dk: Optional[torch.Tensor] = None,
                    dv: Optional[torch.Tensor] = None, *, positions: Optional[torch.Tensor] = None,
                    q: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None,
                    norm_eps: Optional[float] = None, q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None,
                    out: Optional[Tuple[Optional[torch.Tensor], ...]] = None, ws: Optional[torch.Tensor] = None,
                    stream=None):
    """Run bsa_rotary_backward: the gradients dq, dk, dv [B, heads, N, d] that arrive at rotary's results, to
    the gradients [B, N, heads, d] of its inputs. With norm_eps, q and k are rotary's inputs. Returns
    (gq, gk, gv, gq_weight, gk_weight); a weight's gradient (fp32 [d]) where that weight is given."""
    what = "rotary_backward"
    first = dq if dq is not None else dk if dk is not None else dv
    if stream is not None and (there := _elsewhere(stream, first, what)):
        with there:
            return rotary_backward(plan, dq, dk, dv, positions=positions, q=q, k=k, norm_eps=norm_eps,
                                   q_weight=q_weight, k_weight=k_weight, out=out, ws=ws)
    device, dtype, code, B, N, pos, pos_batch, weights = _rotary_args(
        plan, first, positions, dq is not None or dk is not None, norm_eps is not None, q_weight, k_weight, 2, what)
    norm, d = norm_eps is not None, plan.d
    res, desc, dweights = [None, None, None], [None, None, None], [None, None]
    for i, t in enumerate((dq, dk, dv)):
        if t is None:
            continue
        h = t.shape[1] if t.dim() == 4 else 0
        shape = (B, N, h, d)
        at, s = _view(t, (B, h, N, d), dtype, device, what, "dq, dk, dv")
        o = out[i] if out is not None else None
        if o is None:
            o = t.new_empty(shape)
        o_at, r = _view(o, shape, dtype, device, what, "out")
        x_at, x, dw = 0, (0, 0, 0), 0
        if norm and i < 2:
            side = q if i == 0 else k
            if side is None:
                raise BsaError(ERR_INVALID_ARG, "rotary_backward: the norm needs q and k")
            x_at, x = _view(side, shape, dtype, device, what, "q, k")
            if weights[i]:
                dweights[i] = torch.empty_like(q_weight if i == 0 else k_weight)
                dw = dweights[i].data_ptr()
        desc[i] = _HEADS_GRAD.pack(at, s[0], s[2], s[1], x_at, x[0], x[1], x[2], o_at, r[0], r[1], r[2], weights[i], dw, h)
        res[i] = o
    if ws is None and (dweights[0] is not None or dweights[1] is not None):
        ws = rotary_workspace(B, N, plan.d, device)
    _run("bsa_rotary_backward", load().bsa_rotary_backward, device, ctypes.byref(plan), *desc, code, B, N, pos,
         pos_batch, norm, norm_eps if norm else 0.0, _ptr(ws), _workspace_bytes(ws, device, what))
    return (*res, dweights[0], dweights[1])


_KINDS = {"rms": NORM_RMS, "layer": NORM_LAYER}


class NormSpec:
    """A norm over the channels: kind "rms" or "layer", fp32 weight and bias [C] (None: ones, zeros), eps."""

    def __init__(self, kind: str, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 eps: float = 1e-6):
        if kind not in _KINDS:
            raise BsaError(ERR_INVALID_ARG, f"NormSpec: kind {kind!r}")
        self.kind, self.weight, self.bias, self.eps = kind, weight, bias, float(eps)


class GatedNormGrads(NamedTuple):
    """What gated_norm_backward returns; None for what the forward did not have."""
    dx: Optional[torch.Tensor]
    dy: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dshift: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dpost_bias: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dpre_bias: Optional[torch.Tensor]


def _norm_args(n: Optional[NormSpec], C: int, device, what: str):
    if n is None:
        return NORM_NONE, 0.0, 0, 0
    w, b = n.weight, n.bias
    return (_KINDS[n.kind], n.eps, 0 if w is None else _view(w, (C,), torch.float32, device, what, "weight")[0],
            0 if b is None else _view(b, (C,), torch.float32, device, what, "bias")[0])


def _gated_desc(shape, device, stream_dt: int, branch_dt: int, alpha, post, pre, gate, scale, shift, what: str):
    """(bsa_gated_norm_desc as bytes, F)"""
    B, N, C = shape
    F, mod = 1, None
    mods = []
    for m in (gate, scale, shift):
        if m is None:
            mods += _NO_ROWS
            continue
        frames = m.dim() == 3
        if mod is None:
            F, mod = m.shape[1] if frames else 1, m.dtype
        at, s = _view(m, (B, F, C) if frames else (B, C), mod, device, what, "gate, scale, shift")
        if not frames and F != 1:
            raise BsaError(ERR_SHAPE, f"{what}: modulations of shape {tuple(m.shape)} and of {F} frames")
        mods += (at, s[0], s[1] if frames else 0)
    if mod is not None and mod not in _CODES:
        raise BsaError(ERR_DTYPE, f"{what}: modulation dtype {mod}")
    return _DESC.pack(B, N, C, F, stream_dt, branch_dt, _CODES[mod] if mod is not None else BF16, alpha,
                      *_norm_args(post, C, device, what), *_norm_args(pre, C, device, what), *mods), F


def gated_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *, gate: Optional[torch.Tensor] = None,
               alpha: float = 1.0, post: Optional[NormSpec] = None, pre: Optional[NormSpec] = None,
               scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
               out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
               branch_dtype: Optional[torch.dtype] = None, stream=None):
    """Run bsa_gated_norm: h = x + alpha * gate * post(y), z = pre(h) * (1 + scale) + shift, for x, y [B, N, C] and
    modulations [B, C] or [B, F, C] (F frames of N / F tokens). Without y, h is x and is not written; without
    pre there is no z, whose dtype is y's (without y: that of out's z, branch_dtype or x's). Returns (h, z)."""
    what = "gated_norm"
    if stream is not None and (there := _elsewhere(stream, x, what)):
        with there:
            return gated_norm(x, y, gate=gate, alpha=alpha, post=post, pre=pre, scale=scale, shift=shift, out=out,
                              branch_dtype=branch_dtype)
    device = _cuda_device(x, what)
    if x.dim() != 3:
        raise BsaError(ERR_SHAPE, f"gated_norm: x has {x.dim()} dimensions, expected 3")
    shape, dtype = x.shape, x.dtype
    pack = _ROWS.pack
    at, s = _view(x, shape, dtype, device, what, "x")
    rows = [pack(at, s[0], s[1]), None, None, None]
    h, z = out if out is not None else (None, None)
    branch = y if y is not None else z
    branch_dtype = branch.dtype if branch is not None else branch_dtype or dtype
    if y is not None:
        at, s = _view(y, shape, branch_dtype, device, what, "y")
        rows[1] = pack(at, s[0], s[1])
        if h is None:
            h = x.new_empty(shape)
    if pre is not None and z is None:
        z = torch.empty(shape, dtype=branch_dtype, device=device)
    if h is not None:
        at, s = _view(h, shape, dtype, device, what, "out h")
        rows[2] = pack(at, s[0], s[1])
    if z is not None:
        at, s = _view(z, shape, branch_dtype, device, what, "out z")
        rows[3] = pack(at, s[0], s[1])
    desc, _ = _gated_desc(shape, device, _code(x, what), _CODES.get(branch_dtype, -1), alpha, post, pre, gate, scale,
                          shift, what)
    _run("bsa_gated_norm", load().bsa_gated_norm, device, desc, *rows)
    return h, z


def gated_norm_workspace(B: int, N: int, C: int, device="cuda") -> torch.Tensor:
    """Device workspace of gated_norm_backward."""
    return torch.empty(bsa_gated_norm_workspace_size(B, N, C), dtype=torch.uint8, device=device)


def gated_norm_backward(dh: Optional[torch.Tensor], dz: Optional[torch.Tensor], h: Optional[torch.Tensor],
                        y: Optional[torch.Tensor] = None, *, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                        post: Optional[NormSpec] = None, pre: Optional[NormSpec] = None,
                        scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                        out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
                        ws: Optional[torch.Tensor] = None, stream=None) -> GatedNormGrads:
    """Run bsa_gated_norm_backward. dh [B, N, C] is the gradient that arrives at h from where h goes on (None:
    zero), dz the one at z (with pre only), h gated_norm's h (its x without y) and y its y. Without pre, dx is dh
    itself and nothing is written for it. `out`: (dx, dy). Gradients of the modulations have their dtype and
    shape, those of weights and biases are fp32 [C]. A broadcast modulation (an expanded one) is refused: its
    gradient would be a sum over what it is broadcast to."""
    what = "gated_norm_backward"
    first = dh if dh is not None else dz
    if first is None:
        raise BsaError(ERR_INVALID_ARG, f"{what}: neither dh nor dz")
    if stream is not None and (there := _elsewhere(stream, first, what)):
        with there:
            return gated_norm_backward(dh, dz, h, y, gate=gate, alpha=alpha, post=post, pre=pre, scale=scale,
                                       shift=shift, out=out, ws=ws)
    device = _cuda_device(first, what)
    if first.dim() != 3:
        raise BsaError(ERR_SHAPE, f"{what}: {first.dim()} dimensions, expected 3")
    shape = first.shape
    like = dh if dh is not None else h
    if like is None:
        raise BsaError(ERR_INVALID_ARG, f"{what}: no h")
    stream_dtype = like.dtype
    branch_dtype = dz.dtype if dz is not None else y.dtype if y is not None else stream_dtype

    def rows(t, dtype, name):
        if t is None:
            return _NO_ROWS
        at, s = _view(t, shape, dtype, device, what, name)
        return at, s[0], s[1]

    dx, dy = out if out is not None else (None, None)
    if pre is None:
        dx = h = None
    elif dx is None:
        dx = torch.empty(shape, dtype=stream_dtype, device=device)
    if y is None:
        dy = None
    elif dy is None:
        dy = torch.empty(shape, dtype=branch_dtype, device=device)
    views = (*rows(dh, stream_dtype, "dh"), *rows(dz, branch_dtype, "dz"), *rows(h, stream_dtype, "h"),
             *rows(y, branch_dtype, "y"), *rows(dx, stream_dtype, "out dx"), *rows(dy, branch_dtype, "out dy"))
    desc, _ = _gated_desc(shape, device, _code(like, what), _CODES.get(branch_dtype, -1), alpha, post, pre, gate, scale,
                          shift, what)
    dmods, dparams, at = [], [], []
    for m in (gate, scale, shift):
        d = None if m is None else m.new_empty(m.shape)
        dmods.append(d)
        at.append(0 if d is None else d.data_ptr())
    for n in (post, pre):
        for p in (n.weight, n.bias) if n is not None else (None, None):
            d = None if p is None else torch.empty_like(p)
            dparams.append(d)
            at.append(0 if d is None else d.data_ptr())
    if ws is None and any(at):
        ws = gated_norm_workspace(*shape, device)
    args = _GRADS.pack(*views, *at)
    _run("bsa_gated_norm_backward", load().bsa_gated_norm_backward, device, desc, args, _ptr(ws),
         _workspace_bytes(ws, device, what))
    return GatedNormGrads(dx if pre is not None else dh, dy, *dmods, *dparams)
