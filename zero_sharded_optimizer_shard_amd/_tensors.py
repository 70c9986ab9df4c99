"""ctypes binding of include/zs_tensors.h: AdamW over lists of tensors with
states in 32 or 8 bits, the gradients' sum of squares and the conversion of
states.  Argument marshalling only, as in _zs.py; the caller hands over the
table and the workspace, as it does every other buffer.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

from ._muon import ZS_BF16, ZS_F32, _device, _int, _type, _workspace
from ._muon import _on_stream as _muon_stream
from ._zs import _check, zs_adamw
from ._zs import lib as _zs_lib

ZS_STATE_NONE, ZS_STATE_32, ZS_STATE_8 = 0, 32, 8
ZS_STATE8_BLOCK = 256
ZS_TENSORS_MAX_GROUPS = 16

TENSORS_EXPORTS = ["zs_tensors_create", "zs_tensors_free",
                   "zs_tensors_table_bytes", "zs_tensors_upload",
                   "zs_tensors_step", "zs_tensors_sumsq_workspace",
                   "zs_tensors_sumsq", "zs_tensors_convert"]


class zs_tensor(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("grad", ctypes.c_void_p),
                ("grad_stride", ctypes.c_int64), ("param", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("group", ctypes.c_int32)]


_ready = None


def _on_stream(stream):
    """The given stream, or the current one: by its address, where torch has
    it, as making a stream object takes longer than the launch."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if stream is not None or raw is None:
        return _muon_stream(stream)
    return raw(torch.cuda.current_device())


def _lib():
    global _ready
    if _ready is None:
        L = _zs_lib()
        i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        P = ctypes.POINTER
        L.zs_tensors_create.argtypes = [i32, P(zs_tensor), i32, i32, i32,
                                        i32, P(p)]
        L.zs_tensors_free.argtypes = [p]
        L.zs_tensors_table_bytes.argtypes = [p, P(i64)]
        L.zs_tensors_upload.argtypes = [p, p, i64, p]
        L.zs_tensors_step.argtypes = [p, P(zs_adamw), i32, i64, p,
                                      ctypes.c_float, p]
        L.zs_tensors_sumsq_workspace.argtypes = [p, P(i64)]
        L.zs_tensors_sumsq.argtypes = [p, p, p, i64, p]
        L.zs_tensors_convert.argtypes = [p, p, p]
        for name in TENSORS_EXPORTS:
            getattr(L, name).restype = ctypes.c_int
        L.zs_tensors_free.restype = None
        _ready = L
    return _ready


class TensorList:
    """Owning handle of a zs_tensors*.  It keeps the tensors and the table
    alive: keep it as long as its calls may run, replays of captured ones
    included."""

    def __init__(self, handle: int, tensors):
        self._h = ctypes.c_void_p(handle)
        self._tensors = tensors
        self._table = None

    @property
    def handle(self):
        return self._h

    def __del__(self):
        if getattr(self, "_h", None) is not None and self._h.value and _ready:
            _ready.zs_tensors_free(self._h)
            self._h = None


def _one_type(tensors, name, of):
    kinds = {of(t, name) for t in tensors or ()}
    if len(kinds) > 1:
        raise TypeError(f"{name}: one element type for all tensors of a list")
    return kinds.pop() if kinds else None


def _state_type(m, v):
    import torch
    kinds = {(a.dtype, b.dtype) for a, b in zip(m, v)}
    if kinds <= {(torch.float32, torch.float32)}:
        return ZS_STATE_32
    if kinds == {(torch.int8, torch.uint8)}:
        return ZS_STATE_8
    raise TypeError("m, v: need float32, or int8 codes of m and uint8 codes "
                    "of v, for all tensors of a list")


def _slices(g, numel, world):
    """(address, stride) of a tensor's gradients: numel elements, or with
    several ranks [world, ...] with numel elements in each slice."""
    if world == 1:
        if g.numel() != numel or not g.is_contiguous():
            raise ValueError(f"grads: need {numel} contiguous elements")
        return g.data_ptr(), numel
    if g.dim() < 1 or g.shape[0] != world or g.numel() != world * numel:
        raise ValueError(f"grads: need [{world}, ...] with {numel} elements "
                         "in each slice")
    if numel and not g[0].is_contiguous():
        raise ValueError("grads: each slice must be contiguous")
    return g.data_ptr(), g.stride(0) if numel else 0


def zs_tensors_create(*, params: Optional[Sequence] = None,
                      grads: Optional[Sequence] = None,
                      master: Optional[Sequence] = None,
                      m: Optional[Sequence] = None,
                      v: Optional[Sequence] = None,
                      m_scale: Optional[Sequence] = None,
                      v_scale: Optional[Sequence] = None, world: int = 1,
                      groups: Optional[Sequence[int]] = None) -> TensorList:
    """A list of tensors: sequences of device tensors, one entry each.

    params: bf16 or fp32, contiguous, of any shape; grads: bf16 or fp32, of
    as many elements, or [world, ...] slices of several ranks (whose rows may
    be strided); master: fp32, for bf16 params; m, v: fp32, or int8 and uint8
    codes with m_scale and v_scale of ceil(numel / ZS_STATE8_BLOCK) floats;
    groups: each tensor's index into a step's hyper-parameters (0 unless
    given).  A step needs params, grads, m and v; zs_tensors_sumsq grads;
    zs_tensors_convert m and v.  zs_tensors_upload makes the list ready.

    The list keeps these tensors, and every step reads the gradients from the
    same grads: let autograd add into them (each parameter's .grad set to its
    buffer once, and zero_grad(set_to_none=False)), or copy into them.  After
    zero_grad(), whose set_to_none is True by default, a parameter's next .grad
    is another tensor, and a step would take the old values again."""
    import torch
    if (m is None) != (v is None):
        raise ValueError("m and v belong together")
    given = [s for s in (params, m, grads) if s is not None]
    if not given:
        raise ValueError("a list needs params, grads or states")
    n = len(given[0])
    world = _int(world, "world")
    plain = {"param": params, "master": master, "m": m, "v": v}
    scales = {"m_scale": m_scale, "v_scale": v_scale}
    for name, s in {**plain, **scales, "grads": grads,
                    "groups": groups}.items():
        if s is not None and len(s) != n:
            raise ValueError(f"{name}: {len(s)} entries, {n} tensors")
    everything = [t for s in (*plain.values(), *scales.values(), grads)
                  if s is not None for t in s]
    _device(*everything)
    grad_type = _one_type(grads, "grads", _type)
    param_type = _one_type(params, "params", _type)
    state = ZS_STATE_NONE if m is None else _state_type(m, v)
    arr = (zs_tensor * max(n, 1))()
    for i in range(n):
        a = arr[i]
        if params is not None or m is not None:
            a.numel = given[0][i].numel()
        else:
            a.numel = grads[i].numel() // max(world, 1)
        for name, s in plain.items():
            if s is None:
                continue
            t = s[i]
            if t.numel() != a.numel or not t.is_contiguous():
                raise ValueError(f"{name}: tensor {i} needs {a.numel} "
                                 "contiguous elements")
            if name == "master" and t.dtype != torch.float32:
                raise TypeError("master: need float32")
            setattr(a, name, t.data_ptr())
        for name, s in scales.items():
            if s is None:
                continue
            t, need = s[i], -(-a.numel // ZS_STATE8_BLOCK)
            if t.dtype != torch.float32:
                raise TypeError(f"{name}: need float32")
            if t.numel() < need or not t.is_contiguous():
                raise ValueError(f"{name}: tensor {i} needs {need} "
                                 "contiguous elements")
            setattr(a, name, t.data_ptr())
        if grads is not None:
            a.grad, a.grad_stride = _slices(grads[i], a.numel, world)
        a.group = _int(groups[i], "groups") if groups is not None else 0
    out = ctypes.c_void_p()
    _check(_lib().zs_tensors_create(
        n, arr, world, ZS_BF16 if grad_type is None else grad_type,
        ZS_BF16 if param_type is None else param_type, state,
        ctypes.byref(out)), "zs_tensors_create")
    return TensorList(out.value, everything)


def zs_tensors_table_bytes(lst: TensorList) -> int:
    """Bytes of device memory that the list's table takes."""
    out = ctypes.c_int64()
    _check(_lib().zs_tensors_table_bytes(lst.handle, ctypes.byref(out)),
           "zs_tensors_table_bytes")
    return out.value


def zs_tensors_upload(lst: TensorList, table, *, stream=None) -> None:
    """Write the list's table into `table`, a device tensor of
    zs_tensors_table_bytes bytes or more that the list keeps; waits for the
    copy.  Once for a list, before its first use."""
    _device(table)
    ptr, nbytes = _workspace(table, "table")
    _check(_lib().zs_tensors_upload(lst.handle, ptr, nbytes,
                                    _on_stream(stream)), "zs_tensors_upload")
    lst._table = table


def _double(t, name):
    import torch
    if t.dtype != torch.float64 or t.numel() < 1:
        raise TypeError(f"{name}: need one float64")
    return t.data_ptr()


def zs_tensors_step(lst: TensorList, hp, *, step: int, sumsq=None,
                    max_norm: float = math.inf, stream=None) -> None:
    """One AdamW step of every tensor of the list.  hp: a zs_adamw, or one
    for each hyper-parameter group; step: the counter t, from 1.  sumsq: a
    device float64 that zs_tensors_sumsq wrote (or ranks added up): the
    gradients are clipped to the global norm max_norm, and where it is
    negative or not finite the step writes nothing.  With states in 8 bits
    keep beta2 to 0.99: above it the roots of v do not follow gradients that
    fall (include/zs_tensors.h has the figures)."""
    hps = [hp] if isinstance(hp, zs_adamw) else hp
    arr = (zs_adamw * max(len(hps), 1))(*hps)
    ptr = None
    if sumsq is not None:
        _device(sumsq)
        ptr = _double(sumsq, "sumsq")
    _check(_lib().zs_tensors_step(lst.handle, arr, len(hps),
                                  _int(step, "step", 64), ptr, max_norm,
                                  _on_stream(stream)), "zs_tensors_step")


def zs_tensors_sumsq_workspace(lst: TensorList) -> int:
    """Bytes of workspace zs_tensors_sumsq needs for the list."""
    out = ctypes.c_int64()
    _check(_lib().zs_tensors_sumsq_workspace(lst.handle, ctypes.byref(out)),
           "zs_tensors_sumsq_workspace")
    return out.value


def zs_tensors_sumsq(lst: TensorList, out, *, workspace,
                     stream=None) -> None:
    """The sum of the squares of the list's gradients (their mean over the
    ranks) into `out`, a device float64; its root is their global norm.
    workspace: a device tensor of zs_tensors_sumsq_workspace bytes or
    more."""
    _device(out, workspace)
    ws, nbytes = _workspace(workspace)
    _check(_lib().zs_tensors_sumsq(lst.handle, _double(out, "out"), ws,
                                   nbytes, _on_stream(stream)),
           "zs_tensors_sumsq")


def zs_tensors_convert(src: TensorList, dst: TensorList, *,
                       stream=None) -> None:
    """m and v of every tensor of `src` into the form of `dst`: fp32 into
    8-bit codes and scales, or back.  Both lists have the same sizes in the
    same order."""
    _check(_lib().zs_tensors_convert(src.handle, dst.handle,
                                     _on_stream(stream)),
           "zs_tensors_convert")
