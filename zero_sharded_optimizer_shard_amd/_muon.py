"""ctypes binding of include/zs_muon.h: orthogonalisation by Newton-Schulz
products and the whole-tensor Muon step.  Argument marshalling only, as in
_zs.py; the caller hands over the workspace, as it does every other buffer.
"""

from __future__ import annotations

import ctypes
import operator
from typing import Sequence

from ._zs import (ZS_GRADS_TILED, ZS_TILE, Layout, _bf16, _check, _f32,
                  _grads_need, _layout_code, _need, _step_need, _stream,
                  _tiles)
from ._zs import lib as _zs_lib

ZS_NS_FAST, ZS_NS_FULL = 0, 1
ZS_NS_MAX_STEPS = 16
ZS_BF16, ZS_F32 = 0, 1
ZS_MUON_SCALE_NONE, ZS_MUON_SCALE_SHAPE, ZS_MUON_SCALE_RMS = 0, 1, 2
# the usual coefficients: steep at zero, singular values to about [0.7, 1.2]
ZS_NS_COEF = (3.4445, -4.7750, 2.0315)

MUON_EXPORTS = ["zs_orthogonalize_workspace", "zs_orthogonalize",
                "zs_muon_workspace", "zs_muon_step"]

_PRECISION = {"fast": ZS_NS_FAST, "full": ZS_NS_FULL}
_SCALE = {"none": ZS_MUON_SCALE_NONE, "shape": ZS_MUON_SCALE_SHAPE,
          "rms": ZS_MUON_SCALE_RMS}


class zs_newton_schulz(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("eps", ctypes.c_float),
                ("coef", (ctypes.c_float * 3) * ZS_NS_MAX_STEPS)]


class zs_ns_matrices(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64),
                ("x_batch_stride", ctypes.c_int64),
                ("x_row_stride", ctypes.c_int64),
                ("o_batch_stride", ctypes.c_int64),
                ("o_row_stride", ctypes.c_int64)]


class zs_muon(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("ns", zs_newton_schulz)]


class zs_muon_tensor(ctypes.Structure):
    _fields_ = [("bucket_id", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


_ready = False


def _lib():
    global _ready
    L = _zs_lib()
    if not _ready:
        i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        P = ctypes.POINTER
        L.zs_orthogonalize_workspace.argtypes = [i32, P(zs_ns_matrices), i32,
                                                 P(i64)]
        L.zs_orthogonalize.argtypes = [i32, P(zs_ns_matrices), i32, i32,
                                       P(zs_newton_schulz), p, i64, p]
        L.zs_muon_workspace.argtypes = [p, i32, P(zs_muon_tensor), i32,
                                        P(i64)]
        L.zs_muon_step.argtypes = [p, i32, P(zs_muon_tensor), P(p), i32, i64,
                                   p, p, p, P(zs_muon), p, i64, p]
        for name in MUON_EXPORTS:
            getattr(L, name).restype = ctypes.c_int
        _ready = True
    return L


def _int(v, name: str, bits: int = 32) -> int:
    """v, if it has a place in the library's integer (ctypes would drop its
    upper bits without a word)."""
    v = operator.index(v)
    if not -(1 << (bits - 1)) <= v < 1 << (bits - 1):
        raise ValueError(f"{name}: {v} does not fit {bits} bits")
    return v


def _precision(precision) -> int:
    # unknown codes go through unchanged so the library reports them
    return _PRECISION[precision] if precision in _PRECISION \
        else _int(int(precision), "precision")


_Coef = ctypes.c_float * 3


def _newton_schulz(steps: int, coef, eps: float, precision):
    """coef: one (a, b, c) for every step, or one per step."""
    steps = _int(steps, "steps")
    ns = zs_newton_schulz(steps, _precision(precision), eps)
    per_step = len(coef) > 0 and isinstance(coef[0], (tuple, list))
    for row in coef if per_step else [coef]:
        if len(row) != 3:
            raise ValueError(f"coef: {len(row)} coefficients, not 3")
    if per_step and len(coef) != steps:
        raise ValueError(f"coef: {len(coef)} rows for {steps} steps")
    # a number of steps past the last place is the library's to refuse
    rows = [_Coef(*row) for row in coef] if per_step \
        else [_Coef(*coef)] * min(steps, ZS_NS_MAX_STEPS)
    for k, row in enumerate(rows[:ZS_NS_MAX_STEPS]):
        ns.coef[k] = row
    return ns


def _device(*tensors):
    """The library works on the current device: refuse tensors of another."""
    import torch
    current = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("expected a device tensor")
        if current is None:
            current = torch.cuda.current_device()
        if t.device.index != current:
            raise ValueError(f"tensor on {t.device}, the current device is "
                             f"cuda:{current}")


def _on_stream(stream):
    import torch
    if stream is not None and \
            stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream of {stream.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return _stream(stream)


def _type(t, name) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return ZS_BF16
    if t.dtype == torch.float32:
        return ZS_F32
    raise TypeError(f"{name}: need bfloat16 or float32")


def _stack(t, name):
    """(batch, rows, cols, batch stride, row stride) of a 2-D or 3-D tensor
    whose last dimension is contiguous."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name}: need [rows, cols] or [batch, rows, cols]")
    b = t.shape[0] if t.dim() == 3 else 1
    r, c = t.shape[-2:]
    if t.numel() == 0:                  # skipped, whatever its strides
        return b, r, c, r * c, c
    if c > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: columns must be contiguous")
    row = t.stride(-2) if r > 1 else c
    return b, r, c, (t.stride(0) if t.dim() == 3 and b > 1 else r * row), row


def _workspace(workspace, name="workspace"):
    if not workspace.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _matrices(mats, outs=None):
    arr = (zs_ns_matrices * max(len(mats), 1))()
    for i, x in enumerate(mats):
        b, r, c, xb, xr = _stack(x, "mats")
        m = arr[i]
        m.x, m.batch, m.rows, m.cols = x.data_ptr(), b, r, c
        m.x_batch_stride, m.x_row_stride = xb, xr
        if outs is not None:
            if outs[i].shape != x.shape:
                raise ValueError(f"outs[{i}]: shape {tuple(outs[i].shape)}, "
                                 f"the input has {tuple(x.shape)}")
            m.o = outs[i].data_ptr()
            m.o_batch_stride, m.o_row_stride = _stack(outs[i], "outs")[3:]
    return arr


def zs_orthogonalize_workspace(mats: Sequence, precision="fast") -> int:
    """Bytes of workspace zs_orthogonalize needs for these tensors."""
    out = ctypes.c_int64()
    _check(_lib().zs_orthogonalize_workspace(
        len(mats), _matrices(mats), _precision(precision),
        ctypes.byref(out)), "zs_orthogonalize_workspace")
    return out.value


def zs_orthogonalize(mats: Sequence, outs: Sequence, *, workspace,
                     steps: int = 5, coef=ZS_NS_COEF, eps: float = 1e-7,
                     precision="fast", stream=None) -> None:
    """Orthogonalise each matrix of `mats` into `outs` by Newton-Schulz
    steps.  mats, outs: device tensors [rows, cols] or [batch, rows, cols]
    with contiguous columns (rows and stacks may be strided), bf16 or fp32,
    one type for all of mats and one for all of outs.  coef: (a, b, c), or
    one per step.  workspace: a device tensor of zs_orthogonalize_workspace
    bytes or more (for the same precision).

    precision is "fast" unless it is given, for fp32 tensors too: after five
    steps the result is about 1e-3 of its norm off, half of what rounding it
    to bf16 costs.  "full" is level with fp32 products (2e-6), in up to three
    times the time of the products.  include/zs_muon.h has the figures by
    kind of matrix, and for more steps."""
    if len(mats) != len(outs):
        raise ValueError("one output per input")
    _device(*mats, *outs, workspace)
    xt = {_type(t, "mats") for t in mats} or {ZS_F32}
    ot = {_type(t, "outs") for t in outs} or {ZS_F32}
    if len(xt) > 1 or len(ot) > 1:
        raise TypeError("one element type for all inputs and one for all "
                        "outputs of a call")
    ns = _newton_schulz(steps, coef, eps, precision)
    ws, nbytes = _workspace(workspace)
    _check(_lib().zs_orthogonalize(len(mats), _matrices(mats, outs),
                                   xt.pop(), ot.pop(), ctypes.byref(ns), ws,
                                   nbytes, _on_stream(stream)),
           "zs_orthogonalize")


def _tensors(tensors):
    """(bucket_id, rows, cols) or (bucket_id, batch, rows, cols) each."""
    arr = (zs_muon_tensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        if len(t) not in (3, 4):
            raise ValueError("tensors: need (bucket_id, rows, cols) or "
                             "(bucket_id, batch, rows, cols)")
        sizes = (1,) + tuple(t[1:]) if len(t) == 3 else t[1:]
        arr[i] = zs_muon_tensor(_int(t[0], "bucket_id"),
                                *[_int(v, "tensors", 64) for v in sizes])
    return arr


def zs_muon_workspace(layout: Layout, tensors: Sequence,
                      precision="fast") -> int:
    """Bytes of workspace zs_muon_step needs for these tensors."""
    out = ctypes.c_int64()
    _check(_lib().zs_muon_workspace(layout.handle, len(tensors),
                                    _tensors(tensors), _precision(precision),
                                    ctypes.byref(out)), "zs_muon_workspace")
    return out.value


def zs_muon_step(layout: Layout, tensors: Sequence, grads: Sequence, state,
                 param_shard=None, full_flat=None, *, workspace,
                 grad_layout="slices", grad_stride: int = 0, lr: float,
                 momentum: float, weight_decay: float, nesterov: bool = True,
                 scale="rms", steps: int = 5, coef=ZS_NS_COEF,
                 eps: float = 1e-7, precision="fast", stream=None) -> None:
    """Muon step of matrices this rank owns under a whole-tensor layout.
    tensors: (bucket_id, rows, cols) or (bucket_id, batch, rows, cols) each,
    at most ZS_MAX_GROUP; grads: one tensor of W slices each, as
    zs_buckets_step takes them; state: the shard's tiled state, of which row
    1 holds the momentum; scale: "none", "shape" or "rms".

    precision is "fast" unless it is given: the update lr*s*O is about 1e-3
    of its norm off, which leaves a master of 0.02 sigma after a step of lr
    3e-4 about 1e-6 of its norm off, where fp32 products ("full" is level
    with them) leave 4e-8.  The momentum is the same in both."""
    n = len(tensors)
    if len(grads) != n:
        raise ValueError("one gradient tensor per matrix tensor")
    _device(*grads, state, param_shard, full_flat, workspace)
    code = _int(_layout_code(grad_layout), "grad_layout")
    grad_stride = _int(grad_stride, "grad_stride", 64)
    _, _, _, W, buckets = layout.sizes()
    arr = _tensors(tensors)
    for t, g in zip(arr, grads):
        if 0 <= t.bucket_id < len(buckets):  # others: the library's to refuse
            sl = buckets[t.bucket_id].slice_numel
            numel = t.batch * t.rows * t.cols
            # a slice's padding is not read
            need = _tiles(sl) * W * ZS_TILE if code == ZS_GRADS_TILED \
                else _grads_need(W, 0, min(numel, sl), code, grad_stride)
            _need(g, need, "grads")
    _step_need(layout, None, code, grad_stride, state, 3, param_shard,
               full_flat)
    ptrs = (ctypes.c_void_p * max(n, 1))(*[_bf16(g, "grads") for g in grads])
    hp = zs_muon(lr, momentum, weight_decay, int(bool(nesterov)),
                 _SCALE[scale] if scale in _SCALE
                 else _int(int(scale), "scale"),
                 _newton_schulz(steps, coef, eps, precision))
    ws, nbytes = _workspace(workspace)
    _check(_lib().zs_muon_step(layout.handle, n, arr, ptrs, code,
                               grad_stride, _f32(state, "state"),
                               _bf16(param_shard, "param_shard"),
                               _bf16(full_flat, "full_flat"),
                               ctypes.byref(hp), ws, nbytes,
                               _on_stream(stream)), "zs_muon_step")
