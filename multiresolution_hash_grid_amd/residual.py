"""A residual head of any width on the hash-grid encoding, and the step that
trains it: binding of the linear, RMS norm and AdamW entry points of
include/hashgrid.h, their autograd functions, modules and optimizer.

As in ``hashgrid``, the binding only marshals arguments; every computation runs
in the HIP kernels of the library and there is no fallback.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from .hashgrid import (HG_ADAM_ZERO_GRAD, HG_F16, HG_F32, _check, _dev, _keep_for_stream, _stream,
                       _workspace, load_library)

HG_BF16, HG_F8 = 2, 3
HG_ACT = {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3}
F8 = torch.float8_e4m3fn
_CODES = {torch.float32: HG_F32, torch.float16: HG_F16, torch.bfloat16: HG_BF16, F8: HG_F8}
_HALF = (torch.float16, torch.bfloat16)

_P, _I64, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class _Linear(ctypes.Structure):
    _fields_ = [("m", _I64), ("k", _I32), ("n", _I32), ("x", _P), ("x_stride", _I64), ("w", _P), ("w_stride", _I64),
                ("x_scale", _P), ("w_scale", _P), ("bias", _P), ("residual", _P), ("residual_stride", _I64),
                ("y", _P), ("y_stride", _I64), ("pre", _P), ("pre_stride", _I64), ("x_dtype", _I32), ("y_dtype", _I32),
                ("act", _I32)]


class _LinearGrad(ctypes.Structure):
    _fields_ = [("m", _I64), ("k", _I32), ("n", _I32), ("dy", _P), ("dy_stride", _I64), ("pre", _P), ("pre_stride", _I64),
                ("x", _P), ("x_stride", _I64), ("w", _P), ("w_stride", _I64), ("dx", _P), ("dx_stride", _I64),
                ("dw", _P), ("dw_stride", _I64), ("db", _P), ("dtype", _I32), ("dy_dtype", _I32), ("dw_dtype", _I32),
                ("act", _I32), ("accumulate", _I32)]


class _RmsNorm(ctypes.Structure):
    _fields_ = [("m", _I64), ("c", _I32), ("x", _P), ("x_stride", _I64), ("residual", _P), ("residual_stride", _I64),
                ("w", _P), ("y", _P), ("y_stride", _I64), ("y_scale", _P), ("sum", _P), ("sum_stride", _I64), ("rstd", _P),
                ("eps", _F), ("dtype", _I32), ("y_dtype", _I32)]


class _RmsNormGrad(ctypes.Structure):
    _fields_ = [("m", _I64), ("c", _I32), ("dy", _P), ("dy_stride", _I64), ("sum", _P), ("sum_stride", _I64), ("w", _P),
                ("rstd", _P), ("ds", _P), ("ds_stride", _I64), ("dx", _P), ("dx_stride", _I64), ("dw", _P),
                ("dtype", _I32), ("accumulate", _I32)]


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", _P), ("grad", _P), ("m", _P), ("v", _P), ("m_exp", _P), ("v_exp", _P), ("copy", _P),
                ("count", _I64), ("lr", _F), ("weight_decay", _F), ("grad_dtype", _I32), ("copy_dtype", _I32),
                ("state_bits", _I32), ("reserved", _I32)]


class _AdamW(ctypes.Structure):
    _fields_ = [("beta1", _F), ("beta2", _F), ("eps", _F), ("step", _I32), ("seed", ctypes.c_uint32)]


_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        lib = load_library()
        size = ctypes.c_size_t
        for name, args in (
                ("hashgrid_linear_forward", [_P, _P]),
                ("hashgrid_linear_backward_workspace_size", [_P, _P]),
                ("hashgrid_linear_backward", [_P, _P, size, _P]),
                ("hashgrid_rms_norm_forward", [_P, _P]),
                ("hashgrid_rms_norm_backward_workspace_size", [_P, _P]),
                ("hashgrid_rms_norm_backward", [_P, _P, size, _P]),
                ("hashgrid_adamw_step", [_P, _P, _I32, _P, _I32, _P])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _bound = lib
    return _bound


def _rows(t, name, shape, dtype, like) -> int:
    """Row stride of a matrix argument, after its checks."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a tensor on {like.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be [{shape[0]}, {shape[1]}] with unit column stride")
    return t.stride(0)


def _vector(t, name, n, like) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a float32 tensor on {like.device}")
    if t.dim() != 1 or t.shape[0] != n or (t.stride(0) != 1 and n > 1):
        raise ValueError(f"{name} must be a contiguous [{n}] tensor")
    return t.data_ptr()


def _act(act) -> int:
    if act not in HG_ACT:
        raise ValueError(f"act must be one of {', '.join(HG_ACT)}")
    return HG_ACT[act]


def _matrix(t, name) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in _CODES:
        raise ValueError(f"{name} must be a 2-dimensional GPU tensor of float32, float16, bfloat16 or float8_e4m3fn")
    return t


def hashgrid_linear_forward(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *, act: str = "none",
                            residual: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                            weight_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                            save_pre: bool = False, out: torch.Tensor | None = None, stream=None):
    """y = act(x W^T + bias) + residual for x [m, k] and weight [n, k] in float16 or bfloat16, or both in
    float8_e4m3fn with ``x_scale`` [m] and ``weight_scale`` [n].  y has ``out_dtype`` (by default x's, bfloat16 for
    8-bit operands), bias is float32, the residual has y's type.  ``out`` receives y (it may be the residual).
    With ``save_pre`` the call returns (y, z), z being the pre-activation in x's type for the backward."""
    _matrix(x, "x")
    _matrix(weight, "weight")
    m, k = x.shape
    n = weight.shape[0]
    eight = x.dtype == F8
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if eight else x.dtype
    made = out is None
    y = torch.empty((m, n), dtype=out_dtype, device=x.device) if made else out
    pre = torch.empty((m, n), dtype=x.dtype, device=x.device) if save_pre else None
    op = _Linear(m, k, n, x.data_ptr(), _rows(x, "x", (m, k), x.dtype, x),
                 weight.data_ptr(), _rows(weight, "weight", (n, k), x.dtype, x),
                 None if x_scale is None else _vector(x_scale, "x_scale", m, x),
                 None if weight_scale is None else _vector(weight_scale, "weight_scale", n, x),
                 None if bias is None else _vector(bias, "bias", n, x),
                 None if residual is None else residual.data_ptr(),
                 0 if residual is None else _rows(residual, "residual", (m, n), out_dtype, x),
                 y.data_ptr(), y.stride(0) if made else _rows(y, "out", (m, n), out_dtype, x),
                 None if pre is None else pre.data_ptr(), n, _CODES[x.dtype], _CODES.get(out_dtype, -1), _act(act))
    _check(_lib().hashgrid_linear_forward(ctypes.byref(op), _stream(x, stream)))
    if stream is not None:
        _keep_for_stream(x, stream, y if made else None, pre)
    return (y, pre) if save_pre else y


def hashgrid_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, act: str = "none",
                             pre: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True,
                             need_db: bool = True, weight_dtype: torch.dtype = torch.float32,
                             dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, db: torch.Tensor | None = None,
                             accumulate: bool = False, workspace="auto", stream=None) -> tuple:
    """(dx, dw, db) of hashgrid_linear_forward for upstream ``dy`` [m, n] (x's type or float32); dx has x's type,
    dw ``weight_dtype`` (float32 or x's type), db is float32.  ``pre`` is the saved pre-activation (needed unless act
    is "none").  ``need_*`` leave an output out (None).  ``dx``, ``dw``, ``db`` receive the outputs; with
    ``accumulate`` dw and db, which must be given, are added to.  ``workspace``: a uint8 GPU tensor or "auto"."""
    _matrix(dy, "dy")
    _matrix(x, "x")
    _matrix(weight, "weight")
    m, k = x.shape
    n = weight.shape[0]
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate adds to dw and db: pass them")
    made = []

    def output(t, need, shape, dtype):
        if not need:
            return None
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=x.device)
            made.append(t)
        return t

    dw_dtype = weight_dtype if dw is None else dw.dtype
    dx = output(dx, need_dx, (m, k), x.dtype)
    dw = output(dw, need_dw, (n, k), dw_dtype)
    db = output(db, need_db, (n,), torch.float32)
    op = _LinearGrad(m, k, n, dy.data_ptr(), _rows(dy, "dy", (m, n), dy.dtype, x),
                     None if pre is None else pre.data_ptr(),
                     0 if pre is None else _rows(pre, "pre", (m, n), x.dtype, x),
                     x.data_ptr(), _rows(x, "x", (m, k), x.dtype, x),
                     weight.data_ptr(), _rows(weight, "weight", (n, k), x.dtype, x),
                     None if dx is None else dx.data_ptr(), 0 if dx is None else _rows(dx, "dx", (m, k), x.dtype, x),
                     None if dw is None else dw.data_ptr(), 0 if dw is None else _rows(dw, "dw", (n, k), dw_dtype, x),
                     None if db is None else _vector(db, "db", n, x),
                     _CODES[x.dtype], _CODES[dy.dtype], _CODES.get(dw_dtype, -1), _act(act), int(accumulate))
    lib = _lib()
    auto = isinstance(workspace, str)

    def alloc():
        size = ctypes.c_size_t(0)
        _check(lib.hashgrid_linear_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)))
        return torch.empty(size.value, dtype=torch.uint8, device=x.device) if size.value else None

    ws_ptr, ws_bytes, ws = _workspace(workspace, alloc, "workspace")
    _check(lib.hashgrid_linear_backward(ctypes.byref(op), ws_ptr, ws_bytes, _stream(x, stream)))
    if stream is not None:
        _keep_for_stream(x, stream, *made, ws if auto else None)
    return dx, dw, db


class RmsNormOutput(NamedTuple):
    """y; its row scales (8-bit y); the sum s and 1 / rms, where asked for."""
    y: torch.Tensor
    scale: torch.Tensor | None
    sum: torch.Tensor | None
    rstd: torch.Tensor | None


def hashgrid_rms_norm_forward(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None,
                              eps: float = 1e-6, out_dtype: torch.dtype | None = None, save_sum: bool = False,
                              save_rstd: bool = False, out: torch.Tensor | None = None,
                              sum_out: torch.Tensor | None = None, stream=None) -> RmsNormOutput:
    """y = s / sqrt(mean(s^2) + eps) * weight of s = x + residual, row by row, for x [m, c] in float32, float16 or
    bfloat16 and weight [c] in float32.  ``out_dtype`` is x's, or float8_e4m3fn with one scale a row.  ``save_sum``
    (or ``sum_out``, which may be x or the residual) keeps s in x's type, ``save_rstd`` the 1 / rms of each row."""
    _matrix(x, "x")
    m, c = x.shape
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    made = []
    y = out
    if y is None:
        y = torch.empty((m, c), dtype=out_dtype, device=x.device)
        made.append(y)
    scale = rstd = None
    if out_dtype == F8:
        scale = torch.empty(m, dtype=torch.float32, device=x.device)
        made.append(scale)
    s = sum_out
    if s is None and save_sum:
        s = torch.empty((m, c), dtype=x.dtype, device=x.device)
        made.append(s)
    if save_rstd:
        rstd = torch.empty(m, dtype=torch.float32, device=x.device)
        made.append(rstd)
    op = _RmsNorm(m, c, x.data_ptr(), _rows(x, "x", (m, c), x.dtype, x),
                  None if residual is None else residual.data_ptr(),
                  0 if residual is None else _rows(residual, "residual", (m, c), x.dtype, x),
                  _vector(weight, "weight", c, x), y.data_ptr(), _rows(y, "out", (m, c), out_dtype, x),
                  None if scale is None else scale.data_ptr(),
                  None if s is None else s.data_ptr(), 0 if s is None else _rows(s, "sum_out", (m, c), x.dtype, x),
                  None if rstd is None else rstd.data_ptr(), eps, _CODES[x.dtype], _CODES.get(out_dtype, -1))
    _check(_lib().hashgrid_rms_norm_forward(ctypes.byref(op), _stream(x, stream)))
    if stream is not None:
        _keep_for_stream(x, stream, *made)
    return RmsNormOutput(y, scale, s, rstd)


def hashgrid_rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                               ds: torch.Tensor | None = None, need_dw: bool = True, dx: torch.Tensor | None = None,
                               dw: torch.Tensor | None = None, accumulate: bool = False, workspace="auto",
                               stream=None) -> tuple:
    """(dx, dweight) of hashgrid_rms_norm_forward for upstream ``dy``, from the saved sum ``s`` and ``rstd``; ``ds`` is
    the gradient that reaches s itself and is added.  dx is the gradient of x and of the residual; dweight is float32
    (with ``accumulate``, ``dw`` must be given and is added to)."""
    _matrix(s, "s")
    m, c = s.shape
    if accumulate and need_dw and dw is None:
        raise ValueError("accumulate adds to dw: pass it")
    made = []
    if dx is None:
        dx = torch.empty((m, c), dtype=s.dtype, device=s.device)
        made.append(dx)
    if dw is None and need_dw:
        dw = torch.empty(c, dtype=torch.float32, device=s.device)
        made.append(dw)
    if not need_dw:
        dw = None
    op = _RmsNormGrad(m, c, dy.data_ptr(), _rows(dy, "dy", (m, c), s.dtype, s), s.data_ptr(),
                      _rows(s, "s", (m, c), s.dtype, s), _vector(weight, "weight", c, s), _vector(rstd, "rstd", m, s),
                      None if ds is None else ds.data_ptr(), 0 if ds is None else _rows(ds, "ds", (m, c), s.dtype, s),
                      dx.data_ptr(), _rows(dx, "dx", (m, c), s.dtype, s), None if dw is None else _vector(dw, "dw", c, s),
                      _CODES[s.dtype], int(accumulate))
    lib = _lib()
    auto = isinstance(workspace, str)

    def alloc():
        size = ctypes.c_size_t(0)
        _check(lib.hashgrid_rms_norm_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)))
        return torch.empty(size.value, dtype=torch.uint8, device=s.device) if size.value else None

    ws_ptr, ws_bytes, ws = _workspace(workspace, alloc, "workspace")
    _check(lib.hashgrid_rms_norm_backward(ctypes.byref(op), ws_ptr, ws_bytes, _stream(s, stream)))
    if stream is not None:
        _keep_for_stream(s, stream, *made, ws if auto else None)
    return dx, dw


@dataclass
class AdamWTensor:
    """One tensor of an AdamW step: a float32 parameter, its gradient (float32, float16 or bfloat16), its moments --
    both float32, or ``m`` float8_e4m3fn and ``v`` uint8 with the block exponents ``m_exp`` and ``v_exp`` (uint8, one
    per 256 values) -- and, if wanted, a 16-bit ``copy`` that receives the updated values.  All contiguous."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    m_exp: torch.Tensor | None = None
    v_exp: torch.Tensor | None = None
    copy: torch.Tensor | None = None
    lr: float = 1e-3
    weight_decay: float = 0.0

    @staticmethod
    def states(param: torch.Tensor, bits: int) -> dict:
        """Moments of zero for ``param``, ready for step 1."""
        if bits == 32:
            return dict(m=torch.zeros_like(param, memory_format=torch.contiguous_format),
                        v=torch.zeros_like(param, memory_format=torch.contiguous_format))
        if bits != 8:
            raise ValueError("moments have 32 or 8 bits")
        codes = [torch.zeros(param.shape, dtype=torch.uint8, device=param.device) for _ in range(2)]
        exps = [torch.ones(-(-param.numel() // 256), dtype=torch.uint8, device=param.device) for _ in range(2)]
        return dict(m=codes[0].view(F8), v=codes[1], m_exp=exps[0], v_exp=exps[1])


class HashGridAdamWPlan:
    """The tensors of an AdamW step, checked and described once; ``step`` updates them all in one call.  The plan
    holds the tensors; ``set_grads`` exchanges the gradients, ``set_rates`` the rates."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self._c = (_AdamWTensor * max(1, len(self.tensors)))()
        for i, t in enumerate(self.tensors):
            p = t.param
            _dev(p, "param", torch.float32)
            eight = t.m_exp is not None or t.v_exp is not None
            _dev(t.m, "m", F8 if eight else torch.float32)
            _dev(t.v, "v", torch.uint8 if eight else torch.float32)
            parts = [("param", p, p.shape), ("m", t.m, p.shape), ("v", t.v, p.shape)]
            if eight:
                blocks = torch.Size([-(-p.numel() // 256)])
                parts += [("m_exp", _dev(t.m_exp, "m_exp", torch.uint8), blocks),
                          ("v_exp", _dev(t.v_exp, "v_exp", torch.uint8), blocks)]
            if t.copy is not None:
                if t.copy.dtype not in _HALF:
                    raise ValueError("copy must be float16 or bfloat16")
                parts.append(("copy", _dev(t.copy, "copy", t.copy.dtype), p.shape))
            for name, part, shape in parts:
                if part.device != p.device or part.shape != shape or not part.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {p.device}")
            if p.device != self.tensors[0].param.device:
                raise ValueError("the tensors of a plan must be on one device")
            self._c[i] = _AdamWTensor(p.data_ptr(), None, t.m.data_ptr(), t.v.data_ptr(),
                                      t.m_exp.data_ptr() if eight else None, t.v_exp.data_ptr() if eight else None,
                                      None if t.copy is None else t.copy.data_ptr(), p.numel(), t.lr, t.weight_decay,
                                      HG_F32, 0 if t.copy is None else _CODES[t.copy.dtype], 8 if eight else 32, 0)
        self.set_grads([t.grad for t in self.tensors])

    def set_grads(self, grads) -> None:
        if len(grads) != len(self.tensors):
            raise ValueError(f"{len(self.tensors)} gradients are needed")
        for i, (t, g) in enumerate(zip(self.tensors, grads)):
            p = t.param
            if not isinstance(g, torch.Tensor) or g.device != p.device or g.shape != p.shape or not g.is_contiguous():
                raise ValueError(f"grad must be a contiguous {tuple(p.shape)} tensor on {p.device}")
            if g.dtype != torch.float32 and g.dtype not in _HALF:
                raise ValueError(f"grad must be float32, float16 or bfloat16, got {g.dtype}")
            t.grad = g
            self._c[i].grad = g.data_ptr()
            self._c[i].grad_dtype = _CODES[g.dtype]

    def set_rates(self, i: int, lr: float, weight_decay: float) -> None:
        self._c[i].lr, self._c[i].weight_decay = lr, weight_decay

    def step(self, *, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, seed: int = 0,
             grad_scale: torch.Tensor | None = None, zero_grad: bool = False, stream=None) -> None:
        """Update every tensor; ``step`` is the 1-based index of this update, ``seed`` that of the 8-bit moments'
        rounding noise (another one each step).  ``grad_scale``: a float32 GPU scalar the gradients are multiplied
        by; when it is not finite the step changes nothing.  ``zero_grad`` clears the gradients."""
        if not self.tensors:
            return
        p = self.tensors[0].param
        scale = None
        if grad_scale is not None:
            _dev(grad_scale, "grad_scale", torch.float32)
            if grad_scale.numel() != 1 or grad_scale.device != p.device:
                raise ValueError(f"grad_scale must be a scalar on {p.device}")
            scale = grad_scale.data_ptr()
        opt = _AdamW(beta1, beta2, eps, step, seed & 0xFFFFFFFF)
        _check(_lib().hashgrid_adamw_step(ctypes.byref(opt), self._c, len(self.tensors), scale,
                                          HG_ADAM_ZERO_GRAD if zero_grad else 0, _stream(p, stream)))


def hashgrid_adamw_step(tensors, **kw) -> None:
    """One AdamW update of a list of ``AdamWTensor``: ``HashGridAdamWPlan(tensors).step(**kw)``."""
    HashGridAdamWPlan(tensors).step(**kw)
