"""A residual head of any width on the hash-grid encoding, and the step that
trains it: binding of the linear, RMS norm and AdamW entry points of
include/hashgrid.h, their autograd functions, modules and optimizer.

As in ``hashgrid``, the binding only marshals arguments; every computation runs
in the HIP kernels of the library and there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from .hashgrid import (HG_ADAM_ZERO_GRAD, HG_F16, HG_F32, _check, _dev, _keep_for_stream, _stream, load_library)

HG_BF16, HG_F8 = 2, 3
HG_ADAM_ZERO_SKIPPED, HG_ADAM_CLOCK = 4, 8
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
    _fields_ = [("beta1", _F), ("beta2", _F), ("eps", _F), ("step", _I32), ("seed", ctypes.c_uint32), ("clocks", _P)]


def _packer(structure):
    """struct.Struct of a ctypes structure: packing the fields' values into bytes costs a quarter of building it."""
    codes, at = "@", 0
    for name, kind in structure._fields_:
        field = getattr(structure, name)
        codes += f"{field.offset - at}x" if field.offset > at else ""
        codes += {_P: "Q", _I64: "q", _I32: "i", _F: "f", ctypes.c_uint32: "I"}[kind]
        at = field.offset + field.size
    codes += f"{ctypes.sizeof(structure) - at}x" if ctypes.sizeof(structure) > at else ""
    packer = struct.Struct(codes)
    assert packer.size == ctypes.sizeof(structure)
    return packer.pack


_linear, _linear_grad, _rms_norm, _rms_norm_grad = (_packer(t) for t in (_Linear, _LinearGrad, _RmsNorm, _RmsNormGrad))

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


def _rows(t, name, shape, dtype, device) -> int:
    """Row stride of a matrix argument, after its checks."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be [{shape[0]}, {shape[1]}], got {list(t.shape)}")
    row, column = t.stride()
    if column != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return row


def _vector(t, name, n, device) -> int:
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a float32 tensor on {device}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous [{n}] tensor")
    return t.data_ptr()


#: The current stream's handle by device index; building a Stream object for it costs 1.5 us a call more.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _here(device, stream) -> int:
    """The stream of a call as an integer handle."""
    if stream is None:
        return _raw_stream(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


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
    dtype, device, mn = x.dtype, x.device, (m, n)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if dtype == F8 else dtype
    if out is None:
        y, ys = torch.empty(mn, dtype=out_dtype, device=device), n
    else:
        y, ys = out, _rows(out, "out", mn, out_dtype, device)
    pre = torch.empty(mn, dtype=dtype, device=device) if save_pre else None
    op = _linear(m, k, n, x.data_ptr(), _rows(x, "x", (m, k), dtype, device),
                 weight.data_ptr(), _rows(weight, "weight", (n, k), dtype, device),
                 0 if x_scale is None else _vector(x_scale, "x_scale", m, device),
                 0 if weight_scale is None else _vector(weight_scale, "weight_scale", n, device),
                 0 if bias is None else _vector(bias, "bias", n, device),
                 0 if residual is None else residual.data_ptr(),
                 0 if residual is None else _rows(residual, "residual", mn, out_dtype, device),
                 y.data_ptr(), ys, 0 if pre is None else pre.data_ptr(), n, _CODES[dtype], _CODES.get(out_dtype, -1), _act(act))
    if (rc := _lib().hashgrid_linear_forward(op, _here(device, stream))):
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, y if out is None else None, pre)
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
    dtype, device, mn = x.dtype, x.device, (m, n)
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate adds to dw and db: pass them")
    made = []
    dxs = dws = 0
    dw_dtype = weight_dtype if dw is None else dw.dtype
    if not need_dx:
        dx = None
    elif dx is None:
        dx, dxs = torch.empty((m, k), dtype=dtype, device=device), k
        made.append(dx)
    else:
        dxs = _rows(dx, "dx", (m, k), dtype, device)
    if not need_dw:
        dw = None
    elif dw is None:
        dw, dws = torch.empty((n, k), dtype=dw_dtype, device=device), k
        made.append(dw)
    else:
        dws = _rows(dw, "dw", (n, k), dw_dtype, device)
    if not need_db:
        db = None
    elif db is None:
        db = torch.empty((n,), dtype=torch.float32, device=device)
        made.append(db)
    op = _linear_grad(m, k, n, dy.data_ptr(), _rows(dy, "dy", mn, dy.dtype, device),
                      0 if pre is None else pre.data_ptr(), 0 if pre is None else _rows(pre, "pre", mn, dtype, device),
                      x.data_ptr(), _rows(x, "x", (m, k), dtype, device),
                      weight.data_ptr(), _rows(weight, "weight", (n, k), dtype, device),
                      0 if dx is None else dx.data_ptr(), dxs, 0 if dw is None else dw.data_ptr(), dws,
                      0 if db is None else _vector(db, "db", n, device),
                      _CODES[dtype], _CODES[dy.dtype], _CODES.get(dw_dtype, -1), _act(act), accumulate)
    lib = _lib()
    rc, made_ws = _with_workspace(lib.hashgrid_linear_backward_workspace_size, lib.hashgrid_linear_backward, op, workspace,
                                  device, stream)
    if rc:
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, *made, made_ws)
    return dx, dw, db


def _with_workspace(sizer, call, op, workspace, device, stream):
    """(return code of ``call``, the workspace made here if any)."""
    ptr = size = 0
    made = None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, 'auto' or None")
        need = ctypes.c_size_t(0)
        rc = sizer(op, ctypes.byref(need))
        if rc:
            return rc, None
        size = need.value
        if size:
            made = torch.empty(size, dtype=torch.uint8, device=device)
            ptr = made.data_ptr()
    elif workspace is not None:
        _dev(workspace, "workspace", torch.uint8)
        ptr, size = workspace.data_ptr(), workspace.numel()
    return call(op, ptr, size, _here(device, stream)), made


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
    m, c = mc = x.shape
    dtype, device = x.dtype, x.device
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    y = torch.empty(mc, dtype=out_dtype, device=device) if out is None else out
    scale = torch.empty(m, dtype=torch.float32, device=device) if out_dtype == F8 else None
    s = sum_out
    if s is None and save_sum:
        s = torch.empty(mc, dtype=dtype, device=device)
    rstd = torch.empty(m, dtype=torch.float32, device=device) if save_rstd else None
    op = _rms_norm(m, c, x.data_ptr(), _rows(x, "x", mc, dtype, device),
                   0 if residual is None else residual.data_ptr(),
                   0 if residual is None else _rows(residual, "residual", mc, dtype, device),
                   _vector(weight, "weight", c, device), y.data_ptr(), c if out is None else _rows(y, "out", mc, out_dtype, device),
                   0 if scale is None else scale.data_ptr(),
                   0 if s is None else s.data_ptr(), 0 if s is None else _rows(s, "sum_out", mc, dtype, device),
                   0 if rstd is None else rstd.data_ptr(), eps, _CODES[dtype], _CODES.get(out_dtype, -1))
    if (rc := _lib().hashgrid_rms_norm_forward(op, _here(device, stream))):
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, y if out is None else None, scale, s if sum_out is None else None, rstd)
    return RmsNormOutput(y, scale, s, rstd)


def hashgrid_rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                               ds: torch.Tensor | None = None, need_dw: bool = True, dx: torch.Tensor | None = None,
                               dw: torch.Tensor | None = None, accumulate: bool = False, workspace="auto",
                               stream=None) -> tuple:
    """(dx, dweight) of hashgrid_rms_norm_forward for upstream ``dy``, from the saved sum ``s`` and ``rstd``; ``ds`` is
    the gradient that reaches s itself and is added.  dx is the gradient of x and of the residual; dweight is float32
    (with ``accumulate``, ``dw`` must be given and is added to).  ``dx`` receives the gradient; it may be dy, s or ds for
    rows of up to 4096 columns."""
    _matrix(s, "s")
    m, c = mc = s.shape
    dtype, device = s.dtype, s.device
    if accumulate and need_dw and dw is None:
        raise ValueError("accumulate adds to dw: pass it")
    made = []
    if dx is None:
        dx, dxs = torch.empty(mc, dtype=dtype, device=device), c
        made.append(dx)
    else:
        dxs = _rows(dx, "dx", mc, dtype, device)
    if not need_dw:
        dw = None
    elif dw is None:
        dw = torch.empty(c, dtype=torch.float32, device=device)
        made.append(dw)
    op = _rms_norm_grad(m, c, dy.data_ptr(), _rows(dy, "dy", mc, dtype, device), s.data_ptr(), _rows(s, "s", mc, dtype, device),
                        _vector(weight, "weight", c, device), _vector(rstd, "rstd", m, device),
                        0 if ds is None else ds.data_ptr(), 0 if ds is None else _rows(ds, "ds", mc, dtype, device),
                        dx.data_ptr(), dxs, 0 if dw is None else _vector(dw, "dw", c, device), _CODES[dtype], accumulate)
    lib = _lib()
    rc, made_ws = _with_workspace(lib.hashgrid_rms_norm_backward_workspace_size, lib.hashgrid_rms_norm_backward, op, workspace,
                                  device, stream)
    if rc:
        _check(rc)
    if stream is not None:
        _keep_for_stream(s, stream, *made, made_ws)
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

    def step(self, *, step: int = 0, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, seed: int = 0,
             grad_scale: torch.Tensor | None = None, zero_grad: bool = False, zero_skipped: bool = False,
             clocks: torch.Tensor | None = None, stream=None) -> None:
        """Update every tensor; ``step`` is the 1-based index of this update, ``seed`` that of the 8-bit moments'
        rounding noise (another one each step).  With ``clocks``, an int32 [tensors, 4] GPU tensor, ``step`` is not
        needed: column 0 counts each tensor's steps, those that were not skipped, and ``seed`` may stay the same.  ``grad_scale``: a float32 GPU scalar the gradients are multiplied
        by; when it is not finite the step changes nothing.  ``zero_grad`` clears the gradients, with ``zero_skipped``
        also those of a step that grad_scale skips."""
        if not self.tensors:
            return
        p = self.tensors[0].param
        scale = None
        if grad_scale is not None:
            _dev(grad_scale, "grad_scale", torch.float32)
            if grad_scale.numel() != 1 or grad_scale.device != p.device:
                raise ValueError(f"grad_scale must be a scalar on {p.device}")
            scale = grad_scale.data_ptr()
        flags = (HG_ADAM_ZERO_GRAD if zero_grad else 0) | (HG_ADAM_ZERO_SKIPPED if zero_skipped else 0)
        if clocks is not None:
            _dev(clocks, "clocks", torch.int32)
            if clocks.shape != (len(self.tensors), 4) or not clocks.is_contiguous() or clocks.device != p.device:
                raise ValueError(f"clocks must be a contiguous [{len(self.tensors)}, 4] tensor on {p.device}")
            flags |= HG_ADAM_CLOCK
        opt = _AdamW(beta1, beta2, eps, step, seed & 0xFFFFFFFF, None if clocks is None else clocks.data_ptr())
        _check(_lib().hashgrid_adamw_step(ctypes.byref(opt), self._c, len(self.tensors), scale, flags, _stream(p, stream)))


def hashgrid_adamw_step(tensors, **kw) -> None:
    """One AdamW update of a list of ``AdamWTensor``: ``HashGridAdamWPlan(tensors).step(**kw)``."""
    HashGridAdamWPlan(tensors).step(**kw)


class HashGridLinearFunction(torch.autograd.Function):
    """Autograd of hashgrid_linear_forward: x in a 16-bit type, the weight an fp32 master that the products read
    rounded to it, bias fp32, residual in the output's type.  Gradients of the masters are fp32.  The gradients cannot
    be differentiated again: autograd raises."""

    @staticmethod
    def forward(ctx, x, weight, bias, act="none", residual=None, out_dtype=None):
        w = weight.to(x.dtype)
        train = any(ctx.needs_input_grad)
        # ReLU's slope can be read from y itself where no residual was added
        keep = train and act != "none" and not (act == "relu" and residual is None and out_dtype in (None, x.dtype))
        out = hashgrid_linear_forward(x, w, bias, act=act, residual=residual, out_dtype=out_dtype, save_pre=keep)
        y, pre = out if keep else (out, out if train and act == "relu" else None)
        ctx.act = act
        ctx.save_for_backward(x, w, pre)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, pre = ctx.saved_tensors
        need = ctx.needs_input_grad + (False,) * (6 - len(ctx.needs_input_grad))  # arguments may have been left out
        dy = dy.contiguous()
        dx, dw, db = hashgrid_linear_backward(dy, x, w, act=ctx.act, pre=pre, need_dx=need[0], need_dw=need[1],
                                              need_db=need[2])
        return dx, dw, db, None, dy if need[4] else None, None


class HashGridRmsNormFunction(torch.autograd.Function):
    """Autograd of hashgrid_rms_norm_forward: returns y, or (y, s) with a residual, s = x + residual in x's type.
    The gradients cannot be differentiated again: autograd raises."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, eps=1e-6):
        out = hashgrid_rms_norm_forward(x, weight, residual=residual, eps=eps, save_sum=residual is not None, save_rstd=True)
        s = x if residual is None else out.sum
        ctx.save_for_backward(s, weight, out.rstd)
        ctx.set_materialize_grads(False)  # an output that nothing reads has no gradient, not one of zeros
        return out.y if residual is None else (out.y, out.sum)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad + (False,) * (4 - len(ctx.needs_input_grad))
        if dy is None:  # s alone goes on
            return ds, torch.zeros_like(weight) if need[1] else None, ds if need[2] else None, None
        dx, dw = hashgrid_rms_norm_backward(dy.contiguous(), s, weight, rstd, ds=None if ds is None else ds.contiguous(),
                                            need_dw=need[1])
        return dx, dw, dx if need[2] else None, None


class HashGridResidualHead(torch.nn.Module):
    """A residual head of any width on the encoding: ``forward(features [n, in_features]) -> [n, out_features]`` fp32.

        h = stem(features)
        per block: h = h + W2 act(W1 norm(h) + b1) + b2
        y = W norm(h + stem's h) + b

    Weights, biases and norm weights are fp32 masters; activations and the weights' copies that the matrix cores read
    are ``dtype`` (bfloat16 or float16).  ``quantized()`` is the same head for inference with 8-bit operands behind
    the blocks' norms."""

    def __init__(self, in_features=32, width=256, blocks=2, out_features=4, act="silu", dtype=torch.bfloat16,
                 eps=1e-6, device="cuda"):
        super().__init__()
        if dtype not in _HALF:
            raise ValueError("dtype must be torch.float16 or torch.bfloat16")
        _act(act)
        self.act, self.dtype, self.eps, self.blocks = act, dtype, eps, blocks

        def layer(name, fan_in, fan_out):
            w = torch.empty((fan_out, fan_in), device=device)
            torch.nn.init.xavier_uniform_(w)
            b = torch.empty(fan_out, device=device).uniform_(-fan_in ** -0.5, fan_in ** -0.5)
            self.register_parameter(f"{name}_w", torch.nn.Parameter(w))
            self.register_parameter(f"{name}_b", torch.nn.Parameter(b))

        layer("stem", in_features, width)
        for i in range(blocks):
            self.register_parameter(f"norm{i}", torch.nn.Parameter(torch.ones(width, device=device)))
            layer(f"up{i}", width, width)
            layer(f"down{i}", width, width)
        self.register_parameter("norm_out", torch.nn.Parameter(torch.ones(width, device=device)))
        layer("out", width, out_features)

    def _layer(self, name):
        return getattr(self, f"{name}_w"), getattr(self, f"{name}_b")

    def forward(self, features: torch.Tensor) -> torch.Tensor:
        linear, norm = HashGridLinearFunction.apply, HashGridRmsNormFunction.apply
        h = stem = linear(features.to(self.dtype), *self._layer("stem"))
        for i in range(self.blocks):
            u = linear(norm(h, getattr(self, f"norm{i}"), None, self.eps), *self._layer(f"up{i}"), self.act)
            h = linear(u, *self._layer(f"down{i}"), "none", h)
        y, _ = norm(h, self.norm_out, stem, self.eps)
        return linear(y, *self._layer("out"), "none", None, torch.float32)

    def quantized(self) -> "HashGridResidualHead8":
        return HashGridResidualHead8(self)


def quantize_rows(w: torch.Tensor) -> tuple:
    """(e4m3 values, scales) of a matrix, one scale a row: the largest magnitude of a row at 448."""
    w = w.detach().float()
    scale = w.abs().amax(1) / 448.0
    up = torch.where(scale < 2.0 ** -100, 2.0 ** 100, 1.0)  # 1 / scale of a tiny row would not be finite
    inv = torch.where(scale > 0, 1.0 / (scale * up), torch.zeros_like(scale))
    return (w * up[:, None] * inv[:, None]).clamp(-448.0, 448.0).to(F8), scale


class HashGridResidualHead8:
    """A HashGridResidualHead for inference: the blocks' first products read 8-bit rows with scales, which the norm
    writes, and 8-bit weights; the residual stream, the other products and the outputs stay in the head's 16-bit type."""

    def __init__(self, head: HashGridResidualHead):
        self.act, self.dtype, self.eps, self.blocks = head.act, head.dtype, head.eps, head.blocks
        grab = lambda t: t.detach().clone()  # noqa: E731
        self.stem = head.stem_w.detach().to(self.dtype), grab(head.stem_b)
        self.layers = [(grab(getattr(head, f"norm{i}")), *quantize_rows(getattr(head, f"up{i}_w")), grab(getattr(head, f"up{i}_b")),
                        getattr(head, f"down{i}_w").detach().to(self.dtype), grab(getattr(head, f"down{i}_b")))
                       for i in range(self.blocks)]
        self.out = grab(head.norm_out), head.out_w.detach().to(self.dtype), grab(head.out_b)

    def __call__(self, features: torch.Tensor) -> torch.Tensor:
        h = stem = hashgrid_linear_forward(features.to(self.dtype), *self.stem)
        for norm, w8, ws, b1, w2, b2 in self.layers:
            n8, scale, _, _ = hashgrid_rms_norm_forward(h, norm, eps=self.eps, out_dtype=F8)
            u = hashgrid_linear_forward(n8, w8, b1, act=self.act, x_scale=scale, weight_scale=ws, out_dtype=self.dtype)
            h = hashgrid_linear_forward(u, w2, b2, residual=h)
        norm, w, b = self.out
        return hashgrid_linear_forward(hashgrid_rms_norm_forward(h, norm, residual=stem, eps=self.eps).y, w, b,
                                       out_dtype=torch.float32)


class HashGridAdamW(torch.optim.Optimizer):
    """AdamW over the tables and a head's weights, all tensors in one call (hashgrid_adamw_step).  Groups have their own
    ``lr`` and ``weight_decay`` (the pages: no decay on the tables, a rate 5 to 10 times the head's); ``state_bits`` 8
    keeps the moments in 8 bits.  ``grad_scale`` of ``step`` is the float32 GPU scalar gradients are multiplied by; when
    it is not finite the step leaves parameters and moments as they are and does not count: each state's "step" is an
    int32 on the GPU.  ``zero_grad_in_step`` clears the gradients inside the step, a skipped one too, so that the next
    backward can add to them."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.99), eps=1e-15, weight_decay=0.0, state_bits=32, seed=0,
                 zero_grad_in_step=False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits))
        self.seed, self.zero_grad_in_step = seed, zero_grad_in_step

    @torch.no_grad()
    def step(self, closure=None, grad_scale: torch.Tensor | None = None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        calls: dict = {}
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                st = self.state[p]
                if not st:
                    st["step"] = 0
                    st.update(AdamWTensor.states(p, group["state_bits"]))
                tensors, states = calls.setdefault((tuple(group["betas"]), group["eps"]), ([], []))
                tensors.append(AdamWTensor(p, p.grad, st["m"], st["v"], st.get("m_exp"), st.get("v_exp"), None, group["lr"],
                                           group["weight_decay"]))
                states.append(st)
        for ((b1, b2), eps), (tensors, states) in calls.items():
            HashGridAdamWPlan(tensors).step(beta1=b1, beta2=b2, eps=eps, seed=self.seed, grad_scale=grad_scale,
                                            zero_grad=self.zero_grad_in_step, zero_skipped=self.zero_grad_in_step,
                                            clocks=self._clocks(states, tensors[0].param.device))
        return loss

    @staticmethod
    def _clocks(states, device) -> torch.Tensor:
        """The [n, 4] clocks of a call, whose column 0 the states' "step" are: as they lie where the same states came
        together before, else gathered anew (from a checkpoint's numbers too)."""
        steps = [st["step"] for st in states]
        if all(isinstance(s, torch.Tensor) and s.device == device and s.dtype == torch.int32 for s in steps):
            at = steps[0].untyped_storage()
            if at.nbytes() == 16 * len(steps) and all(s.data_ptr() == at.data_ptr() + 16 * i for i, s in enumerate(steps)):
                return torch.as_strided(steps[0], (len(steps), 4), (4, 1), 0)
        clocks = torch.zeros(len(steps), 4, dtype=torch.int32, device=device)
        if any(isinstance(s, torch.Tensor) or s for s in steps):
            clocks[:, 0] = torch.stack([torch.as_tensor(s, device=device).reshape(()).to(torch.int32) for s in steps])
        for i, st in enumerate(states):
            st["step"] = clocks[i, 0]
        return clocks

    def load_state_dict(self, state_dict):
        """Restores 8-bit moments in their own types, which Optimizer.load_state_dict turns into the parameter's, and
        counts of its own, which it would share with the dict."""
        super().load_state_dict(state_dict)
        for st in self.state.values():
            if isinstance(st.get("step"), torch.Tensor):
                st["step"] = st["step"].clone()
            if "m_exp" in st:
                st["m"] = st["m"].to(F8)
                for k in ("v", "m_exp", "v_exp"):
                    st[k] = st[k].to(torch.uint8)
