"""A head with per-image codes, layer norms and gated feed-forward blocks: binding of the embedding, layer norm and
gated entry points of include/hashgrid.h, their autograd functions and modules.

As in ``residual``, the binding only marshals arguments; every computation runs in the HIP kernels of the library and
there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from .hashgrid import _check, _dev, _keep_for_stream
from .residual import (_CODES, _F, _HALF, _I32, _I64, _P, F8, HashGridLinearFunction, _act, _here, _matrix, _packer, _recorded, _rows,
                       _vector, hashgrid_linear_forward, quantize_rows)
from .residual import _lib as _residual_lib

_IDS = {torch.int32: 32, torch.int64: 64}


class _Embedding(ctypes.Structure):
    _fields_ = [("m", _I64), ("rows", _I32), ("c", _I32), ("ids", _P), ("table", _P), ("table_stride", _I64), ("y", _P),
                ("y_stride", _I64), ("scale", _F), ("ids_bits", _I32), ("table_dtype", _I32), ("y_dtype", _I32)]


class _EmbeddingGrad(ctypes.Structure):
    _fields_ = [("m", _I64), ("rows", _I32), ("c", _I32), ("ids", _P), ("dy", _P), ("dy_stride", _I64), ("dtable", _P),
                ("dtable_stride", _I64), ("scale", _F), ("ids_bits", _I32), ("dy_dtype", _I32), ("dtable_dtype", _I32),
                ("accumulate", _I32)]


class _LayerNorm(ctypes.Structure):
    _fields_ = [("m", _I64), ("c", _I32), ("x", _P), ("x_stride", _I64), ("residual", _P), ("residual_stride", _I64), ("w", _P),
                ("b", _P), ("y", _P), ("y_stride", _I64), ("y_scale", _P), ("sum", _P), ("sum_stride", _I64), ("mean", _P),
                ("rstd", _P), ("eps", _F), ("dtype", _I32), ("y_dtype", _I32)]


class _LayerNormGrad(ctypes.Structure):
    _fields_ = [("m", _I64), ("c", _I32), ("dy", _P), ("dy_stride", _I64), ("sum", _P), ("sum_stride", _I64), ("w", _P),
                ("mean", _P), ("rstd", _P), ("ds", _P), ("ds_stride", _I64), ("dx", _P), ("dx_stride", _I64), ("dw", _P),
                ("db", _P), ("dtype", _I32), ("accumulate", _I32)]


class _Gated(ctypes.Structure):
    _fields_ = [("m", _I64), ("k", _I32), ("n", _I32), ("x", _P), ("x_stride", _I64), ("wg", _P), ("wg_stride", _I64), ("wu", _P),
                ("wu_stride", _I64), ("x_scale", _P), ("g_scale", _P), ("u_scale", _P), ("bg", _P), ("bu", _P), ("h", _P),
                ("h_stride", _I64), ("gate", _P), ("up", _P), ("gate_stride", _I64), ("up_stride", _I64), ("x_dtype", _I32),
                ("h_dtype", _I32), ("act", _I32)]


class _GatedGrad(ctypes.Structure):
    _fields_ = [("m", _I64), ("k", _I32), ("n", _I32), ("dh", _P), ("dh_stride", _I64), ("gate", _P), ("up", _P),
                ("gate_stride", _I64), ("up_stride", _I64), ("x", _P), ("x_stride", _I64), ("wg", _P), ("wu", _P),
                ("wg_stride", _I64), ("wu_stride", _I64), ("dx", _P), ("dx_stride", _I64), ("dwg", _P), ("dwu", _P),
                ("dwg_stride", _I64), ("dwu_stride", _I64), ("dbg", _P), ("dbu", _P), ("dtype", _I32), ("dw_dtype", _I32),
                ("act", _I32), ("accumulate", _I32)]


_embedding, _embedding_grad, _layer_norm, _layer_norm_grad, _gated, _gated_grad = (
    _packer(t) for t in (_Embedding, _EmbeddingGrad, _LayerNorm, _LayerNormGrad, _Gated, _GatedGrad))

_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        lib = _residual_lib()
        size = ctypes.c_size_t
        for name in ("embedding", "layer_norm", "gated"):
            for end, args in (("forward", [_P, _P]), ("backward_workspace_size", [_P, _P]), ("backward", [_P, _P, size, _P])):
                fn = getattr(lib, f"hashgrid_{name}_{end}")
                fn.argtypes, fn.restype = args, ctypes.c_int
        _bound = lib
    return _bound


_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(device, call, *args) -> int:
    """``call`` with the tensors' device as the current one."""
    if device.index == _current():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _launch_with_workspace(name, op, workspace, device, stream):
    """(return code of the backward ``name``, the workspace made here if any)."""
    lib = _lib()
    ptr = size = 0
    made = None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, 'auto' or None")
        need = ctypes.c_size_t(0)
        rc = getattr(lib, f"hashgrid_{name}_backward_workspace_size")(op, ctypes.byref(need))
        if rc:
            return rc, None
        size = need.value
        if size:
            made = torch.empty(size, dtype=torch.uint8, device=device)
            ptr = made.data_ptr()
    elif workspace is not None:
        _dev(workspace, "workspace", torch.uint8)
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        ptr, size = workspace.data_ptr(), workspace.numel()
    return _launch(device, getattr(lib, f"hashgrid_{name}_backward"), op, ptr, size, _here(device, stream)), made


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _opt_rows(t, name, shape, dtype, device) -> int:
    return 0 if t is None else _rows(t, name, shape, dtype, device)


def _opt_vector(t, name, n, device) -> int:
    return 0 if t is None else _vector(t, name, n, device)


def _ids(ids, device) -> torch.Tensor:
    if not isinstance(ids, torch.Tensor) or ids.device != device or ids.dtype not in _IDS:
        raise ValueError(f"ids must be an int32 or int64 tensor on {device}")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be one-dimensional and contiguous")
    return ids


def hashgrid_embedding_forward(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out_dtype: torch.dtype | None = None,
                               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """scale * table[ids] for a table [rows, c] in float32, float16 or bfloat16 and ids [m] in int32 or int64; an id
    outside 0 .. rows - 1 (such as -1) names no row and gives zeros.  The result has the table's type, or ``out_dtype``
    float16 or bfloat16 of a float32 table.  ``out`` [m, c] receives it: columns of a wider buffer, for instance."""
    rows, c = _matrix(table, "table").shape
    device = table.device
    m = _ids(ids, device).shape[0]
    if rows >= 1 << 31 or c >= 1 << 31:
        raise ValueError("table has 2^31 rows or columns, or more")
    if out_dtype is None:
        out_dtype = table.dtype if out is None else out.dtype
    y, ys = (torch.empty((m, c), dtype=out_dtype, device=device), c) if out is None else (out, _rows(out, "out", (m, c), out_dtype, device))
    op = _embedding(m, rows, c, ids.data_ptr(), table.data_ptr(), _rows(table, "table", (rows, c), table.dtype, device), y.data_ptr(), ys,
                    scale, _IDS[ids.dtype], _CODES[table.dtype], _CODES.get(out_dtype, -1))
    if (rc := _launch(device, _lib().hashgrid_embedding_forward, op, _here(device, stream))):
        _check(rc)
    if stream is not None:
        _keep_for_stream(table, stream, y if out is None else None)
    return y


def hashgrid_embedding_backward(dy: torch.Tensor, ids: torch.Tensor, rows: int, *, scale: float = 1.0,
                                table_dtype: torch.dtype = torch.float32, dtable: torch.Tensor | None = None,
                                accumulate: bool = False, workspace="auto", stream=None) -> torch.Tensor:
    """Gradient [rows, c] of hashgrid_embedding_forward's table for upstream ``dy`` [m, c]: row v is scale times the sum
    of dy's rows whose id is v, zeros where there is none; ids that name no row are left out.  ``table_dtype`` is
    float32 or dy's type.  ``dtable`` receives the gradient; with ``accumulate`` it must be given and is added to.
    ``workspace``: a uint8 GPU tensor or "auto"."""
    m, c = _matrix(dy, "dy").shape
    device = dy.device
    if _ids(ids, device).shape[0] != m:
        raise ValueError(f"{m} ids are needed, got {ids.shape[0]}")
    rows = int(rows)
    if not 0 <= rows < 1 << 31 or c >= 1 << 31:
        raise ValueError("rows must lie in 0 .. 2^31 - 1")
    if accumulate and dtable is None:
        raise ValueError("accumulate adds to dtable: pass it")
    if dtable is None:
        out, os_ = torch.empty((rows, c), dtype=table_dtype, device=device), c
    else:
        if not isinstance(dtable, torch.Tensor):
            raise ValueError("dtable must be a tensor")
        out, os_ = dtable, _rows(dtable, "dtable", (rows, c), dtable.dtype, device)
    op = _embedding_grad(m, rows, c, ids.data_ptr(), dy.data_ptr(), _rows(dy, "dy", (m, c), dy.dtype, device), out.data_ptr(), os_,
                         scale, _IDS[ids.dtype], _CODES[dy.dtype], _CODES.get(out.dtype, -1), accumulate)
    rc, made = _launch_with_workspace("embedding", op, workspace, device, stream)
    if rc:
        _check(rc)
    if stream is not None:
        _keep_for_stream(dy, stream, out if dtable is None else None, made)
    return out


class LayerNormOutput(NamedTuple):
    """y; its row scales (8-bit y); the sum s, the mean and 1 / deviation of each row, where asked for."""
    y: torch.Tensor
    scale: torch.Tensor | None
    sum: torch.Tensor | None
    mean: torch.Tensor | None
    rstd: torch.Tensor | None


def hashgrid_layer_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                                residual: torch.Tensor | None = None, eps: float = 1e-5, out_dtype: torch.dtype | None = None,
                                save_sum: bool = False, save_stats: bool = False, out: torch.Tensor | None = None,
                                sum_out: torch.Tensor | None = None, stream=None) -> LayerNormOutput:
    """y = (s - mean) / sqrt(var + eps) * weight + bias of s = x + residual, row by row, for x [m, c] in float32, float16
    or bfloat16 and weight and bias [c] in float32 (None: ones, zeros).  ``out_dtype`` is x's, or float8_e4m3fn with one
    scale a row.  ``save_sum`` (or ``sum_out``, which may be x or the residual) keeps s in x's type, ``save_stats`` the
    mean and 1 / sqrt(var + eps) of each row."""
    m, c = mc = _matrix(x, "x").shape
    dtype, device = x.dtype, x.device
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    y = torch.empty(mc, dtype=out_dtype, device=device) if out is None else out
    scale = torch.empty(m, dtype=torch.float32, device=device) if out_dtype == F8 else None
    s = sum_out
    if s is None and save_sum:
        s = torch.empty(mc, dtype=dtype, device=device)
    mean, rstd = (torch.empty(m, dtype=torch.float32, device=device) for _ in range(2)) if save_stats else (None, None)
    op = _layer_norm(m, c, x.data_ptr(), _rows(x, "x", mc, dtype, device), _ptr(residual),
                     _opt_rows(residual, "residual", mc, dtype, device), _opt_vector(weight, "weight", c, device),
                     _opt_vector(bias, "bias", c, device), y.data_ptr(), c if out is None else _rows(y, "out", mc, out_dtype, device),
                     _ptr(scale), _ptr(s), _opt_rows(s, "sum_out", mc, dtype, device), _ptr(mean), _ptr(rstd), eps, _CODES[dtype],
                     _CODES.get(out_dtype, -1))
    if (rc := _launch(device, _lib().hashgrid_layer_norm_forward, op, _here(device, stream))):
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, y if out is None else None, scale, s if sum_out is None else None, mean, rstd)
    return LayerNormOutput(y, scale, s, mean, rstd)


def hashgrid_layer_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                                 rstd: torch.Tensor, *, ds: torch.Tensor | None = None, need_dw: bool = True, need_db: bool = True,
                                 dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, db: torch.Tensor | None = None,
                                 accumulate: bool = False, workspace="auto", stream=None) -> tuple:
    """(dx, dweight, dbias) of hashgrid_layer_norm_forward for upstream ``dy``, from the saved sum ``s``, ``mean`` and
    ``rstd``; ``ds`` is the gradient that reaches s itself and is added.  dx is the gradient of x and of the residual;
    dweight and dbias are float32 (with ``accumulate``, ``dw`` and ``db`` must be given and are added to) or left out
    (None) without ``need_dw``, ``need_db``.  ``dx`` receives the gradient; it may be dy, s or ds for rows of up to 4096
    columns."""
    m, c = mc = _matrix(s, "s").shape
    dtype, device = s.dtype, s.device
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate adds to dw and db: pass them")
    made = []

    def vector(v, need):
        if not need:
            return None
        if v is None:
            made.append(torch.empty(c, dtype=torch.float32, device=device))
            return made[-1]
        return v

    if dx is None:
        dx, dxs = torch.empty(mc, dtype=dtype, device=device), c
        made.append(dx)
    else:
        dxs = _rows(dx, "dx", mc, dtype, device)
    dw, db = vector(dw, need_dw), vector(db, need_db)
    op = _layer_norm_grad(m, c, dy.data_ptr(), _rows(dy, "dy", mc, dtype, device), s.data_ptr(), _rows(s, "s", mc, dtype, device),
                          _opt_vector(weight, "weight", c, device), _vector(mean, "mean", m, device), _vector(rstd, "rstd", m, device),
                          _ptr(ds), _opt_rows(ds, "ds", mc, dtype, device), dx.data_ptr(), dxs, _opt_vector(dw, "dw", c, device),
                          _opt_vector(db, "db", c, device), _CODES[dtype], accumulate)
    rc, made_ws = _launch_with_workspace("layer_norm", op, workspace, device, stream)
    if rc:
        _check(rc)
    if stream is not None:
        _keep_for_stream(s, stream, *made, made_ws)
    return dx, dw, db


def hashgrid_gated_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, b_gate: torch.Tensor | None = None,
                           b_up: torch.Tensor | None = None, *, act: str = "silu", x_scale: torch.Tensor | None = None,
                           gate_scale: torch.Tensor | None = None, up_scale: torch.Tensor | None = None,
                           out_dtype: torch.dtype | None = None, save_pre: bool = False, out: torch.Tensor | None = None, stream=None):
    """h = act(x w_gate^T + b_gate) * (x w_up^T + b_up) for x [m, k] and weights [n, k] in float16 or bfloat16, or all in
    float8_e4m3fn with ``x_scale`` [m], ``gate_scale`` and ``up_scale`` [n].  h has ``out_dtype``: x's or float32, for
    8-bit operands also float16 or bfloat16 (the default).  Biases are float32.  ``out`` receives h.  With ``save_pre``
    the call returns (h, gate, up), the two projections in x's type for the backward."""
    m, k = _matrix(x, "x").shape
    n = _matrix(w_gate, "w_gate").shape[0]
    dtype, device, mn, nk = x.dtype, x.device, (m, n), (n, k)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if dtype == F8 else dtype
    h, hs = (torch.empty(mn, dtype=out_dtype, device=device), n) if out is None else (out, _rows(out, "out", mn, out_dtype, device))
    gate, up = (torch.empty(mn, dtype=dtype, device=device) for _ in range(2)) if save_pre else (None, None)
    op = _gated(m, k, n, x.data_ptr(), _rows(x, "x", (m, k), dtype, device), w_gate.data_ptr(), _rows(w_gate, "w_gate", nk, dtype, device),
                _matrix(w_up, "w_up").data_ptr(), _rows(w_up, "w_up", nk, dtype, device), _opt_vector(x_scale, "x_scale", m, device),
                _opt_vector(gate_scale, "gate_scale", n, device), _opt_vector(up_scale, "up_scale", n, device),
                _opt_vector(b_gate, "b_gate", n, device), _opt_vector(b_up, "b_up", n, device), h.data_ptr(), hs, _ptr(gate), _ptr(up), n, n,
                _CODES[dtype], _CODES.get(out_dtype, -1), _act(act))
    if (rc := _launch(device, _lib().hashgrid_gated_forward, op, _here(device, stream))):
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, h if out is None else None, gate, up)
    return (h, gate, up) if save_pre else h


def hashgrid_gated_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, gate: torch.Tensor,
                            up: torch.Tensor, *, act: str = "silu", need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                            weight_dtype: torch.dtype = torch.float32, dx: torch.Tensor | None = None,
                            dw_gate: torch.Tensor | None = None, dw_up: torch.Tensor | None = None,
                            db_gate: torch.Tensor | None = None, db_up: torch.Tensor | None = None, accumulate: bool = False,
                            workspace="auto", stream=None) -> tuple:
    """(dx, dw_gate, dw_up, db_gate, db_up) of hashgrid_gated_forward for upstream ``dh`` [m, n], from the projections
    ``gate`` and ``up`` it kept, all in x's type.  dx has x's type, the weights' gradients ``weight_dtype`` (float32 or
    x's type), the biases' float32.  ``need_*`` leave outputs out (None).  ``dx``, ``dw_*``, ``db_*`` receive the
    outputs (of a pair both or neither); with ``accumulate`` dw_* and db_*, which must be given, are added to.  The
    gradients of gate and up enter the products in x's type: in float16, upstream gradients below some 2^-14 (a mean
    loss over many points has them) need a loss scale."""
    m, k = _matrix(x, "x").shape
    n = _matrix(w_gate, "w_gate").shape[0]
    dtype, device, mn, nk = x.dtype, x.device, (m, n), (n, k)
    if accumulate and ((need_dw and (dw_gate is None or dw_up is None)) or (need_db and (db_gate is None or db_up is None))):
        raise ValueError("accumulate adds to dw_gate, dw_up, db_gate and db_up: pass them")
    made = []

    def new(shape, kind):
        made.append(torch.empty(shape, dtype=kind, device=device))
        return made[-1]

    dw_dtype = weight_dtype if dw_gate is None else dw_gate.dtype
    dx = None if not need_dx else new((m, k), dtype) if dx is None else dx
    dw_gate, dw_up = (None if not need_dw else new(nk, dw_dtype) if t is None else t for t in (dw_gate, dw_up))
    db_gate, db_up = (None if not need_db else new((n,), torch.float32) if t is None else t for t in (db_gate, db_up))
    op = _gated_grad(m, k, n, _matrix(dh, "dh").data_ptr(), _rows(dh, "dh", mn, dtype, device),
                     _matrix(gate, "gate").data_ptr(), _matrix(up, "up").data_ptr(), _rows(gate, "gate", mn, dtype, device),
                     _rows(up, "up", mn, dtype, device), x.data_ptr(), _rows(x, "x", (m, k), dtype, device), w_gate.data_ptr(),
                     _matrix(w_up, "w_up").data_ptr(), _rows(w_gate, "w_gate", nk, dtype, device), _rows(w_up, "w_up", nk, dtype, device),
                     _ptr(dx), _opt_rows(dx, "dx", (m, k), dtype, device), _ptr(dw_gate), _ptr(dw_up),
                     _opt_rows(dw_gate, "dw_gate", nk, dw_dtype, device), _opt_rows(dw_up, "dw_up", nk, dw_dtype, device),
                     _opt_vector(db_gate, "db_gate", n, device), _opt_vector(db_up, "db_up", n, device), _CODES[dtype],
                     _CODES.get(dw_dtype, -1), _act(act), accumulate)
    rc, made_ws = _launch_with_workspace("gated", op, workspace, device, stream)
    if rc:
        _check(rc)
    if stream is not None:
        _keep_for_stream(x, stream, *made, made_ws)
    return dx, dw_gate, dw_up, db_gate, db_up


# ------------------------------------------------------------------ autograd

def _needs(ctx, n) -> tuple:
    """needs_input_grad of n arguments, some of which may have been left out."""
    return ctx.needs_input_grad + (False,) * (n - len(ctx.needs_input_grad))


_GRAD_STRIDE = 1 << 22  # the longest row stride that every backward takes


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """An upstream gradient as the kernels take it: itself where its rows lie apart and their columns together, as those
    of a slice of a wider gradient do, else a contiguous copy (of one value expanded, for instance)."""
    (m, c), (row, column) = t.shape, t.stride()
    return t if (column == 1 or c == 1) and (m == 1 or c <= row <= _GRAD_STRIDE) else t.contiguous()


class HashGridEmbeddingFunction(torch.autograd.Function):
    """Autograd of hashgrid_embedding_forward in the table; its gradient is dense and of the table's type.  The gradient
    cannot be differentiated again: autograd raises."""

    @staticmethod
    def forward(ctx, table, ids, scale=1.0, out_dtype=None):
        ctx.scale, ctx.table = scale, (table.shape[0], table.dtype)
        ctx.save_for_backward(ids)
        return hashgrid_embedding_forward(table, ids, scale=scale, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, dtype = ctx.table
        return hashgrid_embedding_backward(_as_rows(dy), *ctx.saved_tensors, rows, scale=ctx.scale, table_dtype=dtype), None, None, None


class HashGridCodedInputFunction(torch.autograd.Function):
    """A layer's input of encoded features and codes side by side: [features | scale * table[ids]] in a 16-bit type, the
    codes written in place by the lookup.  The gradients cannot be differentiated again: autograd raises."""

    @staticmethod
    def forward(ctx, features, table, ids, dtype, scale=1.0):
        m, f = features.shape
        x = torch.empty((m, f + table.shape[1]), dtype=dtype, device=features.device)
        x[:, :f].copy_(features)
        hashgrid_embedding_forward(table, ids, scale=scale, out=x[:, f:])
        ctx.scale, ctx.width, ctx.kind, ctx.table = scale, f, features.dtype, (table.shape[0], table.dtype)
        ctx.save_for_backward(ids)
        return x

    @staticmethod
    @once_differentiable
    def backward(ctx, dx):
        (ids,), f, (rows, dtype) = ctx.saved_tensors, ctx.width, ctx.table
        need, dx = _needs(ctx, 5), _as_rows(dx)
        dtable = hashgrid_embedding_backward(dx[:, f:], ids, rows, scale=ctx.scale, table_dtype=dtype) if need[1] else None
        return dx[:, :f].to(ctx.kind) if need[0] else None, dtable, None, None, None


class HashGridLayerNormFunction(torch.autograd.Function):
    """Autograd of hashgrid_layer_norm_forward: returns y, or (y, s) with a residual, s = x + residual in x's type.
    Weight and bias may be None.  The statistics are kept only where autograd records the call.  The gradients cannot be
    differentiated again: autograd raises."""

    @classmethod
    def apply(cls, *args):
        return super().apply(_recorded(*args), *args)

    @staticmethod
    def forward(ctx, keep, x, weight, bias=None, residual=None, eps=1e-5):
        out = hashgrid_layer_norm_forward(x, weight, bias, residual=residual, eps=eps, save_sum=residual is not None, save_stats=keep)
        if keep:
            ctx.save_for_backward(x if residual is None else out.sum, weight, out.mean, out.rstd)
        ctx.set_materialize_grads(False)  # an output that nothing reads has no gradient, not one of zeros
        return out.y if residual is None else (out.y, out.sum)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, mean, rstd = ctx.saved_tensors
        need = _needs(ctx, 6)[1:]
        if dy is None:  # s alone goes on
            zero = lambda n: torch.zeros(s.shape[1], device=s.device) if n else None  # noqa: E731
            return None, ds, zero(need[1]), zero(need[2]), ds if need[3] else None, None
        dx, dw, db = hashgrid_layer_norm_backward(_as_rows(dy), s, weight, mean, rstd, ds=None if ds is None else _as_rows(ds),
                                                  need_dw=need[1], need_db=need[2])
        return None, dx, dw, db, dx if need[3] else None, None


class HashGridGatedFunction(torch.autograd.Function):
    """Autograd of hashgrid_gated_forward: x in a 16-bit type, the weights fp32 masters that the products read rounded to
    it, biases fp32 or None.  Gradients of the masters are fp32.  The projections are kept only where autograd records the
    call.  The gradients cannot be differentiated again: autograd raises."""

    @classmethod
    def apply(cls, *args):
        return super().apply(_recorded(*args), *args)

    @staticmethod
    def forward(ctx, keep, x, w_gate, w_up, b_gate=None, b_up=None, act="silu"):
        wg, wu = w_gate.to(x.dtype), w_up.to(x.dtype)
        ctx.act = act
        if not keep:
            return hashgrid_gated_forward(x, wg, wu, b_gate, b_up, act=act)
        h, gate, up = hashgrid_gated_forward(x, wg, wu, b_gate, b_up, act=act, save_pre=True)
        ctx.save_for_backward(x, wg, wu, gate, up)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, wg, wu, gate, up = ctx.saved_tensors
        need = _needs(ctx, 7)[1:]
        out = hashgrid_gated_backward(_as_rows(dh), x, wg, wu, gate, up, act=ctx.act, need_dx=need[0], need_dw=need[1] or need[2],
                                      need_db=need[3] or need[4])
        return (None,) + tuple(t if n else None for t, n in zip(out, need)) + (None,)


# ------------------------------------------------------------------ modules

class HashGridCodes(torch.nn.Module):
    """A learned code for each of ``count`` images or frames: ``forward(ids [m]) -> [m, width]``, rows of an fp32 table
    times ``scale``, in ``dtype``.  An id outside 0 .. count - 1 gives zeros and gets no gradient."""

    def __init__(self, count: int, width: int, scale: float = 1.0, dtype=torch.float32, device="cuda"):
        super().__init__()
        self.scale, self.dtype = scale, dtype
        self.table = torch.nn.Parameter(torch.randn(count, width, device=device) * 0.01)

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return HashGridEmbeddingFunction.apply(self.table, ids, self.scale, self.dtype)


class HashGridGatedHead(torch.nn.Module):
    """A head of gated feed-forward blocks on the encoding, with a code per image beside the features if ``codes`` is not
    0: ``forward(features [n, in_features], ids [n]) -> [n, out_features]`` fp32.

        h = stem([features | code[ids]])
        per block: h = h + Wd (act(Wg norm(h) + bg) (Wu norm(h) + bu)) + bd
        y = W norm(h + stem's h) + b

    norm is the layer norm.  ``hidden`` is the blocks' width between (2 * width by default).  Weights, biases, codes and
    the norms' weights are fp32 masters; activations and the weights' copies that the matrix cores read are ``dtype``
    (bfloat16 or float16; gradients pass in it too, so in float16 the loss of many points needs a scale, whose inverse
    HashGridAdamW.step takes as ``grad_scale``).  Without a graph to record, as under torch.no_grad(), nothing is kept
    for a backward.  ``quantized()`` is the same head for inference with 8-bit operands behind the blocks' norms."""

    def __init__(self, in_features=32, width=256, blocks=2, out_features=4, hidden=None, act="silu", codes=0, code_width=64,
                 dtype=torch.bfloat16, eps=1e-5, device="cuda"):
        super().__init__()
        if dtype not in _HALF:
            raise ValueError("dtype must be torch.float16 or torch.bfloat16")
        _act(act)
        self.act, self.dtype, self.eps, self.blocks = act, dtype, eps, blocks
        hidden = 2 * width if hidden is None else hidden
        self.codes = HashGridCodes(codes, code_width, dtype=dtype, device=device) if codes else None

        def layer(name, fan_in, fan_out):
            w = torch.empty((fan_out, fan_in), device=device)
            torch.nn.init.xavier_uniform_(w)
            b = torch.empty(fan_out, device=device).uniform_(-fan_in ** -0.5, fan_in ** -0.5)
            self.register_parameter(f"{name}_w", torch.nn.Parameter(w))
            self.register_parameter(f"{name}_b", torch.nn.Parameter(b))

        def norm(name):
            self.register_parameter(f"{name}_w", torch.nn.Parameter(torch.ones(width, device=device)))
            self.register_parameter(f"{name}_b", torch.nn.Parameter(torch.zeros(width, device=device)))

        layer("stem", in_features + (code_width if codes else 0), width)
        for i in range(blocks):
            norm(f"norm{i}")
            layer(f"gate{i}", width, hidden)
            layer(f"up{i}", width, hidden)
            layer(f"down{i}", hidden, width)
        norm("norm_out")
        layer("out", width, out_features)

    def _layer(self, name):
        return getattr(self, f"{name}_w"), getattr(self, f"{name}_b")

    def _input(self, features, ids):
        if (ids is None) != (self.codes is None):
            raise ValueError("ids belong to a head with codes, and such a head needs them")
        if ids is None:
            return features.to(self.dtype)
        return HashGridCodedInputFunction.apply(features, self.codes.table, ids, self.dtype, self.codes.scale)

    def forward(self, features: torch.Tensor, ids: torch.Tensor | None = None) -> torch.Tensor:
        linear, norm, gated = HashGridLinearFunction.apply, HashGridLayerNormFunction.apply, HashGridGatedFunction.apply
        h = stem = linear(self._input(features, ids), *self._layer("stem"))
        for i in range(self.blocks):
            (wg, bg), (wu, bu) = self._layer(f"gate{i}"), self._layer(f"up{i}")
            f = gated(norm(h, *self._layer(f"norm{i}"), None, self.eps), wg, wu, bg, bu, self.act)
            h = linear(f, *self._layer(f"down{i}"), "none", h)
        if _recorded(h, stem, *self._layer("norm_out")):
            y, _ = norm(h, *self._layer("norm_out"), stem, self.eps)
        else:  # nobody reads the sum
            y = hashgrid_layer_norm_forward(h, *self._layer("norm_out"), residual=stem, eps=self.eps).y
        return linear(y, *self._layer("out"), "none", None, torch.float32)

    def quantized(self) -> "HashGridGatedHead8":
        return HashGridGatedHead8(self)


class HashGridGatedHead8:
    """A HashGridGatedHead for inference: the blocks' gated products read 8-bit rows with scales, which the norm writes,
    and 8-bit weights; the residual stream, the other products, the codes and the outputs stay in the head's 16-bit type."""

    def __init__(self, head: HashGridGatedHead):
        self.act, self.dtype, self.eps = head.act, head.dtype, head.eps
        grab = lambda t: t.detach().clone()  # noqa: E731
        half = lambda t: t.detach().clone().to(self.dtype)  # noqa: E731
        self.codes = None if head.codes is None else (grab(head.codes.table), head.codes.scale)
        self.stem = half(head.stem_w), grab(head.stem_b)
        self.layers = [dict(norm=(grab(getattr(head, f"norm{i}_w")), grab(getattr(head, f"norm{i}_b"))),
                            gate=quantize_rows(getattr(head, f"gate{i}_w")), up=quantize_rows(getattr(head, f"up{i}_w")),
                            biases=(grab(getattr(head, f"gate{i}_b")), grab(getattr(head, f"up{i}_b"))),
                            down=(half(getattr(head, f"down{i}_w")), grab(getattr(head, f"down{i}_b")))) for i in range(head.blocks)]
        self.norm_out = grab(head.norm_out_w), grab(head.norm_out_b)
        self.out = half(head.out_w), grab(head.out_b)

    def __call__(self, features: torch.Tensor, ids: torch.Tensor | None = None) -> torch.Tensor:
        if (ids is None) != (self.codes is None):
            raise ValueError("ids belong to a head with codes, and such a head needs them")
        if ids is None:
            x = features.to(self.dtype)
        else:
            x = HashGridCodedInputFunction.apply(features, self.codes[0], ids, self.dtype, self.codes[1])
        h = stem = hashgrid_linear_forward(x, *self.stem)
        for layer in self.layers:
            n8 = hashgrid_layer_norm_forward(h, *layer["norm"], eps=self.eps, out_dtype=F8)
            (wg, gs), (wu, us) = layer["gate"], layer["up"]
            f = hashgrid_gated_forward(n8.y, wg, wu, *layer["biases"], act=self.act, x_scale=n8.scale, gate_scale=gs, up_scale=us,
                                       out_dtype=self.dtype)
            h = hashgrid_linear_forward(f, *layer["down"], residual=h)
        y = hashgrid_layer_norm_forward(h, *self.norm_out, residual=stem, eps=self.eps).y
        return hashgrid_linear_forward(y, *self.out, out_dtype=torch.float32)
