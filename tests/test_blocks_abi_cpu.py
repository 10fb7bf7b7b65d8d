"""Refusals of the embedding, layer norm and gated entry points: the C ABI's
argument checks (nothing is launched, so no GPU is needed) and the binding's."""
import ctypes

import pytest
import torch

import multiresolution_hash_grid_amd as hg
from multiresolution_hash_grid_amd import blocks as K
from multiresolution_hash_grid_amd import hashgrid as B
from multiresolution_hash_grid_amd import residual as R

P, Q = 0x1000, 0x2000
E, U = B.HG_EINVAL, B.HG_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return K._lib()


def refused(lib, name, op, code, word, backward=False):
    if backward:
        size = ctypes.c_size_t(0)
        assert getattr(lib, f"hashgrid_{name}_backward")(ctypes.byref(op), P, 1 << 60, None) == code
        assert word in lib.hashgrid_last_error().decode()
        assert getattr(lib, f"hashgrid_{name}_backward_workspace_size")(ctypes.byref(op), ctypes.byref(size)) == code
    else:
        assert getattr(lib, f"hashgrid_{name}_forward")(ctypes.byref(op), None) == code
        assert word in lib.hashgrid_last_error().decode()


LOOKUP = dict(m=4, rows=9, c=8, ids=P, table=P, table_stride=8, y=Q, y_stride=8, scale=1.0, ids_bits=32, table_dtype=B.HG_F32,
              y_dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(m=(1 << 40) + 1), E, "m ="), (dict(rows=-1), E, "rows ="), (dict(c=0), E, "c ="),
    (dict(c=(1 << 20) + 1), E, "c ="), (dict(ids_bits=16), E, "ids_bits"), (dict(ids=None), E, "ids is NULL"), (dict(ids=P + 2), E, "aligned"),
    (dict(ids_bits=64, ids=P + 4), E, "aligned"), (dict(table=None), E, "table is NULL"), (dict(table=P + 2), E, "aligned"),
    (dict(table_stride=7), E, "stride"), (dict(y=None), E, "y is NULL"), (dict(y_stride=7), E, "stride"),
    (dict(table_dtype=R.HG_F8), U, "table_dtype"), (dict(table_dtype=B.HG_F16, y_dtype=B.HG_F32), U, "y_dtype"),
    (dict(table_dtype=B.HG_F16, y_dtype=R.HG_BF16), U, "y_dtype"), (dict(y_dtype=R.HG_F8), U, "y_dtype"), (dict(y_dtype=9), U, "y_dtype"), (dict(y=P), E, "its own"),
])
def test_embedding_forward_refuses(lib, change, code, word):
    refused(lib, "embedding", K._Embedding(**(LOOKUP | change)), code, word)


SORT = dict(m=4, rows=9, c=8, ids=P, dy=P, dy_stride=8, dtable=Q, dtable_stride=8, scale=1.0, ids_bits=64, dy_dtype=B.HG_F16,
            dtable_dtype=B.HG_F32)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(m=(1 << 30) + 1), E, "m ="), (dict(rows=-2), E, "rows ="), (dict(c=0), E, "c ="),
    (dict(ids_bits=8), E, "ids_bits"), (dict(ids=None), E, "ids is NULL"), (dict(ids=P + 4), E, "aligned"), (dict(dy=None), E, "dy is NULL"),
    (dict(dy=P + 1), E, "aligned"), (dict(dy_stride=4), E, "stride"), (dict(dtable=None), E, "dtable is NULL"),
    (dict(dtable_stride=7), E, "stride"), (dict(dtable=Q + 2), E, "aligned"), (dict(dy_dtype=R.HG_F8), U, "dy_dtype"),
    (dict(dtable_dtype=R.HG_BF16), U, "dtable_dtype"), (dict(dy_dtype=B.HG_F32, dtable_dtype=B.HG_F16), U, "dtable_dtype"),
    (dict(dtable=P), E, "its own"),
])
def test_embedding_backward_refuses(lib, change, code, word):
    refused(lib, "embedding", K._EmbeddingGrad(**(SORT | change)), code, word, True)


NORM = dict(m=4, c=8, x=P, x_stride=8, w=P, b=P, y=Q, y_stride=8, eps=1e-5, dtype=B.HG_F16, y_dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(c=0), E, "c ="), (dict(c=(1 << 20) + 1), E, "c ="), (dict(eps=-1.0), E, "eps"),
    (dict(eps=float("nan")), E, "eps"), (dict(eps=float("inf")), E, "eps"), (dict(dtype=R.HG_F8), U, "dtype"),
    (dict(y_dtype=B.HG_F32), U, "y_dtype"), (dict(x=None), E, "x is NULL"), (dict(y=None), E, "y is NULL"), (dict(w=P + 2), E, "aligned"),
    (dict(b=P + 2), E, "aligned"), (dict(y_dtype=R.HG_F8), E, "y_scale is NULL"), (dict(y_scale=P), E, "y_scale"),
    (dict(x_stride=4), E, "stride"), (dict(residual=P, residual_stride=4), E, "stride"), (dict(sum=P + 1, sum_stride=8), E, "aligned"),
    (dict(mean=P + 1), E, "aligned"), (dict(rstd=P + 1), E, "aligned"), (dict(y=P, y_stride=16), E, "row stride"),
    (dict(sum=P, sum_stride=16), E, "row stride"), (dict(sum=Q, sum_stride=8), E, "one buffer"),
    (dict(y=P, y_dtype=R.HG_F8, y_scale=P), E, "their type"), (dict(mean=0x3000, rstd=0x3000), E, "one buffer"),
])
def test_layer_norm_forward_refuses(lib, change, code, word):
    refused(lib, "layer_norm", K._LayerNorm(**(NORM | change)), code, word)


NGRAD = dict(m=4, c=8, dy=P, dy_stride=8, sum=P, sum_stride=8, w=P, mean=P, rstd=P, dx=Q, dx_stride=8, dw=0x3000, db=0x4000, dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(c=0), E, "c ="), (dict(dtype=R.HG_F8), U, "dtype"), (dict(dy=None), E, "dy is NULL"),
    (dict(sum=None), E, "sum is NULL"), (dict(dx=None), E, "dx is NULL"), (dict(mean=None), E, "mean is NULL"),
    (dict(rstd=None), E, "rstd is NULL"), (dict(ds=P, ds_stride=4), E, "stride"), (dict(dw=P + 2), E, "aligned"), (dict(db=P + 2), E, "aligned"),
    (dict(dx=P, dx_stride=9), E, "row stride"), (dict(dw=0x4000), E, "one buffer"),
    (dict(c=4097, dy_stride=4097, sum_stride=4097, dx=P, dx_stride=4097), E, "in place"),
])
def test_layer_norm_backward_refuses(lib, change, code, word):
    refused(lib, "layer_norm", K._LayerNormGrad(**(NGRAD | change)), code, word, True)


GATED = dict(m=4, k=8, n=8, x=P, x_stride=8, wg=P, wg_stride=8, wu=P, wu_stride=8, h=Q, h_stride=8, x_dtype=B.HG_F16, h_dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(k=0), E, "k ="), (dict(n=65537), E, "n ="), (dict(act=4), E, "activation"),
    (dict(x=None), E, "x is NULL"), (dict(wg=None), E, "wg is NULL"), (dict(wu=None), E, "wu is NULL"), (dict(h=None), E, "h is NULL"),
    (dict(x=P + 1), E, "aligned"), (dict(bg=P + 2), E, "aligned"), (dict(bu=P + 2), E, "aligned"), (dict(x_stride=7), E, "stride"),
    (dict(wg_stride=7), E, "stride"), (dict(wu_stride=7), E, "stride"), (dict(h_stride=7), E, "stride"),
    (dict(gate=P, gate_stride=8), E, "together"), (dict(up=P, up_stride=8), E, "together"),
    (dict(gate=0x3000, gate_stride=4, up=0x4000, up_stride=8), E, "stride"), (dict(gate=0x3000, gate_stride=8, up=0x3000, up_stride=8), E, "their own"),
    (dict(h=P), E, "their own"), (dict(x_dtype=B.HG_F32), U, "x_dtype"), (dict(h_dtype=R.HG_BF16), U, "h_dtype"),
    (dict(x_dtype=R.HG_F8, h_dtype=R.HG_F8), U, "scale"),
    (dict(x_dtype=R.HG_F8, gate=0x3000, up=0x4000, gate_stride=8, up_stride=8), U, "kept"),
    (dict(x_dtype=R.HG_F8, g_scale=P, u_scale=P), E, "x_scale is NULL"), (dict(x_dtype=R.HG_F8, x_scale=P, u_scale=P), E, "g_scale is NULL"),
    (dict(x_dtype=R.HG_F8, x_scale=P, g_scale=P), E, "u_scale is NULL"), (dict(x_scale=P), E, "belong"), (dict(u_scale=P), E, "belong"),
    (dict(x=0x3000, h=P), E, "operands"), (dict(gate=0x3000, up=P, gate_stride=8, up_stride=8), E, "operands"),
])
def test_gated_forward_refuses(lib, change, code, word):
    refused(lib, "gated", K._Gated(**(GATED | change)), code, word)


GGRAD = dict(m=4, k=8, n=8, dh=P, dh_stride=8, gate=P, up=P, gate_stride=8, up_stride=8, x=P, x_stride=8, wg=P, wu=P, wg_stride=8,
             wu_stride=8, dx=Q, dx_stride=8, dwg=0x3000, dwu=0x4000, dwg_stride=8, dwu_stride=8, dbg=0x5000, dbu=0x6000, dtype=B.HG_F16, dw_dtype=B.HG_F32, act=2)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), E, "m ="), (dict(k=-3), E, "k ="), (dict(act=9), E, "activation"), (dict(dtype=R.HG_F8), U, "dtype"),
    (dict(dtype=B.HG_F32), U, "dtype"), (dict(dw_dtype=R.HG_BF16), U, "dw_dtype"), (dict(dh=None), E, "dh is NULL"),
    (dict(gate=None), E, "gate is NULL"), (dict(up=None), E, "up is NULL"), (dict(x=None), E, "x is NULL"), (dict(wg=None), E, "wg is NULL"),
    (dict(wu=None), E, "wu is NULL"), (dict(dwg=None), E, "together"), (dict(dbu=None), E, "together"), (dict(dwg_stride=4), E, "stride"),
    (dict(dx_stride=4), E, "stride"), (dict(dbg=P + 1), E, "aligned"), (dict(dh=P + 1), E, "aligned"),
    (dict(x_stride=(1 << 22) + 1), E, "stride"), (dict(gate_stride=(1 << 22) + 1), E, "stride"), (dict(dx=P), E, "their own"),
    (dict(dwg=P), E, "their own"), (dict(dwu=P), E, "their own"), (dict(dwu=0x3000), E, "two buffers"), (dict(dbu=0x5000), E, "two buffers"),
])
def test_gated_backward_refuses(lib, change, code, word):
    refused(lib, "gated", K._GatedGrad(**(GGRAD | change)), code, word, True)


@pytest.mark.parametrize("name,op", [
    ("embedding", K._EmbeddingGrad(**(SORT | dict(m=100000)))), ("layer_norm", K._LayerNormGrad(**NGRAD)),
    ("gated", K._GatedGrad(**(GGRAD | dict(m=100000)))),
])
def test_workspaces(lib, name, op):
    call, size = getattr(lib, f"hashgrid_{name}_backward"), ctypes.c_size_t(0)
    sizer = getattr(lib, f"hashgrid_{name}_backward_workspace_size")
    assert sizer(ctypes.byref(op), None) == E
    assert sizer(ctypes.byref(op), ctypes.byref(size)) == B.HG_OK and size.value > 0
    for ws, n in ((None, 0), (P, size.value - 1), (P + 16, size.value)):
        assert call(ctypes.byref(op), ws, n, None) == E and "workspace" in lib.hashgrid_last_error().decode()


def test_without_rows_nothing_is_looked_at(lib):
    for name, op in (("embedding", K._Embedding(**(LOOKUP | dict(m=0, ids=None, table=None, y=None)))),
                     ("layer_norm", K._LayerNorm(**(NORM | dict(m=0, x=None, y=None)))),
                     ("gated", K._Gated(**(GATED | dict(m=0, x=None, wg=None, h=None))))):
        call = getattr(lib, f"hashgrid_{name}_forward")
        assert call(ctypes.byref(op), None) == B.HG_OK and lib.hashgrid_last_error() == b""
        assert call(None, None) == E
        assert getattr(lib, f"hashgrid_{name}_backward")(None, None, 0, None) == E
    op = K._EmbeddingGrad(**(SORT | dict(rows=0, dtable=None)))
    assert lib.hashgrid_embedding_backward(ctypes.byref(op), None, 0, None) == B.HG_OK


def test_binding_refuses_tensors_off_the_gpu():
    x, w, i = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: hg.hashgrid_embedding_forward(x, i), lambda: hg.hashgrid_embedding_backward(x, i, 3),
                 lambda: hg.hashgrid_layer_norm_forward(x, w, w), lambda: hg.hashgrid_layer_norm_backward(x, x, w, w, w),
                 lambda: hg.hashgrid_gated_forward(x, x, x), lambda: hg.hashgrid_gated_backward(x, x, x, x, x, x)):
        with pytest.raises(ValueError):
            call()


def test_heads_refuse():
    with pytest.raises(ValueError):
        hg.HashGridGatedHead(dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError):
        hg.HashGridGatedHead(act="tanh", device="cpu")
    for head, ids in ((hg.HashGridGatedHead(8, 8, 1, device="cpu"), torch.zeros(2, dtype=torch.int64)),
                      (hg.HashGridGatedHead(8, 8, 1, codes=3, code_width=4, device="cpu"), None)):
        for form in (head, head.quantized()):
            with pytest.raises(ValueError, match="ids"):
                form(torch.zeros(2, 8), ids)
