"""Refusals of the residual head's entry points: the C ABI's argument checks
(nothing is launched, so no GPU is needed) and the Python binding's."""
import ctypes

import pytest
import torch

import multiresolution_hash_grid_amd as hg
from multiresolution_hash_grid_amd import hashgrid as B
from multiresolution_hash_grid_amd import residual as R

P = 0x1000


@pytest.fixture(scope="module")
def lib():
    return R._lib()


def message(lib):
    return lib.hashgrid_last_error().decode()


LINEAR = dict(m=4, k=8, n=8, x=P, x_stride=8, w=P, w_stride=8, y=P, y_stride=8, x_dtype=B.HG_F16, y_dtype=B.HG_F16, act=0)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), B.HG_EINVAL, "m ="), (dict(k=0), B.HG_EINVAL, "k ="), (dict(n=65537), B.HG_EINVAL, "n ="),
    (dict(act=4), B.HG_EINVAL, "activation"), (dict(act=-1), B.HG_EINVAL, "activation"),
    (dict(x=None), B.HG_EINVAL, "x is NULL"), (dict(w=None), B.HG_EINVAL, "w is NULL"), (dict(y=None), B.HG_EINVAL, "y is NULL"),
    (dict(x=P + 1), B.HG_EINVAL, "aligned"), (dict(bias=P + 2), B.HG_EINVAL, "aligned"),
    (dict(x_stride=7), B.HG_EINVAL, "stride"), (dict(w_stride=7), B.HG_EINVAL, "stride"), (dict(y_stride=-8), B.HG_EINVAL, "stride"),
    (dict(residual=P, residual_stride=7), B.HG_EINVAL, "stride"), (dict(pre=P, pre_stride=0), B.HG_EINVAL, "stride"),
    (dict(m=1 << 39, x_stride=1 << 40), B.HG_EINVAL, "too large"),
    (dict(x_dtype=B.HG_F32), B.HG_EUNSUPPORTED, "x_dtype"), (dict(y_dtype=R.HG_BF16), B.HG_EUNSUPPORTED, "y_dtype"),
    (dict(y_dtype=R.HG_F8), B.HG_EUNSUPPORTED, "y_dtype"), (dict(x_dtype=R.HG_F8, y_dtype=R.HG_F8), B.HG_EUNSUPPORTED, "scale"),
    (dict(x_dtype=R.HG_F8, x_scale=P, w_scale=P, pre=P, pre_stride=8), B.HG_EUNSUPPORTED, "pre"),
    (dict(x_dtype=R.HG_F8, w_scale=P), B.HG_EINVAL, "x_scale is NULL"), (dict(x_dtype=R.HG_F8, x_scale=P), B.HG_EINVAL, "w_scale is NULL"),
    (dict(x_scale=P), B.HG_EINVAL, "x_scale"), (dict(w_scale=P), B.HG_EINVAL, "w_scale"),
])
def test_linear_forward_refuses(lib, change, code, word):
    op = R._Linear(**(LINEAR | change))
    assert lib.hashgrid_linear_forward(ctypes.byref(op), None) == code
    assert word in message(lib)


def test_linear_forward_without_rows_does_nothing(lib):
    op = R._Linear(**(LINEAR | dict(m=0, x=None, y=None, w=None)))
    assert lib.hashgrid_linear_forward(ctypes.byref(op), None) == B.HG_OK and message(lib) == ""
    assert lib.hashgrid_linear_forward(None, None) == B.HG_EINVAL


GRAD = dict(m=4, k=8, n=8, dy=P, dy_stride=8, pre=P, pre_stride=8, x=P, x_stride=8, w=P, w_stride=8, dx=P, dx_stride=8, dw=P,
            dw_stride=8, db=P, dtype=B.HG_F16, dy_dtype=B.HG_F16, dw_dtype=B.HG_F32, act=2)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), B.HG_EINVAL, "m ="), (dict(k=-3), B.HG_EINVAL, "k ="), (dict(act=9), B.HG_EINVAL, "activation"),
    (dict(dtype=R.HG_F8), B.HG_EUNSUPPORTED, "dtype"), (dict(dtype=B.HG_F32), B.HG_EUNSUPPORTED, "dtype"),
    (dict(dy_dtype=R.HG_BF16), B.HG_EUNSUPPORTED, "dy_dtype"), (dict(dw_dtype=R.HG_F8), B.HG_EUNSUPPORTED, "dw_dtype"),
    (dict(dy=None), B.HG_EINVAL, "dy is NULL"), (dict(pre=None), B.HG_EINVAL, "pre is NULL"), (dict(x=None), B.HG_EINVAL, "x is NULL"),
    (dict(w=None), B.HG_EINVAL, "w is NULL"), (dict(dw_stride=4), B.HG_EINVAL, "stride"), (dict(dx_stride=4), B.HG_EINVAL, "stride"),
    (dict(db=P + 1), B.HG_EINVAL, "aligned"), (dict(dy=P + 1), B.HG_EINVAL, "aligned"), (dict(x_stride=(1 << 22) + 1), B.HG_EINVAL, "stride"),
])
def test_linear_backward_refuses(lib, change, code, word):
    op = R._LinearGrad(**(GRAD | change))
    size = ctypes.c_size_t(0)
    assert lib.hashgrid_linear_backward(ctypes.byref(op), P, 1 << 40, None) == code
    assert word in message(lib)
    assert lib.hashgrid_linear_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)) == code


def test_linear_backward_workspace(lib):
    op = R._LinearGrad(**(GRAD | dict(m=100000)))
    size = ctypes.c_size_t(0)
    assert lib.hashgrid_linear_backward_workspace_size(ctypes.byref(op), None) == B.HG_EINVAL
    assert lib.hashgrid_linear_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)) == B.HG_OK
    if size.value:
        assert lib.hashgrid_linear_backward(ctypes.byref(op), None, 0, None) == B.HG_EINVAL
        assert lib.hashgrid_linear_backward(ctypes.byref(op), P, size.value - 1, None) == B.HG_EINVAL
        assert "workspace" in message(lib)
        assert lib.hashgrid_linear_backward(ctypes.byref(op), P + 16, size.value, None) == B.HG_EINVAL


NORM = dict(m=4, c=8, x=P, x_stride=8, w=P, y=P, y_stride=8, eps=1e-6, dtype=B.HG_F16, y_dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), B.HG_EINVAL, "m ="), (dict(c=0), B.HG_EINVAL, "c ="), (dict(c=(1 << 20) + 1), B.HG_EINVAL, "c ="),
    (dict(eps=-1.0), B.HG_EINVAL, "eps"), (dict(eps=float("nan")), B.HG_EINVAL, "eps"), (dict(eps=float("inf")), B.HG_EINVAL, "eps"),
    (dict(dtype=R.HG_F8), B.HG_EUNSUPPORTED, "dtype"), (dict(y_dtype=B.HG_F32), B.HG_EUNSUPPORTED, "y_dtype"),
    (dict(x=None), B.HG_EINVAL, "x is NULL"), (dict(w=None), B.HG_EINVAL, "w is NULL"), (dict(y=None), B.HG_EINVAL, "y is NULL"),
    (dict(y_dtype=R.HG_F8), B.HG_EINVAL, "y_scale is NULL"), (dict(y_scale=P), B.HG_EINVAL, "y_scale"),
    (dict(x_stride=4), B.HG_EINVAL, "stride"), (dict(residual=P, residual_stride=4), B.HG_EINVAL, "stride"),
    (dict(sum=P + 1, sum_stride=8), B.HG_EINVAL, "aligned"), (dict(rstd=P + 1), B.HG_EINVAL, "aligned"),
])
def test_rms_norm_forward_refuses(lib, change, code, word):
    op = R._RmsNorm(**(NORM | change))
    assert lib.hashgrid_rms_norm_forward(ctypes.byref(op), None) == code
    assert word in message(lib)


NGRAD = dict(m=4, c=8, dy=P, dy_stride=8, sum=P, sum_stride=8, w=P, rstd=P, dx=P, dx_stride=8, dw=P, dtype=B.HG_F16)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), B.HG_EINVAL, "m ="), (dict(c=0), B.HG_EINVAL, "c ="), (dict(dtype=R.HG_F8), B.HG_EUNSUPPORTED, "dtype"),
    (dict(dy=None), B.HG_EINVAL, "dy is NULL"), (dict(sum=None), B.HG_EINVAL, "sum is NULL"), (dict(dx=None), B.HG_EINVAL, "dx is NULL"),
    (dict(w=None), B.HG_EINVAL, "w is NULL"), (dict(rstd=None), B.HG_EINVAL, "rstd is NULL"),
    (dict(ds=P, ds_stride=4), B.HG_EINVAL, "stride"), (dict(dw=P + 2), B.HG_EINVAL, "aligned"),
])
def test_rms_norm_backward_refuses(lib, change, code, word):
    op = R._RmsNormGrad(**(NGRAD | change))
    size = ctypes.c_size_t(0)
    assert lib.hashgrid_rms_norm_backward(ctypes.byref(op), P, 1 << 40, None) == code
    assert word in message(lib)
    assert lib.hashgrid_rms_norm_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)) == code


def test_rms_norm_backward_workspace(lib):
    op, size = R._RmsNormGrad(**NGRAD), ctypes.c_size_t(0)
    assert lib.hashgrid_rms_norm_backward_workspace_size(ctypes.byref(op), ctypes.byref(size)) == B.HG_OK and size.value > 0
    assert lib.hashgrid_rms_norm_backward(ctypes.byref(op), None, 0, None) == B.HG_EINVAL
    assert lib.hashgrid_rms_norm_backward(ctypes.byref(op), P + 4, size.value, None) == B.HG_EINVAL


TENSOR = dict(param=P, grad=P, m=P, v=P, count=8, lr=1e-3, grad_dtype=B.HG_F32, state_bits=32)


@pytest.mark.parametrize("opt,tensor,word", [
    (dict(step=0), {}, "step"), (dict(beta1=1.0), {}, "betas"), (dict(beta2=-0.1), {}, "betas"), (dict(eps=-1.0), {}, "eps"),
    (dict(eps=float("nan")), {}, "eps"),
    ({}, dict(count=-1), "count"), ({}, dict(state_bits=16), "state_bits"), ({}, dict(grad_dtype=R.HG_F8), "grad_dtype"),
    ({}, dict(copy=P, copy_dtype=B.HG_F32), "copy_dtype"), ({}, dict(lr=float("inf")), "lr"), ({}, dict(weight_decay=-1.0), "weight_decay"),
    ({}, dict(reserved=1), "reserved"), ({}, dict(param=None), "device pointers"), ({}, dict(grad=None), "device pointers"),
    ({}, dict(state_bits=8), "device pointers"), ({}, dict(param=P + 2), "misaligned"), ({}, dict(v=P + 2), "misaligned"),
    ({}, dict(copy=P + 1, copy_dtype=B.HG_F16), "misaligned"),
])
def test_adamw_refuses(lib, opt, tensor, word):
    o = R._AdamW(**(dict(beta1=0.9, beta2=0.99, eps=1e-8, step=1) | opt))
    t = (R._AdamWTensor * 2)(R._AdamWTensor(**TENSOR), R._AdamWTensor(**(TENSOR | tensor)))
    assert lib.hashgrid_adamw_step(ctypes.byref(o), t, 2, None, 0, None) == B.HG_EINVAL
    assert word in message(lib)


def test_adamw_refuses_bad_lists(lib):
    o = R._AdamW(0.9, 0.99, 1e-8, 1, 0)
    assert lib.hashgrid_adamw_step(None, None, 0, None, 0, None) == B.HG_EINVAL
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 1, None, 0, None) == B.HG_EINVAL
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, -1, None, 0, None) == B.HG_EINVAL
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 0, None, 2, None) == B.HG_EINVAL
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 0, P + 1, 0, None) == B.HG_EINVAL
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 0, None, 0, None) == B.HG_OK


def test_binding_refuses_tensors_off_the_gpu():
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8)
    for call in (lambda: hg.hashgrid_linear_forward(x, x), lambda: hg.hashgrid_linear_backward(x, x, x),
                 lambda: hg.hashgrid_rms_norm_forward(x, w), lambda: hg.hashgrid_rms_norm_backward(x, x, w, w),
                 lambda: hg.hashgrid_adamw_step([hg.AdamWTensor(w, w, w, w)], step=1)):
        with pytest.raises(ValueError):
            call()


def test_moments_of_zero():
    p = torch.zeros(300)
    s = hg.AdamWTensor.states(p, 8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["v"].dtype == torch.uint8 and s["m_exp"].numel() == s["v_exp"].numel() == 2
    assert hg.AdamWTensor.states(p, 32)["m"].dtype == torch.float32
    with pytest.raises(ValueError):
        hg.AdamWTensor.states(p, 16)
