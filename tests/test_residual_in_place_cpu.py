"""Refusals of outputs in place of inputs that the kernels cannot take (nothing
is launched, so no GPU is needed)."""
import ctypes

import pytest

from multiresolution_hash_grid_amd import hashgrid as B
from multiresolution_hash_grid_amd import residual as R

P, Q, S, T = 0x10000, 0x20000, 0x30000, 0x40000


def refused(call, op, *rest):
    lib = R._lib()
    rc = getattr(lib, call)(ctypes.byref(op), *rest, None)
    return rc == B.HG_EINVAL and "in place" in lib.hashgrid_last_error().decode()


NGRAD = dict(m=4, c=8, dy=P, dy_stride=8, sum=Q, sum_stride=8, ds=S, ds_stride=8, w=T, rstd=T, dx=P, dx_stride=8, dtype=B.HG_F16)


@pytest.mark.parametrize("at", [P, Q, S])
def test_norm_backward_of_long_rows(at):
    # Above 4096 columns the row is read again after dx of it is written, and dw after all of dx.
    assert refused("hashgrid_rms_norm_backward", R._RmsNormGrad(**(NGRAD | dict(c=4097, dy_stride=5000, sum_stride=5000, ds_stride=5000,
                                                                                dx_stride=5000, dx=at))), None, 0)


@pytest.mark.parametrize("at,stride", [(P, "dy_stride"), (Q, "sum_stride"), (S, "ds_stride")])
def test_norm_backward_of_other_strides(at, stride):
    assert refused("hashgrid_rms_norm_backward", R._RmsNormGrad(**(NGRAD | {"dx": at, stride: 16})), None, 0)


NORM = dict(m=4, c=8, x=P, x_stride=8, residual=Q, residual_stride=8, w=T, y=S, y_stride=8, eps=1e-6, dtype=B.HG_F16, y_dtype=B.HG_F16)


@pytest.mark.parametrize("change", [dict(y=P, y_stride=16), dict(y=Q, y_stride=16), dict(sum=P, sum_stride=16), dict(sum=Q, sum_stride=9),
                                    dict(y=P, y_dtype=R.HG_F8, y_scale=T), dict(y=Q, y_dtype=R.HG_F8, y_scale=T)])
def test_norm_forward(change):
    assert refused("hashgrid_rms_norm_forward", R._RmsNorm(**(NORM | change)))


def test_linear_forward():
    op = dict(m=4, k=8, n=8, x=P, x_stride=8, w=T, w_stride=8, y=Q, y_stride=16, residual=Q, residual_stride=8, x_dtype=B.HG_F16,
              y_dtype=B.HG_F16)
    assert refused("hashgrid_linear_forward", R._Linear(**op))
