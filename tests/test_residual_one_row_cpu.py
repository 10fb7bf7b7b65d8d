"""Row strides of the linear backward where there is one row, or no matrix: not
looked at (the C ABI's checks; nothing is launched)."""
import ctypes

import pytest

from multiresolution_hash_grid_amd import hashgrid as B
from multiresolution_hash_grid_amd import residual as R

P = 0x1000
GRAD = dict(m=1, k=8, n=8, dy=P, dy_stride=8, pre=P, pre_stride=8, x=P, x_stride=8, w=P, w_stride=8, dx=P, dx_stride=8, dw=P,
            dw_stride=8, db=P, dtype=B.HG_F16, dy_dtype=B.HG_F16, dw_dtype=B.HG_F32, act=2)


def size(**change):
    out = ctypes.c_size_t(0)
    op = R._LinearGrad(**(GRAD | change))
    return R._lib().hashgrid_linear_backward_workspace_size(ctypes.byref(op), ctypes.byref(out))


@pytest.mark.parametrize("name", ["dy_stride", "pre_stride", "x_stride", "dx_stride"])
@pytest.mark.parametrize("stride", [(1 << 22) + 1, 1 << 40, -5, 0])
def test_one_row_has_no_stride(name, stride):
    assert size(**{name: stride}) == B.HG_OK
    if stride > 0:
        assert size(m=2, **{name: stride}) == B.HG_EINVAL


def test_a_matrix_that_is_left_out_has_no_stride():
    assert size(m=100, pre=None, pre_stride=1 << 30, act=0) == B.HG_OK
    assert size(m=100, dx=None, dx_stride=1 << 30) == B.HG_OK
