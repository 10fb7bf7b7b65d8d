"""The linear backward of one row of matrices with very long rows."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("k,n", [(96, 64), (35, 7), (300, 520)])
def test_one_row_of_very_long_ones(k, n):
    g = torch.Generator(device=DEV).manual_seed(k)
    long = lambda c: torch.randn(1, (1 << 22) + 64, generator=g, device=DEV).half()[:, 1:1 + c]  # noqa: E731
    x, dy, pre, dx = long(k), long(n), long(n), long(k)
    w = torch.randn(n, k, generator=g, device=DEV).half()
    want = hg.hashgrid_linear_backward(dy.contiguous(), x.contiguous(), w, act="silu", pre=pre.contiguous())
    got = hg.hashgrid_linear_backward(dy, x, w, act="silu", pre=pre, dx=dx)
    assert x.stride(0) > 1 << 22 and all(torch.equal(a, b) for a, b in zip(got, want))
