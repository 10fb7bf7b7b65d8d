"""Linear layers of very many outputs (or, in the backward, inputs): weights
that are cut into more slices than the card has compute units."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def normal(g, m, n, dtype, scale=1.0):
    return (torch.randn(m, n, generator=g, device=DEV) * scale).to(dtype)


def near_product(got, x, w, b, scales, dtype):
    """got is x w^T + b in every row and column, columns taken in parts: the bound is the reference's, act none."""
    x = x.double() if scales is None else x.double() * scales[0].double()[:, None]
    for at in range(0, w.shape[0], 8192):
        c = slice(at, at + 8192)
        wc = w[c].double() if scales is None else w[c].double() * scales[1][c].double()[:, None]
        z, size = x @ wc.t().contiguous(), x.abs() @ wc.abs().t().contiguous()
        if b is not None:
            z, size = z + b[c].double(), size + b[c].double().abs()
        err = R.rounded(z, (x.shape[1] + 4) * R.EPS32 * size, dtype)
        bad = ~((got[:, c].double() - z).abs() <= err)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off from column {at}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,k,n,dtype", [
    (4096, 512, 50257, F16), (33, 512, 33000, F16), (32, 256, 20000, F16), (32, 256, 32768, BF16), (16, 64, 65536, BF16),
    (12, 64, 65536, F16), (700, 500, 40001, BF16), (2000, 384, 50304, F16), (20, 1024, 17000, F8), (300, 1024, 20000, F8),
    (5000, 7, 65535, F16), (100, 600, 65536, BF16)])
def test_forward_of_many_outputs(m, k, n, dtype):
    g = torch.Generator(device=DEV).manual_seed(m + k + n)
    x, w = normal(g, m, k, dtype), normal(g, n, k, dtype, 20.0 if dtype == F8 else k ** -0.5)
    b = torch.randn(n, generator=g, device=DEV)
    scales = (torch.rand(m, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV) * k ** -0.5) if dtype == F8 else None
    sc = dict(x_scale=scales[0], weight_scale=scales[1]) if scales else {}
    y = hg.hashgrid_linear_forward(x, w, b, **sc)
    near_product(y, x, w, b, scales, y.dtype)


@pytest.mark.parametrize("m,k,n,dtype", [(700, 33001, 500, F16), (40, 50304, 512, BF16)])
def test_backward_of_many_inputs(m, k, n, dtype):
    # dx goes through the forward's kernels with k outputs; with accumulate an error after dW would have added to it already.
    g = torch.Generator(device=DEV).manual_seed(m + k + n)
    x, w, dy = normal(g, m, k, dtype), normal(g, n, k, dtype, n ** -0.5), normal(g, m, n, dtype)
    old, ob = torch.randn(n, k, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)
    dw, db = old.clone(), ob.clone()
    dx, _, _ = hg.hashgrid_linear_backward(dy, x, w, dw=dw, db=db, accumulate=True)
    near_product(dx, dy, w.t().contiguous(), None, None, dtype)
    # one more rounding than the product's, that of the addition
    size = dy.double().abs().t() @ x.double().abs()
    err = (m + 4) * R.EPS32 * size
    want = dy.double().t() @ x.double() + old.double()
    assert ((dw.double() - want).abs() <= R.rounded(want, err, F32)).all()
    want = dy.double().sum(0) + ob.double()
    assert ((db.double() - want).abs() <= R.rounded(want, (m + 4) * R.EPS32 * dy.double().abs().sum(0), F32)).all()
