"""8-bit outputs of the RMS norm for rows whose largest value is near or below
fp32's smallest normal one."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -149  # fp32's smallest value


@pytest.mark.parametrize("c", [5, 40, 101, 256, 1000, 4096, 5000, 5003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tiny_rows_keep_their_values_and_zeros(c, dtype):
    g = torch.Generator().manual_seed(c)
    powers = [-10.0, -33.0, -36.0, -38.0, -39.0, -40.0, -41.0, -42.0, -45.0, -46.0]
    x = torch.randn(len(powers), c, generator=g, dtype=torch.float64) * 10.0 ** torch.tensor(powers, dtype=torch.float64)[:, None]
    x[:, 1::3] = 0
    x = x.to(dtype).to(DEV)
    w = torch.ones(c, device=DEV)
    eps = 1e-6  # the rows' own squares vanish beside it: y = 1000 x
    y, scale, _, _ = hg.hashgrid_rms_norm_forward(x, w, eps=eps, out_dtype=F8)
    _, _, want, rel = R.norm(x, None, w, eps)
    got, sc = y.float().double().cpu(), scale.double().cpu()
    assert got.isfinite().all() and sc.isfinite().all()
    assert not got[want == 0].any()
    # each product and the scale itself round to fp32's steps there, and the scale counts 448 times at most
    top = want.abs().amax(1)
    assert ((sc - top / 448).abs() <= (rel + 4 * R.EPS32) * top / 448 + TINY).all()
    assert not got[sc == 0].any()
    err = want.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10 * sc[:, None] * (1 + 4 * rel) + (448 / 2 + 4) * TINY
    assert ((got * sc[:, None] - want).abs() <= err).all()
    # rows that keep fp32's precision hold their values, not just their signs
    for row in range(4):
        assert got[row].unique().numel() > min(c // 4, 3) and got[row].abs().max() == 448
