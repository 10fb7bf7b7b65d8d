"""8-bit gated layers whose scales' product leaves fp32 although every result lies in
it: a row's scale and a unit's are applied one after the other, by every kernel."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F8 = torch.float32, torch.float8_e4m3fn

# few rows (tiles), fewer inputs than a piece, weights in LDS, in registers, in blocks
SIZES = [(1, 256, 40), (33, 100, 70), (5, 7, 9), (9001, 64, 100), (33001, 128, 400), (20001, 600, 130)]


def operands(m, k, n, zeros=False):
    g = torch.Generator().manual_seed(m + k + n)
    x, wg, wu = (torch.randn(i, k, generator=g) * 100 for i in (m, n, n))
    if zeros:
        wg[::2] = 0.0
    at = torch.cat([torch.arange(min(m, 200)), torch.randint(0, m, (200,), generator=g), torch.arange(max(0, m - 200), m)])
    return (g, at.to(DEV)) + tuple(t.to(F8).to(DEV) for t in (x, wg, wu))


def within(h, want, err):
    """R.within, and NaN where a NaN is due (a few values lie past 448 and have no other code)."""
    bad = want.isnan()
    assert torch.equal(h.isnan().cpu(), bad) and not bad.all()
    R.within(h.cpu().masked_fill(bad, 0.0), want.masked_fill(bad, 0.0), err.masked_fill(bad, 0.0))


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("row,unit", [(2.0 ** -110, 2.0 ** -39), (2.0 ** -126, 2.0 ** -20), (2.0 ** -60, 2.0 ** -80)])
def test_small_scales(m, k, n, row, unit):
    # The gate's two scales multiply to 2^-149 .. 2^-140, where fp32 has one bit to ten; its sums of some 2^15 bring it
    # back to where there are 15 and more, and the other projection, scaled to its sums' size, brings h to 2^-120 and up.
    g, at, x, wg, wu = operands(m, k, n)
    xs = (row * (1 + torch.rand(m, generator=g))).to(DEV)
    gs = (unit * (1 + torch.rand(n, generator=g))).to(DEV)
    us = (0.5 / row * (1 + torch.rand(n, generator=g))).to(DEV)
    h = hg.hashgrid_gated_forward(x, wg, wu, act="none", x_scale=xs, gate_scale=gs, up_scale=us, out_dtype=F32)
    wh, zg, zu, eh, _, _ = K.gated(x[at], wg, wu, None, None, "none", xs[at], gs, us, F32)
    # Below 2^-126 a rounding is off by up to 2^-150 whatever the value: of the row's scaled sum, multiplied by the
    # unit's scale then, and of the gate itself
    scaled = 2.0 ** -150
    e_g, e_u = scaled * gs.double().cpu() + 2.0 ** -150, scaled * us.double().cpu()
    within(h[at], wh, eh + 1.001 * (e_g * zu.abs() + e_u * (zg.abs() + e_g)))


@pytest.mark.parametrize("m,k,n", SIZES)
def test_large_scales(m, k, n):
    # 2^100 times 2^40 is no fp32 number; a unit whose weights are zeros has its bias all the same
    g, at, x, wg, wu = operands(m, k, n, zeros=True)
    xs, gs, us = torch.full((m,), 2.0 ** 100, device=DEV), torch.full((n,), 2.0 ** 40, device=DEV), torch.full((n,), 2.0 ** -100, device=DEV)
    bg = torch.randn(n, generator=g).to(DEV)
    h = hg.hashgrid_gated_forward(x, wg, wu, bg, act="none", x_scale=xs, gate_scale=gs, up_scale=us, out_dtype=F32)
    wh, _, _, eh, _, _ = K.gated(x[at], wg[::2], wu[::2], bg[::2], None, "none", xs[at], gs[::2], us[::2], F32)
    within(h[at][:, ::2], wh, eh)
