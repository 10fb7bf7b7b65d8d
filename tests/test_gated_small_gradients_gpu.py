"""Gated layers' gradients of upstream ones as small as a mean loss over many points
makes them: what binary16 keeps of dg and du, with a loss scale and without."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def operands(m, k, n, dtype, size):
    g = torch.Generator().manual_seed(m + k + n)
    make = lambda i, j, s=1.0: (torch.randn(i, j, generator=g) * s).to(dtype).to(DEV)  # noqa: E731
    return make(m, n, size), [make(m, k), make(n, k, k ** -0.5), make(n, k, k ** -0.5), make(m, n), make(m, n)]


# one pass of one tile, two passes, units in slices
@pytest.mark.parametrize("m,k,n", [(5000, 64, 96), (3000, 300, 140), (256, 256, 512)])
@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** -18, 2.0 ** -20])
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_small_upstream_gradients(monkeypatch, m, k, n, size, act):
    # in binary16 as it stands: each value of dg and du is off by 2^-11 of itself, or by half the smallest step, 2^-25
    dh, rest = operands(m, k, n, F16, size)
    bounds = K.gated_grad(dh, *rest, act)
    for t, (want, err), kept in zip(hg.hashgrid_gated_backward(dh, *rest, act=act), bounds, (F16, F32, F32, F32, F32)):
        R.within(t, want, R.rounded(want, err, kept))
    # with the loss scaled by 2^14 (exact: dh's values are whole multiples of 2^-24 of 11 bits and fewer) they are off by
    # 2^-11 of themselves down to 2^-28: the bound without the steps' end, and those values' half step of 2^-39 beside it
    scale, half = 2.0 ** 14, 2.0 ** -39
    scaled = (dh.double() * scale).to(F16)
    assert torch.equal(scaled.double() / scale, dh.double())
    got = hg.hashgrid_gated_backward(scaled, *rest, act=act)
    monkeypatch.setitem(R.TINY, F16, 0.0)
    x = rest[0].double().cpu().abs()
    ends = [None, half * x.sum(0), half * x.sum(0), 0.0, 0.0]
    for i, (want, err) in enumerate(K.gated_grad(dh, *rest, act)):
        if i:  # (dx is binary16 itself: it is unscaled where it is used)
            R.within(got[i].double() / scale, want, R.rounded(want, err + ends[i], F32))
    dx = torch.stack([w.double().cpu().abs().sum(0) for w in rest[1:3]]).sum(0) * half
    want, err = K.gated_grad(dh, *rest, act)[0]
    R.within(got[0].double() / scale, want, R.rounded(want, err + dx, F16) + 2.0 ** -25 / scale)


@pytest.mark.parametrize("m,k,n", [(5000, 64, 96), (3000, 300, 140)])
def test_bfloat16_needs_no_scale(m, k, n):
    # its exponents are fp32's: dh times a power of two gives the same gradients times it
    dh, rest = operands(m, k, n, BF16, 1.0)
    want = hg.hashgrid_gated_backward(dh, *rest)
    for power in (-20, 14):
        got = hg.hashgrid_gated_backward(dh * 2.0 ** power, *rest)
        assert all(torch.equal(a, (b.double() * 2.0 ** power).to(a.dtype)) for a, b in zip(got, want))
