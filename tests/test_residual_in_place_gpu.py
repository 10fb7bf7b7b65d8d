"""Outputs that take the place of an input, as the residual head's operators
allow it."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def part(t, pad):
    """The same values as columns 1.. of a wider buffer, if pad."""
    if not pad:
        return t.clone()
    buf = torch.full((t.shape[0], t.shape[1] + pad), 3.0, device=DEV, dtype=t.dtype)
    buf[:, 1:1 + t.shape[1]] = t
    return buf[:, 1:1 + t.shape[1]]


@pytest.mark.parametrize("m,k,n", [(5, 7, 3), (40, 1024, 512), (1000, 32, 256), (3001, 96, 65), (5003, 256, 256), (20000, 256, 4),
                                   (4001, 500, 330), (3000, 700, 64), (2000, 520, 300)])
@pytest.mark.parametrize("dtype", [F16, BF16, F8])
@pytest.mark.parametrize("pad", [0, 3])
def test_linear_over_its_residual(m, k, n, dtype, pad):
    g = torch.Generator(device=DEV).manual_seed(m + k + n)
    x, w = (torch.randn(s, k, generator=g, device=DEV).to(dtype) for s in (m, n))
    sc = dict(x_scale=torch.rand(m, generator=g, device=DEV), weight_scale=torch.rand(n, generator=g, device=DEV)) if dtype == F8 else {}
    for out in (BF16 if dtype == F8 else dtype, F32):
        r = torch.randn(m, n, generator=g, device=DEV).to(out)
        want = hg.hashgrid_linear_forward(x, w, act="silu", residual=r, out_dtype=out, **sc)
        y = part(r, pad)
        hg.hashgrid_linear_forward(x, w, act="silu", residual=y, out=y, **sc)
        assert torch.equal(y, want)


@pytest.mark.parametrize("c", [3, 31, 96, 101, 256, 513, 1000, 2000, 2049, 4091, 4096])
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_norm_backward_over_its_inputs(c, dtype, pad):
    g = torch.Generator(device=DEV).manual_seed(c)
    m = 3000 if c < 600 else 300
    dy, s, ds = (torch.randn(m, c, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(c, generator=g, device=DEV)
    q = (s.float().square().mean(1) + 1e-6).rsqrt()
    want = hg.hashgrid_rms_norm_backward(dy, s, w, q, ds=ds)
    for i in range(3):
        args = [dy, s, ds]
        args[i] = part(args[i], pad)
        got = hg.hashgrid_rms_norm_backward(args[0], args[1], w, q, ds=args[2], dx=args[i])
        assert got[0] is args[i] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_longer_rows_refuse():
    dy, s = (torch.randn(4, 4097, device=DEV) for _ in range(2))
    w, q = torch.ones(4097, device=DEV), torch.ones(4, device=DEV)
    for dx in (dy, s):
        with pytest.raises(hg.HashGridError, match="in place"):
            hg.hashgrid_rms_norm_backward(dy, s, w, q, dx=dx)
