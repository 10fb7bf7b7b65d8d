"""Layer norms and gated layers over more rows than one round of workgroups takes, so
that a workgroup goes on to a second row or tile in every form of its kernel."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5


def rows(g, m, n, dtype, scale=1.0, pad=0):
    """[m, n] as columns of a buffer that is ``pad`` wider, at an odd place for odd ones."""
    t = (torch.randn(m, n + pad, generator=g) * scale).clamp(-448.0, 448.0).to(dtype).to(DEV)
    return t[:, (pad & 1):(pad & 1) + n]


def spans(m, most):
    """Stretches of ``most`` rows that cover m; the last one ends with them."""
    return [(a, a + most) for a in range(0, m - most, most)] + [(max(0, m - most), m)]


# dx by a kernel of its own: 256 rows a tile.  More tiles than workgroups (256 over the columns' tiles, 512 for inputs
# that 64 columns hold), the last one ragged: all of a row's inputs in one tile, in two, in narrower ones, and inputs or
# units of rows shorter than a piece.
@pytest.mark.parametrize("m,k,n,tiles_k", [(70001, 256, 136, 1), (40001, 300, 140, 2), (70001, 100, 200, 1), (140001, 40, 136, 1),
                                           (140001, 5, 136, 1), (70001, 100, 5, 2)])
@pytest.mark.parametrize("dtype,act", [(F16, "gelu_tanh"), (BF16, "silu")])
def test_gated_backward_of_more_tiles_than_workgroups(m, k, n, tiles_k, dtype, act):
    g = torch.Generator().manual_seed(m + k + n)
    x, wg, wu = rows(g, m, k, dtype, 1.0, 8), rows(g, n, k, dtype, k ** -0.5), rows(g, n, k, dtype, k ** -0.5)
    dh, gate, up = (rows(g, m, n, dtype, 1.0, p) for p in (3, 0, 6))
    got = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=act)
    for t, (want, err), kept in zip(got, K.gated_grad(dh, x, wg, wu, gate, up, act), (dtype, F32, F32, F32, F32)):
        R.within(t, want, R.rounded(want, err, kept))
    again = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # a row's dx in calls whose workgroups have a tile each (and as many as leave the units uncut)
    for a, z in spans(m, 128 // tiles_k * 256):
        part = hg.hashgrid_gated_backward(dh[a:z], x[a:z], wg, wu, gate[a:z], up[a:z], act=act, need_dw=False, need_db=False)[0]
        assert torch.equal(part, got[0][a:z])


def gated_rows(g, m, k, n, dtype):
    """(operands, scales) of a forward."""
    eight = dtype == F8
    x, wg, wu = rows(g, m, k, dtype, 20.0 if eight else 1.0, 5), *(rows(g, n, k, dtype, 20.0 if eight else k ** -0.5) for _ in range(2))
    b = [torch.randn(n, generator=g).to(DEV) for _ in range(2)]
    sc = [(torch.rand(i, generator=g) * s).to(DEV) for i, s in ((m, 0.1), (n, k ** -0.5), (n, k ** -0.5))] if eight else [None] * 3
    return (x, wg, wu, *b), sc


# weights that LDS does not hold, in registers: 66001 rows leave the units uncut, and so do 33001 of them
@pytest.mark.parametrize("k,n", [(60, 700), (128, 1024), (192, 200), (250, 300), (384, 160), (512, 300)])
@pytest.mark.parametrize("out", [F32, F16])
def test_gated_8bit_forward_with_weights_in_registers(k, n, out):
    m = 66001
    g = torch.Generator().manual_seed(k + n)
    ops, (xs, gs, us) = gated_rows(g, m, k, n, F8)
    h = hg.hashgrid_gated_forward(*ops, act="gelu_tanh", out_dtype=out, x_scale=xs, gate_scale=gs, up_scale=us)
    at = torch.cat([torch.arange(300), torch.randint(0, m, (2000,), generator=g), torch.arange(m - 300, m)]).to(DEV)
    wh, _, _, eh, _, _ = K.gated(ops[0][at], *ops[1:], "gelu_tanh", xs[at], gs, us, out)
    R.within(h[at], wh, eh)
    for a, z in spans(m, 33001):
        part = hg.hashgrid_gated_forward(ops[0][a:z], *ops[1:], act="gelu_tanh", out_dtype=out, x_scale=xs[a:z], gate_scale=gs, up_scale=us)
        assert torch.equal(part, h[a:z])


@pytest.mark.parametrize("k,n", [(32, 1200), (64, 700), (96, 420), (128, 310), (192, 230), (256, 300)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("wide", [True, False])
def test_gated_forward_with_weights_in_registers(k, n, dtype, wide):
    m, out = 66001, F32 if wide else dtype
    g = torch.Generator().manual_seed(k + n)
    ops, _ = gated_rows(g, m, k, n, dtype)
    h, gate, up = hg.hashgrid_gated_forward(*ops, out_dtype=out, save_pre=True)
    assert torch.equal(hg.hashgrid_gated_forward(*ops, out_dtype=out), h)
    at = torch.cat([torch.arange(300), torch.randint(0, m, (2000,), generator=g), torch.arange(m - 300, m)]).to(DEV)
    wh, zg, zu, eh, eg, eu = K.gated(ops[0][at], *ops[1:], "silu", None, None, None, out)
    R.within(h[at], wh, eh)
    R.within(gate[at], zg, R.rounded(zg, eg, dtype))
    R.within(up[at], zu, R.rounded(zu, eu, dtype))
    for a, z in spans(m, 33001):
        part = hg.hashgrid_gated_forward(ops[0][a:z], *ops[1:], out_dtype=out, save_pre=True)
        assert all(torch.equal(p, t[a:z]) for p, t in zip(part, (h, gate, up)))


# 2048 workgroups of 256 threads: of 64 rows, of 32, 16, 8, 4 and 4 of two pieces a lane, of one, and of one whose
# columns come in rounds
NORMS = [(140003, 32), (70001, 64), (33001, 100), (17001, 200), (9001, 384), (9001, 513), (2500, 2000), (2100, 4091), (2500, 4100)]


@pytest.mark.parametrize("m,c", NORMS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_layer_norm_forward(m, c, dtype):
    g = torch.Generator().manual_seed(m + c)
    x, r = rows(g, m, c, dtype, 1.0, 3), rows(g, m, c, dtype, 1.0, 4)
    w, b = torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
    out = hg.hashgrid_layer_norm_forward(x, w, b, residual=r, eps=EPS, save_sum=True, save_stats=True)
    ws, wm, wq, wy, (em, eq, ey) = K.layer_norm(x, r, w, b, EPS)
    R.within(out.y, wy, R.rounded(wy, ey, dtype))
    R.within(out.sum, ws, R.rounded(ws, R.EPS32 * ws.abs(), dtype))
    R.within(out.mean, wm, em)
    R.within(out.rstd, wq, eq)
    eight = hg.hashgrid_layer_norm_forward(x, w, b, residual=r, eps=EPS, out_dtype=F8)
    K.check_8bit(eight.y, eight.scale, wy, ey)
    # the same rows in calls whose workgroups have one round of them
    for a, z in spans(m, m // 2 + 1):
        part = hg.hashgrid_layer_norm_forward(x[a:z], w, b, residual=r[a:z], eps=EPS, save_sum=True, save_stats=True)
        assert all(torch.equal(getattr(part, f), getattr(out, f)[a:z]) for f in ("y", "sum", "mean", "rstd"))
        part = hg.hashgrid_layer_norm_forward(x[a:z], w, b, residual=r[a:z], eps=EPS, out_dtype=F8)
        assert torch.equal(part.y.view(torch.uint8), eight.y[a:z].view(torch.uint8)) and torch.equal(part.scale, eight.scale[a:z])


@pytest.mark.parametrize("m,c", NORMS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_layer_norm_backward(m, c, dtype):
    g = torch.Generator().manual_seed(m + c + 1)
    dy, s, ds = (rows(g, m, c, dtype, 1.0, p) for p in (5, 0, 2))
    w = torch.randn(c, generator=g).to(DEV)
    mu = s.float().mean(1)
    q = ((s.float() - mu[:, None]).square().mean(1) + EPS).rsqrt()
    got = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, ds=ds)
    for t, (want, err), kept in zip(got, K.layer_norm_grad(dy, s, w, mu, q, ds), (dtype, F32, F32)):
        R.within(t, want, R.rounded(want, err, kept))
    again = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, ds=ds)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for a, z in spans(m, 500):  # a row at most for each workgroup
        part = hg.hashgrid_layer_norm_backward(dy[a:z], s[a:z], w, mu[a:z], q[a:z], ds=ds[a:z], need_dw=False, need_db=False)[0]
        assert torch.equal(part, got[0][a:z])
