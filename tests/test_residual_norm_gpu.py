"""The RMS norm with the residual's addition (hashgrid_rms_norm_*) on the GPU
against its 64-bit form, within the error its roundings allow."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6
COLUMNS = [1, 7, 8, 31, 32, 33, 64, 96, 100, 128, 200, 256, 384, 512, 513, 1000, 1024, 2048, 3000, 4096, 4097, 6001, 10240]


def wide(g, m, n, dtype, pad):
    t = torch.randn(m, n + pad, generator=g).to(dtype).to(DEV)
    return t[:, (pad & 1):(pad & 1) + n]


def gen(*key):
    return torch.Generator().manual_seed(hash(key) & 0x7FFFFFFF)


def check_8bit(y, scale, want, rel):
    # |y| <= 448 scale; a code is within half its step (2^-4 of the value, 2^-10 of the scale below 2^-6) of its value.
    top = want.abs().amax(1)
    assert ((scale.double().cpu() - top / 448).abs() <= (rel + 4 * R.EPS32) * top / 448).all()
    sc = scale.double().cpu()[:, None]
    R.within(y.float().double() * scale.double()[:, None], want, want.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10 * sc * (1 + 4 * rel))


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_forward(c, dtype, pad):
    for m in (1, 37) if c > 600 else (1, 130, 700):
        g = gen(c, m, pad)
        x, r = wide(g, m, c, dtype, pad), wide(g, m, c, dtype, pad)
        w = torch.randn(c, generator=g).to(DEV)
        for res in (None, r):
            y, scale, s, q = hg.hashgrid_rms_norm_forward(x, w, residual=res, eps=EPS, save_sum=True, save_rstd=True)
            ws, wq, wy, rel = R.norm(x, res, w, EPS)
            assert scale is None
            R.within(y, wy, R.rounded(wy, rel * wy.abs(), dtype))
            R.within(s, ws, R.rounded(ws, R.EPS32 * ws.abs(), dtype))
            R.within(q, wq, rel * wq)
            y8, scale, _, _ = hg.hashgrid_rms_norm_forward(x, w, residual=res, eps=EPS, out_dtype=F8)
            check_8bit(y8, scale, wy, rel)


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_backward(c, dtype, pad):
    for m in (1, 37) if c > 600 else (1, 130, 5000):
        g = gen(c, m, pad, 1)
        s, dy, ds = (wide(g, m, c, dtype, pad) for _ in range(3))
        w = torch.randn(c, generator=g).to(DEV)
        q = (s.float().square().mean(1) + EPS).rsqrt()
        for d in (None, ds):
            dx, dw = hg.hashgrid_rms_norm_backward(dy, s, w, q, ds=d)
            (rx, ex), (rw, ew) = R.norm_grad(dy, s, w, q, d)
            R.within(dx, rx, R.rounded(rx, ex, dtype))
            R.within(dw, rw, R.rounded(rw, ew, F32))
            again = hg.hashgrid_rms_norm_backward(dy, s, w, q, ds=d)
            assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
        old = torch.randn(c, generator=g).to(DEV)
        got = hg.hashgrid_rms_norm_backward(dy, s, w, q, ds=ds, dw=old.clone(), accumulate=True)[1]
        assert torch.equal(got, old + dw)
        assert hg.hashgrid_rms_norm_backward(dy, s, w, q, need_dw=False)[1] is None


def test_in_place():
    g = gen(3)
    for c in (3, 96, 101, 5000, 5003):
        x, r = wide(g, 50, c, BF16, 0), wide(g, 50, c, BF16, 0)
        w = torch.randn(c, generator=g).to(DEV)
        want = hg.hashgrid_rms_norm_forward(x, w, residual=r, save_sum=True)
        a, b = x.clone(), r.clone()
        hg.hashgrid_rms_norm_forward(a, w, residual=b, out=a, sum_out=b)
        assert torch.equal(a, want.y) and torch.equal(b, want.sum)


def test_rows_of_zeros_and_values_that_are_not_finite():
    for c in (40, 256, 5000):
        x = torch.randn(8, c, generator=gen(c)).to(F16)
        x[0] = 0
        x[1, 3] = float("nan")
        x[2, 5] = float("inf")
        x = x.to(DEV)
        w = torch.ones(c, device=DEV)
        y = hg.hashgrid_rms_norm_forward(x, w).y
        assert not y[0].any() and y[1].isnan().all()
        assert y[2, 5].isnan() and not y[2, :5].any()      # inf / inf, and finite / inf
        good = hg.hashgrid_rms_norm_forward(x[3:].contiguous(), w).y
        assert torch.equal(y[3:], good)
        y8, scale, _, _ = hg.hashgrid_rms_norm_forward(x, w, out_dtype=F8)
        assert scale[0] == 0 and not y8[0].float().any() and scale[1].isnan() and scale[2].isnan()
        assert scale[3:].isfinite().all() and y8[3:].float().isfinite().all()
        # a row of zeros with eps = 0: 0 * inf
        assert hg.hashgrid_rms_norm_forward(x[:1], w, eps=0.0).y.isnan().all()


def test_the_norm_feeds_the_8bit_product():
    g = gen(4)
    x, r = wide(g, 300, 96, BF16, 0), wide(g, 300, 96, BF16, 0)
    w = torch.rand(96, generator=g).to(DEV) + 0.5
    y8, scale, _, _ = hg.hashgrid_rms_norm_forward(x, w, residual=r, out_dtype=F8)
    w8, ws = torch.randn(64, 96, generator=g).to(F8).to(DEV), torch.rand(64, generator=g).to(DEV)
    y = hg.hashgrid_linear_forward(y8, w8, x_scale=scale, weight_scale=ws)
    wy, _, ey, _ = R.linear(y8, w8, None, "none", None, scale, ws, BF16)
    R.within(y, wy, ey)


def test_gradient_against_differences():
    g = gen(6)
    m, c = 9, 21
    x, dy, w = wide(g, m, c, F32, 0), wide(g, m, c, F32, 0), torch.randn(c, generator=g).to(DEV)
    _, _, s, q = hg.hashgrid_rms_norm_forward(x, w, eps=EPS, save_sum=True, save_rstd=True)
    dx, dw = hg.hashgrid_rms_norm_backward(dy, s, w, q)
    X, W, D = (t.double().cpu() for t in (x, w, dy))
    h = 1e-5

    def loss(X, W):
        return (D * X * (X.square().mean(1, keepdim=True) + EPS).rsqrt() * W).sum()

    for t, got in ((X, dx), (W, dw)):
        for i in range(t.numel()):
            d = torch.zeros_like(t)
            d.view(-1)[i] = h
            want = (loss(X + d, W) - loss(X - d, W)) / (2 * h) if t is X else (loss(X, W + d) - loss(X, W - d)) / (2 * h)
            assert abs(got.double().cpu().view(-1)[i] - want) <= 1e-4


def test_no_rows_another_stream_and_graph_replay():
    w = torch.ones(96, device=DEV)
    e = torch.empty(0, 96, dtype=F16, device=DEV)
    assert hg.hashgrid_rms_norm_forward(e, w).y.shape == (0, 96)
    dx, dw = hg.hashgrid_rms_norm_backward(e, e, w, torch.empty(0, device=DEV))
    assert dx.shape == (0, 96) and not dw.any()
    g = gen(8)
    x, dy = wide(g, 3000, 96, F16, 0), wide(g, 3000, 96, F16, 0)

    def both(stream=None):
        o = hg.hashgrid_rms_norm_forward(x, w, residual=dy, save_sum=True, save_rstd=True, stream=stream)
        return (o.y, o.sum, o.rstd) + hg.hashgrid_rms_norm_backward(dy, o.sum, w, o.rstd, ds=o.y, stream=stream)

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g).to(F16).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both()))
