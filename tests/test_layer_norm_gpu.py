"""The layer norm with the residual's addition (hashgrid_layer_norm_*) on the GPU
against its 64-bit form, within the error its roundings allow."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5
COLUMNS = [1, 2, 7, 8, 31, 32, 33, 64, 96, 100, 128, 200, 256, 384, 512, 513, 1000, 1024, 2048, 3000, 4096, 4097, 6001, 10240]


def wide(g, m, n, dtype, pad, shift=0.0):
    t = (torch.randn(m, n + pad, generator=g) + shift).to(dtype).to(DEV)
    return t[:, (pad & 1):(pad & 1) + n]


def gen(*key):
    return torch.Generator().manual_seed(hash(key) & 0x7FFFFFFF)


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_forward(c, dtype, pad):
    for m in (1, 37) if c > 600 else (1, 130, 700):
        g = gen(c, m, pad)
        x, r = wide(g, m, c, dtype, pad, 0.5), wide(g, m, c, dtype, pad)
        w, b = torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
        for res, ww, bb in ((None, w, b), (r, w, None), (r, None, b)):
            y, scale, s, mu, q = hg.hashgrid_layer_norm_forward(x, ww, bb, residual=res, eps=EPS, save_sum=True, save_stats=True)
            ws, wm, wq, wy, (em, eq, ey) = K.layer_norm(x, res, ww, bb, EPS)
            assert scale is None
            R.within(y, wy, R.rounded(wy, ey, dtype))
            R.within(s, ws, R.rounded(ws, R.EPS32 * ws.abs(), dtype))
            R.within(mu, wm, em)
            R.within(q, wq, eq)
            y8, scale, _, _, _ = hg.hashgrid_layer_norm_forward(x, ww, bb, residual=res, eps=EPS, out_dtype=F8)
            K.check_8bit(y8, scale, wy, ey)


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_backward(c, dtype, pad):
    for m in (1, 37) if c > 600 else (1, 130, 5000):
        g = gen(c, m, pad, 1)
        s, dy, ds = wide(g, m, c, dtype, pad, 0.5), wide(g, m, c, dtype, pad), wide(g, m, c, dtype, pad)
        w = torch.randn(c, generator=g).to(DEV)
        mu = s.float().mean(1)
        q = ((s.float() - mu[:, None]).square().mean(1) + EPS).rsqrt()
        for d, ww in ((None, w), (ds, w), (ds, None)):
            dx, dw, db = hg.hashgrid_layer_norm_backward(dy, s, ww, mu, q, ds=d)
            (rx, ex), (rw, ew), (rb, eb) = K.layer_norm_grad(dy, s, ww, mu, q, d)
            R.within(dx, rx, R.rounded(rx, ex, dtype))
            R.within(dw, rw, R.rounded(rw, ew, F32))
            R.within(db, rb, R.rounded(rb, eb, F32))
            again = hg.hashgrid_layer_norm_backward(dy, s, ww, mu, q, ds=d)
            assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
        ow, ob = torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
        got = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, dw=ow.clone(), db=ob.clone(), accumulate=True)
        _, dw, db = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q)
        assert torch.equal(got[1], ow + dw) and torch.equal(got[2], ob + db)
        # each output alone is the same output
        only = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, need_db=False)
        assert torch.equal(only[1], dw) and only[2] is None
        only = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, need_dw=False)
        assert torch.equal(only[2], db) and only[1] is None
        only = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, need_dw=False, need_db=False)
        assert torch.equal(only[0], got[0]) and only[1:] == (None, None)


def test_a_large_mean_costs_no_variance():
    # rows at 1000 whose values are 1/16 apart: fp32 squares of the values would leave nothing of the variance
    g = gen(5)
    for c in (64, 300, 5000):
        x = (1000 + torch.randint(-8, 9, (20, c), generator=g) / 16).to(DEV)
        y, _, _, mu, q = hg.hashgrid_layer_norm_forward(x, save_stats=True)
        _, wm, wq, wy, (em, eq, ey) = K.layer_norm(x, None, None, None, EPS)
        R.within(y, wy, R.rounded(wy, ey, F32))
        R.within(q, wq, eq)
        assert float((q.double().cpu() / wq - 1).abs().max()) < 1e-5


def test_in_place():
    g = gen(3)
    for c in (3, 96, 101, 5000, 5003):
        x, r = wide(g, 50, c, BF16, 0), wide(g, 50, c, BF16, 0)
        w, b = torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
        want = hg.hashgrid_layer_norm_forward(x, w, b, residual=r, save_sum=True)
        a, e = x.clone(), r.clone()
        hg.hashgrid_layer_norm_forward(a, w, b, residual=e, out=a, sum_out=e)
        assert torch.equal(a, want.y) and torch.equal(e, want.sum)
    for c in (3, 96, 101, 513, 2000, 4091):
        for pad in (0, 3):
            dy, s, ds = (wide(g, 300, c, F16, pad) for _ in range(3))
            w = torch.randn(c, generator=g).to(DEV)
            mu = s.float().mean(1)
            q = ((s.float() - mu[:, None]).square().mean(1) + EPS).rsqrt()
            want = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q, ds=ds)
            for i in range(3):
                args = [dy, s, ds]
                args[i] = args[i].clone() if not pad else torch.nn.functional.pad(args[i], (1, 2))[:, 1:-2]
                got = hg.hashgrid_layer_norm_backward(args[0], args[1], w, mu, q, ds=args[2], dx=args[i])
                assert got[0] is args[i] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_constant_rows_and_values_that_are_not_finite():
    for c in (5, 40, 256, 5000):
        x = torch.randn(8, c, generator=gen(c)).to(F16)
        x[0] = 2.0
        x[1, 3] = float("nan")
        x[2, 4] = float("inf")
        x = x.to(DEV)
        w, b = torch.ones(c, device=DEV), torch.full((c,), 0.25, device=DEV)
        y = hg.hashgrid_layer_norm_forward(x, w, b).y
        assert (y[0] == 0.25).all() and y[1].isnan().all() and y[2].isnan().all()  # a constant row has no deviation
        assert torch.equal(y[3:], hg.hashgrid_layer_norm_forward(x[3:].contiguous(), w, b).y)
        y8, scale, _, _, _ = hg.hashgrid_layer_norm_forward(x, w, out_dtype=F8)
        assert scale[0] == 0 and not y8[0].float().any() and scale[1].isnan() and scale[2].isnan()
        assert scale[3:].isfinite().all() and y8[3:].float().isfinite().all()
        assert hg.hashgrid_layer_norm_forward(x[:1], w, eps=0.0).y.isnan().all()  # 0 * inf
        # rows next to one that is not finite keep their gradients
        mu, q = x.float().mean(1), torch.ones(8, device=DEV)
        dx = hg.hashgrid_layer_norm_backward(x, x, w, mu, q)[0]
        assert dx[1].isnan().all() and torch.equal(dx[3:], hg.hashgrid_layer_norm_backward(x[3:], x[3:], w, mu[3:], q[3:])[0])


def test_rows_of_one_column_have_no_gradient():
    g = gen(9)
    s, dy, w = wide(g, 500, 1, F32, 0), wide(g, 500, 1, F32, 0), torch.randn(1, generator=g).to(DEV)
    out = hg.hashgrid_layer_norm_forward(s, w, save_stats=True)
    assert not out.y.any()
    assert not hg.hashgrid_layer_norm_backward(dy, s, w, out.mean, out.rstd)[0].any()


def test_the_norm_feeds_the_8bit_product():
    g = gen(4)
    x, r = wide(g, 300, 96, BF16, 0), wide(g, 300, 96, BF16, 0)
    w, b = torch.rand(96, generator=g).to(DEV) + 0.5, torch.randn(96, generator=g).to(DEV)
    y8, scale, _, _, _ = hg.hashgrid_layer_norm_forward(x, w, b, residual=r, out_dtype=F8)
    w8, ws = torch.randn(64, 96, generator=g).to(F8).to(DEV), torch.rand(64, generator=g).to(DEV)
    y = hg.hashgrid_linear_forward(y8, w8, x_scale=scale, weight_scale=ws)
    wy, _, ey, _ = R.linear(y8, w8, None, "none", None, scale, ws, BF16)
    R.within(y, wy, ey)


def test_gradient_against_differences():
    g = gen(6)
    m, c = 9, 21
    x, dy, w, b = wide(g, m, c, F32, 0), wide(g, m, c, F32, 0), torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
    _, _, s, mu, q = hg.hashgrid_layer_norm_forward(x, w, b, eps=EPS, save_sum=True, save_stats=True)
    got = hg.hashgrid_layer_norm_backward(dy, s, w, mu, q)
    X, W, B, D = (t.double().cpu() for t in (x, w, b, dy))
    h = 1e-5

    def loss(t):
        d = t[0] - t[0].mean(1, keepdim=True)
        return (D * (d * (d.square().mean(1, keepdim=True) + EPS).rsqrt() * t[1] + t[2])).sum()

    for k in range(3):
        for i in range((X, W, B)[k].numel()):
            a, z = [t.clone() for t in (X, W, B)], [t.clone() for t in (X, W, B)]
            a[k].view(-1)[i] += h
            z[k].view(-1)[i] -= h
            assert abs(got[k].double().cpu().view(-1)[i] - (loss(a) - loss(z)) / (2 * h)) <= 1e-4


def test_no_rows_another_stream_and_graph_replay():
    w = torch.ones(96, device=DEV)
    e, n = torch.empty(0, 96, dtype=F16, device=DEV), torch.empty(0, device=DEV)
    assert hg.hashgrid_layer_norm_forward(e, w, w).y.shape == (0, 96)
    for c in (96, 5000):
        e, w2 = torch.empty(0, c, dtype=F16, device=DEV), torch.ones(c, device=DEV)
        dx, dw, db = hg.hashgrid_layer_norm_backward(e, e, w2, n, n)
        assert dx.shape == (0, c) and not dw.any() and not db.any()
    g = gen(8)
    x, dy = wide(g, 3000, 96, F16, 0), wide(g, 3000, 96, F16, 0)

    def both(stream=None):
        o = hg.hashgrid_layer_norm_forward(x, w, w, residual=dy, save_sum=True, save_stats=True, stream=stream)
        return (o.y, o.sum, o.mean, o.rstd) + hg.hashgrid_layer_norm_backward(dy, o.sum, w, o.mean, o.rstd, ds=o.y, stream=stream)

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
