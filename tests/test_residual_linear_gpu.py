"""The linear layer (hashgrid_linear_forward and _backward) on the GPU against
its 64-bit form, within the error its roundings allow (residual_reference)."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
ACTS = ["none", "relu", "silu", "gelu_tanh"]


def wide(g, m, n, dtype, pad, scale=1.0):
    """[m, n] as columns 1.. of a wider buffer when pad is odd (so that no row is aligned), 0.. otherwise."""
    at = pad & 1
    t = (torch.randn(m, n + pad, generator=g) * scale).to(dtype).to(DEV)
    return t[:, at:at + n] if pad else t


def gen(*key):
    return torch.Generator().manual_seed(hash(key) & 0x7FFFFFFF)


SIZES = [(1, 1, 1), (1, 96, 64), (3, 7, 5), (16, 32, 16), (17, 33, 19), (64, 64, 4), (65, 35, 64), (127, 31, 129), (130, 256, 256),
         (257, 96, 33), (1000, 130, 70), (300, 520, 300), (40, 1024, 512), (33, 8, 1024), (5000, 35, 64), (9000, 256, 4)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_forward(m, k, n, dtype, pad):
    g = gen(m, k, n, pad)
    x, w = wide(g, m, k, dtype, pad), wide(g, n, k, dtype, pad, k ** -0.5)
    b = torch.randn(n, generator=g).to(DEV)
    for i, kind in enumerate(ACTS):
        out = F32 if (i + m) % 3 == 0 else dtype
        r = wide(g, m, n, out, pad) if i % 2 else None
        bias = None if kind == "none" else b
        y, z = hg.hashgrid_linear_forward(x, w, bias, act=kind, residual=r, out_dtype=out, save_pre=True)
        wy, wz, ey, ez = R.linear(x, w, bias, kind, r, None, None, out)
        assert y.dtype == out and z.dtype == dtype
        R.within(y, wy, ey)
        R.within(z, wz, R.rounded(wz, ez, dtype))
        assert torch.equal(y, hg.hashgrid_linear_forward(x, w, bias, act=kind, residual=r, out_dtype=out))


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("pad", [0, 3])
def test_forward_8bit(m, k, n, pad):
    g = gen(m, k, n, pad, 8)
    x, w = wide(g, m, k, F8, pad, 20.0), wide(g, n, k, F8, pad, 20.0)
    xs, ws = (torch.rand(m, generator=g) * 0.1).to(DEV), (torch.rand(n, generator=g) * k ** -0.5).to(DEV)
    b = torch.randn(n, generator=g).to(DEV)
    for i, kind in enumerate(ACTS):
        out = (BF16, F16, F32)[(i + k) % 3]
        r = wide(g, m, n, out, pad) if i % 2 else None
        y = hg.hashgrid_linear_forward(x, w, b, act=kind, residual=r, x_scale=xs, weight_scale=ws, out_dtype=out)
        wy, _, ey, _ = R.linear(x, w, b, kind, r, xs, ws, out)
        R.within(y, wy, ey)


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_backward(m, k, n, dtype, pad):
    g = gen(m, k, n, pad, 1)
    x, w = wide(g, m, k, dtype, pad), wide(g, n, k, dtype, pad, k ** -0.5)
    for i, kind in enumerate(ACTS):
        dy = wide(g, m, n, F32 if (i + n) % 3 == 0 else dtype, pad)
        pre = wide(g, m, n, dtype, pad) if kind != "none" else None
        wd = F32 if i % 2 else dtype
        dx, dw, db = hg.hashgrid_linear_backward(dy, x, w, act=kind, pre=pre, weight_dtype=wd)
        (rx, ex), (rw, ew), (rb, eb) = R.linear_grad(dy, x, w, pre, kind)
        R.within(dx, rx, R.rounded(rx, ex, dtype))
        R.within(dw, rw, R.rounded(rw, ew, wd))
        R.within(db, rb, R.rounded(rb, eb, F32))
        again = hg.hashgrid_linear_backward(dy, x, w, act=kind, pre=pre, weight_dtype=wd)
        assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
        # each output alone is the same output
        only = hg.hashgrid_linear_backward(dy, x, w, act=kind, pre=pre, weight_dtype=wd, need_dx=False, need_db=False)
        assert only[0] is None and only[2] is None and torch.equal(only[1], dw)
        only = hg.hashgrid_linear_backward(dy, x, w, act=kind, pre=pre, need_dw=False, need_db=False)
        assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
        only = hg.hashgrid_linear_backward(dy, x, w, act=kind, pre=pre, need_dw=False, need_dx=False)
        assert torch.equal(only[2], db)


def test_backward_accumulates():
    g = gen(11)
    for dtype, wd in ((F16, F32), (BF16, BF16)):
        x, w, dy = wide(g, 333, 40, dtype, 0), wide(g, 24, 40, dtype, 0), wide(g, 333, 24, dtype, 0)
        old, ob = torch.randn(24, 40, generator=g).to(wd).to(DEV), torch.randn(24, generator=g).to(DEV)
        _, dw0, db0 = hg.hashgrid_linear_backward(dy, x, w, weight_dtype=F32)
        dw, db = old.clone(), ob.clone()
        hg.hashgrid_linear_backward(dy, x, w, dw=dw, db=db, accumulate=True, need_dx=False)
        assert torch.equal(dw, (old.float() + dw0).to(wd)) and torch.equal(db, ob + db0)


@pytest.mark.parametrize("m", [1, 20, 32])
@pytest.mark.parametrize("k,n", [(40, 24), (5, 300), (300, 3), (256, 200)])
def test_backward_of_few_rows_accumulates(m, k, n):
    # One workgroup a tile: dW and db are added to where they lie, in a matrix with a stride of its own.
    g = gen(m, k, n, 12)
    for dtype, wd in ((F16, F32), (BF16, BF16)):
        x, w, dy = wide(g, m, k, dtype, 3), wide(g, n, k, dtype, 0), wide(g, m, n, dtype, 3)
        buf = torch.randn(n, k + 5, generator=g).to(wd).to(DEV)
        old, ob = buf.clone(), torch.randn(n, generator=g).to(DEV)
        dx0, dw0, db0 = hg.hashgrid_linear_backward(dy, x, w, weight_dtype=F32)
        dw, db = buf[:, 2:2 + k], ob.clone()
        dx, _, _ = hg.hashgrid_linear_backward(dy, x, w, dw=dw, db=db, accumulate=True)
        assert torch.equal(dx, dx0)
        assert torch.equal(dw, (old[:, 2:2 + k].float() + dw0).to(wd)) and torch.equal(db, ob + db0)
        assert torch.equal(buf[:, :2], old[:, :2]) and torch.equal(buf[:, 2 + k:], old[:, 2 + k:])


def test_no_rows():
    x, w = torch.empty(0, 32, dtype=F16, device=DEV), torch.ones(8, 32, dtype=F16, device=DEV)
    assert hg.hashgrid_linear_forward(x, w).shape == (0, 8)
    dy = torch.empty(0, 8, dtype=F16, device=DEV)
    dx, dw, db = hg.hashgrid_linear_backward(dy, x, w)
    assert dx.shape == (0, 32) and not dw.any() and not db.any()
    kept = torch.ones(8, 32, device=DEV)
    hg.hashgrid_linear_backward(dy, x, w, dw=kept, db=torch.ones(8, device=DEV), accumulate=True)
    assert (kept == 1).all()


@pytest.mark.parametrize("m,k,n", [(4000, 513, 3), (5001, 640, 16), (3000, 1027, 32), (2500, 1000, 61), (2049, 900, 128), (1500, 5100, 9),
                                   (1037, 1300, 64), (2000, 2040, 25)])
@pytest.mark.parametrize("dtype", [F16, BF16, F8])
def test_long_rows_to_few_outputs(m, k, n, dtype):
    # Contractions longer than a wave's registers hold, whole fragments and cut ones, between columns of NaN.
    g = gen(m, k, n, 9)
    out = F32 if n % 2 else (BF16 if dtype == F8 else dtype)

    def between(rows, scale):
        buf = torch.full((rows, k + 3), float("nan")).to(dtype)
        buf[:, 2:-1] = (torch.randn(rows, k, generator=g) * scale).to(dtype)
        return buf.to(DEV)[:, 2:-1]

    x, w = between(m, 1.0), between(n, 20.0 if dtype == F8 else k ** -0.5)
    xs, ws = ((torch.rand(m, generator=g) * 0.1).to(DEV), (torch.rand(n, generator=g) * k ** -0.5).to(DEV)) if dtype == F8 else (None, None)
    b, r = torch.randn(n, generator=g).to(DEV), wide(g, m, n, out, 3)
    for kind, res in (("silu", r), ("none", None)):
        got = hg.hashgrid_linear_forward(x, w, b, act=kind, residual=res, x_scale=xs, weight_scale=ws, out_dtype=out,
                                         save_pre=dtype != F8)
        y, z = got if dtype != F8 else (got, None)
        wy, wz, ey, ez = R.linear(x, w, b, kind, res, xs, ws, out)
        R.within(y, wy, ey)
        if z is not None:
            R.within(z, wz, R.rounded(wz, ez, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16, F8])
@pytest.mark.parametrize("m,k,n", [(40, 35, 20), (700, 64, 40), (6000, 96, 64)])
def test_bytes_around_the_rows_are_not_touched_or_used(dtype, m, k, n):
    # The buffer around x, w and r holds NaN, the one around y a mark.
    g = gen(m, k, n, 5)

    def inside(t, fill):
        buf = torch.full((t.shape[0] + 2, t.shape[1] + 5), fill, device=DEV).to(t.dtype)
        buf[1:-1, 2:-3] = t
        return buf, buf[1:-1, 2:-3]

    nan = float("nan")
    out = BF16 if dtype == F8 else dtype
    x, w = (torch.randn(s, k, generator=g).to(dtype).to(DEV) for s in (m, n))
    r = torch.randn(m, n, generator=g).to(out).to(DEV)
    sc = dict(x_scale=torch.rand(m, generator=g).to(DEV), weight_scale=torch.rand(n, generator=g).to(DEV)) if dtype == F8 else {}
    want = hg.hashgrid_linear_forward(x, w, act="silu", residual=r, **sc)
    buf, y = inside(torch.zeros_like(want), 7.0)
    hg.hashgrid_linear_forward(inside(x, nan)[1], inside(w, nan)[1], act="silu", residual=inside(r, nan)[1], out=y, **sc)
    assert torch.equal(y, want)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[1:-1, 2:-3] = False
    assert (buf[mask] == 7.0).all()
    if dtype == F8:
        return
    dy = r
    want = hg.hashgrid_linear_backward(dy, x, w, act="gelu_tanh", pre=r, weight_dtype=dtype)
    bx, dx = inside(torch.zeros_like(x), 7.0)
    bw, dw = inside(torch.zeros_like(w), 7.0)
    hg.hashgrid_linear_backward(inside(dy, nan)[1], inside(x, nan)[1], inside(w, nan)[1], act="gelu_tanh", pre=inside(r, nan)[1],
                                dx=dx, dw=dw)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    for b in (bx, bw):
        mask = torch.ones_like(b, dtype=torch.bool)
        mask[1:-1, 2:-3] = False
        assert (b[mask] == 7.0).all()


def test_values_that_are_not_finite():
    # z of +-inf: silu and GELU give inf and 0; NaN reaches its own outputs alone.
    x = torch.zeros(20, 32, dtype=BF16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = float("inf"), -float("inf"), float("nan")
    w = torch.eye(4, 32, device=DEV).to(BF16) + 1
    for kind in ACTS:
        y = hg.hashgrid_linear_forward(x, w, act=kind).float()
        assert (y[0] == float("inf")).all()
        assert (y[1] == (-float("inf") if kind == "none" else 0)).all()
        assert y[2].isnan().all()
        assert not y[3:].any()
    # a blocked ReLU passes nothing on, whatever arrives
    dy = torch.full((20, 4), float("inf"), dtype=BF16, device=DEV)
    pre = torch.full((20, 4), -1.0, dtype=BF16, device=DEV)
    dx, dw, db = hg.hashgrid_linear_backward(dy, x[3:4].expand(20, 32).contiguous(), w, act="relu", pre=pre)
    assert not dx.any() and not dw.any() and not db.any()
    # far out, the slopes are 0 and 1
    pre = torch.tensor([-3e38, -200.0, 200.0, 3e38], device=DEV).to(BF16).expand(20, 4).contiguous()
    for kind in ("silu", "gelu_tanh"):
        _, _, db = hg.hashgrid_linear_backward(torch.ones(20, 4, dtype=BF16, device=DEV), x[3:4].expand(20, 32).contiguous(), w,
                                               act=kind, pre=pre)
        assert db.tolist() == [0.0, 0.0, 20.0, 20.0]


def test_gradient_against_differences():
    # dL/dx, dL/dW and dL/db of L = sum(c y) by central differences of the 64-bit form, through the kernels' own z.
    g = gen(21)
    m, k, n = 24, 12, 10
    for kind in ("silu", "gelu_tanh"):
        x, w = wide(g, m, k, F16, 0), wide(g, n, k, F16, 0, 0.5)
        b, c = torch.randn(n, generator=g).to(DEV), wide(g, m, n, F16, 0)
        _, pre = hg.hashgrid_linear_forward(x, w, b, act=kind, save_pre=True)
        dx, dw, db = hg.hashgrid_linear_backward(c, x, w, act=kind, pre=pre)
        X, W, B, C = (t.double().cpu() for t in (x, w, b, c))

        def loss(X, W, B):
            return (C * R.act(X @ W.t() + B, kind)).sum()

        h = 1e-4
        for t, got in ((X, dx), (W, dw), (B, db)):
            for i in range(0, t.numel(), 7):
                d = torch.zeros_like(t)
                d.view(-1)[i] = h
                args = [tuple(s + sgn * d if s is t else s for s in (X, W, B)) for sgn in (1, -1)]
                want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
                # z rounded to binary16 moves a slope by 2^-11 |z| at most, dz is rounded too; sums of at most 24 terms
                assert abs(got.double().cpu().view(-1)[i] - want) <= 24 * 3 * 4 * 2 ** -10 + 1e-6


def test_another_stream_and_graph_replay():
    g = gen(31)
    x, w, b = wide(g, 5000, 96, F16, 0), wide(g, 64, 96, F16, 0, 0.1), torch.randn(64, generator=g).to(DEV)
    want = hg.hashgrid_linear_forward(x, w, b, act="silu", save_pre=True)
    wg = hg.hashgrid_linear_backward(want[0], x, w, act="silu", pre=want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, z = hg.hashgrid_linear_forward(x, w, b, act="silu", save_pre=True, stream=s)
    grads = hg.hashgrid_linear_backward(y, x, w, act="silu", pre=z, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want[0]) and all(torch.equal(p, q) for p, q in zip(grads, wg))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = hg.hashgrid_linear_forward(x, w, b, act="silu", save_pre=True)
        grads = hg.hashgrid_linear_backward(y, x, w, act="silu", pre=z)
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=g).to(F16).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = hg.hashgrid_linear_forward(x, w, b, act="silu", save_pre=True)
        wg = hg.hashgrid_linear_backward(want[0], x, w, act="silu", pre=want[1])
        assert torch.equal(y, want[0]) and all(torch.equal(p, q) for p, q in zip(grads, wg))


@pytest.mark.parametrize("m,k,n,dtype", [(100001, 256, 256, BF16), (70000, 35, 64, F16), (70001, 512, 300, F16), (65541, 1000, 72, BF16)])
def test_many_rows(m, k, n, dtype):
    # Whole outputs against a 64-bit product on sampled rows (dx, y) and in full (dw, db).
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(m, k, generator=g, device=DEV).to(dtype)
    w = (torch.randn(n, k, generator=g, device=DEV) * k ** -0.5).to(dtype)
    b = torch.randn(n, generator=g, device=DEV)
    dy = torch.randn(m, n, generator=g, device=DEV).to(dtype)
    y, z = hg.hashgrid_linear_forward(x, w, b, act="silu", residual=dy, save_pre=True)
    dx, dw, db = hg.hashgrid_linear_backward(dy, x, w, act="silu", pre=z)
    at = torch.cat([torch.arange(0, m, 997), torch.arange(m - 40, m)]).to(DEV)
    wy, wz, ey, ez = R.linear(x[at], w, b, "silu", dy[at], None, None, dtype)
    R.within(y[at], wy, ey)
    (rx, ex), _, _ = R.linear_grad(dy[at], x[at], w, z[at], "silu")
    R.within(dx[at], rx, R.rounded(rx, ex, dtype))
    _, (rw, ew), (rb, eb) = R.linear_grad(dy, x, w, z, "silu")
    R.within(dw, rw, R.rounded(rw, ew, F32))
    R.within(db, rb, R.rounded(rb, eb, F32))


def test_offsets_past_32_bits():
    # Rows of a buffer of more than 2^32 elements: the last rows of every operand lie past 32-bit offsets.
    m, stride, k, n = 70000, 65536, 32, 16
    g = torch.Generator(device=DEV).manual_seed(9)
    big = torch.empty(m * stride, dtype=F16, device=DEV).view(m, stride)
    x = big[:, :k]
    x.copy_(torch.randn(m, k, generator=g, device=DEV))
    w = torch.randn(n, k, generator=g, device=DEV).to(F16)
    dy = torch.randn(m, n, generator=g, device=DEV).to(F16)
    y = big[:, 64:64 + n]
    hg.hashgrid_linear_forward(x, w, act="relu", out=y)
    xc = x.contiguous()
    assert torch.equal(y, hg.hashgrid_linear_forward(xc, w, act="relu"))
    pre = big[:, 128:128 + n]
    pre.copy_(y)
    dx = big[:, 256:256 + k]
    got = hg.hashgrid_linear_backward(dy, x, w, act="relu", pre=pre, dx=dx)
    want = hg.hashgrid_linear_backward(dy, xc, w, act="relu", pre=y.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
