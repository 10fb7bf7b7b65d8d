"""The gated feed-forward product (hashgrid_gated_forward and _backward) on the
GPU against its 64-bit form, within the error its roundings allow."""
import pytest
import torch

import blocks_reference as K
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


SIZES = [(1, 1, 1), (1, 256, 512), (3, 7, 5), (16, 32, 16), (17, 33, 19), (64, 64, 4), (65, 35, 64), (127, 31, 129), (130, 256, 256),
         (257, 96, 33), (1000, 130, 70), (300, 520, 300), (40, 1024, 512), (33, 8, 1024), (5000, 35, 93), (4100, 64, 40),
         (2500, 256, 100), (2048, 384, 200), (1030, 640, 260), (1100, 32, 1300), (1300, 64, 700), (2100, 96, 450), (1025, 120, 300),
         (1200, 192, 170), (3000, 250, 300)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_forward(m, k, n, dtype, pad):
    g = gen(m, k, n, pad)
    x, wg, wu = wide(g, m, k, dtype, pad), wide(g, n, k, dtype, pad, k ** -0.5), wide(g, n, k, dtype, 0, k ** -0.5)
    bg, bu = torch.randn(n, generator=g).to(DEV), torch.randn(n, generator=g).to(DEV)
    for i, kind in enumerate(ACTS):
        out = F32 if (i + m) % 3 == 0 else dtype
        b = (None, bu) if kind == "none" else (bg, None) if kind == "relu" else (bg, bu)
        h, gate, up = hg.hashgrid_gated_forward(x, wg, wu, *b, act=kind, out_dtype=out, save_pre=True)
        wh, zg, zu, eh, eg, eu = K.gated(x, wg, wu, *b, kind, None, None, None, out)
        assert h.dtype == out and gate.dtype == up.dtype == dtype
        R.within(h, wh, eh)
        R.within(gate, zg, R.rounded(zg, eg, dtype))
        R.within(up, zu, R.rounded(zu, eu, dtype))
        buf = torch.full((m, n + pad + 1), 3.0, dtype=out, device=DEV)
        hg.hashgrid_gated_forward(x, wg, wu, *b, act=kind, out=buf[:, 1:1 + n])
        assert torch.equal(buf[:, 1:1 + n], h) and (buf[:, :1] == 3).all() and (buf[:, 1 + n:] == 3).all()


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("pad", [0, 3])
def test_forward_8bit(m, k, n, pad):
    g = gen(m, k, n, pad, 8)
    x, wg, wu = wide(g, m, k, F8, pad, 20.0), wide(g, n, k, F8, pad, 20.0), wide(g, n, k, F8, 0, 20.0)
    xs = (torch.rand(m, generator=g) * 0.1).to(DEV)
    gs, us = ((torch.rand(n, generator=g) * k ** -0.5).to(DEV) for _ in range(2))
    bg, bu = torch.randn(n, generator=g).to(DEV), torch.randn(n, generator=g).to(DEV)
    for i, kind in enumerate(ACTS):
        out = (BF16, F16, F32)[(i + k) % 3]
        h = hg.hashgrid_gated_forward(x, wg, wu, bg, bu, act=kind, x_scale=xs, gate_scale=gs, up_scale=us, out_dtype=out)
        wh, _, _, eh, _, _ = K.gated(x, wg, wu, bg, bu, kind, xs, gs, us, out)
        R.within(h, wh, eh)


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_backward(m, k, n, dtype, pad):
    g = gen(m, k, n, pad, 1)
    x, wg, wu = wide(g, m, k, dtype, pad), wide(g, n, k, dtype, pad, k ** -0.5), wide(g, n, k, dtype, 0, k ** -0.5)
    dh, gate, up = (wide(g, m, n, dtype, pad) for _ in range(3))
    for i, kind in enumerate(ACTS):
        wd = F32 if i % 2 else dtype
        got = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=kind, weight_dtype=wd)
        for t, (want, err), kept in zip(got, K.gated_grad(dh, x, wg, wu, gate, up, kind), (dtype, wd, wd, F32, F32)):
            assert t.dtype == kept
            R.within(t, want, R.rounded(want, err, kept))
        again = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=kind, weight_dtype=wd)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        # each output alone is the same output
        for need in ((True, False, False), (False, True, False), (False, False, True)):
            only = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=kind, weight_dtype=wd,
                                              **dict(zip(("need_dx", "need_dw", "need_db"), need)))
            for t, a, n_ in zip(only, got, (need[0], need[1], need[1], need[2], need[2])):
                assert torch.equal(t, a) if n_ else t is None


@pytest.mark.parametrize("m,k,n", [(1, 40, 24), (333, 40, 24), (20, 5, 300), (1500, 300, 3), (900, 256, 200)])
def test_backward_accumulates(m, k, n):
    g = gen(m, k, n, 11)
    for dtype, wd in ((F16, F32), (BF16, BF16)):
        x, wg, wu = wide(g, m, k, dtype, 3), wide(g, n, k, dtype, 0), wide(g, n, k, dtype, 0)
        dh, gate, up = (wide(g, m, n, dtype, 0) for _ in range(3))
        want = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, weight_dtype=F32)
        bufs = [torch.randn(n, k + 5, generator=g).to(wd).to(DEV) for _ in range(2)]
        old, ob = [b.clone() for b in bufs], [torch.randn(n, generator=g).to(DEV) for _ in range(2)]
        db = [b.clone() for b in ob]
        dxb = torch.full((m, k + 7), 3.0, dtype=dtype, device=DEV)
        dx = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, dx=dxb[:, 3:3 + k], dw_gate=bufs[0][:, 2:2 + k], dw_up=bufs[1][:, 2:2 + k],
                                        db_gate=db[0], db_up=db[1], accumulate=True)[0]
        assert torch.equal(dx, want[0]) and (dxb[:, :3] == 3).all() and (dxb[:, 3 + k:] == 3).all()
        for b, o, w in zip(bufs, old, want[1:3]):
            assert torch.equal(b[:, 2:2 + k], (o[:, 2:2 + k].float() + w).to(wd))
            assert torch.equal(b[:, :2], o[:, :2]) and torch.equal(b[:, 2 + k:], o[:, 2 + k:])
        for b, o, w in zip(db, ob, want[3:]):
            assert torch.equal(b, o + w)


def test_no_rows():
    x, w = torch.empty(0, 32, dtype=F16, device=DEV), torch.ones(8, 32, dtype=F16, device=DEV)
    h, gate, up = hg.hashgrid_gated_forward(x, w, w, save_pre=True)
    assert h.shape == gate.shape == up.shape == (0, 8)
    dx, dg, du, bg, bu = hg.hashgrid_gated_backward(h, x, w, w, gate, up)
    assert dx.shape == (0, 32) and not dg.any() and not du.any() and not bg.any() and not bu.any()
    one = [torch.ones(8, 32, device=DEV) for _ in range(2)] + [torch.ones(8, device=DEV) for _ in range(2)]
    hg.hashgrid_gated_backward(h, x, w, w, gate, up, dw_gate=one[0], dw_up=one[1], db_gate=one[2], db_up=one[3], accumulate=True)
    assert all((t == 1).all() for t in one)


@pytest.mark.parametrize("m,k,n", [(5, 40, 24), (3000, 64, 48), (600, 600, 130)])
def test_rows_that_are_not_finite_stay_alone(m, k, n):
    g = gen(m, k, 5)
    x, wg, wu = wide(g, m, k, F16, 0), wide(g, n, k, F16, 0, 0.1), wide(g, n, k, F16, 0, 0.1)
    want = hg.hashgrid_gated_forward(x, wg, wu)
    bad = x.clone()
    bad[1, 2], bad[m - 1] = float("nan"), float("inf")
    h = hg.hashgrid_gated_forward(bad, wg, wu)
    assert h[1].isnan().all() and not h[m - 1].isfinite().all()
    keep = [i for i in range(m) if i not in (1, m - 1)]
    assert torch.equal(h[keep], want[keep])
    dh, gate, up = (wide(g, m, n, F16, 0) for _ in range(3))
    want = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up)[0]
    bad = gate.clone()
    bad[1, 2] = float("nan")
    dx = hg.hashgrid_gated_backward(dh, x, wg, wu, bad, up)[0]
    assert dx[1].isnan().all()
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(dx[keep], want[keep])


def test_gates_at_the_ends():
    # what a gate of minus infinity, of the type's lowest value and of plus infinity lets through
    gate = torch.tensor([[float("-inf")], [torch.finfo(F16).min], [torch.finfo(F16).max], [float("inf")]], dtype=F16, device=DEV).repeat(1, 8)
    up, dh = torch.full_like(gate, 2.0), torch.full_like(gate, 0.5)
    x, w = torch.ones(4, 8, dtype=F16, device=DEV), torch.eye(8, dtype=F16, device=DEV)
    for kind in ("relu", "silu", "gelu_tanh"):
        _, _, _, bg, bu = hg.hashgrid_gated_backward(dh[:2], x[:2], w, w, gate[:2], up[:2], act=kind)
        assert not bg.any() and not bu.any()
        _, _, _, bg, bu = hg.hashgrid_gated_backward(dh[2:3], x[2:3], w, w, gate[2:3], up[2:3], act=kind)
        assert (bg == 1).all() and (bu == 0.5 * torch.finfo(F16).max).all()
        _, _, _, bg, bu = hg.hashgrid_gated_backward(dh[3:], x[3:], w, w, gate[3:], up[3:], act=kind)
        assert (bg == 1).all() and (bu == float("inf")).all()
    # a relu that is shut lets nothing through, whatever meets it
    bad = torch.full_like(gate, float("inf"))
    shut = torch.full_like(gate, -1.0)
    dx, dg, du, bg, bu = hg.hashgrid_gated_backward(bad, x, w, w, shut, bad, act="relu")
    assert not dx.any() and not dg.any() and not du.any() and not bg.any() and not bu.any()


def test_gradient_against_differences():
    g = gen(6)
    m, k, n = 5, 9, 6
    x, wg, wu = wide(g, m, k, F16, 0), wide(g, n, k, F16, 0), wide(g, n, k, F16, 0)
    dh = wide(g, m, n, F16, 0)
    X, G, U, D = (t.double().cpu() for t in (x, wg, wu, dh))
    for kind in ("none", "silu", "gelu_tanh"):
        # the projections in binary16 are what the backward reads: differences go through the same values
        gate, up = ((X @ w.t()).to(F16).to(DEV) for w in (G, U))
        got = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act=kind)
        h = 1e-5

        def loss(X, G, U, BG, BU):
            zg, zu = gate.double().cpu() + (X @ G.t() - X0 @ G0.t()) + BG, up.double().cpu() + (X @ U.t() - X0 @ U0.t()) + BU
            return (D * R.act(zg, kind) * zu).sum()

        X0, G0, U0 = X, G, U
        base = [X, G, U, torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)]
        for i, t in enumerate(base):
            for j in range(t.numel()):
                a, z = [b.clone() for b in base], [b.clone() for b in base]
                a[i].view(-1)[j] += h
                z[i].view(-1)[j] -= h
                want = (loss(*a) - loss(*z)) / (2 * h)
                # dg and du are rounded to 2^-11 of themselves on the way into a product of up to 12 terms of size 20
                assert abs(got[i].double().cpu().view(-1)[j] - want) <= 12 * 20 * 2.0 ** -11


@pytest.mark.parametrize("m,k,n", [(3000, 96, 100), (200, 520, 70)])
def test_another_stream_and_graph_replay(m, k, n):
    g = gen(8, m)
    x, wg, wu = wide(g, m, k, BF16, 0), wide(g, n, k, BF16, 0, 0.1), wide(g, n, k, BF16, 0, 0.1)

    def both(stream=None):
        h, gate, up = hg.hashgrid_gated_forward(x, wg, wu, save_pre=True, stream=stream)
        return (h, gate, up) + hg.hashgrid_gated_backward(h, x, wg, wu, gate, up, stream=stream)

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
        x.copy_(torch.randn(x.shape, generator=g).to(BF16).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_refusals_of_the_binding():
    x, w = torch.ones(4, 8, dtype=F16, device=DEV), torch.ones(6, 8, dtype=F16, device=DEV)
    h = torch.ones(4, 6, dtype=F16, device=DEV)
    for call in (lambda: hg.hashgrid_gated_forward(x, w, w[:5]), lambda: hg.hashgrid_gated_forward(x, w, w.to(BF16)),
                 lambda: hg.hashgrid_gated_forward(x, w, w, torch.ones(5, device=DEV)), lambda: hg.hashgrid_gated_forward(x, w, w.cpu()),
                 lambda: hg.hashgrid_gated_forward(x, w, w, act="tanh"), lambda: hg.hashgrid_gated_forward(x, w, w, out=h[:, :5]),
                 lambda: hg.hashgrid_gated_backward(h, x, w, w, h, h[:3]), lambda: hg.hashgrid_gated_backward(h.float(), x, w, w, h, h),
                 lambda: hg.hashgrid_gated_backward(h, x, w, w, h, h, accumulate=True),
                 lambda: hg.hashgrid_gated_backward(h, x, w, w, h, h, dx=w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(hg.HashGridError, match="workspace"):
        xs, hs = x.repeat(100, 1), h.repeat(100, 1)
        hg.hashgrid_gated_backward(hs, xs, w, w, hs, hs, workspace=None)
    with pytest.raises(hg.HashGridError, match="together"):
        R_ = torch.empty(6, 8, device=DEV)
        hg.blocks._check(hg.blocks._lib().hashgrid_gated_backward(hg.blocks._gated_grad(
            4, 8, 6, h.data_ptr(), 6, h.data_ptr(), h.data_ptr(), 6, 6, x.data_ptr(), 8, w.data_ptr(), w.data_ptr(), 8, 8, 0, 0,
            R_.data_ptr(), 0, 8, 0, 0, 0, 1, 0, 2, 0), None, 0, None))
    with pytest.raises(hg.HashGridError, match="h_dtype"):
        hg.hashgrid_gated_forward(x, w, w, out_dtype=BF16)
