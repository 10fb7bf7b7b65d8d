"""Rows of a table by their numbers (hashgrid_embedding_*) on the GPU against
their 64-bit form, within the error the roundings allow."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def gen(*key):
    return torch.Generator().manual_seed(hash(key) & 0x7FFFFFFF)


def wide(g, m, n, dtype, pad):
    t = torch.randn(m, n + pad, generator=g).to(dtype).to(DEV)
    return t[:, (pad & 1):(pad & 1) + n]


def make_ids(g, m, rows, kind, dtype=torch.int64):
    if kind == "one":
        ids = torch.full((m,), rows // 2)
    elif kind == "runs":
        ids = torch.randint(0, rows, (-(-m // 50),), generator=g).repeat_interleave(50)[:m]
    elif kind == "skewed":
        ids = (torch.rand(m, generator=g) ** 6 * rows).long().clamp_max(rows - 1)
    else:
        ids = torch.randint(0, rows, (m,), generator=g)
    if kind == "odd":  # some name no row
        ids[torch.rand(m, generator=g) < 0.3] = -1
        ids[torch.rand(m, generator=g) < 0.1] = rows
        ids[:1] = torch.iinfo(dtype).max
        ids[1:2] = torch.iinfo(dtype).min
    return ids.to(dtype).to(DEV)


TYPES = [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)]
COLUMNS = [1, 3, 7, 8, 9, 16, 31, 64, 96, 100, 257, 512, 520, 1100]


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("table_dtype,out", TYPES)
def test_forward(c, table_dtype, out):
    for m, rows, kind, bits, pad, scale in ((1, 1, "uniform", torch.int64, 0, 1.0), (77, 5, "odd", torch.int32, 3, 22.627417),
                                            (1500, 1000, "odd", torch.int64, 8, 0.125)):
        g = gen(c, m)
        table, ids = wide(g, rows, c, table_dtype, pad), make_ids(g, m, rows, kind, bits)
        y = hg.hashgrid_embedding_forward(table, ids, scale=scale, out_dtype=out)
        want, err = K.lookup(table, ids, torch.tensor(scale).item(), out)
        R.within(y, want, err)
        # into columns of a wider buffer, whose others stay
        buf = torch.full((m, c + 9), 3.0, dtype=out, device=DEV)
        got = hg.hashgrid_embedding_forward(table, ids, scale=scale, out=buf[:, 5:5 + c])
        assert got.data_ptr() == buf[:, 5:].data_ptr() and torch.equal(buf[:, 5:5 + c], y)
        assert (buf[:, :5] == 3).all() and (buf[:, 5 + c:] == 3).all()


def test_values_that_are_not_finite_and_rows_without_an_id():
    table = torch.tensor([[float("nan"), 1.0], [float("inf"), -2.0], [3.0, 4.0]], device=DEV)
    y = hg.hashgrid_embedding_forward(table, torch.tensor([-1, 0, 1, 2, 3], device=DEV))
    assert not y[0].any() and y[1, 0].isnan() and y[1, 1] == 1 and y[2, 0] == float("inf") and not y[4].any()
    dy = torch.tensor([[float("nan")], [1.0], [float("inf")], [2.0], [5.0]], device=DEV)
    d = hg.hashgrid_embedding_backward(dy, torch.tensor([0, 1, 2, 1, -1], device=DEV), 4)[:, 0].tolist()
    assert d[0] != d[0] and d[1:] == [3.0, float("inf"), 0.0]


@pytest.mark.parametrize("c", COLUMNS)
@pytest.mark.parametrize("dtype,table_dtype", [(F32, F32), (F16, F32), (F16, F16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("kind", ["uniform", "odd", "skewed", "one", "runs"])
def test_backward(c, dtype, table_dtype, kind):
    for m, rows, bits, pad in ((1, 3, torch.int64, 0), (130, 7, torch.int32, 3), (5000 if c < 300 else 2100, 600, torch.int64, 8)):
        g = gen(c, m, kind)
        dy, ids = wide(g, m, c, dtype, pad), make_ids(g, m, rows, kind, bits)
        scale = 1.0 if m == 130 else 22.627417
        d = hg.hashgrid_embedding_backward(dy, ids, rows, scale=scale, table_dtype=table_dtype)
        want, err = K.lookup_grad(dy, ids, rows, torch.tensor(scale).item())
        R.within(d, want, R.rounded(want, err, table_dtype))
        assert torch.equal(d, hg.hashgrid_embedding_backward(dy, ids, rows, scale=scale, table_dtype=table_dtype))
        # added to a table that is part of a wider one; rows without an id stay
        buf = torch.randn(rows, c + 5, generator=g).to(table_dtype).to(DEV)
        old = buf.clone()
        hg.hashgrid_embedding_backward(dy, ids, rows, scale=scale, dtable=buf[:, 2:2 + c], accumulate=True)
        want = want + old[:, 2:2 + c].double().cpu()
        R.within(buf[:, 2:2 + c], want, R.rounded(want, err + R.EPS32 * want.abs(), table_dtype))
        assert torch.equal(buf[:, :2], old[:, :2]) and torch.equal(buf[:, 2 + c:], old[:, 2 + c:])
        gone = torch.bincount(ids[(ids >= 0) & (ids < rows)].long(), minlength=rows) == 0
        assert torch.equal(buf[gone], old[gone])
        # written, not added to, in place of what was there
        hg.hashgrid_embedding_backward(dy, ids, rows, scale=scale, dtable=buf[:, 2:2 + c])
        assert torch.equal(buf[:, 2:2 + c], d) and torch.equal(buf[:, :2], old[:, :2])


@pytest.mark.parametrize("rows", [1, 2, 255, 256, 511, 512, 513, 50304, 1 << 17, (1 << 18) - 1, 1 << 20])
@pytest.mark.parametrize("m", [4096, 4097, 70000])
def test_sizes_of_the_sort(rows, m):
    # one pass of up to 9 bits and several; one tile of keys and several; small whole numbers, whose sums are exact
    g = gen(rows, m)
    ids = make_ids(g, m, rows, "odd")
    dy = torch.randint(-8, 9, (m, 4), generator=g).to(F16).to(DEV)
    want = torch.zeros(rows, 4, dtype=torch.float64)
    known = ((ids >= 0) & (ids < rows)).cpu()
    want.index_add_(0, ids.cpu()[known], dy.double().cpu()[known])
    assert torch.equal(hg.hashgrid_embedding_backward(dy, ids, rows).double().cpu(), want)


@pytest.mark.parametrize("c,dtype", [(64, BF16), (8, F16), (1, F32), (513, F16)])
@pytest.mark.parametrize("kind", ["one", "runs", "skewed"])
def test_many_rows_of_few_ids(c, dtype, kind):
    m = (1 << 19) + 3 if c <= 64 else 1 << 15
    g = gen(c, kind)
    ids = make_ids(g, m, 40, kind, torch.int32)
    dy = (torch.randint(-4, 5, (m, c), generator=g) / 4).to(dtype).to(DEV)  # sums below 2^21 quarters: exact in any order
    want = torch.zeros(40, c, dtype=torch.float64, device=DEV).index_add_(0, ids.long(), dy.double())
    assert torch.equal(hg.hashgrid_embedding_backward(dy, ids, 40).double(), want)


def test_nothing_to_do():
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert hg.hashgrid_embedding_forward(torch.ones(3, 4, device=DEV), none).shape == (0, 4)
    d = hg.hashgrid_embedding_backward(torch.empty(0, 4, device=DEV), none, 3)
    assert d.shape == (3, 4) and not d.any()
    old = torch.ones(3, 4, device=DEV)
    assert (hg.hashgrid_embedding_backward(torch.empty(0, 4, device=DEV), none, 3, dtable=old, accumulate=True) == 1).all()
    ids = torch.tensor([0, -1], device=DEV)
    y = hg.hashgrid_embedding_forward(torch.empty(0, 4, device=DEV), ids)  # a table without rows
    assert y.shape == (2, 4) and not y.any()
    assert hg.hashgrid_embedding_backward(torch.ones(2, 4, device=DEV), ids, 0).shape == (0, 4)
    d = hg.hashgrid_embedding_backward(torch.ones(2, 4, device=DEV), torch.tensor([-1, 7], device=DEV), 5)
    assert d.shape == (5, 4) and not d.any()


def test_refusals_of_the_binding():
    t, i = torch.ones(3, 4, device=DEV), torch.tensor([0, 1], device=DEV)
    for call in (lambda: hg.hashgrid_embedding_forward(t, i.float()), lambda: hg.hashgrid_embedding_forward(t, i[None]),
                 lambda: hg.hashgrid_embedding_forward(t, torch.zeros(4, dtype=torch.int64, device=DEV)[::2]),
                 lambda: hg.hashgrid_embedding_forward(t, i.cpu()), lambda: hg.hashgrid_embedding_forward(t, i, out=t),
                 lambda: hg.hashgrid_embedding_forward(t[0], i), lambda: hg.hashgrid_embedding_backward(t, i, 3),
                 lambda: hg.hashgrid_embedding_backward(t[:2], i, -1), lambda: hg.hashgrid_embedding_backward(t[:2], i, 1 << 31),
                 lambda: hg.hashgrid_embedding_backward(t[:2], i, 3, accumulate=True),
                 lambda: hg.hashgrid_embedding_backward(t[:2], i, 3, dtable=t[:2]),
                 lambda: hg.hashgrid_embedding_backward(t[:2], i, 3, workspace="none")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(hg.HashGridError, match="workspace"):
        hg.hashgrid_embedding_backward(t[:2], i, 3, workspace=None)
    with pytest.raises(hg.HashGridError, match="y_dtype"):
        hg.hashgrid_embedding_forward(t.to(F16), i, out_dtype=F32)


def test_another_stream_and_graph_replay():
    g = gen(1)
    m, rows, c = 9000, 700, 24
    table, dy = wide(g, rows, c, F32, 0), wide(g, m, c, BF16, 0)
    ids = make_ids(g, m, rows, "skewed")

    def both(stream=None):
        return (hg.hashgrid_embedding_forward(table, ids, scale=3.0, out_dtype=F16, stream=stream),
                hg.hashgrid_embedding_backward(dy, ids, rows, stream=stream))

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for kind in ("one", "odd", "uniform", "runs"):
        ids.copy_(make_ids(g, m, rows, kind))
        dy.copy_(wide(g, m, c, BF16, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_autograd():
    g = gen(2)
    codes = hg.HashGridCodes(9, 6, scale=2.0)
    ids = torch.tensor([3, 3, -1, 8, 0, 3], device=DEV)
    w = torch.randn(6, 6, generator=g).to(DEV)
    (codes(ids) * w).sum().backward()
    want, err = K.lookup_grad(w, ids, 9, 2.0)
    R.within(codes.table.grad, want, R.rounded(want, err, F32))
    # a gradient that is one value everywhere
    codes.table.grad = None
    codes(ids).sum().backward()
    assert codes.table.grad[:, 0].tolist() == [2.0, 0, 0, 6.0, 0, 0, 0, 0, 2.0]
    # features and codes side by side
    f = torch.randn(6, 5, generator=g).to(DEV).requires_grad_()
    x = hg.HashGridCodedInputFunction.apply(f, codes.table, ids, F16, 2.0)
    assert torch.equal(x[:, :5], f.detach().to(F16)) and torch.equal(x[:, 5:], hg.hashgrid_embedding_forward(codes.table.detach(), ids, scale=2.0, out_dtype=F16))
    codes.table.grad = None
    up = torch.randn(6, 11, generator=g).to(F16).to(DEV)
    (x * up).sum().backward()
    assert torch.equal(f.grad, up[:, :5].float())
    want, err = K.lookup_grad(up[:, 5:], ids, 9, 2.0)
    R.within(codes.table.grad, want, R.rounded(want, err, F32))
