"""Embedding and gated operators over more rows than a round of workgroups takes,
with offsets past 32 bits, and in calls that overlap."""
import pytest
import torch

import blocks_reference as K
import multiresolution_hash_grid_amd as hg
import residual_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def rows(g, m, n, dtype, scale=1.0):
    return (torch.randn(m, n, generator=g) * scale).to(dtype).to(DEV)


# weights in LDS, in registers (both sets of units, and idle waves), in blocks
@pytest.mark.parametrize("m,k,n", [(70001, 64, 100), (40003, 256, 300), (70001, 32, 1100), (33001, 120, 290), (70000, 264, 300)])
@pytest.mark.parametrize("dtype", [F16, BF16, F8])
def test_gated_forward(m, k, n, dtype):
    g = torch.Generator().manual_seed(m + k)
    eight = dtype == F8
    x, wg, wu = rows(g, m, k, dtype, 20.0 if eight else 1.0), rows(g, n, k, dtype, 20.0 if eight else k ** -0.5), rows(g, n, k, dtype, 20.0 if eight else k ** -0.5)
    b = [torch.randn(n, generator=g).to(DEV) for _ in range(2)]
    sc = {}
    if eight:
        sc = dict(x_scale=(torch.rand(m, generator=g) * 0.1).to(DEV), gate_scale=(torch.rand(n, generator=g) * k ** -0.5).to(DEV),
                  up_scale=(torch.rand(n, generator=g) * k ** -0.5).to(DEV))
    out = BF16 if eight else dtype
    h = hg.hashgrid_gated_forward(x, wg, wu, *b, act="silu", out_dtype=out, **sc)
    pick = torch.cat([torch.arange(300), torch.randint(0, m, (3000,), generator=g), torch.arange(m - 300, m)])
    at = pick.to(DEV)
    wh, zg, zu, eh, eg, eu = K.gated(x[at], wg, wu, *b, "silu", sc["x_scale"][at] if eight else None, sc.get("gate_scale"), sc.get("up_scale"), out)
    R.within(h[at], wh, eh)
    if not eight:
        h2, gate, up = hg.hashgrid_gated_forward(x, wg, wu, *b, act="silu", save_pre=True)
        assert torch.equal(h2, h)
        R.within(gate[at], zg, R.rounded(zg, eg, dtype))
        R.within(up[at], zu, R.rounded(zu, eu, dtype))
    # every row, not the picked ones alone: the same rows one workgroup at a time
    for a in range(0, m, 16384):
        one = dict(sc, x_scale=sc["x_scale"][a:a + 16384]) if eight else {}
        part = hg.hashgrid_gated_forward(x[a:a + 16384], wg, wu, *b, act="silu", out_dtype=out, **one)
        assert (part.float() - h[a:a + 16384].float()).abs().max() <= 2.0 ** -6 * h.float().abs().max()


@pytest.mark.parametrize("m,k,n", [(40001, 256, 300), (70000, 64, 100), (20001, 300, 140), (64, 256, 512), (300, 96, 1000), (1000, 520, 700)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated_backward(m, k, n, dtype):
    g = torch.Generator().manual_seed(m + k + 1)
    x, wg, wu = rows(g, m, k, dtype), rows(g, n, k, dtype, k ** -0.5), rows(g, n, k, dtype, k ** -0.5)
    dh, gate, up = (rows(g, m, n, dtype) for _ in range(3))
    got = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act="gelu_tanh")
    for t, (want, err), kept in zip(got, K.gated_grad(dh, x, wg, wu, gate, up, "gelu_tanh"), (dtype, F32, F32, F32, F32)):
        R.within(t, want, R.rounded(want, err, kept))
    again = hg.hashgrid_gated_backward(dh, x, wg, wu, gate, up, act="gelu_tanh")
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_embedding_of_more_keys_than_are_held():
    m = (1 << 20) + 5003
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(-1, 3000, (m,), generator=g, dtype=torch.int32).to(DEV)
    dy = torch.randint(-8, 9, (m, 8), generator=g).to(F16).to(DEV)
    want = torch.zeros(3000, 8, dtype=torch.float64, device=DEV).index_add_(0, ids.long().clamp_min(0), dy.double() * (ids >= 0)[:, None])
    assert torch.equal(hg.hashgrid_embedding_backward(dy, ids, 3000).double(), want)
    table = torch.randn(3000, 8, generator=g).to(DEV)
    y = hg.hashgrid_embedding_forward(table, ids)
    assert torch.equal(y, torch.where((ids >= 0)[:, None], table[ids.long().clamp_min(0)], torch.zeros((), device=DEV)))


def test_codes_past_the_caches_into_columns():
    # an output larger than the caches takes stores of its own; what lies beside the columns stays
    for m, c, dtype in ((300001, 70, BF16), (200003, 96, F32), (2000001, 8, F16)):
        g = torch.Generator().manual_seed(c)
        table = torch.randn(50, c, generator=g).to(DEV)
        ids = torch.randint(-1, 50, (m,), generator=g).to(DEV)
        buf = torch.full((m, c + 5), 3.0, dtype=dtype, device=DEV)
        hg.hashgrid_embedding_forward(table, ids, out=buf[:, 3:3 + c])
        want = torch.where((ids >= 0)[:, None], table[ids.clamp_min(0)], torch.zeros((), device=DEV)).to(dtype)
        assert torch.equal(buf[:, 3:3 + c], want) and (buf[:, :3] == 3).all() and (buf[:, 3 + c:] == 3).all()


def test_offsets_past_32_bits():
    stride = (1 << 30) + 8  # elements between rows: row 2 begins past 2^31 elements, 2^32 bytes
    buf = torch.zeros(2 * stride + 64, dtype=F16, device=DEV)
    wide = buf.as_strided((3, 16), (stride, 1))
    wide.copy_(torch.randn(3, 16, generator=torch.Generator().manual_seed(1)).to(F16))
    ids = torch.tensor([2, 0, 1, 2, -1], device=DEV)
    assert torch.equal(hg.hashgrid_embedding_forward(wide, ids), hg.hashgrid_embedding_forward(wide.contiguous(), ids))
    ids = torch.tensor([1, 0, 1], device=DEV)
    want = hg.hashgrid_embedding_backward(wide.contiguous(), ids, 2, table_dtype=F16)
    assert torch.equal(hg.hashgrid_embedding_backward(wide, ids, 2, table_dtype=F16), want)
    x, w = torch.randn(3, 16, device=DEV).to(F16), torch.randn(16, 16, device=DEV).to(F16)
    want = [hg.hashgrid_gated_forward(x, w, w), hg.hashgrid_layer_norm_forward(x).y]
    wide.copy_(x)
    assert torch.equal(hg.hashgrid_gated_forward(wide, w, w), want[0])
    assert torch.equal(hg.hashgrid_layer_norm_forward(wide).y, want[1])
    hg.hashgrid_gated_forward(x, w, w, out=wide)
    assert torch.equal(wide, want[0])
    hg.hashgrid_embedding_backward(x, torch.tensor([2, 0, 2], device=DEV), 3, dtable=wide)
    assert torch.equal(wide, hg.hashgrid_embedding_backward(x, torch.tensor([2, 0, 2], device=DEV), 3, table_dtype=F16))


def test_calls_on_two_streams():
    g = torch.Generator().manual_seed(9)
    sets = [(rows(g, 30000, 96, BF16), rows(g, 200, 96, BF16, 0.1), torch.randint(0, 90, (30000,), generator=g).to(DEV)) for _ in range(2)]

    def work(x, w, ids):
        h, gate, up = hg.hashgrid_gated_forward(x, w, w, save_pre=True)
        return (h,) + hg.hashgrid_gated_backward(h, x, w, w, gate, up) + (hg.hashgrid_embedding_backward(x, ids, 90),) + \
            hg.hashgrid_layer_norm_forward(x, save_stats=True)[:1]

    want = [work(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(work(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))


@pytest.mark.parametrize("m,k,n", [(9001, 128, 1024), (5003, 100, 700), (3001, 512, 300), (4001, 64, 1100)])
def test_gated_8bit_to_f32(m, k, n):
    g = torch.Generator().manual_seed(k)
    x, wg, wu = rows(g, m, k, F8, 20.0), rows(g, n, k, F8, 20.0), rows(g, n, k, F8, 20.0)
    b = [torch.randn(n, generator=g).to(DEV) for _ in range(2)]
    xs, gs, us = ((torch.rand(i, generator=g) * s).to(DEV) for i, s in ((m, 0.1), (n, k ** -0.5), (n, k ** -0.5)))
    h = hg.hashgrid_gated_forward(x, wg, wu, *b, act="gelu_tanh", out_dtype=F32, x_scale=xs, gate_scale=gs, up_scale=us)
    wh, _, _, eh, _, _ = K.gated(x, wg, wu, *b, "gelu_tanh", xs, gs, us, F32)
    R.within(h, wh, eh)


# rows shorter than a piece (8 values, 16 of 8 bits): with weights that LDS holds, and without
@pytest.mark.parametrize("k", [1, 3, 7, 15])
@pytest.mark.parametrize("m,n", [(70001, 64), (9001, 35), (5003, 1300)])
@pytest.mark.parametrize("dtype", [F16, BF16, F8])
def test_gated_of_few_inputs(m, k, n, dtype):
    g = torch.Generator().manual_seed(m + k)
    eight = dtype == F8
    x, wg, wu = (rows(g, i, k, dtype, 20.0 if eight else 1.0) for i in (m, n, n))
    b = [torch.randn(n, generator=g).to(DEV) for _ in range(2)]
    sc = [(torch.rand(i, generator=g) * 0.1).to(DEV) for i in (m, n, n)] if eight else [None] * 3
    out = BF16 if eight else dtype
    h = hg.hashgrid_gated_forward(x, wg, wu, *b, out_dtype=out, x_scale=sc[0], gate_scale=sc[1], up_scale=sc[2])
    at = torch.cat([torch.arange(500), torch.randint(0, m, (1500,), generator=g), torch.arange(m - 500, m)]).to(DEV)
    wh, zg, zu, eh, eg, eu = K.gated(x[at], wg, wu, *b, "silu", sc[0][at] if eight else None, sc[1], sc[2], out)
    R.within(h[at], wh, eh)
    if not eight:
        h2, gate, up = hg.hashgrid_gated_forward(x, wg, wu, *b, save_pre=True)
        assert torch.equal(h2, h)
        R.within(gate[at], zg, R.rounded(zg, eg, dtype))
        R.within(up[at], zu, R.rounded(zu, eu, dtype))
