"""Operands and outputs of layer norms and gated layers, each with a row stride of its
own, up to the longest that a gated backward takes."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
LONGEST = 1 << 22


def like(t, pad, at):
    """t's values in rows that are ``pad`` columns apart more, from column ``at`` on."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device=DEV)
    wide[:, at:at + t.shape[1]] = t
    return wide[:, at:at + t.shape[1]]


def operands(m, k, n, dtype):
    g = torch.Generator().manual_seed(m + k + n)
    make = lambda i, j, s=1.0: (torch.randn(i, j, generator=g) * s).to(dtype).to(DEV)  # noqa: E731
    return [make(m, n), make(m, k), make(n, k, k ** -0.5), make(n, k, k ** -0.5), make(m, n), make(m, n)]  # dh, x, wg, wu, gate, up


# one pass of one tile; two passes; few rows in slices; rows shorter than a piece; many rows
@pytest.mark.parametrize("m,k,n", [(700, 40, 24), (301, 300, 140), (64, 256, 512), (500, 5, 200), (40001, 264, 136)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated_backward(m, k, n, dtype):
    ops = operands(m, k, n, dtype)
    want = hg.hashgrid_gated_backward(*ops, act="silu")
    for pads in ((1, 2, 3, 4, 5, 6), (24, 8, 0, 16, 40, 32), (0, 0, 0, 0, 0, 9), (0, 0, 0, 0, 9, 0), (9, 0, 0, 0, 0, 0), (0, 9, 0, 0, 0, 0)):
        apart = [like(t, p, p // 2) for t, p in zip(ops, pads)]
        dx = torch.full((m, k + 11), 7.0, dtype=dtype, device=DEV)
        dwg, dwu = (torch.full((n, k + p), 7.0, device=DEV) for p in (3, 12))
        got = hg.hashgrid_gated_backward(*apart, act="silu", dx=dx[:, 4:4 + k], dw_gate=dwg[:, 1:1 + k], dw_up=dwu[:, 8:8 + k])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (dx[:, :4] == 7).all() and (dx[:, 4 + k:] == 7).all() and (dwg[:, :1] == 7).all() and (dwg[:, 1 + k:] == 7).all()
        assert (dwu[:, :8] == 7).all() and (dwu[:, 8 + k:] == 7).all()


@pytest.mark.parametrize("k,n", [(40, 24), (300, 140), (64, 500), (100, 5)])
def test_gated_backward_of_the_longest_strides(k, n):
    # 300 rows 2^22 values apart: the last ones of a tile begin past 2^31 bytes.  All matrices lie beside each other in
    # one buffer, and then one at a time.
    m = 300
    ops = operands(m, k, n, BF16)
    want = hg.hashgrid_gated_backward(*ops, act="gelu_tanh")
    buf = torch.empty(m * LONGEST, dtype=BF16, device=DEV)
    at = 1

    def far(t):
        nonlocal at
        v = buf.as_strided(t.shape, (LONGEST, 1), at)
        at += t.shape[1] + 3
        return v

    moved = {i: far(ops[i]).copy_(ops[i]) for i in (0, 1, 4, 5)}
    dx = far(ops[1])
    got = hg.hashgrid_gated_backward(*(moved.get(i, t) for i, t in enumerate(ops)), act="gelu_tanh", dx=dx)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, want))
    for i in moved:
        one = [moved[i] if j == i else t for j, t in enumerate(ops)]
        assert all(torch.equal(a, b) for a, b in zip(hg.hashgrid_gated_backward(*one, act="gelu_tanh"), want))
        far_ = moved[i].as_strided(ops[i].shape, (LONGEST + 1, 1))
        with pytest.raises(hg.HashGridError, match="stride"):
            hg.hashgrid_gated_backward(*(far_[:299] if j == i else t[:299] if j in moved else t for j, t in enumerate(ops)))


@pytest.mark.parametrize("m,c", [(130, 7), (130, 100), (60, 600), (40, 2000), (30, 4500)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_layer_norm(m, c, dtype):
    g = torch.Generator().manual_seed(m + c)
    x, r, dy, ds = ((torch.randn(m, c, generator=g)).to(dtype).to(DEV) for _ in range(4))
    w, b = torch.randn(c, generator=g).to(DEV), torch.randn(c, generator=g).to(DEV)
    want = hg.hashgrid_layer_norm_forward(x, w, b, residual=r, save_sum=True, save_stats=True)
    grads = hg.hashgrid_layer_norm_backward(dy, want.sum, w, want.mean, want.rstd, ds=ds)
    for pads in ((1, 2, 3, 4), (8, 0, 16, 24), (0, 5, 0, 0)):
        y, s = like(x, pads[2], 0), like(x, pads[3], pads[3] // 2)
        out = hg.hashgrid_layer_norm_forward(like(x, pads[0], 0), w, b, residual=like(r, pads[1], pads[1]), out=y, sum_out=s, save_stats=True)
        assert out.y is y and out.sum is s
        assert all(torch.equal(getattr(out, f), getattr(want, f)) for f in ("y", "sum", "mean", "rstd"))
        dx = like(x, pads[3], 0)
        got = hg.hashgrid_layer_norm_backward(like(dy, pads[0], 0), like(s, pads[1], pads[1]), w, out.mean, out.rstd,
                                              ds=like(ds, pads[2], 0), dx=dx)
        assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, grads))
