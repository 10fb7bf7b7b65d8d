"""Upstream gradients reach the kernels as they lie where the kernels take them so: a
slice of a wider gradient is not copied.  Stand-ins that note their arguments take
the kernels' place."""
import pytest
import torch

from multiresolution_hash_grid_amd import blocks as K

IDS = torch.tensor([2, 0, -1, 2, 7])


@pytest.fixture
def seen(monkeypatch):
    """The upstream gradients that the backwards were called with."""
    got = []

    def embedding(dy, ids, rows, **_):
        got.append(dy)
        return torch.zeros(rows, dy.shape[1])

    def norm(dy, s, w, mean, q, *, ds=None, need_dw, need_db):
        got.extend(t for t in (dy, ds) if t is not None)
        return (torch.zeros(s.shape),) + tuple(torch.zeros(s.shape[1]) if n else None for n in (need_dw, need_db))

    def gated(dh, x, wg, wu, gate, up, **_):
        got.append(dh)
        return tuple(torch.zeros(t) for t in (x.shape, wg.shape, wu.shape, wg.shape[:1], wg.shape[:1]))

    def forward(shape, n=1):
        return tuple(torch.zeros(shape) for _ in range(n))

    for name, f in (("embedding_backward", embedding), ("layer_norm_backward", norm), ("gated_backward", gated),
                    ("embedding_forward", lambda t, i, out=None, **_: forward((len(i), t.shape[1]))[0] if out is None else out.zero_()),
                    ("layer_norm_forward", lambda x, *_, **__: K.LayerNormOutput(x.clone(), None, x.clone(), x[:, 0].clone(), x[:, 0].clone())),
                    ("gated_forward", lambda x, wg, *_, save_pre=False, **__: forward((x.shape[0], wg.shape[0]), 3) if save_pre else None)):
        monkeypatch.setattr(K, "hashgrid_" + name, torch.no_grad()(f))
    return got


def leaf(*shape):
    return torch.ones(*shape, requires_grad=True)


FORMS = dict(embedding=lambda: K.HashGridEmbeddingFunction.apply(leaf(3, 8), IDS),
             coded=lambda: K.HashGridCodedInputFunction.apply(leaf(5, 6), leaf(3, 8), IDS, torch.float32),
             norm=lambda: K.HashGridLayerNormFunction.apply(leaf(5, 6), leaf(6)),
             gated=lambda: K.HashGridGatedFunction.apply(leaf(5, 6), leaf(4, 6), leaf(4, 6), None, None))


@pytest.mark.parametrize("name", FORMS)
def test_a_slice_of_a_wider_gradient_is_not_copied(seen, name):
    y = FORMS[name]()
    wide = torch.randn(5, y.shape[1] + 7)
    up = wide[:, 3:3 + y.shape[1]]
    y.backward(up)
    dy, = seen
    at = up[:, 6:] if name == "coded" else up  # the codes' columns
    assert dy.data_ptr() == at.data_ptr() and dy.stride() == at.stride() and torch.equal(dy, at)


def test_both_gradients_of_a_norm_with_a_residual(seen):
    y, s = K.HashGridLayerNormFunction.apply(leaf(5, 6), leaf(6), None, leaf(5, 6))
    wide = torch.randn(5, 20)
    torch.autograd.backward([y, s], [wide[:, :6], wide[:, 11:17]])
    assert [t.data_ptr() for t in seen] == [wide.data_ptr(), wide[:, 11:].data_ptr()]


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("kind", ["one value", "one row", "columns apart", "transposed", "too far apart"])
def test_what_the_kernels_do_not_take_is_copied(seen, name, kind):
    y = FORMS[name]()
    m, c = y.shape
    up = {"one value": lambda: torch.ones(()).expand(m, c), "one row": lambda: torch.randn(1, c).expand(m, c),
          "columns apart": lambda: torch.randn(m, 2 * c)[:, ::2], "transposed": lambda: torch.randn(c, m).t(),
          "too far apart": lambda: torch.empty(5, (1 << 22) + 1)[:, :c].fill_(2.0)}[kind]()
    y.backward(up)
    dy, = seen
    assert dy.stride(1) == 1 and c - (6 if name == "coded" else 0) <= dy.stride(0) <= 1 << 22
    assert torch.equal(dy, up[:, 6:] if name == "coded" else up)


def test_one_row_or_one_column_are_taken_at_any_stride():
    a = torch.empty(64).as_strided((1, 6), (1, 1))
    b = torch.empty(64).as_strided((5, 1), (9, 4))
    assert K._as_rows(a) is a and K._as_rows(b) is b
    assert K._as_rows(torch.empty(64).as_strided((2, 6), (5, 1))).is_contiguous()  # rows that overlap
    assert K._as_rows(torch.empty(0, 6)).shape == (0, 6)
