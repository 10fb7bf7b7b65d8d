"""What the autograd functions ask their kernels to keep: everything the backward
reads where autograd records the call, nothing where it does not.  Stand-ins that
note their arguments take the kernels' place."""
import pytest
import torch

from multiresolution_hash_grid_amd import blocks as K
from multiresolution_hash_grid_amd import residual as R


@pytest.fixture
def kept(monkeypatch):
    """(name, what the call kept) of the forwards, in the order of their calls."""
    seen = []

    def product(x, n):
        return x.float().sum(1, keepdim=True).expand(-1, n).to(x.dtype).clone()

    def gated(x, wg, wu, bg=None, bu=None, *, save_pre=False, **_):
        seen.append(("gated", {"pre"} if save_pre else set()))
        h = product(x, wg.shape[0])
        return (h, h.clone(), h.clone()) if save_pre else h

    def layer_norm(x, w=None, b=None, *, residual=None, save_sum=False, save_stats=False, **_):
        seen.append(("layer_norm", ({"sum"} if save_sum else set()) | ({"stats"} if save_stats else set())))
        row = torch.zeros(x.shape[0]) if save_stats else None
        return K.LayerNormOutput(x.clone(), None, x.clone() if save_sum else None, row, row)

    def linear(x, w, b=None, *, out_dtype=None, save_pre=False, **_):
        seen.append(("linear", {"pre"} if save_pre else set()))
        y = product(x, w.shape[0]).to(out_dtype or x.dtype)
        return (y, y.clone()) if save_pre else y

    def rms_norm(x, w, *, residual=None, save_sum=False, save_rstd=False, **_):
        seen.append(("rms_norm", ({"sum"} if save_sum else set()) | ({"stats"} if save_rstd else set())))
        return R.RmsNormOutput(x.clone(), None, x.clone() if save_sum else None, torch.zeros(x.shape[0]) if save_rstd else None)

    for module, name, f in ((K, "gated", gated), (K, "layer_norm", layer_norm), (R, "linear", linear), (R, "rms_norm", rms_norm)):
        monkeypatch.setattr(module, f"hashgrid_{name}_forward", torch.no_grad()(f))
    return seen


def leaf(*shape, dtype=torch.float32):
    return torch.ones(*shape, dtype=dtype, requires_grad=True)


MODES = [torch.no_grad, torch.inference_mode]


@pytest.mark.parametrize("mode", MODES)
def test_gated_layer_keeps_its_projections_for_a_backward_only(kept, mode):
    args = [leaf(5, 6, dtype=torch.float16)] + [leaf(4, 6), leaf(4, 6), leaf(4), leaf(4)]
    with mode():
        assert not K.HashGridGatedFunction.apply(*args, "silu").requires_grad
    assert K.HashGridGatedFunction.apply(*args).requires_grad
    K.HashGridGatedFunction.apply(*(t.detach() for t in args))  # nothing asks for a gradient
    assert K.HashGridGatedFunction.apply(args[0].detach(), *args[1:3]).requires_grad
    assert [k for _, k in kept] == [set(), {"pre"}, set(), {"pre"}]


@pytest.mark.parametrize("mode", MODES)
def test_layer_norm_keeps_its_statistics_for_a_backward_only(kept, mode):
    x, w, b, r = leaf(5, 6), leaf(6), leaf(6), leaf(5, 6)
    with mode():
        assert not K.HashGridLayerNormFunction.apply(x, w, b).requires_grad
        y, s = K.HashGridLayerNormFunction.apply(x, w, b, r)  # the sum is an output
    assert s.shape == x.shape
    K.HashGridLayerNormFunction.apply(x, w, b)
    K.HashGridLayerNormFunction.apply(x.detach(), None, None, r)
    K.HashGridLayerNormFunction.apply(x.detach(), w.detach(), b.detach())
    assert [k for _, k in kept] == [set(), {"sum"}, {"stats"}, {"sum", "stats"}, set()]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("blocks", [1, 3])
def test_gated_head_keeps_nothing_in_inference(kept, mode, blocks):
    head, x = K.HashGridGatedHead(8, 16, blocks, 4, device="cpu"), torch.ones(5, 8)
    with mode():
        assert head(x).shape == (5, 4)
    names = ["linear"] + ["layer_norm", "gated", "linear"] * blocks + ["layer_norm", "linear"]
    assert [n for n, _ in kept] == names and not any(k for _, k in kept)
    del kept[:]
    assert head(x).requires_grad
    assert [n for n, _ in kept] == names
    assert [k for n, k in kept if n == "gated"] == [{"pre"}] * blocks
    assert [k for n, k in kept if n == "layer_norm"] == [{"stats"}] * blocks + [{"sum", "stats"}]


@pytest.mark.parametrize("mode", MODES)
def test_linear_layer_keeps_its_pre_activation_for_a_backward_only(kept, mode):
    x, w, b = leaf(5, 6, dtype=torch.float16), leaf(4, 6), leaf(4)
    with mode():
        for act in ("silu", "relu", "none"):
            assert not R.HashGridLinearFunction.apply(x, w, b, act).requires_grad
    assert R.HashGridLinearFunction.apply(x, w, b, "silu").requires_grad
    R.HashGridLinearFunction.apply(x.detach(), w.detach(), b.detach(), "silu")
    assert R.HashGridLinearFunction.apply(x.detach(), w, None, "gelu_tanh").requires_grad
    assert [k for _, k in kept] == [set()] * 3 + [{"pre"}, set(), {"pre"}]


@pytest.mark.parametrize("mode", MODES)
def test_rms_norm_keeps_its_statistics_for_a_backward_only(kept, mode):
    x, w, r = leaf(5, 6), leaf(6), leaf(5, 6)
    with mode():
        assert not R.HashGridRmsNormFunction.apply(x, w).requires_grad
        assert R.HashGridRmsNormFunction.apply(x, w, r)[1].shape == x.shape  # the sum is an output
    R.HashGridRmsNormFunction.apply(x, w)
    R.HashGridRmsNormFunction.apply(x.detach(), w.detach(), r)
    R.HashGridRmsNormFunction.apply(x.detach(), w.detach())
    assert [k for _, k in kept] == [set(), {"sum"}, {"stats"}, {"sum", "stats"}, set()]


@pytest.mark.parametrize("mode", MODES)
def test_residual_head_keeps_nothing_in_inference(kept, mode):
    head, x = R.HashGridResidualHead(8, 16, 2, 4, device="cpu"), torch.ones(5, 8)
    with mode():
        assert head(x).shape == (5, 4)
    names = ["linear"] + ["rms_norm", "linear", "linear"] * 2 + ["rms_norm", "linear"]
    assert [n for n, _ in kept] == names and not any(k for _, k in kept)
    del kept[:]
    assert head(x).requires_grad
    assert [k for n, k in kept if n == "rms_norm"] == [{"stats"}] * 2 + [{"sum", "stats"}]
    assert [k for n, k in kept if n == "linear"] == [set(), {"pre"}, set()] + [{"pre"}, set()] + [set()]
