"""The residual head's autograd functions around stand-ins for their kernels in
plain torch, so that what they hand to the kernels and to autograd shows
without a GPU."""
import pytest
import torch

from multiresolution_hash_grid_amd import residual as R


@pytest.fixture
def calls(monkeypatch):
    """The backwards' arguments, in the order of their calls."""
    seen = []

    def linear_forward(x, w, b=None, *, act="none", residual=None, out_dtype=None, save_pre=False, **_):
        z = x.float() @ w.float().t() + (0 if b is None else b)
        y = torch.nn.functional.silu(z) if act == "silu" else z.relu() if act == "relu" else z
        y = (y if residual is None else y + residual.float()).to(out_dtype or x.dtype)
        return (y, z.to(x.dtype)) if save_pre else y

    def linear_backward(dy, x, w, *, act="none", pre=None, need_dx=True, need_dw=True, need_db=True, **_):
        seen.append(dict(dy=dy, need_dx=need_dx, need_dw=need_dw, need_db=need_db))
        dz = dy.float()
        if act == "silu":
            p = torch.sigmoid(pre.float())
            dz = dz * (p + pre.float() * p * (1 - p))
        elif act == "relu":
            dz = dz * (pre > 0)
        return (dz @ w.float()).to(x.dtype) if need_dx else None, dz.t() @ x.float() if need_dw else None, dz.sum(0) if need_db else None

    def norm_forward(x, w, *, residual=None, eps=1e-6, save_sum=False, save_rstd=False, **_):
        s = x.float() if residual is None else x.float() + residual.float()
        q = (s.square().mean(1) + eps).rsqrt()
        return R.RmsNormOutput((s * q[:, None] * w).to(x.dtype), None, s.to(x.dtype) if save_sum else None, q if save_rstd else None)

    def norm_backward(dy, s, w, q, *, ds=None, need_dw=True, **_):
        seen.append(dict(dy=dy, ds=ds, need_dw=need_dw))
        h, g = s.float() * q[:, None], dy.float() * w
        dx = q[:, None] * (g - h * (g * h).mean(1, keepdim=True))
        return (dx if ds is None else dx + ds.float()).to(s.dtype), (dy.float() * h).sum(0) if need_dw else None

    for name, f in (("linear_forward", linear_forward), ("linear_backward", linear_backward),
                    ("rms_norm_forward", norm_forward), ("rms_norm_backward", norm_backward)):
        monkeypatch.setattr(R, "hashgrid_" + name, torch.no_grad()(f))  # kernels leave no graph
    return seen


def leaf(*shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).requires_grad_()


def refuses_second_derivatives(y, inputs):
    """A loss of y and of its gradients: the gradients' part must not be left out without a word."""
    grads = torch.autograd.grad(y.float().square().sum(), inputs, create_graph=True)
    for g in grads:
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.float().square().sum() + y.float().sum()).backward(retain_graph=True)


@pytest.mark.parametrize("act,residual", [("silu", False), ("none", True), ("relu", False)])
def test_linear_cannot_be_differentiated_twice(calls, act, residual):
    x, w, b = leaf(5, 8, dtype=torch.float16), leaf(4, 8), leaf(4)
    r = leaf(5, 4, dtype=torch.float16) if residual else None
    refuses_second_derivatives(R.HashGridLinearFunction.apply(x, w, b, act, r), [x, w, b] + ([r] if residual else []))


@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_cannot_be_differentiated_twice(calls, residual):
    x, w = leaf(5, 8), leaf(8)
    r = leaf(5, 8) if residual else None
    out = R.HashGridRmsNormFunction.apply(x, w, r)
    refuses_second_derivatives(out[0] + out[1] if residual else out, [x, w] + ([r] if residual else []))


def plain_norm(x, w, r, eps=1e-6):
    s = x + r
    return s * (s.square().mean(1, keepdim=True) + eps).rsqrt() * w, s


@pytest.mark.parametrize("use_y,use_s", [(True, False), (False, True), (True, True)])
def test_rms_norm_passes_on_only_the_gradients_there_are(calls, use_y, use_s):
    # An output without a gradient (the sum in front of a head's last layer) is not one of zeros: those would be written and read.
    x, w, r, c = leaf(6, 8), leaf(8), leaf(6, 8), torch.randn(6, 8)
    want = torch.autograd.grad(sum(t.mul(c).sum() for t, u in zip(plain_norm(x, w, r), (use_y, use_s)) if u), [x, w, r],
                               allow_unused=True)
    y, s = R.HashGridRmsNormFunction.apply(x, w, r)
    sum(t.mul(c).sum() for t, u in zip((y, s), (use_y, use_s)) if u).backward()
    for t, g in zip((x, w, r), want):
        assert t.grad.shape == t.shape
        assert torch.allclose(t.grad, torch.zeros_like(t) if g is None else g, atol=1e-5)
    assert len(calls) == (1 if use_y else 0)
    if use_y:
        assert (calls[0]["ds"] is not None) == use_s
