"""The residual head on the encoder, its training step and its 8-bit form, run
together as the example runs them."""
import os
import sys

import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
DEV = "cuda"


def plain(head, features, rounding):
    """The head in float64 torch operations; ``rounding`` is applied where the head rounds to its 16-bit type."""
    r = rounding
    lin = lambda x, n: r(x) @ r(getattr(head, n + "_w").double()).t() + getattr(head, n + "_b").double()  # noqa: E731
    norm = lambda s, w: s * (s.square().mean(1, keepdim=True) + head.eps).rsqrt() * w.double()  # noqa: E731
    act = {"silu": torch.nn.functional.silu, "relu": torch.relu,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[head.act]
    h = stem = r(lin(features.double(), "stem"))
    for i in range(head.blocks):
        u = r(act(lin(r(norm(h, getattr(head, f"norm{i}"))), f"up{i}")))
        h = r(lin(u, f"down{i}") + h)
    return lin(r(norm(h + stem, head.norm_out)), "out")


class Straight(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dtype):
        return x.to(dtype).double()

    @staticmethod
    def backward(ctx, g):
        return g, None


@pytest.mark.parametrize("act", ["silu", "relu", "gelu_tanh"])
@pytest.mark.parametrize("width,blocks,n", [(256, 2, 3000), (64, 1, 777), (40, 3, 50)])
def test_outputs_and_gradients(act, width, blocks, n):
    torch.manual_seed(1)
    head = hg.HashGridResidualHead(32, width, blocks, 4, act=act, dtype=torch.float16)
    x = torch.randn(n, 32, device=DEV).requires_grad_()
    c = torch.randn(n, 4, device=DEV)
    y = head(x)
    (y * c).sum().backward()
    got = [x.grad] + [p.grad for p in head.parameters()]
    x64 = x.detach().clone().requires_grad_()
    for p in head.parameters():
        p.grad = None
    want_y = plain(head, x64, lambda t: Straight.apply(t, torch.float16))
    (want_y * c).sum().backward()
    want = [x64.grad] + [p.grad for p in head.parameters()]
    # binary16 rounds each activation and gradient by 2^-11 at most; some 6 roundings a block on the way, each
    # amplified at most a few times; in the 2-norm of a whole tensor they add like independent errors
    tol = 2.0 ** -11 * 6 * (blocks + 2)
    assert float((y - want_y).detach().norm() / want_y.detach().norm()) <= tol
    for a, b in zip(got, want):
        assert float((a - b).norm() / b.norm()) <= (tol if act != "relu" else 2 * tol)  # ReLUs within rounding of 0 may flip


def test_the_8bit_head_is_near_the_16bit_one():
    torch.manual_seed(2)
    head = hg.HashGridResidualHead(32, 256, 2, 4)
    x = torch.randn(5000, 32, device=DEV)
    with torch.no_grad():
        y, y8 = head(x), head.quantized()(x)
    # e4m3 values and weights: 2^-4 at most, about 2^-5.5 rms each, in two products on the way
    assert float((y - y8).norm() / y.norm()) <= 2.0 ** -4


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_fits(bits):
    import fit_field
    enc, head, losses = fit_field.fit(steps=120, points=1 << 14, width=64, blocks=1, state_bits=bits)
    assert losses.isfinite().all()
    assert float(losses[-10:].mean()) < 0.1 * float(losses[:3].mean())


@pytest.mark.parametrize("bits", [8, 32])
def test_checkpoint_and_resume(bits):
    def build():
        torch.manual_seed(3)
        head = hg.HashGridResidualHead(32, 64, 1, 4)
        opt = hg.HashGridAdamW([dict(params=list(head.parameters()), weight_decay=0.1)], lr=1e-2, state_bits=bits, seed=5)
        return head, opt

    data = torch.randn(6, 500, 32, device=DEV)

    def steps(head, opt, rows):
        for x in rows:
            opt.zero_grad()
            head(x).square().mean().backward()
            opt.step()

    head, opt = build()
    steps(head, opt, data[:3])
    kept = {k: v.clone() for k, v in head.state_dict().items()}, opt.state_dict()
    import io
    buf = io.BytesIO()
    torch.save(kept, buf)
    steps(head, opt, data[3:])
    other, opt2 = build()
    buf.seek(0)
    weights, state = torch.load(buf, weights_only=True)
    other.load_state_dict(weights)
    opt2.load_state_dict(state)
    steps(other, opt2, data[3:])
    for a, b in zip(head.parameters(), other.parameters()):
        assert torch.equal(a, b)
    for s in opt2.state.values():
        assert s["m"].dtype == (torch.float8_e4m3fn if bits == 8 else torch.float32)


def test_optimizer_matches_torch_adamw():
    torch.manual_seed(4)
    a = [torch.nn.Parameter(torch.randn(n, device=DEV)) for n in (1000, 7, 70000)]
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    oa = hg.HashGridAdamW(a, lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    ob = torch.optim.AdamW(b, lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    for _ in range(5):
        for p, q in zip(a, b):
            p.grad = torch.randn_like(p)
            q.grad = p.grad.clone()
        oa.step()
        ob.step()
    for p, q in zip(a, b):
        assert float((p - q).abs().max()) <= 1e-6 * float(q.abs().max()) + 1e-7
