"""HashGridAdamW steps that a gradient scale which is not finite skips."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def scale(v):
    return torch.tensor(v, device=DEV)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_a_skipped_step_that_zeroes_gradients_leaves_none_behind(bits, bad):
    # The caller relies on the step to clear the gradients: an inf that stayed would make every later step skip too.
    g = torch.Generator(device=DEV).manual_seed(1)
    params = [torch.nn.Parameter(torch.randn(n, generator=g, device=DEV)) for n in (1, 5, 1024, 70001)]
    opt = hg.HashGridAdamW(params, lr=1e-2, state_bits=bits, zero_grad_in_step=True)
    for p in params:
        p.grad = torch.full_like(p, INF)
    kept, held = [p.detach().clone() for p in params], [p.grad for p in params]
    opt.step(grad_scale=scale(bad))
    for p, old, grad in zip(params, kept, held):
        assert torch.equal(p, old) and p.grad is grad and not grad.any()
    for p in params:
        p.grad += 1.0
    opt.step(grad_scale=scale(1.0))
    for p, old in zip(params, kept):
        assert p.isfinite().all() and not (p == old).any() and not p.grad.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_plan_clears_the_gradients_of_a_skipped_step_when_asked(dtype, offset):
    buf = torch.full((1000 + offset + 3,), 7.0, device=DEV, dtype=dtype)
    p = torch.randn(1000, device=DEV)
    t = hg.AdamWTensor(param=p, grad=buf[offset:offset + 1000], **hg.AdamWTensor.states(p, 32))
    old = p.clone()
    plan = hg.HashGridAdamWPlan([t])
    plan.step(step=1, grad_scale=scale(INF), zero_grad=True)
    assert (buf == 7).all()
    plan.step(step=1, grad_scale=scale(INF), zero_grad=True, zero_skipped=True)
    assert torch.equal(p, old) and not t.m.any() and not t.v.any() and not t.grad.any()
    assert (buf[:offset] == 7).all() and (buf[offset + 1000:] == 7).all()
