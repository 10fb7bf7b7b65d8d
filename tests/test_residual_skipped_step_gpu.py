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


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("zero", [False, True])
def test_skipped_steps_do_not_count(bits, zero):
    # The overflows a loss scale starts with: afterwards all is as if they had not been (a step counted for nothing
    # would take 1 - b^t for too large a t, and other rounding noise).
    g = torch.Generator(device=DEV).manual_seed(2)
    start = [torch.randn(n, generator=g, device=DEV) for n in (3, 1000, 70001)] + [torch.randn(50, generator=g, device=DEV)] * 40
    grads = [[torch.randn(p.shape, generator=g, device=DEV) for p in start] for _ in range(3)]

    def run(scales):
        params = [torch.nn.Parameter(p.clone()) for p in start]
        opt = hg.HashGridAdamW([dict(params=params[:2]), dict(params=params[2:], lr=1e-2, weight_decay=0.1)], lr=1e-3,
                               state_bits=bits, seed=7, zero_grad_in_step=zero)
        todo = iter(grads)
        for s in scales:
            new = next(todo) if s == 1.0 else [torch.full_like(p, INF) for p in start]
            for p, d in zip(params, new):
                p.grad = d.clone()
            opt.step(grad_scale=scale(s))
        return params, opt

    a, oa = run([INF, float("nan"), 1.0, -INF, 1.0, 1.0])
    b, ob = run([1.0, 1.0, 1.0])
    for p, q in zip(a, b):
        assert torch.equal(p, q)
        for k in ("m", "v"):
            assert torch.equal(oa.state[p][k].view(torch.uint8), ob.state[q][k].view(torch.uint8))
        assert int(oa.state[p]["step"]) == int(ob.state[q]["step"]) == 3


def test_counts_follow_each_parameter():
    # Parameters without a gradient do not step; a refused step counts for nothing; a checkpoint keeps the counts.
    g = torch.Generator(device=DEV).manual_seed(3)
    start = [torch.randn(100, generator=g, device=DEV) for _ in range(3)]
    grads = [[torch.randn(100, generator=g, device=DEV) for _ in start] for _ in range(4)]
    have = [(0, 1), (1, 2), (0, 1, 2), (2,)]

    def build(values):
        params = [torch.nn.Parameter(p.clone()) for p in values]
        return params, hg.HashGridAdamW(params, lr=1e-2, state_bits=8, seed=9)

    def step(params, opt, k):
        for i, p in enumerate(params):
            p.grad = grads[k][i].clone() if i in have[k] else None
        opt.step(grad_scale=scale(1.0))

    a, oa = build(start)
    for k in range(2):
        step(a, oa, k)
    wrong = torch.randn(200, device=DEV)[::2]
    a[0].grad, a[1].grad, a[2].grad = torch.ones_like(a[0]), torch.ones_like(a[1]), wrong
    with pytest.raises(ValueError):
        oa.step()
    assert [int(oa.state[p]["step"]) for p in a] == [1, 2, 1]
    b, ob = build([p.detach() for p in a])
    for p in b:
        p.grad = torch.zeros_like(p)
    import io
    buf = io.BytesIO()
    torch.save(oa.state_dict(), buf)
    buf.seek(0)
    ob.load_state_dict(torch.load(buf, weights_only=True, map_location="cpu"))
    for k in range(2, 4):
        step(a, oa, k)
    assert [int(ob.state[p]["step"]) for p in b] == [1, 2, 1]
    for k in range(2, 4):
        step(b, ob, k)
    for p, q in zip(a, b):
        assert torch.equal(p, q) and int(oa.state[p]["step"]) == int(ob.state[q]["step"])
    assert [int(oa.state[p]["step"]) for p in a] == [2, 3, 3]
    # a checkpoint whose counts are plain numbers
    c, oc = build([p.detach() for p in b])
    state = ob.state_dict()
    for st in state["state"].values():
        st["step"] = int(st["step"])
        for k in ("m", "v"):
            st[k] = st[k].clone()
    oc.load_state_dict(state)
    step(c, oc, 2)
    step(b, ob, 2)
    for p, q in zip(c, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("bits", [8, 32])
def test_counted_steps_are_the_numbered_ones(bits):
    g = torch.Generator(device=DEV).manual_seed(4)
    start = [torch.randn(n, generator=g, device=DEV) for n in (300, 5)] + [torch.randn(20, generator=g, device=DEV)] * 40
    grads = [torch.randn(p.shape, generator=g, device=DEV) for p in start]
    make = lambda: [hg.AdamWTensor(param=p.clone(), grad=d, lr=1e-2, weight_decay=0.1, **hg.AdamWTensor.states(p, bits))  # noqa: E731
                    for p, d in zip(start, grads)]
    a, b = make(), make()
    pa, pb = hg.HashGridAdamWPlan(a), hg.HashGridAdamWPlan(b)
    clocks = torch.zeros(len(a), 4, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    for t in range(1, 120):
        if t == 60:  # a step in a graph counts each replay
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                pa.step(clocks=clocks, beta2=0.99, eps=1e-15, seed=5)
        if t < 60:
            pa.step(clocks=clocks, beta2=0.99, eps=1e-15, seed=5)
        else:
            graph.replay()
        pb.step(step=t, beta2=0.99, eps=1e-15, seed=5 + t)
        assert (clocks[:, 0] == t).all()
        for x, y in zip(a, b):
            assert torch.equal(x.m.view(torch.uint8), y.m.view(torch.uint8)) and torch.equal(x.v.view(torch.uint8), y.v.view(torch.uint8))
            # the corrections' powers may differ in a double's last bit, and their floats then in one of 2^-23
            assert ((x.param - y.param).abs() <= t * 2.0 ** -22 * (y.param.abs() + 2e-2)).all()
