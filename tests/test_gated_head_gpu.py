"""The head of gated blocks with codes, its training step and its 8-bit form, run
together as a program runs them."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Straight(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dtype):
        return x.to(dtype).double()

    @staticmethod
    def backward(ctx, g):
        return g, None


def plain(head, features, ids, r):
    """The head in float64 torch operations; ``r`` is applied where the head rounds to its 16-bit type."""
    p = lambda n: getattr(head, n).double()  # noqa: E731
    lin = lambda x, n: r(x) @ r(p(n + "_w")).t() + p(n + "_b")  # noqa: E731
    act = {"silu": torch.nn.functional.silu, "relu": torch.relu, "none": lambda z: z,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[head.act]

    def norm(s, n):
        d = s - s.mean(1, keepdim=True)
        return d * (d.square().mean(1, keepdim=True) + head.eps).rsqrt() * p(n + "_w") + p(n + "_b")

    x = features.double()
    if ids is not None:
        code = torch.where((ids >= 0)[:, None], head.codes.table.double()[ids.clamp_min(0)] * head.codes.scale, 0.0)
        x = torch.cat([x, code], 1)
    h = stem = r(lin(x, "stem"))
    for i in range(head.blocks):
        n = r(norm(h, f"norm{i}"))
        f = r(act(lin(n, f"gate{i}")) * lin(n, f"up{i}"))
        h = r(lin(f, f"down{i}") + h)
    return lin(r(norm(h + stem, "norm_out")), "out")


@pytest.mark.parametrize("act", ["silu", "relu", "gelu_tanh", "none"])
@pytest.mark.parametrize("width,hidden,blocks,n,codes", [(256, None, 2, 3000, 20), (64, 93, 1, 777, 0), (40, 100, 3, 50, 7)])
def test_outputs_and_gradients(act, width, hidden, blocks, n, codes):
    torch.manual_seed(1)
    head = hg.HashGridGatedHead(32, width, blocks, 4, hidden=hidden, act=act, codes=codes, code_width=24, dtype=torch.float16)
    if codes:
        torch.nn.init.normal_(head.codes.table)
    x = torch.randn(n, 32, device=DEV).requires_grad_()
    ids = torch.randint(-1, codes, (n,), device=DEV) if codes else None
    c = torch.randn(n, 4, device=DEV)
    y = head(x, ids)
    (y * c).sum().backward()
    got = [x.grad] + [p.grad for p in head.parameters()]
    x64 = x.detach().clone().requires_grad_()
    for p in head.parameters():
        p.grad = None
    want_y = plain(head, x64, ids, lambda t: Straight.apply(t, torch.float16))
    (want_y * c).sum().backward()
    want = [x64.grad] + [p.grad for p in head.parameters()]
    # binary16 rounds each activation and gradient by 2^-11 at most; some 8 roundings a block on the way, each
    # amplified at most a few times; in the 2-norm of a whole tensor they add like independent errors
    tol = 2.0 ** -11 * 8 * (blocks + 2)
    assert float((y - want_y).detach().norm() / want_y.detach().norm()) <= tol
    # relu's slope steps from 0 to 1 at 0. A gate that the rounding moves across it has its whole slope wrong: gates
    # that are normal have a density of 0.4 at 0 in units of their deviation, so of them at most 2 x 0.4 x tol lie
    # within tol of 0, and a share p of terms that are wrong as a whole is sqrt(p) of a sum in the 2-norm
    grad_tol = tol + (0.8 * tol) ** 0.5 if act == "relu" else tol
    for (name, _), a, b in zip([("x", None)] + list(head.named_parameters()), got, want):
        assert float((a - b).norm()) <= grad_tol * float(b.norm()) + 1e-6, name


def test_the_8bit_head_is_near_and_takes_single_points():
    torch.manual_seed(2)
    head = hg.HashGridGatedHead(32, 128, 2, 4, codes=9, code_width=16)
    torch.nn.init.normal_(head.codes.table)
    x, ids = torch.randn(2000, 32, device=DEV), torch.randint(0, 9, (2000,), device=DEV)
    eight = head.quantized()
    with torch.no_grad():
        y, y8 = head(x, ids), eight(x, ids)
        # e4m3 rounds each operand of the gated products by 2^-4 of itself at most: some per cent of the blocks' outputs
        assert float((y - y8).norm() / y.norm()) <= 0.15
        # points do not see each other: one alone, as in the batch up to another order of its sums
        for i in (0, 7, 1999):
            one = head(x[i:i + 1], ids[i:i + 1])
            assert float((one - y[i:i + 1]).abs().max()) <= 2.0 ** -5 * float(y.abs().max())
        assert head(x[:0], ids[:0]).shape == (0, 4) and eight(x[:0], ids[:0]).shape == (0, 4)


def test_a_training_step_and_its_frozen_parts():
    torch.manual_seed(3)
    enc = hg.HashGridEncoder(n_levels=4, n_features_per_level=2, log2_hashmap_size=12)
    head = hg.HashGridGatedHead(enc.cfg.out_features, 64, 1, 4, codes=5, code_width=8)
    opt = hg.HashGridAdamW([dict(params=[enc.embeddings], lr=1e-2), dict(params=list(head.parameters()), lr=1e-3)], state_bits=8)
    x, ids = torch.rand(5000, 3, device=DEV), torch.randint(0, 5, (5000,), device=DEV)
    before = [p.detach().clone() for p in head.parameters()]
    for _ in range(2):
        opt.zero_grad()
        head(enc(x), ids).square().mean().backward()
        opt.step()
    assert all(not torch.equal(a, b) and b.isfinite().all() for a, b in zip(before, head.parameters()))
    # parameters that ask for no gradient get none, the others the same as before
    opt.zero_grad()
    head(enc(x), ids).square().mean().backward()
    want = head.up0_w.grad.clone(), enc.embeddings.grad.clone()
    opt.zero_grad()
    for n in ("gate0_w", "gate0_b", "norm0_w", "norm_out_b"):
        getattr(head, n).requires_grad_(False)
    head.codes.table.requires_grad_(False)
    head(enc(x), ids).square().mean().backward()
    assert head.gate0_w.grad is None and head.norm0_w.grad is None and head.codes.table.grad is None
    assert torch.equal(head.up0_w.grad, want[0])
    assert float((enc.embeddings.grad - want[1]).abs().max()) <= 1e-6 * float(want[1].abs().max())


def test_inference_in_a_graph():
    torch.manual_seed(4)
    head = hg.HashGridGatedHead(32, 64, 2, 4, codes=6, code_width=8)
    x, ids = torch.randn(3000, 32, device=DEV), torch.randint(0, 6, (3000,), device=DEV)
    for form in (head, head.quantized()):
        with torch.no_grad():
            form(x, ids)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = form(x, ids)
            for _ in range(3):
                x.normal_()
                ids.random_(0, 6)
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(y, form(x, ids))


def test_a_captured_training_pass():
    torch.manual_seed(5)
    head = hg.HashGridGatedHead(32, 64, 1, 4, codes=6, code_width=8)
    x, ids = torch.randn(5000, 32, device=DEV, requires_grad=True), torch.randint(0, 6, (5000,), device=DEV)
    c = torch.randn(5000, 4, device=DEV)
    leaves = [x] + list(head.parameters())

    def step():
        y = head(x, ids)
        return (y.detach(),) + torch.autograd.grad(y, leaves, c)  # (no graph lives on)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(3):
        with torch.no_grad():
            x.normal_()
            ids.random_(-1, 6)
            c.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in kept]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
