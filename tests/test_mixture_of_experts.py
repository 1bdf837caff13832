"""The operators together: a mixture-of-experts block's forward and backward pass against the
same formulas in 64 bits, its training step captured into a graph, and its 8-bit serving with
adapters.

Tolerances: an output that went through k stages, each rounded to bf16 (2^-8 of its
size) and summed with random signs, is off by a few 2^-8 of its root mean square; the bounds
below are 2-norms, k 2^-8 each, and for the server 2^-4 for the codes' rounding in the
product's result, which the other terms dilute."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
from examples.mixture_of_experts import MixtureOfExperts, Server, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


def _rel(got, want):
    return float((O.f64(got) - want).norm() / want.norm())


def _formula(x, r, w, index, top, eps):
    """The block in 64 bits, the experts as chosen."""
    h = x + r
    n = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps) * w["gain"]
    weight = torch.softmax((n @ w["router"].T).gather(1, index), dim=1)
    y = h + n @ w["shared"].T
    for j in range(top):
        e = index[:, j]
        u = O.act(torch.einsum("tw,thw->th", n, w["w1"][e]) + w["b1"][e], "gelu")
        y = y + weight[:, j:j + 1] * torch.einsum("th,twh->tw", u, w["w2"][e])
    return y


@pytest.mark.parametrize("tokens,width,hidden,experts,top", [(1, 64, 128, 4, 1), (37, 136, 264, 5, 3),
                                                             (300, 256, 512, 8, 2), (64, 72, 40, 16, 1)])
def test_block_against_64_bits(gemm, tokens, width, hidden, experts, top):
    block = MixtureOfExperts(gemm, width, hidden, experts, top, tokens, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy = (torch.randn(tokens, width, generator=gen, device="cuda").bfloat16() for _ in range(3))
    y = block.forward(x, r)
    dx = block.backward(dy)
    assert gemm.sync_status()[0] == G.GEMM_OK
    w = {k: O.f64(v).requires_grad_() for k, v in block.weights.items()}
    xs = O.f64(x).requires_grad_()
    y64 = _formula(xs, O.f64(r), w, block.routing.index.cpu(), top, block.eps)
    (y64 * O.f64(dy)).sum().backward()
    assert _rel(y, y64.detach()) < 4 * U
    assert _rel(dx, xs.grad) < 6 * U
    for k in w:
        if float(w[k].grad.norm()) > 0:          # (with one choice a token the router has none)
            assert _rel(block.grads[k], w[k].grad) < 6 * U, k


def test_gradients_against_differences(gemm):
    """The formula's central difference along the computed gradient, over the gradient's squared
    norm: 1 up to the gradient's own error, 6 2^-8 as above (0.05 with the difference's)."""
    tokens, width = 256, 128
    block = MixtureOfExperts(gemm, width, 256, 4, 2, tokens, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, r, dy = (torch.randn(tokens, width, generator=gen, device="cuda").bfloat16() for _ in range(3))
    block.forward(x, r)
    block.backward(dy)
    index = block.routing.index.cpu()
    grad = {k: O.f64(v) for k, v in block.grads.items()}
    w0 = {k: O.f64(v) for k, v in block.weights.items()}
    for k in ("w1", "w2", "b1", "shared"):
        e = 1e-4 / float(grad[k].norm())
        loss = lambda s: float((_formula(O.f64(x), O.f64(r), {**w0, k: w0[k] + s * grad[k]}, index, 2,
                                         block.eps) * O.f64(dy)).sum())
        slope = (loss(e) - loss(-e)) / (2 * e)
        assert abs(slope / float(grad[k].square().sum()) - 1) < 0.05, k


def test_training_runs_and_changes_every_weight(gemm):
    block, losses = train(gemm, width=128, hidden=256, experts=4, top=2, tokens=256, steps=4)
    assert all(torch.isfinite(torch.tensor(losses))) and len(losses) == 4
    fresh = MixtureOfExperts(gemm, 128, 256, 4, 2, 256, seed=1)
    assert all(not torch.equal(block.master[k], fresh.master[k]) for k in fresh.master)


def test_a_captured_step_follows_its_inputs(gemm):
    """Forward and backward pass in one graph: other inputs choose other experts."""
    tokens, width = 200, 136
    block, eager = (MixtureOfExperts(gemm, width, 264, 6, 2, tokens, seed=7) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda: torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
    x, r, dy = rnd(), rnd(), rnd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x, r)
        block.backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, r)
        block.backward(dy)
    for _ in range(2):
        for t in (x, r, dy):
            t.copy_(rnd())
        for k in block.grads:
            block.grads[k].zero_()
            eager.grads[k].zero_()
        graph.replay()
        eager.forward(x, r)
        eager.backward(dy)
        torch.cuda.synchronize()
        assert gemm.sync_status()[0] == G.GEMM_OK
        assert torch.equal(block.y, eager.y) and torch.equal(block.dx, eager.dx)
        assert all(torch.equal(block.grads[k], eager.grads[k]) for k in block.grads)


@pytest.mark.parametrize("tokens", [1, 13])
def test_server_follows_the_block(gemm, tokens):
    block = MixtureOfExperts(gemm, 256, 512, 6, 2, tokens, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    x, r = rnd(tokens, 256), rnd(tokens, 256)
    n, rank = 3, 8
    a, b, scale = rnd(n, rank, 256), rnd(n, 256, rank), torch.rand(n, generator=gen, device="cuda") * 0.02
    bounds = torch.arange(tokens + 1, dtype=torch.int32, device="cuda")
    index = torch.arange(tokens, dtype=torch.int32, device="cuda") % (n + 1) - 1
    want = O.f64(block.forward(x, r))
    for i, e in enumerate(index.tolist()):
        if e >= 0:
            want[i] += float(scale[e]) * O.f64(b[e]) @ (O.f64(a[e]) @ O.f64(block.n[i]))
    got = Server(block, tokens, (a, b, scale))(x, r, bounds, index)
    assert gemm.sync_status()[0] == G.GEMM_OK
    assert _rel(got, want) < 2.0 ** -4
