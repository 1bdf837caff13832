"""The operators together: a feed-forward block's forward and backward pass against the
same formulas in 64 bits, its training, and its 8-bit decoding.

Tolerances: an output that went through k stages, each rounded to bf16 (2^-8 of
its size) and summed with random signs, is off by a few 2^-8 of its root mean
square; the bounds below are 2-norms, k 2^-8 each, and for the 8-bit decoder
2^-4 for the codes' rounding in the product's result, which the residual dilutes."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
from examples.feed_forward import Decoder, FeedForward, train

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


@pytest.mark.parametrize("rows,width,hidden", [(1, 64, 128), (37, 136, 264), (300, 512, 1024)])
def test_block_against_64_bits(gemm, rows, width, hidden):
    block = FeedForward(gemm, width, hidden, rows, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy = (torch.randn(rows, width, generator=gen, device="cuda").bfloat16() for _ in range(3))
    y = block.forward(x, r)
    dx = block.backward(dy)
    assert gemm.sync_status()[0] == G.GEMM_OK
    w = {k: O.f64(v).requires_grad_() for k, v in block.weights.items()}
    xs = O.f64(x).requires_grad_()
    h = xs + O.f64(r)
    n = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + block.eps) * w["gain"]
    y64 = h + O.act(n @ w["w1"].T + w["b1"], "gelu") @ w["w2"].T + w["b2"]
    (y64 * O.f64(dy)).sum().backward()
    assert _rel(y, y64.detach()) < 3 * U
    assert _rel(dx, xs.grad) < 4 * U
    for k in w:
        assert _rel(block.grads[k], w[k].grad) < 4 * U, k


def test_training_lowers_the_loss(gemm):
    _, losses = train(gemm, width=256, hidden=512, rows=256, steps=12)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.7 * losses[0], losses


@pytest.mark.parametrize("tokens", [1, 5])
def test_decoder_follows_the_block(gemm, tokens):
    block = FeedForward(gemm, 256, 1024, tokens, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, r = (torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = O.f64(block.forward(x, r))
    assert _rel(Decoder(block, tokens)(x, r), want) < 2.0 ** -4
