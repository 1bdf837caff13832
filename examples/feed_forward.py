"""A pre-norm feed-forward block of a transformer on the library's operators.

    h = x + r                        the residual stream
    n = rmsnorm(h) * g
    u = gelu(n W1^T + b1)
    y = h + u W2^T + b2              the stream's next value

FeedForward trains it in bf16 (forward, backward, a plain SGD step on fp32
master weights); Decoder serves it token by token with 8-bit weights: the
normalisation writes E4M3 codes and row scales, which the first product reads
together with the weights' per-feature scales.  Every step of the computation is
a call of one library handle; torch holds the tensors and updates the weights.

    python examples/feed_forward.py      trains on synthetic data, then decodes
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_epilogue_persistent_gb300 as G  # noqa: E402

E4M3_TOP = 448.0


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class FeedForward:
    """One block's weights, activations and gradients for `rows` tokens."""

    def __init__(self, gemm, width, hidden, rows, seed=0, eps=1e-6):
        self.gemm, self.eps, self.rows, self.width, self.hidden = gemm, eps, rows, width, hidden
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, scale: torch.randn(*s, generator=gen, device="cuda") * scale
        # fp32 master weights and their bf16 copies, which the products read
        self.master = {"gain": torch.ones(width, device="cuda"),
                       "w1": rnd(hidden, width, scale=width ** -0.5),
                       "b1": torch.zeros(hidden, device="cuda"),
                       "w2": rnd(width, hidden, scale=hidden ** -0.5),
                       "b2": torch.zeros(width, device="cuda")}
        self.weights = {k: v.bfloat16() for k, v in self.master.items()}
        self.grads = {k: torch.zeros_like(v) for k, v in self.master.items()}
        # activations the backward pass reads, and its own
        self.h, self.n = _empty(rows, width), _empty(rows, width)
        self.rstd = _empty(rows, dtype=torch.float32)
        self.z, self.u, self.y = _empty(rows, hidden), _empty(rows, hidden), _empty(rows, width)
        self.du, self.dz = _empty(rows, hidden), _empty(rows, hidden)
        self.dn, self.dx = _empty(rows, width), _empty(rows, width)
        self.workspace = _empty(max(1, G.gemm_rmsnorm_bwd_workspace(rows, width)),
                                dtype=torch.uint8)

    def forward(self, x, r, stream=None):
        w, g = self.weights, self.gemm
        g.rmsnorm(x, w["gain"], self.n, residual=r, h=self.h, rstd=self.rstd, eps=self.eps,
                  stream=stream)
        g.linear(self.n, w["w1"], self.u, bias=w["b1"], activation="gelu", z=self.z, stream=stream)
        g.linear(self.u, w["w2"], self.y, bias=w["b2"], residual=self.h, stream=stream)
        return self.y

    def backward(self, dy, stream=None):
        """Weight gradients (added to self.grads' products; biases and gain overwritten) and
        the gradient of x and r, from the gradient of y."""
        w, g, d = self.weights, self.gemm, self.grads
        g.linear_bwd(dy, self.u, w["w2"], da=self.du, db=d["w2"], dbias=d["b2"], accumulate=True,
                     stream=stream)
        g.linear_bwd(self.du, self.n, w["w1"], z=self.z, activation="gelu", dz=self.dz, da=self.dn,
                     db=d["w1"], dbias=d["b1"], accumulate=True, stream=stream)
        g.rmsnorm_bwd(self.dn, self.h, w["gain"], self.rstd, self.dx, d["gain"], dh=dy,
                      workspace=self.workspace, stream=stream)
        return self.dx

    def step(self, rate):
        for k, v in self.master.items():
            v.add_(self.grads[k], alpha=-rate)
            self.weights[k].copy_(v)
            self.grads[k].zero_()


class Decoder:
    """The block for a few tokens at a time, its first product in 8 bits."""

    def __init__(self, block, tokens=1):
        w = block.weights
        self.gemm, self.eps = block.gemm, block.eps
        self.gain, self.b1, self.w2, self.b2 = w["gain"], w["b1"], w["w2"], w["b2"]
        # per-feature scales of the 8-bit weights
        w1 = block.master["w1"]
        self.s1 = w1.abs().amax(dim=1).clamp(min=2.0 ** -100) / E4M3_TOP
        self.w1 = (w1 / self.s1[:, None]).to(torch.float8_e4m3fn)
        self.h = _empty(tokens, block.width)
        self.n = _empty(tokens, block.width, dtype=torch.float8_e4m3fn)
        self.scale = _empty(tokens, dtype=torch.float32)
        self.u, self.y = _empty(tokens, block.hidden), _empty(tokens, block.width)

    def __call__(self, x, r, stream=None):
        g = self.gemm
        g.rmsnorm(x, self.gain, self.n, residual=r, h=self.h, scale=self.scale, eps=self.eps,
                  stream=stream)
        g.linear(self.n, self.w1, self.u, bias=self.b1, activation="gelu", row_scale=self.scale,
                 col_scale=self.s1, stream=stream)
        g.linear(self.u, self.w2, self.y, bias=self.b2, residual=self.h, stream=stream)
        return self.y


def train(gemm, width=512, hidden=2048, rows=1024, steps=30, rate=0.02, seed=1):
    """Fits the block to another one's outputs; returns (block, the loss before each step)."""
    block, target = FeedForward(gemm, width, hidden, rows, seed), FeedForward(gemm, width, hidden,
                                                                              rows, seed + 1)
    gen = torch.Generator(device="cuda").manual_seed(seed + 2)
    x, r = (torch.randn(rows, width, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = target.forward(x, r).float()
    losses = []
    for _ in range(steps):
        err = block.forward(x, r).float() - want
        losses.append(float(err.square().mean()))
        block.backward((err * (2.0 / rows)).bfloat16())
        block.step(rate)
    return block, losses


def main():
    gemm = G.Gemm(torch.cuda.current_device())
    block, losses = train(gemm)
    print("loss: " + " ".join(f"{v:.4f}" for v in losses[::5]))
    decoder = Decoder(block)
    x, r = (torch.randn(1, block.width, device="cuda").bfloat16() for _ in range(2))
    decoder(x, r)                                # the first call plans its launches
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decoder(x, r, torch.cuda.current_stream())
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(1000):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"decode: {start.elapsed_time(end):.2f} us a token")
    status, detail = gemm.sync_status()
    assert status == G.GEMM_OK, (G.gemm_status_string(status), hex(detail))
    gemm.close()


if __name__ == "__main__":
    main()
