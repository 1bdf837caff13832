"""A pre-norm mixture-of-experts block of a transformer on the library's operators.

    h = x + r                                   the residual stream
    n = rmsnorm(h) * g
    w, e = softmax and numbers of the `top` largest of n Wr^T
    y = h + n Ws^T + sum_j w_j (gelu(n W1[e_j]^T + b1[e_j]) W2[e_j]^T)

(Ws: a projection that all tokens share.)  MixtureOfExperts trains it in bf16 (forward,
backward, a plain SGD step on fp32 master weights); Server decodes a batch of requests with
8-bit first products and a low-rank adapter of Ws for each request that has one.  Every
step of the computation but the choice of experts is a call of one library handle; torch
holds the tensors, picks the largest logits and updates the weights.  Nothing is read back
to the host: a captured graph of a step serves whatever the router decides.

    python examples/mixture_of_experts.py      trains on synthetic data, then decodes
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_epilogue_persistent_gb300 as G  # noqa: E402

E4M3_TOP = 448.0


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Routing:
    """The choices of `tokens` tokens and where their rows lie."""

    def __init__(self, tokens, experts, top):
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.top, self.offsets, self.slot = top, i32(experts + 1), i32(tokens, top)
        whole = -(-experts // 8) * 8                 # (rows of whole 16-byte pieces)
        self.logits = _empty(tokens, whole, dtype=torch.float32)[:, :experts]
        self.dlogits = _empty(tokens, whole)[:, :experts]
        self.weight, self.index = _empty(tokens, top, dtype=torch.float32), None

    def choose(self, gemm, stream=None):
        best, self.index = torch.topk(self.logits, self.top, dim=1)
        self.weight.copy_(torch.softmax(best, dim=1))
        gemm.route(self.index, self.offsets, self.slot, stream=stream)

    def logits_grad(self, dweight):
        """Gradient of the logits from that of the weights, bf16."""
        d = self.weight * (dweight - (dweight * self.weight).sum(dim=1, keepdim=True))
        return self.dlogits.zero_().scatter_(1, self.index, d.bfloat16())


class MixtureOfExperts:
    """One block's weights, activations and gradients for `tokens` tokens.  Its calls run on
    torch's current stream."""

    def __init__(self, gemm, width, hidden, experts, top, tokens, seed=0, eps=1e-6):
        self.gemm, self.eps, self.width, self.hidden = gemm, eps, width, hidden
        self.experts, self.top, self.tokens = experts, top, tokens
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, scale: torch.randn(*s, generator=gen, device="cuda") * scale
        # fp32 master weights and their bf16 copies, which the products read
        self.master = {"gain": torch.ones(width, device="cuda"),
                       "router": rnd(experts, width, scale=width ** -0.5),
                       "shared": rnd(width, width, scale=width ** -0.5),
                       "w1": rnd(experts, hidden, width, scale=width ** -0.5),
                       "b1": torch.zeros(experts, hidden, device="cuda"),
                       "w2": rnd(experts, width, hidden, scale=hidden ** -0.5)}
        self.weights = {k: v.bfloat16() for k, v in self.master.items()}
        self.grads = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.routing = Routing(tokens, experts, top)
        rows = tokens * top
        # activations the backward pass reads, and its own
        self.h, self.n, self.y = (_empty(tokens, width) for _ in range(3))
        self.rstd = _empty(tokens, dtype=torch.float32)
        self.xs, self.ys = _empty(rows, width), _empty(rows, width)
        self.z, self.u = _empty(rows, hidden), _empty(rows, hidden)
        self.dweight = _empty(tokens, top, dtype=torch.float32)
        self.dys, self.dxs = _empty(rows, width), _empty(rows, width)
        self.du, self.dz = _empty(rows, hidden), _empty(rows, hidden)
        self.dn, self.dn_shared, self.dx = (_empty(tokens, width) for _ in range(3))
        self.workspace = _empty(max(1, G.gemm_rmsnorm_bwd_workspace(tokens, width)),
                                dtype=torch.uint8)

    def forward(self, x, r):
        w, g, t, s = self.weights, self.gemm, self.routing, torch.cuda.current_stream()
        g.rmsnorm(x, w["gain"], self.n, residual=r, h=self.h, rstd=self.rstd, eps=self.eps, stream=s)
        g.linear(self.n, w["router"], t.logits, stream=s)
        t.choose(g, s)
        g.dispatch(self.n, t.slot, self.xs, stream=s)
        g.grouped_linear(self.xs, w["w1"], t.offsets, self.u, bias=w["b1"], activation="gelu",
                         z=self.z, stream=s)
        g.grouped_linear(self.u, w["w2"], t.offsets, self.ys, stream=s)
        g.linear(self.n, w["shared"], self.y, residual=self.h, stream=s)
        g.combine(self.ys, t.slot, self.y, weight=t.weight, residual=self.y, stream=s)
        return self.y

    def backward(self, dy):
        """Weight gradients (added to self.grads' products; biases and gain overwritten) and
        the gradient of x and r, from the gradient of y."""
        w, g, t, d, s = self.weights, self.gemm, self.routing, self.grads, torch.cuda.current_stream()
        g.combine_bwd(dy, t.slot, self.dys, weight=t.weight, ys=self.ys, dweight=self.dweight,
                      stream=s)
        g.grouped_linear_bwd(self.dys, self.u, w["w2"], t.offsets, da=self.du, db=d["w2"],
                             accumulate=True, stream=s)
        g.grouped_linear_bwd(self.du, self.xs, w["w1"], t.offsets, z=self.z, activation="gelu",
                             dz=self.dz, da=self.dxs, db=d["w1"], dbias=d["b1"], accumulate=True,
                             stream=s)
        # n's gradient: by way of the experts, the shared projection and the router
        g.linear_bwd(dy, self.n, w["shared"], da=self.dn_shared, db=d["shared"], accumulate=True,
                     stream=s)
        g.combine(self.dxs, t.slot, self.dn, residual=self.dn_shared, stream=s)
        g.linear_bwd(t.logits_grad(self.dweight), self.n, w["router"], da=self.dn_shared,
                     db=d["router"], accumulate=True, stream=s)
        self.dn += self.dn_shared
        g.rmsnorm_bwd(self.dn, self.h, w["gain"], self.rstd, self.dx, d["gain"], dh=dy,
                      workspace=self.workspace, stream=s)
        return self.dx

    def step(self, rate):
        for k, v in self.master.items():
            v.add_(self.grads[k], alpha=-rate)
            self.weights[k].copy_(v)
            self.grads[k].zero_()


class Server:
    """The block for a batch of requests, its experts' first product in 8 bits, with a
    low-rank adapter of the shared projection for each request that has one: a [adapters, rank,
    width], b [adapters, width, rank], scale [adapters].  `tokens`: rows of the batch; request i
    has the rows bounds[i] .. bounds[i + 1] - 1 and the adapter index[i] (-1: none)."""

    def __init__(self, block, tokens, adapters):
        w = block.weights
        self.gemm, self.eps, self.w = block.gemm, block.eps, w
        self.a, self.b, self.scale = adapters
        # per-feature scales of the 8-bit weights
        w1 = block.master["w1"]
        self.s1 = w1.abs().amax(dim=2).clamp(min=2.0 ** -100) / E4M3_TOP
        self.w1 = (w1 / self.s1[:, :, None]).to(torch.float8_e4m3fn)
        self.routing = Routing(tokens, block.experts, block.top)
        rows, width = tokens * block.top, block.width
        self.h, self.n, self.y = (_empty(tokens, width) for _ in range(3))
        self.q, self.qs = (_empty(r, width, dtype=torch.float8_e4m3fn) for r in (tokens, rows))
        self.row, self.rows = (_empty(r, dtype=torch.float32) for r in (tokens, rows))
        self.u, self.ys = _empty(rows, block.hidden), _empty(rows, width)
        self.low = _empty(tokens, self.a.shape[1])

    def __call__(self, x, r, bounds, index):
        g, w, t, s = self.gemm, self.w, self.routing, torch.cuda.current_stream()
        g.rmsnorm(x, w["gain"], self.n, residual=r, h=self.h, eps=self.eps, stream=s)
        g.rmsnorm(x, w["gain"], self.q, residual=r, scale=self.row, eps=self.eps, stream=s)
        g.linear(self.n, w["router"], t.logits, stream=s)
        t.choose(g, s)
        g.dispatch(self.q, t.slot, self.qs, scale=self.row, y_scale=self.rows, stream=s)
        g.grouped_linear(self.qs, self.w1, t.offsets, self.u, bias=w["b1"], activation="gelu",
                         row_scale=self.rows, col_scale=self.s1, stream=s)
        g.grouped_linear(self.u, w["w2"], t.offsets, self.ys, stream=s)
        g.linear(self.n, w["shared"], self.y, residual=self.h, stream=s)
        g.adapters(self.n, self.a, self.b, bounds, index, self.low, self.y, residual=self.y,
                   scale=self.scale, stream=s)
        g.combine(self.ys, t.slot, self.y, weight=t.weight, residual=self.y, stream=s)
        return self.y


def train(gemm, width=512, hidden=1024, experts=8, top=2, tokens=2048, steps=30, rate=0.02, seed=1):
    """Fits the block to another one's outputs; returns (block, the loss before each step)."""
    block, target = (MixtureOfExperts(gemm, width, hidden, experts, top, tokens, s)
                     for s in (seed, seed + 1))
    gen = torch.Generator(device="cuda").manual_seed(seed + 2)
    x, r = (torch.randn(tokens, width, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = target.forward(x, r).float()
    losses = []
    for _ in range(steps):
        err = block.forward(x, r).float() - want
        losses.append(float(err.square().mean()))
        block.backward((err * (2.0 / tokens)).bfloat16())
        block.step(rate)
    return block, losses


def main():
    gemm = G.Gemm(torch.cuda.current_device())
    block, losses = train(gemm)
    print("loss: " + " ".join(f"{v:.4f}" for v in losses[::5]))
    requests, n, rank = 16, 4, 8
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    server = Server(block, requests, (rnd(n, rank, block.width), rnd(n, block.width, rank),
                                      torch.full((n,), 0.01, device="cuda")))
    x, r = rnd(requests, block.width), rnd(requests, block.width)
    bounds = torch.arange(requests + 1, dtype=torch.int32, device="cuda")
    index = torch.arange(requests, dtype=torch.int32, device="cuda") % (n + 1) - 1
    server(x, r, bounds, index)                  # the first call plans its launches
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        server(x, r, bounds, index)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(200):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"decode: {start.elapsed_time(end) * 5:.1f} us a step of {requests} requests")
    status, detail = gemm.sync_status()
    assert status == G.GEMM_OK, (G.gemm_status_string(status), hex(detail))
    gemm.close()


if __name__ == "__main__":
    main()
