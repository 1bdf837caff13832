"""The layer operators on values where arithmetic goes wrong first.

A pre-activation reaches the activation exactly as a test gives it: as the bias of a
product of zeros (forward), and as z (backward)."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
ROWS = [1, 40, 300]          # the split-K kernel with one and with several CTAs, the persistent one


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


def _forward(gemm, z, act, rows, dtype=torch.float32, K=64):
    """(act(z), z) as the layer computes them, on the last of `rows` rows."""
    a = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
    b = torch.zeros(len(z), K, dtype=torch.float16, device="cuda")
    d, kept = (O.strided(torch.zeros(rows, len(z)), t)[0] for t in (NAMES[dtype], "f32"))
    gemm.linear(a, b, d, bias=z.cuda(), activation=act, z=kept)
    assert gemm.sync_status()[0] == G.GEMM_OK
    return d[rows - 1].cpu(), kept[rows - 1].cpu()


def _slope(gemm, z, act, rows=3):
    """act'(z) as the backward pass computes it, in z's type, on the last of `rows` rows."""
    t = NAMES[z.dtype]
    zs, dz, one = (O.strided(v.expand(rows, len(z)), t)[0] for v in (z, 0 * z, torch.ones_like(z)))
    a = torch.zeros(rows, 64, dtype=z.dtype, device="cuda")
    b = torch.zeros(len(z), 64, dtype=z.dtype, device="cuda")
    gemm.linear_bwd(one, a, b, z=zs, activation=act, dz=dz)
    assert gemm.sync_status()[0] == G.GEMM_OK
    return dz[rows - 1].cpu()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("act", ACTS)
def test_nan_passes_every_activation(gemm, act, rows):
    """A NaN comes out where it went in and nowhere else; infinities keep their limits."""
    z = torch.linspace(-3, 3, 77)
    z[[0, 31, 40, 76]] = float("nan")
    z[50] = float("inf")
    d, kept = _forward(gemm, z, act, rows)
    assert torch.equal(torch.isnan(d), torch.isnan(z)) and torch.equal(torch.isnan(kept), torch.isnan(z))
    assert d[50] == float("inf")
    if act == "relu":
        low = torch.tensor([-float("inf"), -1.0, -0.0, 0.0, 2.0])
        assert _forward(gemm, low, act, rows)[0].tolist() == [0.0, 0.0, 0.0, 0.0, 2.0]


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_nan_passes_every_derivative(gemm, act, dtype):
    z = torch.linspace(-3, 3, 77).to(dtype)
    z[[0, 31, 40, 76]] = float("nan")
    z[50], z[51] = float("inf"), -float("inf")
    dz = _slope(gemm, z, act)
    assert torch.equal(torch.isnan(dz), torch.isnan(z))
    assert dz[50] == 1 and dz[51] == 0


# The tails.  Beside the result's own rounding: the fitted distribution function's 2.2e-6, and
# twice that for fp32's rounding of the exponent (at most 128 before 2^x, two roundings of
# 2^-24, times log 2: 1.1e-5) and a few roundings more, together below 2^-15 of the result.
TAIL = 2.0 ** -15
ENDS = {"gelu": 13.0, "gelu_tanh": 10.0, "silu": 80.0}     # results stay normal fp32 numbers


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("act", sorted(ENDS))
def test_small_results_keep_their_digits(gemm, act, rows):
    """Left of the minimum the result falls off to 1e-35: each is right to its own size."""
    z = -torch.linspace(1.0, ENDS[act], 501)
    d, _ = _forward(gemm, z, act, rows)
    want = O.act(z.double(), act)
    O.within(d, want, want.abs() * TAIL, "d")


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_small_16_bit_results_are_the_nearest(gemm, dtype, rows):
    z = -torch.linspace(1.0, 13.0 if dtype == torch.bfloat16 else 5.2, 501)
    d, _ = _forward(gemm, z, "gelu", rows, dtype)
    want = O.act(z.double(), "gelu")
    O.within(d, want, O.rounding(want, NAMES[dtype]) + want.abs() * TAIL, "d")


@pytest.mark.parametrize("act", sorted(ENDS))
def test_small_derivatives_keep_their_digits(gemm, act):
    """act' = p + z p' with p the sigmoid or distribution function: right to the size of its
    two terms."""
    z = -torch.linspace(1.0, ENDS[act] - 1, 501).bfloat16()
    dz = _slope(gemm, z, act)
    v = z.double()
    want = O.act_grad(v, act)
    size = want.abs() + 2 * O.act(v, act).abs() / v.abs()
    O.within(dz, want, O.rounding(want, "bf16") * (1 + 2 * TAIL) + size * TAIL, "dz")


@pytest.mark.parametrize("rows", ROWS)
def test_gelu_near_zero(gemm, rows):
    """In the middle gelu is right to 2^-21 of z: the distribution function to 2^-22."""
    z = torch.linspace(-4, 4, 1001)
    d, _ = _forward(gemm, z, "gelu", rows)
    O.within(d, O.act(z.double(), "gelu"), z.double().abs() * 2.0 ** -21 + 1e-30, "d")


@pytest.mark.parametrize("M,N,K", [(1, 136, 260), (40, 200, 1031), (300, 520, 264)])
def test_ordinary_fp32_operands(gemm, M, N, K):
    """fp32 operands that are no tf32 values lose less than 2^-10 each to the dropped bits: 2^-9 +
    2^-20 of the terms' magnitudes in the product, beside its accumulation's 2^-10.  Their dropping
    alone, in 64 bits, is what the kernels do: then only the accumulation's error is left."""
    gen = torch.Generator().manual_seed(K)
    a, b = torch.randn(M, K, generator=gen), torch.randn(N, K, generator=gen)
    d = O.strided(torch.zeros(M, N), "f32")[0]
    gemm.linear(O.strided(a, "f32")[0], O.strided(b, "f32")[0], d)
    assert gemm.sync_status()[0] == G.GEMM_OK
    S = a.double().abs() @ b.double().abs().T
    O.within(d, a.double() @ b.double().T, S * (2.0 ** -9 + 2.0 ** -20 + 2.0 ** -10), "d")
    ten = lambda t: (t.view(torch.int32) & ~0x1FFF).view(torch.float32).double()
    O.within(d, ten(a) @ ten(b).T, S * 2.0 ** -10, "d of ten fraction bits")


def test_two_handles_at_once():
    """Two handles on two streams, their calls interleaved without ordering between them: each
    result as from one handle alone."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    handles, streams = [G.Gemm(0) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    try:
        gen = torch.Generator().manual_seed(2)
        rnd = lambda *s: torch.randn(*s, generator=gen).to("cuda", torch.bfloat16)
        sets = [(rnd(m, 1024), rnd(776, 1024), rnd(m, 776)) for m in (1, 24, 90, 300)]
        w = rnd(1024)

        def outputs():
            e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
            return [dict(n=e(*a.shape), d=e(*dd.shape), z=e(*dd.shape), dz=e(*dd.shape),
                         da=e(*a.shape), db=e(*b.shape)) for a, b, dd in sets]

        def layer(g, i, o, stream):
            a, b, dd = sets[i]
            g.rmsnorm(a, w, o["n"], stream=stream)
            g.linear(o["n"], b, o["d"], activation="gelu", z=o["z"], stream=stream)
            g.linear_bwd(dd, o["n"], b, z=o["z"], activation="gelu", dz=o["dz"], da=o["da"],
                         db=o["db"], stream=stream)

        want, got = outputs(), [outputs() for _ in handles]
        for i in range(len(sets)):
            layer(handles[0], i, want[i], None)
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(len(sets)):
                for g, stream, outs in zip(handles, streams, got):
                    layer(g, i, outs[i], stream)
        torch.cuda.synchronize()
        for g, outs in zip(handles, got):
            assert g.sync_status()[0] == G.GEMM_OK
            for o, ref in zip(outs, want):
                for k in ref:
                    assert torch.equal(o[k], ref[k]), k
    finally:
        for g in handles:
            g.close()


@pytest.mark.parametrize("rows", ROWS)
def test_minus_infinity(gemm, rows):
    """0 times an infinity, NaN, for the tanh form and silu; the limit 0 for relu and gelu."""
    z = torch.tensor([-float("inf"), -1.0, 1.0])
    for act, want in (("none", -float("inf")), ("relu", 0.0), ("gelu", 0.0)):
        assert _forward(gemm, z, act, rows)[0][0] == want, act
    for act in ("gelu_tanh", "silu"):
        d = _forward(gemm, z, act, rows)[0]
        assert torch.isnan(d).tolist() == [True, False, False], act
