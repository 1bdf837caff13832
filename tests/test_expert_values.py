"""Values of the low-rank adapters and of weight gradients over groups that the other tests' bounds and
shapes let through.  Tolerances as in test_adapters and test_grouped."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
import test_adapters as A
from test_grouped import ACCUM, NAN, _i32, _operand, _rows, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


@pytest.mark.parametrize("t,bits", [(torch.bfloat16, 8), (torch.float16, 11)])
@pytest.mark.parametrize("rank", [1, 5, 16, 40, 300])
def test_few_rows_keep_u_in_32_bits(gemm, t, bits, rank):
    """u of a few rows goes through no workspace and is not rounded: of powers of two whose sum has a bit more than
    the type holds, and B a unit vector, d is u itself."""
    M, K, N = 3, 72, 40
    x = torch.zeros(M, K, dtype=t, device="cuda")
    x[:, 0] = x[:, 65] = 1.0
    a = torch.zeros(2, rank, (K + 7) // 8 * 8, dtype=t, device="cuda")[:, :, :K]
    j = torch.arange(rank, device="cuda")
    a[:, :, 0], a[:, :, 65] = 2.0 ** (j % 3).float(), 2.0 ** (j % 3 - bits).float()
    b = torch.zeros(2, N, (rank + 7) // 8 * 8, dtype=t, device="cuda")[:, :, :rank]
    n = torch.arange(N, device="cuda")
    b[:, n, n % rank] = 1.0
    u = torch.full((M, (rank + 7) // 8 * 8), NAN, dtype=t, device="cuda")[:, :rank]
    d = torch.full((M, N), NAN, device="cuda")
    gemm.adapters(x, a, b, _i32([0, 1, 2, 3]), _i32([1, 0, 1]), u, d)
    assert gemm.sync_status()[0] == G.GEMM_OK
    want = 2.0 ** (n % rank % 3).double() * (1.0 + 2.0 ** -bits)
    assert (want.to(t).double() != want).all()
    assert torch.equal(d.double(), want.expand(M, N))


@pytest.mark.parametrize("cfg", [None, dict(cta_group=1), dict(cta_group=2)])
def test_adapters_in_place_by_either_way_against_64_bits(gemm, cfg):
    """d on r, requests without an adapter among them: by the kernel of few rows and by products."""
    gemm.set_config(**cfg) if cfg else gemm.set_config(None)
    try:
        A._check(gemm, [1] * 40, [(3 * i) % 6 - 1 for i in range(40)], 5, 1032, 520, 24, r_t="f32", d_t="f32",
                 in_place=True)
        A._check(gemm, [2, 0, 5, 1], [1, 0, -1, 2], 3, 77, 130, 40, "f16", r_t="f16", d_t="f16", in_place=True,
                 before=1, behind=2)
    finally:
        gemm.set_config(None)


@pytest.mark.parametrize("offsets", [[-5, 3, 7], [0, 9, 4], [10, 4, 4], [6, 2, 8], [5, 8, 0, 3, 1, 2],
                                     [1 << 30, -(1 << 31), (1 << 31) - 1]])
@pytest.mark.parametrize("cfg", [None, dict(cta_group=1), dict(cta_group=2)])
def test_adapters_values_with_offsets_out_of_range(gemm, offsets, cfg):
    """Each request's rows against the formula, every element of the others as it was."""
    M, N, K, rank, n = 8, 72, 64, 8, len(offsets) - 1
    gen = torch.Generator().manual_seed(5)
    x, X = _operand(gen, M, K, "f16")
    a, Ad = _weights(gen, 3, rank, K, "f16", scale=K ** -0.5)
    b, Bd = _weights(gen, 3, N, rank, "f16")
    r = torch.randn(M, N, generator=gen).double()
    R = O.strided(r.float(), "f32")[0]
    r = O.f64(R)
    index = [(2 * i + 1) % 3 for i in range(n)]
    d, u = O.strided(torch.full((M, N), NAN), "f32"), O.strided(torch.full((M, rank), NAN), "f16")
    gemm.set_config(**cfg) if cfg else gemm.set_config(None)
    try:
        gemm.adapters(X, Ad, Bd, _i32(offsets), _i32(index), u[0], d[0], residual=R)
        assert gemm.sync_status()[0] == G.GEMM_OK
    finally:
        gemm.set_config(None)
    bounds = [min(max(o, 0), M) for o in offsets]
    got, owners = O.f64(d[0]), torch.zeros(M, dtype=torch.int64)
    for g in range(n):
        owners[_rows(bounds, g)] += 1
    for g, e in enumerate(index):
        rows = torch.zeros(M, dtype=torch.bool)
        rows[_rows(bounds, g)] = True
        rows &= owners == 1                       # (requests may not share rows)
        u64, eu = x[rows] @ a[e].T, x[rows].abs() @ a[e].abs().T * ACCUM
        eu = eu + O.rounding(u64.abs() + eu, "f16")
        want = r[rows] + u64 @ b[e].T
        err = eu @ b[e].abs().T + (u64.abs() + eu) @ b[e].abs().T * (ACCUM + 4 * O.U32) + want.abs() * 2 * O.U32
        O.within(got[rows], want, err, f"request {g}")
    assert torch.isnan(got[owners == 0]).all() and O.padding_untouched(*d) and O.padding_untouched(*u)


@pytest.mark.parametrize("cfg", [None, dict(cta_group=1, tile_n=64), dict(cta_group=2, tile_n=256, stages=1)])
@pytest.mark.parametrize("sizes,N,K", [([1], 8, 1), ([3, 0, 40], 129, 77), ([130, 257, 15], 264, 301),
                                       ([300, 0, 65, 513], 520, 701)])
@pytest.mark.parametrize("t,db_t", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
def test_odd_weight_gradients_added_to_in_16_bits(gemm, cfg, sizes, N, K, t, db_t):
    """A residual whose last feature has no neighbour: with da, whose epilogue it does not share, and alone."""
    from test_grouped import _check_backward
    gemm.set_config(**cfg) if cfg else gemm.set_config(None)
    try:
        for give in (("dz", "da", "db"), ("db",)):
            _check_backward(gemm, sizes, N, K, t, "silu" if "dz" in give else "none", da_t="f32", db_t=db_t,
                            accumulate=True, give=give, alpha=0.5, before=1, behind=2)
    finally:
        gemm.set_config(None)
