"""Sizes of the operators over groups of rows at which 32 bits end on the way to an index."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()
    torch.cuda.empty_cache()             # (of many GB)


def test_both_gradients_of_very_many_features(gemm):
    """One row of 224 million features, both gradients in one launch: an inner size whose estimated cycles
    pass 2^31.  Of small whole numbers the results are exact: da sums 4000 products of at most 9, the rest
    are 0; db is one product an element."""
    N, K = 224_000_000, 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    gen = torch.Generator(device="cuda").manual_seed(0)
    small = lambda *s: torch.randint(-3, 4, s, generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    dd = torch.zeros(1, N, dtype=torch.bfloat16, device="cuda")
    at = torch.randperm(N, generator=gen, device="cuda", dtype=torch.int32)[:4000].long()
    at[0], at[1] = 0, N - 1
    dd[0, at] = small(4000)
    a, b = small(1, K), small(1, N, K)
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    da = torch.full((1, K), float("nan"), device="cuda")
    db = torch.full((1, N, K), float("nan"), device="cuda")
    gemm.set_config(cta_group=1, tile_n=64)
    try:
        gemm.grouped_linear_bwd(dd, a, b, offsets, da=da, db=db)
        st, detail = gemm.sync_status()
    finally:
        gemm.set_config(None)
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    some = dd[0].nonzero()[:, 0]
    assert torch.equal(da[0], (dd[0, some, None].float() * b[0, some].float()).sum(0))
    assert int((db != 0).any(2).sum()) == (some.numel() if bool((a != 0).any()) else 0)
    assert torch.equal(db[0, some], dd[0, some, None].float() * a.float())


def _whole_numbers(gen, *shape):
    t = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    return t.random_(-3, 4, generator=gen)


def test_most_rows(gemm):
    """As many rows as a call takes, in 67 groups: every element of the product and of its gradients.  Sums of
    8 products of at most 9 are exact, and so is each group's db: 32 million terms of random signs, whose sum
    stays a whole number below 2^24 (their standard deviation is 23000)."""
    M, N, K, E = (1 << 31) - 8193, 8, 8, 67
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("not enough memory")
    gen = torch.Generator(device="cuda").manual_seed(0)
    a, b = _whole_numbers(gen, M, K), _whole_numbers(gen, E, N, K)
    bounds = [5 + (M - 5) * g // E - (g * 7) % 5 * (0 < g < E) for g in range(E + 1)]
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    nan = lambda *s, dtype=torch.bfloat16: torch.full(s, float("nan"), dtype=dtype, device="cuda")
    d = nan(M, N)
    gemm.grouped_linear(a, b, offsets, d)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    assert torch.isnan(d[:5]).all()
    for g in range(E):
        rows = slice(bounds[g], bounds[g + 1])
        assert torch.equal(d[rows].float(), a[rows].float() @ b[g].float().t()), g
    dd = d.random_(-3, 4, generator=gen)
    da, db, dz = nan(M, K), nan(E, N, K, dtype=torch.float32), nan(M, N)
    gemm.grouped_linear_bwd(dd, a, b, offsets, dz=dz, da=da)
    gemm.grouped_linear_bwd(dd, a, None, offsets, db=db)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    assert torch.isnan(da[:5]).all() and torch.isnan(dz[:5]).all()
    for g in range(E):
        rows = slice(bounds[g], bounds[g + 1])
        assert torch.equal(dz[rows], dd[rows]), g
        assert torch.equal(da[rows].float(), dd[rows].float() @ b[g].float()), g
        want = dd[rows].double().t() @ a[rows].double()
        assert int(want.abs().max()) < 1 << 24
        assert torch.equal(db[g].double(), want), g
