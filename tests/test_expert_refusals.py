"""Calls of the operators whose weights change from row to row at the edge of what is taken: sizes of
nothing, and arguments that would make a result silently wrong, which are refused (CPU)."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
from test_grouped import _bwd, P

INVALID, ALIGN = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.library()


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


# ---------------------------------------------------------------- no features

@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(offsets=None), 0), (dict(da=None), 0), (dict(M=0, da=P[5] + 8), 0), (dict(K=0, da=P[5] + 8), 0),
    (dict(groups=0, da=P[5] + 8), 0), (dict(offsets=P[8] + 2), ALIGN), (dict(da=P[5] + 8), ALIGN),
    (dict(ldda=48), INVALID)])
def test_check_gradients_of_no_features(lib, kw, code):
    assert G.gemm_grouped_linear_bwd_check(
        _bwd(**{**dict(N=0, dd=None, z=None, b=None, dz=None, db=None), **kw})) == code


@pytest.mark.gpu
@pytest.mark.parametrize("K,da_t", [(72, torch.bfloat16), (7, torch.float32), (264, torch.float16)])
@pytest.mark.parametrize("offsets", [[2, 5, 5, 8], [6, 3, 9, 9]])
def test_gradients_of_no_features(gemm, offsets, K, da_t):
    """da, a sum over the features, is 0 in the groups' rows as without groups; others keep what they hold."""
    M, groups = 10, len(offsets) - 1
    e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    da = torch.full((M, (K + 15) // 16 * 16), float("nan"), dtype=da_t, device="cuda")[:, :K]
    db, dbias = e(groups, 0, K), e(groups, 0)
    gemm.grouped_linear_bwd(e(M, 0), e(M, K), e(groups, 0, K), torch.tensor(offsets, dtype=torch.int32).cuda(),
                            z=e(M, 0), activation="silu", dz=e(M, 0), da=da, db=db, dbias=dbias)
    assert gemm.sync_status()[0] == G.GEMM_OK
    mine = torch.zeros(M, dtype=torch.bool)
    for a, b in zip(offsets, offsets[1:]):
        mine[a:b] = True
    assert not da[mine.cuda()].any() and torch.isnan(da[~mine.cuda()]).all()
    one = torch.full((M, (K + 15) // 16 * 16), float("nan"), dtype=da_t, device="cuda")[:, :K]
    gemm.linear_bwd(e(M, 0), None, e(0, K), da=one)
    assert gemm.sync_status()[0] == G.GEMM_OK
    assert not one.any()
