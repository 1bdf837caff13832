"""Calls of the operators whose weights change from row to row at the edge of what is taken: sizes of
nothing, and arguments that would make a result silently wrong, which are refused (CPU)."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
from test_grouped import _bwd, P
from test_layer_arguments import Library, Placed, _handle

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


# ---------------------------------------------------------------- outputs that another argument is

_DISPATCH = dict(T=5, k=3, H=32, R=9, type=G.GEMM_E4M3, x=P[0], ldx=32, slot=P[1], scale=P[2], y=P[3], ldy=32,
                 y_scale=P[4])
_COMBINE = dict(T=5, k=3, H=30, R=9, type=G.GEMM_F16, r_type=G.GEMM_F16, y_type=G.GEMM_F16, ys=P[0],
                ldys=32, slot=P[1], weight=P[2], r=P[3], ldr=32, y=P[4], ldy=32)
_COMBINE_BWD = dict(T=5, k=3, H=30, R=9, type=G.GEMM_F16, dy=P[0], lddy=32, slot=P[1], weight=P[2],
                    ys=P[3], ldys=32, dys=P[4], lddys=32, dweight=P[5])
_ROUTE = dict(T=5, k=2, E=4, index_bytes=4, index=P[0], ldi=2, offsets=P[1], slot=P[2], source=P[3])
_ADAPTERS = dict(M=5, N=96, K=96, rank=96, requests=3, adapters=4, type=G.GEMM_F16, r_type=G.GEMM_F16,
                 d_type=G.GEMM_F16, offsets=P[0], index=P[1], x=P[2], ldx=96, A=P[3], lda=96, strideA=96 * 96,
                 B=P[4], ldb=96, strideB=96 * 96, scale=P[5], u=P[6], ldu=96, r=P[7], ldr=96, d=P[8], ldd=96)
_GROUPED = dict(M=5, N=96, K=96, groups=3, sets=4, a_type=G.GEMM_F16, b_type=G.GEMM_F16, bias_type=G.GEMM_F16,
                r_type=G.GEMM_F16, z_type=G.GEMM_F16, d_type=G.GEMM_F16, alpha=1.0, offsets=P[0], index=P[1],
                A=P[2], lda=96, B=P[3], ldb=96, strideB=96 * 96, row_scale=P[4], col_scale=P[5], bias=P[6],
                R=P[7], ldr=96, Z=P[8], ldz=96, D=P[9], ldd=96)
_GROUPED_BWD = dict(M=5, N=96, K=96, groups=3, type=G.GEMM_F16, da_type=G.GEMM_F16, db_type=G.GEMM_F16,
                    dbias_type=G.GEMM_F16, activation=G.GEMM_ACT_SILU, alpha=1.0, offsets=P[0], dd=P[1], lddd=96,
                    z=P[2], ldz=96, a=P[3], lda=96, b=P[4], ldb=96, strideb=96 * 96, dz=P[5], lddz=96, da=P[6],
                    ldda=96, db=P[7], lddb=96, stridedb=96 * 96, dbias=P[8])
# operator: its structure, a call of it with every tensor (all of one width, so that no size or stride
# refuses any of them in another's place), outputs, and what may be one tensor
CALLS = {
    "route": (G.gemm_route_t, _ROUTE, ("offsets", "slot", "source"), ()),
    "dispatch": (G.gemm_dispatch_t, _DISPATCH, ("y", "y_scale"), ()),
    "combine": (G.gemm_combine_t, _COMBINE, ("y",), ({"y", "r"},)),
    "combine_bwd": (G.gemm_combine_bwd_t, _COMBINE_BWD, ("dys", "dweight"), ({"dys", "ys"},)),
    "grouped_linear": (G.gemm_grouped_linear_t, _GROUPED, ("Z", "D"), ({"D", "R"},)),
    "grouped_linear_bwd": (G.gemm_grouped_linear_bwd_t, _GROUPED_BWD, ("dz", "da", "db", "dbias"),
                           ({"dz", "dd"}, {"dz", "z"})),
    "adapters": (G.gemm_adapters_t, _ADAPTERS, ("u", "d"), ({"d", "r"},)),
}
PAIRS = [(name, out, other) for name, (_, call, outs, _) in CALLS.items() for out in outs
         for other in call if call[other] in P and other != out]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_check_an_output_that_is_another_argument(lib, name, out, other):
    """Each output at every other tensor's address: only what may be in place passes."""
    struct, call, _, in_place = CALLS[name]
    check = getattr(G, f"gemm_{name}_check")
    assert check(struct(**call)) == 0
    want = 0 if {out, other} in in_place else INVALID
    assert check(struct(**{**call, out: call[other]})) == want


_LINEAR_BWD = {k: v for k, v in _GROUPED_BWD.items() if k not in ("groups", "offsets", "strideb", "stridedb")}


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(dz=P[1]), 0), (dict(dz=P[2]), 0), (dict(dz=P[3], db=None), 0), (dict(dz=P[4], da=None), 0),
    (dict(dz=P[3]), INVALID), (dict(dz=P[4]), INVALID), (dict(dz=P[8]), INVALID), (dict(dbias=P[1]), INVALID),
    (dict(dbias=P[2]), INVALID), (dict(dbias=P[3]), INVALID), (dict(dbias=P[4]), INVALID),
    (dict(dbias=P[6]), INVALID), (dict(dbias=P[7]), INVALID)])
def test_check_the_same_without_groups(lib, kw, code):
    assert G.gemm_linear_bwd_check(G.gemm_linear_bwd_t(**{**_LINEAR_BWD, **kw})) == code


@pytest.mark.parametrize("kw", [dict(dz=P[3], db=None), dict(dz=P[4], da=None), dict(dbias=P[4], da=None),
                                dict(dbias=P[3], db=None)])
def test_check_what_is_not_read_may_be_an_output(lib, kw):
    """a is read for db only, b for da only."""
    assert G.gemm_grouped_linear_bwd_check(G.gemm_grouped_linear_bwd_t(**{**_GROUPED_BWD, **kw})) == 0


# ---------------------------------------------------------------- a gradient without what it is made from

def test_the_weights_gradient_without_the_rows_is_refused():
    """combine's dweight is made from ys: without, there is no number of rows to read off it, and no places in
    0 rows would give 0."""
    e = lambda *s: Placed(torch.zeros(*s), 0)
    slot = Placed(torch.zeros(4, 2, dtype=torch.int32), 0)
    lib = Library()
    for kw in (dict(), dict(dys=e(8, 64)), dict(weight=e(4, 2))):
        with pytest.raises(G.GemmError) as err:
            _handle(lib).combine_bwd(e(4, 64), slot, dweight=e(4, 2), **kw)
        assert err.value.status == INVALID and "ys" in str(err.value)
    assert lib.calls == 0
    _handle(lib).combine_bwd(e(4, 64), slot, dweight=e(4, 2), ys=e(0, 64))
    _handle(lib).combine_bwd(e(4, 64), slot, dys=e(8, 64))
    assert lib.calls == 2
