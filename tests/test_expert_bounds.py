"""Bounds of groups that the operators over groups of rows have to take as they come (out of order, out
of range), against the formulas in 64 bits.  Tolerances as in test_grouped."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
from test_grouped import ACCUM, EVAL, NAN, _i32, _operand, _rows, _weights, backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


def _owners(bounds, M):
    """How many groups have each row."""
    n = torch.zeros(M, dtype=torch.int64)
    for g in range(len(bounds) - 1):
        n[_rows(bounds, g)] += 1
    return n


def _check_backward(gemm, offsets, M, N, K, act, give, t="bf16", in_place=None):
    """The gradients over groups of any offsets.  Rows of no group keep what they hold; da of rows that
    groups share is either's and not compared."""
    bounds = [min(max(o, 0), M) for o in offsets]
    E = len(offsets) - 1
    gen = torch.Generator().manual_seed(M + N + K + E)
    dd, DD = _operand(gen, M, N, t)
    z, Z = _operand(gen, M, N, t)
    a, A = _operand(gen, M, K, t)
    b, Bd = _weights(gen, E, N, K, t, scale=K ** -0.5)
    dz64, da64, db64, dbias64 = backward(dd, z, a, b, bounds, act, 1.0, lambda v: v.to(O.TYPES[t]).double())
    own = _owners(bounds, M)
    kept = {"dd": DD, "z": Z}.get(in_place)
    kept = O.f64(kept) if in_place else None
    out = {"dz": {None: None, "dd": (DD, None), "z": (Z, None)}[in_place] or
           O.strided(torch.full((M, N), NAN), t),
           "da": O.strided(torch.full((M, K), NAN), "f32"),
           "db": (torch.full((E, N, K), NAN, device="cuda"), None),
           "dbias": (torch.full((E, N), NAN, device="cuda"), None)}
    out = {k: v for k, v in out.items() if k in give}
    gemm.grouped_linear_bwd(DD, A if "db" in give else None, Bd if "da" in give else None, _i32(offsets),
                            z=Z if act != "none" else None, activation=act, **{k: v[0] for k, v in out.items()})
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    some, one = own > 0, own == 1
    smooth = act not in ("none", "relu")
    ez = dd.abs() * EVAL * smooth + dz64.abs() * O.U32
    # (a dz that rounds the other way differs by one step of its type)
    flip = torch.nan_to_num(ez + 2 * O.rounding(dz64.abs() + ez, t)) * smooth
    mag = torch.nan_to_num(dz64).abs()
    if "dz" in out:
        O.within(out["dz"][0][some.cuda()], dz64[some], (ez + O.rounding(dz64.abs() + ez, t))[some], "dz")
        rest = O.f64(out["dz"][0])[~some]
        assert torch.equal(rest, kept[~some]) if in_place else torch.isnan(rest).all()
    if "da" in out:
        got = O.f64(out["da"][0])
        for g in range(E):
            rows = torch.zeros(M, dtype=torch.bool)
            rows[_rows(bounds, g)] = True
            rows &= one
            S = mag[rows] @ b[g].abs()
            O.within(got[rows], da64[rows], S * (ACCUM + 4 * O.U32) + flip[rows] @ b[g].abs() +
                     O.rounding(da64[rows].abs(), "f32"), "da")
        assert torch.isnan(got[~some]).all() and O.padding_untouched(*out["da"])
    for g in range(E):
        r = _rows(bounds, g)
        if "db" in out:
            S = mag[r].T @ a[r].abs()
            O.within(out["db"][0][g], db64[g], S * (ACCUM + 4 * O.U32) + flip[r].T @ a[r].abs() +
                     O.rounding(db64[g].abs(), "f32"), f"db {g}")
        if "dbias" in out:
            n = r.stop - r.start
            O.within(out["dbias"][0][g], dbias64[g], ez[r].sum(0) + mag[r].sum(0) * (n + 8) * O.U32 +
                     O.rounding(dbias64[g].abs(), "f32"), f"dbias {g}")


OFFSETS = [[-5, 3, 70], [0, 200, 90], [10, 4, 4], [60, 20, 65], [64, 64, 64],
           [1 << 30, -(1 << 31), (1 << 31) - 1], [-9, -5, -1], [65, 0], [40, 65, 3, 9, 9, 20, 0, 2],
           [0, 50, 20, 60]]
PARTS = [("dz",), ("dz", "da"), ("dz", "db"), ("dz", "da", "db"), ("dz", "da", "db", "dbias")]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("give", PARTS)
@pytest.mark.parametrize("act", ["gelu", "none"])
def test_backward_offsets_out_of_order(gemm, offsets, give, act):
    """With a bias's gradient or without, a group has the rows that it has forward."""
    _check_backward(gemm, offsets, 65, 72, 64, act, give)


@pytest.mark.parametrize("give", PARTS)
def test_backward_offsets_out_of_order_of_many_rows(gemm, give):
    _check_backward(gemm, [500, 600, 100, 300, 300, 0, 50, 7, 1], 1000, 1003, 136, "silu", give, "f16")
    _check_backward(gemm, [0, 200, 90], 1000, 520, 72, "relu", give)


@pytest.mark.parametrize("turn", [0, 1, 1100, 2998])
def test_backward_offsets_out_of_order_somewhere(gemm, turn):
    """Of many groups one alone begins again from below, wherever it stands in their order."""
    offsets = [3000 - turn + i if i <= turn else i - turn - 1 for i in range(3001)]
    M = max(offsets) + 2
    for give in (("dz",), ("dz", "dbias")):
        _check_backward(gemm, offsets, M, 40, 8, "gelu_tanh", give)


@pytest.mark.parametrize("in_place", ["dd", "z"])
def test_backward_offsets_out_of_order_in_place(gemm, in_place):
    for offsets in ([60, 20, 55], [40, 65, 3, 9, 9, 20, 0, 2]):
        _check_backward(gemm, offsets, 65, 136, 72, "silu", ("dz", "da", "db"), in_place=in_place)
