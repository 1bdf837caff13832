"""The linear layer's two gradients in one launch, and its products with nothing behind
them, which run on the same kernel, against 64 bits (tolerances as in test_linear): either product first, several rounds of tiles, extra rounds for the
clusters with one tile less, half-width last rounds, every tile shape, and rows
that end inside a 16-byte piece."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
from test_linear import _check_backward, _check_forward


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


def _tiles(M, N, K, cfg):
    cdiv = lambda a, b: -(-a // b)
    return (cdiv(M, cfg.tile_m) + cdiv(N, cfg.tile_m)) * cdiv(K, cfg.tile_n)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [
    (128, 8, 8), (128, 1000, 40), (200, 520, 1100), (1001, 300, 77), (1300, 700, 1500),
    (500, 1800, 1000), (2600, 260, 900), (1920, 1920, 520)])
@pytest.mark.parametrize("da_t,db_t,add", [("f16", "f16", False), ("f16", "f32", True),
                                           ("f32", "f16", True), ("bf16", "f32", False)])
def test_both_gradients(gemm, M, N, K, da_t, db_t, add):
    _check_backward(gemm, M, N, K, "f16", "silu", da_t=da_t, db_t=db_t, accumulate=add)
    cfg = gemm.last_config()
    if M > 200 and not cfg.split_k:  # (few tokens or features: each may have its own launch)
        assert cfg.tiles == _tiles(M, N, K, cfg)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [
    dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=64, epi_warps=1),
    dict(cta_group=1, tile_n=128), dict(cta_group=1, tile_n=192), dict(cta_group=1, tile_n=256),
    dict(cta_group=2, tile_n=128, epi_warps=1), dict(cta_group=2, tile_n=128),
    dict(cta_group=2, tile_n=256, epi_warps=1), dict(cta_group=2, tile_n=256),
    dict(cta_group=2, tile_n=256, tail_split=1), dict(cta_group=1, tile_n=128, stages=2)])
@pytest.mark.parametrize("M,N,K,db_t,add", [(1500, 1100, 1301, "f32", True),
                                            (700, 2900, 900, "bf16", False)])
def test_forced_tiles(gemm, cfg, M, N, K, db_t, add):
    gemm.set_config(**cfg)
    try:
        _check_backward(gemm, M, N, K, "bf16", "none", db_t=db_t, accumulate=add, alpha=0.5,
                        give=("da", "db"))
        last = gemm.last_config()
        assert last.tiles == _tiles(M, N, K, last)
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
def test_watchdog_ends_stalled_gradients():
    """An injected stall with a 100 ms limit: the launch ends by itself and the next computes."""
    g = G.Gemm(0)
    try:
        G.gemm_set_timeout_ns(g.handle, 100_000_000)
        g.set_config(inject_stall=1)
        one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
        dd, a, b, da, db = one(256, 512), one(256, 136), one(512, 136), one(256, 136), one(512, 136)
        g.linear_bwd(dd, a, b, da=da, db=db)
        st, detail = g.sync_status()
        assert st == G.GEMM_ERR_DEVICE_TIMEOUT and (detail >> 24) == 0xE0, hex(detail)
        G.gemm_set_timeout_ns(g.handle, 0)
        g.set_config(None)
        g.linear_bwd(dd, a, b, da=da, db=db)
        assert g.sync_status()[0] == G.GEMM_OK and (da == 512).all() and (db == 256).all()
    finally:
        g.close()


@pytest.mark.gpu
def test_plans_of_one_shape_do_not_reach_another(gemm):
    """Layers planned on different kernels in turn, then one with a forced tile: each by its
    own plan."""
    for _ in range(3):
        for M in (1, 300, 16, 1000, 64, 130):
            _check_forward(gemm, M, 520, 264, "bf16")
        for M in (3, 200, 700):
            _check_backward(gemm, M, 264, 136)
    for M in (2, 40, 900):
        gemm.set_config(cta_group=2, tile_n=96)
        try:
            for N in range(100, 420, 20):
                _check_forward(gemm, M, N, 72, "bf16")
        finally:
            gemm.set_config(None)
        for N in range(100, 420, 20):
            _check_forward(gemm, M, N, 72, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 7, 8, 9, 31, 33, 60, 63, 65, 97, 127, 130, 255, 260])
@pytest.mark.parametrize("d_t,z_t", [("f16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_rows_ending_inside_a_piece(gemm, N, d_t, z_t):
    """Every place of a row's end in a 32-column chunk's pieces; the row's padding is kept."""
    gemm.set_config(cta_group=1, tile_n=64)
    try:
        _check_forward(gemm, 150, N, 40, "f16", d_t=d_t, z_t=z_t, act="gelu", r_t="f16")
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(300, 1003, 520), (1200, 1100, 64), (2100, 700, 301), (150, 7, 8),
                                   (129, 4000, 1)])
@pytest.mark.parametrize("ab,d_t,r_t", [("bf16", "bf16", None), ("f16", "f32", None),
                                        ("bf16", "f16", "f32"), ("f16", "f32", "bf16")])
def test_products_with_nothing_behind(gemm, M, N, K, ab, d_t, r_t):
    _check_forward(gemm, M, N, K, ab, d_t=d_t, bias_t=None, r_t=r_t, alpha=0.75)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=256),
                                 dict(cta_group=2, tile_n=96), dict(cta_group=2, tile_n=256),
                                 dict(cta_group=2, tile_n=128, epi_warps=1)])
def test_products_with_nothing_behind_forced(gemm, cfg):
    """One shape through both kernels in turn: each by its own plan."""
    gemm.set_config(**cfg)
    try:
        for bias_t, r_t in ((None, None), ("f32", None), (None, "bf16"), ("bf16", "bf16")):
            _check_forward(gemm, 1000, 1500, 136, "bf16", bias_t=bias_t, r_t=r_t,
                           in_place=r_t is not None)
    finally:
        gemm.set_config(None)
