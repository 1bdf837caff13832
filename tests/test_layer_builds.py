"""The layer operators in the library's other builds, each in a subprocess so that the test
process keeps the product library: against 64 bits, as in test_linear and test_norm, in
the debug build (whose checks of shared-memory ranges, tensor-memory columns, coordinates,
exchanged pieces and register stores all hold) and in the one without multicast; and the ring
statistics of the layer's launches."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
kind = sys.argv[1]
sys.path.insert(0, "tests")
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind=kind))
import test_linear as L
import test_norm as N
g = G.Gemm(0)
n = 0
def run(check, *args, cfg=None, **kw):
    global n
    g.set_config(**cfg) if cfg else g.set_config(None)
    check(g, *args, **kw)
    st, detail = g.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail), args, cfg)
    n += 1
# the layer: automatic, then every kind of tile of both kernels, row ends inside a piece
for M, N_, K in ((1, 257, 129), (17, 100, 300), (129, 257, 65), (513, 771, 129), (300, 520, 0)):
    for ab in ("bf16", "e4m3", "tf32"):
        run(L._check_forward, M, N_, K, ab, d_t="f16", act="gelu", r_t="bf16", z_t="f32",
            scales=ab == "e4m3")
for cfg in (dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=256), dict(cta_group=2, tile_n=96),
            dict(cta_group=2, tile_n=256), dict(cta_group=2, tile_n=128, epi_warps=1),
            dict(cta_group=2, tile_n=224, epi_warps=2)):
    run(L._check_forward, 1000, 1003, 136, "bf16", cfg=cfg, act="silu", r_t="f32", z_t="bf16")
    run(L._check_forward, 1000, 1003, 136, "bf16", cfg=cfg, bias_t=None, r_t="bf16", in_place=False)
    if cfg["tile_n"] // cfg["cta_group"] % 64 == 0:      # (whole atoms of MN-major operands)
        run(L._check_backward, 1500, 1100, 301, "bf16", "none", cfg=cfg, db_t="f32",
            accumulate=True, give=("da", "db"))
for bn, split in ((16, 1), (16, 8), (48, 5), (64, 7), (96, 8), (128, 1), (128, 8)):
    for ab in ("bf16", "e4m3", "tf32"):
        run(L._check_forward, bn + 3, 203, 1100, ab, cfg=dict(split_k=split, tile_n=bn), act="gelu",
            r_t="bf16", z_t="f32", scales=True)
for feats in (8, 56, 120):
    run(L._check_forward, 60, 203, 1100, "f16", cfg=dict(split_k=4, tile_n=64, tile_m=feats), r_t="f32")
for a_mn, b_mn in ((True, False), (False, True), (True, True)):
    run(L._check_forward, 150, 203, 1100, "f16", cfg=dict(split_k=3, tile_n=128), a_mn=a_mn, b_mn=b_mn)
    run(L._check_forward, 260, 264, 100, "f16", a_mn=a_mn, b_mn=b_mn)
for M, N_, K in ((3, 77, 130), (130, 257, 129), (300, 1003, 520), (2049, 136, 264)):
    run(L._check_backward, M, N_, K, "f16", "gelu")
for M, H in ((3, 7), (5, 1031), (300, 520), (2, 40001)):
    run(N._check_forward, *N._inputs(M, H, "bf16", M + H), "bf16", "e4m3")
    run(N._check_backward, M, H, "bf16")
g.close()
maps = open("/proc/self/maps").read()
assert f"libgemm_gb300_{kind}.so" in maps and "libgemm_gb300.so" not in maps
print("BUILD_OK", n)
'''


@pytest.mark.parametrize("kind", ["debug", "nomc"])
def test_layer_operators_in_another_build(kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD, kind], cwd=ROOT, capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0 and "BUILD_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


STATS = r'''
import sys
sys.path.insert(0, "tests")
import torch
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind="stats"))
g = G.Gemm(0)
one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
cdiv = lambda a, b: -(-a // b)

def stages():
    """Ring stages the last launch issued, and every wait within its loop."""
    rows = g.ring_stats()
    for r in rows:
        assert r[0] + r[1] <= r[2], r
    return sum(r[3] for r in rows), len(rows)

for M, N, K, cfg in ((700, 1000, 300, None), (300, 520, 1000, dict(cta_group=1, tile_n=128, tail_split=1)),
                     (1000, 1500, 136, dict(cta_group=2, tile_n=256, tail_split=1)), (300, 520, 0, None)):
    for act in (None, "gelu"):                 # (no bias, no activation: the kernel of two products)
        g.set_config(**cfg) if cfg else g.set_config(None)
        pad = max(8, cdiv(K, 8) * 8)
        g.linear(one(M, pad)[:, :K], one(N, pad)[:, :K], one(M, cdiv(N, 8) * 8)[:, :N], activation=act)
        c = g.last_config()
        items = c.tiles + c.tail_split
        got, n = stages()
        assert n == c.grid_ctas and got == items * cdiv(K, c.tile_k), (got, items, c.as_dict())
g.set_config(cta_group=2, tile_n=256, tail_split=1)
M, N, K = 1000, 1500, 136
g.linear_bwd(one(M, N + 4)[:, :N], one(M, K), one(N, K), da=one(M, K), db=one(N, K))
c = g.last_config()
want = cdiv(M, 256) * cdiv(K, 256) * cdiv(N, c.tile_k) + cdiv(N, 256) * cdiv(K, 256) * cdiv(M, c.tile_k)
assert stages() == (want, c.grid_ctas), (stages(), want)
g.set_config(split_k=2)
g.linear(one(4, 512), one(256, 512), one(4, 256))
assert g.ring_stats() == [] and g.sync_status()[0] == G.GEMM_OK
g.set_config(None)
g.close()
print("STATS_OK")
'''


def test_ring_statistics_count_the_layer_s_stages():
    """Each launch's own counters: as many stages as its items have k-blocks; none of a split-K
    launch."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", STATS], cwd=ROOT, capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0 and "STATS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
