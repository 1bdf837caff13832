"""The operators whose weights change from row to row in the library's other builds, each in a
subprocess so that the test process keeps the product library: against 64 bits, as in
test_grouped, test_adapters and test_routing, in the debug build (whose checks of
shared-memory ranges, tensor-memory columns, coordinates and stores all hold) and in the one
without multicast; and the ring statistics, which count none of their launches."""
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
import torch
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind=kind))
import test_adapters as A
import test_grouped as L
import test_routing as R
g = G.Gemm(0)
n = 0
def run(check, *args, cfg=None, **kw):
    global n
    g.set_config(**cfg) if cfg else g.set_config(None)
    check(g, *args, **kw)
    st, detail = g.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail), args, cfg)
    n += 1
# the whole epilogue, of each operand type; the lean ones, of each type, residuals and odd widths
for sizes, N, K in (([1], 257, 129), ([1, 6, 0, 17], 100, 300), ([40, 7, 200], 257, 65), ([300, 513], 771, 129),
                    ([3, 2], 72, 0)):
    for ab in ("bf16", "e4m3", "tf32"):
        run(L._check_forward, sizes, N, K, ab, d_t="f16", act="gelu", r_t="bf16", z_t="f32", bias_t="f16",
            scales=ab == "e4m3")
    for d_t, r_t in (("bf16", "bf16"), ("f16", None), ("f32", "f32")):
        run(L._check_forward, sizes, N, K, "bf16", d_t=d_t, r_t=r_t, before=3, behind=5)
        run(L._check_forward, sizes, N + 1, K, "bf16", d_t=d_t, r_t=r_t)
    run(L._check_forward, sizes, N, K, "f16", d_t="f16", b_mn=True)
for cfg in (dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=256), dict(cta_group=2, tile_n=64),
            dict(cta_group=2, tile_n=128, stages=2), dict(cta_group=2, tile_n=256)):
    run(L._check_forward, [300, 0, 5, 129, 400], 520, 264, "bf16", cfg=cfg, act="silu", r_t="f32", z_t="bf16")
    run(L._check_forward, [300, 0, 5, 129, 400], 520, 264, "f16", cfg=cfg, d_t="f16")
    if cfg["tile_n"] // cfg["cta_group"] % 64 == 0:      # (whole atoms of MN-major operands)
        for db_t, odd in (("f32", 0), ("bf16", 0), ("bf16", 1)):
            run(L._check_backward, [300, 0, 5, 129, 400], 520, 264 + odd, cfg=cfg, act="gelu", db_t=db_t,
                accumulate=not odd)
for rows in (1, 15, 16, 17, 127, 128, 129, 143, 144, 145):
    run(L._check_backward, [rows, 3], 136, 72, "f16", da_t="f16", db_t="f16", act="relu")
# adapters: by the kernels for few rows and by products
for sizes in ([1] * 5, [13, 0, 0, 1], [100, 0, 3, 400]):
    for N, K, rank in ((300, 129, 7), (513, 1100, 16), (264, 520, 40), (520, 136, 300)):
        index = [(5 * i) % 4 - 1 for i in range(len(sizes))]
        run(A._check, sizes, index, 3, N, K, rank)
# sorting and back
for T, k, E in ((1, 8, 64), (33, 3, 7), (5000, 2, 300), (70, 2, 4096)):
    gen = torch.Generator().manual_seed(T)
    run(R._check_route, torch.randint(-1, E + 1, (T, k), generator=gen), E)
for T, k, H, r_t in ((33, 3, 1031, "f32"), (2100, 2, 4136, "bf16"), (800, 8, 2571, "f16")):
    run(R.test_combine, T, k, H, "bf16", r_t, "bf16", True)
    run(R.test_combine_bwd, T, k, H, "bf16", True)
g.close()
maps = open("/proc/self/maps").read()
assert f"libgemm_gb300_{kind}.so" in maps and "libgemm_gb300.so" not in maps
print("BUILD_OK", n)
'''


@pytest.mark.parametrize("kind", ["debug", "nomc"])
def test_operators_in_another_build(kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD, kind], cwd=ROOT, capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0 and "BUILD_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


STATS = r'''
import torch
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind="stats"))
g = G.Gemm(0)
one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
bounds = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
for call in (lambda: g.grouped_linear(one(300, 136), one(2, 264, 136), bounds, one(300, 264)),
             lambda: g.grouped_linear_bwd(one(300, 264), one(300, 136), one(2, 264, 136), bounds,
                                          da=one(300, 136), db=one(2, 264, 136)),
             lambda: g.adapters(one(300, 136), one(2, 16, 136), one(2, 264, 16), bounds, which,
                                one(300, 16), one(300, 264))):
    g.linear(one(300, 136), one(264, 136), one(300, 264))
    assert len(g.ring_stats()) == g.last_config().grid_ctas
    call()
    assert g.ring_stats() == []
assert g.sync_status()[0] == G.GEMM_OK
g.close()
print("STATS_OK")
'''


def test_ring_statistics_of_uncounted_launches():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", STATS], cwd=ROOT, capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0 and "STATS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
