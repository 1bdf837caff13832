"""What a handle reports of its latest product when the adapters of few rows, a kernel without tiles and
counters, came after it; and further forms of the gradients, and bounds, in the debug build."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STATS = r'''
import torch
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind="stats"))
g = G.Gemm(0)
one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
none = G.gemm_config_t()
for rows in (2, 300):                    # by the kernel of few rows, by products
    g.linear(one(300, 136), one(264, 136), one(300, 264))
    assert len(g.ring_stats()) == g.last_config().grid_ctas > 0
    g.adapters(one(rows, 136), one(2, 16, 136), one(2, 264, 16), i32(0, 1, rows), i32(1, 0), one(rows, 16),
               one(rows, 264))
    assert g.ring_stats() == [], rows
    c = g.last_config()
    assert (c.tile_n == 0 and bytes(c) == bytes(none)) if rows == 2 else c.tile_n > 0, rows
    # a call with nothing to do is no launch
    g.linear(one(300, 136), one(264, 136), one(300, 264))
    g.adapters(one(0, 136), one(2, 16, 136), one(2, 264, 16), i32(0, 0), i32(1), one(0, 16), one(0, 264))
    assert len(g.ring_stats()) == g.last_config().grid_ctas > 0
assert g.sync_status()[0] == G.GEMM_OK
g.close()
print("STATS_OK")
'''


def test_reports_after_adapters():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", STATS], cwd=ROOT, capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0 and "STATS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


DEBUG = r'''
import sys
sys.path.insert(0, "tests")
import torch
import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
G.select_library(B.build(kind=sys.argv[1]))
import test_expert_bounds as L
import test_grouped as F
g = G.Gemm(0)
for sizes, N, K in (([1], 8, 1), ([3, 0, 40], 129, 77), ([300, 0, 65, 513], 520, 701)):
    for cfg in (None, dict(cta_group=1, tile_n=64), dict(cta_group=2, tile_n=256)):
        g.set_config(**cfg) if cfg else g.set_config(None)
        F._check_backward(g, sizes, N, K, "bf16", "gelu", db_t="bf16", accumulate=True)
g.set_config(None)
for offsets in ([60, 20, 65], [0, 200, 90], [40, 65, 3, 9, 9, 20, 0, 2]):
    for give in (("dz", "da", "db"), ("dz", "da", "db", "dbias")):
        L._check_backward(g, offsets, 65, 136, 72, "silu", give)
st, detail = g.sync_status()
assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
g.close()
maps = open("/proc/self/maps").read()
assert f"libgemm_gb300_{sys.argv[1]}.so" in maps and "libgemm_gb300.so" not in maps
print("BUILD_OK")
'''


@pytest.mark.parametrize("kind", ["debug", "nomc"])
def test_gradients_in_another_build(kind):
    """Odd gradients added to in 16 bits, and offsets out of order, with every access checked."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", DEBUG, kind], cwd=ROOT, capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0 and "BUILD_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
