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
