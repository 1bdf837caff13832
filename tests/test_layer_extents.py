"""The layer operators past 2^31 elements a tensor, checked on the first, middle and last
rows (those past 2^31 among them), and with a row stride that alone exceeds 2^31 bytes.
Tolerances as in test_norm.py and test_linear.py."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O

pytestmark = pytest.mark.gpu
ROWS, COLS = 270_000, 8192                       # 2.2e9 elements
PICK = [0, 1, 131_071, 131_072, 262_143, 262_144, 262_145, ROWS - 1]


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    h = G.Gemm(0)
    yield h
    h.close()
    torch.cuda.empty_cache()


def _big(seed, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(ROWS, COLS, dtype=dtype, device="cuda")
    for i in range(0, ROWS, 30_000):
        t[i:i + 30_000] = torch.randn(min(30_000, ROWS - i), COLS, generator=gen, device="cuda")
    return t


def test_normalisation_and_its_gradient(gemm):
    x = _big(1)
    w = torch.linspace(0.5, 1.5, COLS, device="cuda").bfloat16()
    q = torch.empty(ROWS, COLS, dtype=torch.float8_e4m3fn, device="cuda")
    scale, rstd = torch.empty(ROWS, device="cuda"), torch.empty(ROWS, device="cuda")
    gemm.rmsnorm(x, w, q, scale=scale, rstd=rstd)
    h, r64, y64 = O.rmsnorm(O.f64(x[PICK]), None, O.f64(w), 1e-6)
    e = ((COLS / 32 + 45) / 2 + 6) * O.U32
    O.within(rstd[PICK], r64, r64 * e, "rstd")
    s64 = y64.abs().amax(dim=1) / 448.0
    q64 = y64 / s64[:, None]
    got = torch.stack([q[i].float() for i in PICK])
    O.within(got, q64, O.rounding(q64, "e4m3") * (1 + 4 * e) + q64.abs() * 3 * e, "q")
    del q
    dy = _big(2)
    dx, dw = torch.empty_like(x), torch.empty(COLS, device="cuda")
    ws = torch.empty(G.gemm_rmsnorm_bwd_workspace(ROWS, COLS), dtype=torch.uint8, device="cuda")
    gemm.rmsnorm_bwd(dy, x, w, rstd, dx, dw, workspace=ws)
    d = O.f64(dy[PICK])
    dx64, _ = O.rmsnorm_bwd(d, h, O.f64(w), O.f64(rstd[PICK]), None)
    n, g = h * O.f64(rstd[PICK])[:, None], d * O.f64(w)
    size = O.f64(rstd[PICK])[:, None] * (g.abs() + 2 * n.abs() * (g * n).abs().mean(1, keepdim=True))
    err = size * (COLS / 32 + 53) * O.U32
    O.within(dx[PICK], dx64, O.rounding(dx64.abs() + err, "bf16") + err, "dx")
    # column sums in 64 bits on the GPU, a part of the rows at a time
    want = torch.zeros(COLS, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(0, ROWS, 10_000):
        t = dy[i:i + 10_000].double() * x[i:i + 10_000].double() * rstd[i:i + 10_000, None].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    # a thread's chain holds at most 1800 rows (152 blocks), the rest are 304 block sums
    O.within(dw, O.f64(want), O.f64(size) * 2200 * O.U32, "dweight")


def test_linear_and_the_activation_gradient(gemm):
    K = 64
    gen = torch.Generator().manual_seed(3)
    a, b = torch.randn(ROWS, K, generator=gen).half(), torch.randn(COLS, K, generator=gen).half()
    r = _big(4, torch.float16)
    d, z = (torch.empty(ROWS, COLS, dtype=torch.float16, device="cuda") for _ in range(2))
    gemm.linear(a.cuda(), b.cuda(), d, residual=r, z=z, activation="silu")
    assert gemm.sync_status()[0] == G.GEMM_OK
    z64 = a[PICK].double() @ b.double().T
    ez = a[PICK].double().abs() @ b.double().abs().T * (2.0 ** -10 + 6 * O.U32)
    O.within(z[PICK], z64, ez + O.rounding(z64.abs() + ez, "f16"), "z")
    d64 = O.act(z64, "silu") + O.f64(r[PICK])
    ed = ez * 1.13 + 2.0 ** -21 * z64.abs().clamp(min=1.0) + d64.abs() * 2 * O.U32
    O.within(d[PICK], d64, ed + O.rounding(d64.abs() + ed, "f16"), "d")
    del d
    # dz over z, dd = r
    zs, rs = O.f64(z[PICK]), O.f64(r[PICK])
    gemm.linear_bwd(r, a.cuda(), b.cuda(), z=z, activation="silu", dz=z)
    dz64 = rs * O.act_grad(zs, "silu")
    e = rs.abs() * 2.0 ** -20 + dz64.abs() * 2 * O.U32
    O.within(z[PICK], dz64, e + O.rounding(dz64.abs() + e, "f16"), "dz")


@pytest.mark.parametrize("M", [2, 40])
def test_row_strides_past_2_31_bytes(gemm, M):
    """A few rows of a tensor whose rows are 2.2 GB apart (M = 40 is 88 GB of address range:
    only where the memory is free)."""
    stride, N, K = 1_100_000_000 // 16 * 16, 200, 128
    if torch.cuda.mem_get_info()[0] < (M * stride * 2) + (8 << 30):
        pytest.skip("not enough free device memory")
    buf = torch.empty(M * stride, dtype=torch.float16, device="cuda")
    d = torch.as_strided(buf, (M, N), (stride, 1))
    gen = torch.Generator().manual_seed(M)
    a, b = torch.randn(M, K, generator=gen).half(), torch.randn(N, K, generator=gen).half()
    gemm.linear(a.cuda(), b.cuda(), d)
    want = a.double() @ b.double().T
    err = a.double().abs() @ b.double().abs().T * (2.0 ** -10 + 6 * O.U32)
    O.within(d, want, err + O.rounding(want.abs() + err, "f16"), "d")
    x = torch.randn(M, N, generator=gen).half()
    gemm.rmsnorm(x.cuda(), torch.ones(N, device="cuda"), d)
    y64 = O.rmsnorm(x.double(), None, torch.ones(N, dtype=torch.float64), 1e-6)[2]
    e = ((N / 32 + 45) / 2 + 6) * O.U32
    O.within(d, y64, O.rounding(y64, "f16") * (1 + 2 * e) + y64.abs() * e, "y")
    del buf, d
    torch.cuda.empty_cache()
