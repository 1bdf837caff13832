"""Values of the low-rank adapters and of weight gradients over groups that the other tests' bounds and
shapes let through.  Tolerances as in test_adapters and test_grouped."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
import layer_oracle as O
import test_adapters as A
from test_grouped import ACCUM, NAN, _i32, _operand, _rows, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


@pytest.mark.parametrize("t,bits", [(torch.bfloat16, 8), (torch.float16, 11)])
@pytest.mark.parametrize("rank", [1, 5, 16, 40, 300])
def test_few_rows_keep_u_in_32_bits(gemm, t, bits, rank):
    """u of a few rows goes through no workspace and is not rounded: of powers of two whose sum has a bit more than
    the type holds, and B a unit vector, d is u itself."""
    M, K, N = 3, 72, 40
    x = torch.zeros(M, K, dtype=t, device="cuda")
    x[:, 0] = x[:, 65] = 1.0
    a = torch.zeros(2, rank, (K + 7) // 8 * 8, dtype=t, device="cuda")[:, :, :K]
    j = torch.arange(rank, device="cuda")
    a[:, :, 0], a[:, :, 65] = 2.0 ** (j % 3).float(), 2.0 ** (j % 3 - bits).float()
    b = torch.zeros(2, N, (rank + 7) // 8 * 8, dtype=t, device="cuda")[:, :, :rank]
    n = torch.arange(N, device="cuda")
    b[:, n, n % rank] = 1.0
    u = torch.full((M, (rank + 7) // 8 * 8), NAN, dtype=t, device="cuda")[:, :rank]
    d = torch.full((M, N), NAN, device="cuda")
    gemm.adapters(x, a, b, _i32([0, 1, 2, 3]), _i32([1, 0, 1]), u, d)
    assert gemm.sync_status()[0] == G.GEMM_OK
    want = 2.0 ** (n % rank % 3).double() * (1.0 + 2.0 ** -bits)
    assert (want.to(t).double() != want).all()
    assert torch.equal(d.double(), want.expand(M, N))
