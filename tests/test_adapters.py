"""Low-rank adapters of many requests: refusals (CPU) and the kernels against the formula in 64
bits.

Tolerance: u is off by 2^-10 of the sum of its terms' magnitudes (the bound of every product of this
library) and its rounding; the second product carries that on and adds 2^-10 of its own
terms; scale and residual add 4 u of the magnitudes, u = 2^-24; d is rounded once."""
import ctypes

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
import layer_oracle as O
from test_grouped import _bounds, _i32, _operand, _rows, _weights

NAN, INF, ACCUM = float("nan"), float("inf"), 2.0 ** -10


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


P = [(i + 1) << 20 for i in range(10)]     # fake, aligned device addresses
INVALID, DTYPE, ALIGN = (G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE,
                         G.GEMM_ERR_MISALIGNED)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(M=0, d=None, offsets=None, index=None), 0), (dict(N=0), 0), (dict(requests=0), 0),
    (dict(K=0, x=None, A=None), 0), (dict(rank=0, A=None, B=None, u=None), 0),
    (dict(adapters=0, A=None, B=None, u=None, x=None), 0), (dict(r=None, scale=None), 0),
    (dict(r=P[7]), 0), (dict(rank=5), 0), (dict(adapters=1, strideA=1, strideB=1), 0),
    (dict(d_type=G.GEMM_F32), 0), (dict(scale=P[4] + 4), 0),
    (dict(M=-1), INVALID), (dict(rank=-1), INVALID), (dict(requests=4097), INVALID),
    (dict(adapters=5000), INVALID), (dict(offsets=None), INVALID), (dict(index=None), INVALID),
    (dict(x=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(u=None), INVALID),
    (dict(d=None), INVALID), (dict(ldx=48), INVALID), (dict(ldu=0), INVALID), (dict(ldd=80), INVALID),
    (dict(ldr=80), INVALID), (dict(u=P[0]), INVALID), (dict(u=P[7]), INVALID), (dict(d=P[0]), INVALID),
    (dict(d=P[2]), INVALID), (dict(r=P[7], ldr=104), INVALID),
    (dict(r=P[7], r_type=G.GEMM_F16), INVALID),
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(type=G.GEMM_F32), DTYPE), (dict(d_type=3), DTYPE),
    (dict(r_type=4), DTYPE),
    (dict(x=P[0] + 8), ALIGN), (dict(lda=68), ALIGN), (dict(ldb=20), ALIGN), (dict(strideA=1028), ALIGN),
    (dict(strideB=-8), ALIGN), (dict(u=P[3] + 2), ALIGN), (dict(scale=P[4] + 2), ALIGN),
    (dict(offsets=P[5] + 1), ALIGN), (dict(index=P[6] + 2), ALIGN),
])
def test_check_adapters(lib, kw, code):
    base = dict(M=5, N=96, K=64, rank=16, requests=3, adapters=4, type=G.GEMM_BF16,
                r_type=G.GEMM_BF16, d_type=G.GEMM_BF16, offsets=P[5], index=P[6], x=P[0], ldx=64,
                A=P[1], lda=64, strideA=16 * 64, B=P[2], ldb=16, strideB=96 * 16, scale=P[4], u=P[3],
                ldu=16, r=P[8], ldr=96, d=P[7], ldd=96)
    assert G.gemm_adapters_check(G.gemm_adapters_t(**{**base, **kw})) == code


def test_packed_calls_match_the_structures():
    values = [i + 1 for i, _ in enumerate(G.gemm_adapters_t._fields_)]
    assert G._ADAPTERS.size == ctypes.sizeof(G.gemm_adapters_t)
    assert G._ADAPTERS.pack(*values) == bytes(G.gemm_adapters_t(*values))


def test_null_arguments(lib):
    assert lib.gemm_adapters(None, None, None) == INVALID
    assert lib.gemm_adapters_check(None) == INVALID


# ---------------------------------------------------------------- GPU

def _check(gemm, sizes, index, n, N, K, rank, t="bf16", r_t="bf16", d_t="bf16", scaled=True,
           in_place=False, before=0, behind=0, pad=16, seed=0):
    bounds = _bounds(None, sizes, before)
    M = bounds[-1] + behind
    gen = torch.Generator().manual_seed(seed + M + N + K + rank)
    x, X = _operand(gen, M, K, t, pad)
    a, A = _weights(gen, n, rank, K, t, False, pad, scale=max(1, K) ** -0.5)
    b, Bd = _weights(gen, n, N, rank, t, False, pad)
    r = torch.randn(M, N, generator=gen).to(O.TYPES[r_t]).double() if r_t else None
    scale = (0.5 + torch.rand(n, generator=gen)) if scaled else torch.ones(n)
    R = O.strided(r, r_t, pad) if r_t else None
    D = R if in_place else O.strided(torch.full((M, N), NAN), d_t, pad)
    u = O.strided(torch.full((M, rank), NAN), t, pad)
    gemm.adapters(X, A, Bd, _i32(bounds), _i32(index), u[0], D[0], residual=R[0] if R else None,
                  scale=scale.cuda() if scaled else None)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    assert O.padding_untouched(*u) and O.padding_untouched(*D)
    others = torch.ones(M, dtype=torch.bool)
    others[bounds[0]:bounds[-1]] = False
    for g, e in enumerate(index):
        rows = _rows(bounds, g)
        want = r[rows].clone() if r_t else torch.zeros(rows.stop - rows.start, N, dtype=torch.float64)
        err = torch.zeros_like(want)
        if 0 <= e < n:
            s = float(scale[e])
            u64 = x[rows] @ a[e].T
            eu = x[rows].abs() @ a[e].abs().T * ACCUM
            eu = eu + O.rounding(u64.abs() + eu, t)
            v, S = s * u64 @ b[e].T, s * (u64.abs() + eu) @ b[e].abs().T
            want = want + v
            err = s * eu @ b[e].abs().T + S * (ACCUM + 4 * O.U32) + want.abs() * 2 * O.U32
        O.within(D[0][rows], want, err + O.rounding(want.abs() + err, d_t), f"request {g}")
    if in_place:
        assert torch.equal(O.f64(D[0])[others], r[others])
    else:
        assert torch.isnan(O.f64(D[0])[others]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,n,N,K,rank", [
    ([1], 1, 8, 16, 1), ([1] * 64, 5, 520, 264, 16), ([1, 0, 3], 2, 72, 77, 8),
    ([5, 1, 200, 0, 31], 4, 264, 130, 12), ([300, 17], 3, 1003, 520, 64), ([129, 1, 1], 9, 257, 65, 128),
    ([70, 260], 2, 300, 136, 200)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_adapters(gemm, sizes, n, N, K, rank, t):
    index = [(3 * i) % (n + 1) - 1 for i in range(len(sizes))]
    _check(gemm, sizes, index, n, N, K, rank, t, r_t=t, d_t=t, behind=len(sizes) % 3)
    _check(gemm, sizes, [i % n for i in range(len(sizes))], n, N, K, rank, t, r_t=None, d_t="f32",
           scaled=False, before=2)
    _check(gemm, sizes, index, n, N, K, rank, t, r_t="f32", d_t="f32", in_place=True, before=1,
           behind=1, pad=0 if N % 16 == 0 else 16)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1), dict(cta_group=2), dict(cta_group=1, tile_n=128)])
@pytest.mark.parametrize("sizes,n,N,K,rank", [([1] * 40, 5, 520, 264, 16), ([1, 0, 3, 9], 2, 73, 77, 9),
                                              ([5, 1, 200, 0, 31], 4, 264, 130, 12)])
def test_adapters_on_the_matrix_units(gemm, cfg, sizes, n, N, K, rank):
    """Whatever the number of rows: a forced configuration takes the products over groups."""
    gemm.set_config(**cfg)
    try:
        index = [(3 * i) % (n + 1) - 1 for i in range(len(sizes))]
        for t, r_t, d_t in (("f16", "f16", "f16"), ("bf16", "f32", "bf16"), ("f16", None, "f32")):
            _check(gemm, sizes, index, n, N, K, rank, t, r_t=r_t, d_t=d_t, behind=2)
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[1] * 5, [0, 0, 4, 0], [2, 1, 0, 4], [5, 3, 4], [0] * 9 + [19], [13, 0, 0, 1]])
@pytest.mark.parametrize("N,K,rank", [(8, 8, 1), (300, 129, 7), (513, 4200, 16), (264, 520, 40),
                                      (100, 1000, 300), (257, 9000, 33)])
def test_adapters_of_few_rows(gemm, sizes, N, K, rank):
    """Few rows, of uneven shares: kernels of their own."""
    index = [(2 * i) % 4 - 1 for i in range(len(sizes))]
    _check(gemm, sizes, index, 3, N, K, rank, "f16", r_t="bf16", d_t="f32", before=1)
    _check(gemm, sizes, index, 3, N, K, rank, "bf16", r_t="bf16", d_t="bf16", in_place=True, behind=2)


@pytest.mark.gpu
@pytest.mark.parametrize("offsets", [[-5, 3, 7], [0, 9, 4], [10, 4, 4], [6, 2, 8],
                                     [1 << 30, -(1 << 31), (1 << 31) - 1]])
def test_adapters_offsets_out_of_range(gemm, offsets):
    M, N, K, rank = 8, 72, 64, 8
    gen = torch.Generator().manual_seed(5)
    x, X = _operand(gen, M, K, "f16")
    a, A = _weights(gen, 2, rank, K, "f16", scale=K ** -0.5)
    b, Bd = _weights(gen, 2, N, rank, "f16")
    for cfg in (None, dict(cta_group=1)):
        d, u = O.strided(torch.full((M, N), NAN), "f32"), O.strided(torch.zeros(M, rank), "f16")
        gemm.set_config(**cfg) if cfg else gemm.set_config(None)
        try:
            gemm.adapters(X, A, Bd, _i32(offsets), _i32([0, 1]), u[0], d[0])
            assert gemm.sync_status()[0] == G.GEMM_OK
        finally:
            gemm.set_config(None)
        clamped = [min(max(o, 0), M) for o in offsets]
        rest = torch.ones(M, dtype=torch.bool)
        for g in range(2):
            rest[clamped[g]:max(clamped[g], clamped[g + 1])] = False
        assert torch.equal(torch.isnan(O.f64(d[0])).all(dim=1), rest) and O.padding_untouched(*d)


@pytest.mark.gpu
@pytest.mark.parametrize("index", [[-1, -1], [7, 1 << 30], [-(1 << 31), 0]])
def test_requests_without_an_adapter(gemm, index):
    for r_t, in_place in (("bf16", False), ("bf16", True), (None, False)):
        _check(gemm, [3, 40], index, 2, 136, 72, 16, r_t=r_t, in_place=in_place, behind=4)


@pytest.mark.gpu
def test_no_adapters_no_rank_no_inner(gemm):
    """Nothing to add: d = r."""
    for n, rank, K in ((0, 16, 64), (2, 0, 64), (2, 16, 0)):
        e = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
        r = torch.randn(5, 40).half().cuda()
        d = torch.full((5, 40), NAN, device="cuda")
        gemm.adapters(e(5, K), e(n, rank, K), e(n, 40, rank), _i32([0, 2, 5]), _i32([0, 1]),
                      e(5, rank), d, residual=r)
        assert gemm.sync_status()[0] == G.GEMM_OK
        assert torch.equal(d, r.float())


@pytest.mark.gpu
def test_a_request_s_infinities_stay_its_own(gemm):
    x = torch.randn(6, 64).half().cuda()
    a, b = torch.randn(2, 8, 64).half().cuda(), torch.randn(2, 40, 8).half().cuda()
    a[1] = INF
    x[2:4] = NAN
    u, d = torch.zeros(6, 8).half().cuda(), torch.zeros(6, 40, device="cuda")
    gemm.adapters(x, a, b, _i32([0, 2, 3, 4, 6]), _i32([0, 1, -1, 0]), u, d)
    torch.cuda.synchronize()
    assert torch.isfinite(d[:2]).all() and torch.isfinite(d[4:]).all() and (d[:2] != 0).any()
    assert torch.isnan(d[2]).all() and not d[3].any()


@pytest.mark.gpu
def test_beside_a_shared_layer_in_a_graph(gemm):
    """The layer's output is adapted in place; the graph follows the requests."""
    M, N, K, rank, n = 40, 264, 136, 16, 3
    gen = torch.Generator().manual_seed(3)
    x, X = _operand(gen, M, K, "bf16")
    w, W = _operand(gen, N, K, "bf16", scale=K ** -0.5)
    a, A = _weights(gen, n, rank, K, "bf16", scale=K ** -0.5)
    b, Bd = _weights(gen, n, N, rank, "bf16")
    u, d = torch.zeros(M, rank).bfloat16().cuda(), torch.empty(M, N, device="cuda")
    off, idx = _i32([0, 10, 20, 40]), _i32([0, 1, 2])

    def step(stream=None):
        gemm.linear(X, W, d, stream=stream)
        gemm.adapters(X, A, Bd, off, idx, u, d, residual=d, stream=stream)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for bounds, index in (([0, 1, 39, 40], [2, -1, 1]), ([0, 0, 40, 40], [1, 0, 2])):
        off.copy_(_i32(bounds))
        idx.copy_(_i32(index))
        graph.replay()
        torch.cuda.synchronize()
        want = x @ w.T
        err = x.abs() @ w.abs().T * (ACCUM + 4 * O.U32)
        for g, e in enumerate(index):
            rows = _rows(bounds, g)
            if e >= 0:
                u64 = x[rows] @ a[e].T
                eu = x[rows].abs() @ a[e].abs().T * ACCUM
                eu = eu + O.rounding(u64.abs() + eu, "bf16")
                want[rows] += u64 @ b[e].T
                err[rows] += eu @ b[e].abs().T + (u64.abs() + eu) @ b[e].abs().T * (ACCUM + 4 * O.U32)
        O.within(d, want, err + O.rounding(want.abs() + err, "f32"), "d")


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [255, 256, 257, 1000, 1024, 1025])
@pytest.mark.parametrize("sizes,N,K", [([1, 1], 264, 136), ([0, 3, 1], 77, 40), ([1], 2310, 8)])
def test_adapters_of_few_rows_and_large_ranks(gemm, sizes, N, K, rank):
    index = [(i + 1) % 2 for i in range(len(sizes))]
    _check(gemm, sizes, index, 2, N, K, rank, t="f16", r_t="f32", d_t="bf16", before=1, behind=2)


@pytest.mark.gpu
def test_adapters_in_place_by_either_way_agree(gemm):
    """d on r, requests without an adapter among them: by the kernel of few rows and by products the
    results are the same but for the order of the sums (each within 2^-10 of its terms)."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    x, a, b, r = rnd(40, 520), rnd(5, 24, 520), rnd(5, 1032, 24), rnd(40, 1032).float()
    index = torch.randint(-1, 5, (40,), generator=gen, device="cuda", dtype=torch.int32)
    bounds, u, got = _i32(list(range(41))), torch.empty(40, 24, device="cuda").bfloat16(), []
    for cfg in (None, dict(cta_group=1)):
        gemm.set_config(**cfg) if cfg else gemm.set_config(None)
        d = r.clone()
        gemm.adapters(x, a, b, bounds, index, u, d, residual=d)
        assert gemm.sync_status()[0] == G.GEMM_OK
        got.append(d)
    gemm.set_config(None)
    none = index < 0
    assert torch.equal(got[0][none], r[none]) and torch.equal(got[1][none], r[none])
    # |u| terms: 24 of |x a| sums, each off by 2^-10 of 520 terms of about 0.64 and a rounding
    size = torch.einsum("mk,mrk->mr", x.double().abs(), a[index.clamp(min=0).long()].double().abs())
    mag = torch.einsum("mr,mnr->mn", size, b[index.clamp(min=0).long()].double().abs())
    assert ((got[0] - got[1]).double().abs() <= mag * (2 * 2.0 ** -10 + 2 * 2.0 ** -8) + 1e-6).all()
