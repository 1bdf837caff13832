"""The linear layer and its backward pass: refusals (CPU), the 64-bit formulas
against differences (CPU), and the kernels against them.

Tolerances.  A product's fp32 accumulation is off by at most 2^-10 of the sum of
its terms' magnitudes (the bound every product of this library is held to), S
below; the scales' and bias's arithmetic by at most 6 u of S and the bias, u = 2^-24.  An
activation of slope at most 1.13 carries an error of z on at 1.13 times its size,
and its own evaluation is off by at most 2^-21 of max(1, |z|): the exponential's
2^-22 and the published 1.5e-7 of the distribution function.  Results are rounded
once."""
import ctypes
import itertools

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
import layer_oracle as O

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
SLOPE, EVAL, ACCUM = 1.13, 2.0 ** -21, 2.0 ** -10


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


# ---------------------------------------------------------------- CPU

P = [(i + 1) << 20 for i in range(10)]     # fake, aligned device addresses
INVALID, DTYPE, ALIGN = (G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE,
                         G.GEMM_ERR_MISALIGNED)


def _fwd(**kw):
    base = dict(M=5, N=96, K=64, a_type=G.GEMM_E4M3, b_type=G.GEMM_E5M2, bias_type=G.GEMM_F32,
                r_type=G.GEMM_BF16, z_type=G.GEMM_F16, d_type=G.GEMM_BF16,
                activation=G.GEMM_ACT_GELU, alpha=1.0, A=P[0], lda=64, B=P[1], ldb=64,
                row_scale=P[2], col_scale=P[3], bias=P[4], R=P[5], ldr=96, Z=P[6], ldz=96,
                D=P[7], ldd=96)
    base.update(kw)
    return G.gemm_linear_t(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(M=0, A=None, D=None), 0), (dict(N=0), 0), (dict(K=0, A=None, B=None), 0),
    (dict(R=None, Z=None, bias=None, row_scale=None, col_scale=None), 0),
    (dict(R=P[7]), 0), (dict(bias=P[4] + 4), 0), (dict(N=95, K=61, M=1), 0),
    (dict(a_type=G.GEMM_TF32, b_type=G.GEMM_TF32), 0),
    (dict(layoutA=G.GEMM_MN_MAJOR, lda=16, layoutB=G.GEMM_MN_MAJOR, ldb=96), 0),
    (dict(M=-1), INVALID), (dict(K=1 << 31), INVALID), (dict(A=None), INVALID),
    (dict(D=None), INVALID), (dict(lda=48), INVALID), (dict(ldd=88), INVALID),
    (dict(ldz=80), INVALID), (dict(layoutA=2), INVALID), (dict(activation=5), INVALID),
    (dict(activation=-1), INVALID), (dict(R=P[7], ldr=104), INVALID),
    (dict(R=P[7], r_type=G.GEMM_F16), INVALID), (dict(Z=P[7]), INVALID), (dict(Z=P[5]), INVALID),
    (dict(D=P[0]), INVALID), (dict(Z=P[1]), INVALID), (dict(ldb=1 << 40), INVALID),
    (dict(a_type=G.GEMM_F16), DTYPE), (dict(a_type=G.GEMM_F32, b_type=G.GEMM_F32), DTYPE),
    (dict(a_type=G.GEMM_F16, b_type=G.GEMM_BF16), DTYPE), (dict(d_type=G.GEMM_E4M3), DTYPE),
    (dict(r_type=G.GEMM_E4M3), DTYPE), (dict(bias_type=G.GEMM_TF32), DTYPE),
    (dict(z_type=9), DTYPE),
    (dict(a_type=G.GEMM_TF32, b_type=G.GEMM_TF32, layoutB=G.GEMM_MN_MAJOR), DTYPE),
    (dict(A=P[0] + 8), ALIGN), (dict(lda=72), ALIGN), (dict(D=P[7] + 2), ALIGN),
    (dict(ldd=100), ALIGN), (dict(ldr=100), ALIGN), (dict(bias=P[4] + 2), ALIGN),
    (dict(row_scale=P[2] + 2), ALIGN), (dict(col_scale=P[3] + 1), ALIGN),
])
def test_check_linear(lib, kw, code):
    assert G.gemm_linear_check(_fwd(**kw)) == code


def _bwd(**kw):
    base = dict(M=5, N=96, K=64, type=G.GEMM_F16, da_type=G.GEMM_F16, db_type=G.GEMM_F32,
                dbias_type=G.GEMM_F32, activation=G.GEMM_ACT_SILU, accumulate=1, alpha=1.0,
                dd=P[0], lddd=96, z=P[1], ldz=96, a=P[2], lda=64, b=P[3], ldb=64, dz=P[4], lddz=96,
                da=P[5], ldda=64, db=P[6], lddb=64, dbias=P[7])
    base.update(kw)
    return G.gemm_linear_bwd_t(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(da=None, b=None), 0), (dict(db=None, a=None), 0), (dict(dbias=None), 0),
    (dict(M=0, dd=None, z=None, a=None, dz=None, da=None), 0),
    (dict(N=0, dd=None, z=None, b=None, dz=None, db=None), 0),
    (dict(activation=0, z=None, dz=None), 0), (dict(da=None, db=None, dz=None), 0),
    (dict(dz=P[0]), 0), (dict(dz=P[1]), 0),
    (dict(M=-1), INVALID), (dict(dd=None), INVALID), (dict(z=None), INVALID),
    (dict(dz=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID),
    (dict(activation=7), INVALID), (dict(lddz=88), INVALID), (dict(dz=P[0], lddz=104), INVALID),
    (dict(dz=P[1], lddz=104), INVALID), (dict(da=P[4]), INVALID), (dict(db=P[4]), INVALID),
    (dict(da=P[2]), INVALID), (dict(db=P[3]), INVALID), (dict(da=P[6]), INVALID),
    (dict(db=P[2]), INVALID), (dict(da=P[3]), INVALID),
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(type=G.GEMM_F32), DTYPE),
    (dict(da_type=G.GEMM_E4M3), DTYPE), (dict(dbias_type=5), DTYPE),
    (dict(dd=P[0] + 8), ALIGN), (dict(lddz=100), ALIGN), (dict(a=P[2] + 2), ALIGN),
    (dict(ldb=68), ALIGN), (dict(dbias=P[7] + 2), ALIGN),
])
def test_check_linear_bwd(lib, kw, code):
    assert G.gemm_linear_bwd_check(_bwd(**kw)) == code


def test_packed_calls_match_the_structures():
    """The tensor calls pack the C structures by format: same size, every field in its place."""
    for fmt, cls in ((G._LINEAR, G.gemm_linear_t), (G._LINEAR_BWD, G.gemm_linear_bwd_t),
                     (G._RMSNORM, G.gemm_rmsnorm_t), (G._RMSNORM_BWD, G.gemm_rmsnorm_bwd_t)):
        values = [float(i + 1) if t is ctypes.c_float else i + 1
                  for i, (_, t) in enumerate(cls._fields_)]
        assert fmt.size == ctypes.sizeof(cls)
        assert fmt.pack(*values) == bytes(cls(*values)), cls


def test_null_arguments(lib):
    assert lib.gemm_linear(None, None, None) == INVALID
    assert lib.gemm_linear_check(None) == INVALID
    assert lib.gemm_linear_bwd(None, None, None) == INVALID
    assert lib.gemm_linear_bwd_check(None) == INVALID


@pytest.mark.parametrize("name", ACTS)
def test_derivatives_against_differences(name):
    """Central differences of step 1e-6 in 64 bits are off by at most 1e-9."""
    v = torch.linspace(-9, 9, 2001, dtype=torch.float64) + 1e-3
    e = 1e-6
    d = (O.act(v + e, name) - O.act(v - e, name)) / (2 * e)
    assert float((d - O.act_grad(v, name)).abs().max()) < 1e-8
    assert float(O.act_grad(v, name).abs().max()) < SLOPE


def test_backward_formula_against_differences():
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    a, b, bias, dd = rnd(3, 4), rnd(5, 4), rnd(5), rnd(3, 5)
    loss = lambda a, b, bias: float((O.act(0.5 * a @ b.T + bias, "gelu") * dd).sum())
    dz = dd * O.act_grad(0.5 * a @ b.T + bias, "gelu")
    e = 1e-6
    for args, i, grad in (((a, b, bias), 0, 0.5 * dz @ b), ((a, b, bias), 1, 0.5 * dz.T @ a),
                          ((a, b, bias), 2, dz.sum(0))):
        for at in itertools.product(*(range(n) for n in args[i].shape)):
            up, down = list(args), list(args)
            up[i], down[i] = args[i].clone(), args[i].clone()
            up[i][at] += e
            down[i][at] -= e
            assert abs((loss(*up) - loss(*down)) / (2 * e) - float(grad[at])) < 1e-8


# ---------------------------------------------------------------- GPU

def _operand(gen, R, K, t, mn=False, pad=16, scale=1.0):
    """(values in 64 bits, device view [R, K]) of an operand whose padding is NaN."""
    v = torch.randn(R, K, generator=gen) * scale
    if t in O.TOP8:
        v = (v * O.TOP8[t] / 4.5).clamp(-O.TOP8[t], O.TOP8[t])
    if t == "tf32":
        import workloads as W
        v = W.round_to_tf32(v)
        t = "f32"
    v = v.to(O.TYPES[t]).float()
    if mn:
        return v.double(), O.strided(v.T.contiguous(), t, pad)[0].T
    return v.double(), O.strided(v, t, pad)[0]


def _check_forward(gemm, M, N, K, ab="bf16", b_t=None, d_t="bf16", act="none", bias_t="f32", r_t=None,
                   z_t=None, scales=False, alpha=1.0, a_mn=False, b_mn=False, pad=16,
                   in_place=False, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * M + 13 * N + K)
    b_t = b_t or ab
    a, A = _operand(gen, M, K, ab, a_mn, pad)
    b, Bd = _operand(gen, N, K, b_t, b_mn, pad, scale=max(K, 1) ** -0.5)
    rs = cs = None
    factor = torch.full((M, N), float(torch.tensor(alpha)), dtype=torch.float64)
    if scales:
        unit = lambda t: 4.5 / O.TOP8[t] if t in O.TOP8 else 1.0
        rs = ((0.5 + torch.rand(M, generator=gen)) * unit(ab)).float()
        cs = ((0.5 + torch.rand(N, generator=gen)) * unit(b_t)).float()
        factor = factor * torch.outer(rs.double(), cs.double())
    bias = (torch.randn(N, generator=gen)).to(O.TYPES[bias_t]) if bias_t else None
    r = torch.randn(M, N, generator=gen).to(O.TYPES[r_t]).double() if r_t else None
    z64 = (a @ b.T) * factor + (bias.double() if bias_t else 0.0)
    S = (a.abs() @ b.abs().T) * factor.abs()
    R = O.strided(r, r_t, pad) if r_t else None
    nan = torch.full((M, N), float("nan"))
    D = R if in_place else O.strided(nan, d_t, pad)
    Z = O.strided(nan, z_t, pad) if z_t else None
    cuda = lambda v: None if v is None else v.cuda()
    gemm.linear(A, Bd, D[0], bias=cuda(bias), activation=act, residual=R[0] if R else None,
                z=Z[0] if Z else None, row_scale=cuda(rs), col_scale=cuda(cs), alpha=alpha)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    ez = S * (ACCUM + 6 * O.U32) + (bias.double().abs() * O.U32 if bias_t else 0.0) + \
        z64.abs() * 2 * O.U32
    d64 = O.act(z64, act)
    ed = ez * SLOPE + (0 if act in ("none", "relu") else EVAL * z64.abs().clamp(min=1.0))
    if r_t:
        d64 = d64 + r
        ed = ed + (d64.abs() + r.abs()) * O.U32
    O.within(D[0], d64, ed + O.rounding(d64.abs() + ed, d_t), "d")
    assert O.padding_untouched(*D)
    if z_t:
        O.within(Z[0], z64, ez + O.rounding(z64.abs() + ez, z_t), "z")
        assert O.padding_untouched(*Z)
    if r_t and not in_place:
        assert torch.equal(O.f64(R[0]), r) and O.padding_untouched(*R)


SIZES = [(1, 1, 1), (1, 8, 16), (1, 257, 129), (2, 64, 100), (3, 1000, 77), (7, 33, 520),
         (8, 129, 64), (9, 300, 65), (16, 512, 1000), (17, 100, 300), (33, 77, 1031),
         (64, 640, 512), (100, 1003, 260), (128, 128, 128), (129, 257, 65), (300, 520, 1000),
         (513, 771, 129), (700, 1100, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ab,d_t", [("f16", "f16"), ("bf16", "f32"), ("e4m3", "bf16"),
                                    ("tf32", "f32")])
def test_forward_sizes(gemm, M, N, K, ab, d_t):
    i = M + N + K
    _check_forward(gemm, M, N, K, ab, d_t=d_t, act=ACTS[i % 5], r_t=[None, "bf16", "f32"][i % 3],
                   z_t=[None, "f16", "f32", "bf16"][i % 4], scales=ab == "e4m3" or i % 7 == 0,
                   bias_t=[None, "f32", "f16", "bf16"][(i // 2) % 4])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 5, 16, 40, 200])
def test_forward_activations(gemm, M, act):
    _check_forward(gemm, M, 264, 200, "f16", d_t="f32", act=act, z_t="f32", alpha=2.0)


@pytest.mark.gpu
@pytest.mark.parametrize("ab,b_t", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M", [1, 12, 50, 150])
def test_forward_8bit_pairs(gemm, M, ab, b_t):
    _check_forward(gemm, M, 200, 528, ab, b_t, scales=True, r_t="bf16", act="silu")


@pytest.mark.gpu
@pytest.mark.parametrize("a_mn,b_mn", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (5, 136, 200), (40, 300, 133), (260, 264, 100)])
def test_forward_layouts(gemm, M, N, K, a_mn, b_mn):
    for ab in ("bf16", "e4m3"):
        _check_forward(gemm, M, N, K, ab, a_mn=a_mn, b_mn=b_mn, scales=ab == "e4m3", act="relu",
                       r_t="f16", z_t="bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 6, 48, 300])
def test_forward_in_place_residual_and_tight_rows(gemm, M):
    _check_forward(gemm, M, 512, 256, "bf16", d_t="bf16", r_t="bf16", in_place=True, pad=0,
                   act="gelu")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 9, 130])
@pytest.mark.parametrize("b_mn", [False, True])
def test_forward_no_inner_dimension(gemm, M, b_mn):
    """K = 0: d = act(bias) + residual, z = bias."""
    bias = torch.randn(72).cuda()
    r = torch.randn(M, 72).half()
    a = torch.empty(M, 0, dtype=torch.float16, device="cuda")
    b = torch.empty(72, 0, dtype=torch.float16, device="cuda")
    d, z = (torch.full((M, 72), float("nan"), device="cuda") for _ in range(2))
    gemm.linear(a, b.T.contiguous().T if b_mn else b, d, bias=bias, activation="silu",
                residual=r.cuda(), z=z)
    want = O.act(O.f64(bias), "silu") + r.double()
    O.within(z, O.f64(bias).expand(M, 72), torch.full((M, 72), 1e-12, dtype=torch.float64), "z")
    O.within(d, want, (want.abs() + r.double().abs()) * 2 * O.U32 + EVAL, "d")


@pytest.mark.gpu
def test_forward_empty_is_a_no_op(gemm):
    e = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    gemm.linear(e(0, 64), e(32, 64), e(0, 32))
    gemm.linear(e(8, 64), e(0, 64), e(8, 0))
    assert gemm.sync_status()[0] == G.GEMM_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 30, 140])
def test_forward_nan_and_infinity_stay_in_their_rows(gemm, M):
    """A row of a with a NaN or an infinity spoils its own outputs alone, whatever NaN lies
    in the padding of every tensor."""
    K, N = 200, 72
    gen = torch.Generator().manual_seed(M)
    a, b = torch.randn(M, K, generator=gen).half(), torch.randn(N, K, generator=gen).half()
    a[0, K - 1] = float("nan")
    if M > 1:
        a[M - 1, 3] = float("inf")
    d = O.strided(torch.zeros(M, N), "f32")[0]
    gemm.linear(O.strided(a, "f16")[0], O.strided(b, "f16")[0], d, activation="none")
    out = d.cpu()
    assert torch.isnan(out[0]).all()
    if M > 1:
        assert not torch.isfinite(out[M - 1]).any()
        want = a[1:M - 1].double() @ b.double().T
        S = a[1:M - 1].double().abs() @ b.double().abs().T
        O.within(out[1:M - 1], want, S * (ACCUM + 4 * O.U32), "other rows")


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1, tile_n=128), dict(cta_group=1, tile_n=256),
                                 dict(cta_group=2, tile_n=256), dict(cta_group=2, tile_n=96),
                                 dict(cta_group=1, tile_n=64, epi_warps=2),
                                 dict(cta_group=2, tile_n=224, epi_warps=2),
                                 dict(cta_group=1, tile_n=192, epi_warps=2, epi_slots=2)])
@pytest.mark.parametrize("ab", ["bf16", "e4m3", "tf32"])
def test_forward_forced_configurations(gemm, cfg, ab):
    gemm.set_config(**cfg)
    try:
        for M, N, K in ((40, 1003, 260), (1000, 1500, 136)):
            _check_forward(gemm, M, N, K, ab, d_t="f16", act="gelu", r_t="bf16", z_t="f32",
                           scales=True)
            c = gemm.last_config()
            assert all(getattr(c, k) == v for k, v in cfg.items())
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("bn,split", [(16, 1), (16, 2), (16, 8), (32, 3), (48, 5), (64, 4), (64, 7),
                                      (80, 2), (96, 8), (112, 3), (128, 1), (128, 6), (128, 8)])
@pytest.mark.parametrize("ab", ["bf16", "e4m3", "tf32"])
def test_forward_split_over_a_cluster(gemm, bn, split, ab):
    """The split-K kernel at every tile width class and cluster size, ragged, one tile and
    several, K from one k-block per CTA up."""
    gemm.set_config(split_k=split, tile_n=bn)
    try:
        for M, N, K in ((1, 1, 1030), (37, 203, 1033), (bn + 3, 264, 1500)):
            _check_forward(gemm, M, N, K, ab, d_t="f16", act="gelu", r_t="bf16", z_t="f32",
                           scales=True)
            c = gemm.last_config()
            assert (c.split_k, c.tile_n) == (split, bn)
        if split > 1:                            # more CTAs than k-blocks
            with pytest.raises(G.GemmError) as e:
                _check_forward(gemm, 4, 8, 16 if ab == "tf32" else 32, ab)
            assert e.value.status == G.GEMM_ERR_UNSUPPORTED_CONFIG
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("feats", [8, 24, 56, 96, 120])
@pytest.mark.parametrize("bn,split", [(16, 1), (16, 3), (64, 4), (96, 2), (128, 1)])
def test_forward_split_narrow_feature_tiles(gemm, feats, bn, split):
    gemm.set_config(split_k=split, tile_n=bn, tile_m=feats)
    try:
        for ab, N in (("f16", 203), ("e4m3", 88)):
            _check_forward(gemm, bn - 3, N, 1100, ab, act="silu", r_t="f32", z_t="bf16",
                           scales=ab == "e4m3")
            assert gemm.last_config().tile_m == feats
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("a_mn,b_mn", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("bn,split", [(64, 2), (128, 3), (128, 8), (128, 1)])
def test_forward_split_layouts(gemm, bn, split, a_mn, b_mn):
    gemm.set_config(split_k=split, tile_n=bn)
    try:
        for ab in ("f16", "e5m2"):
            if ab == "e5m2" and a_mn and bn % 128:
                continue
            _check_forward(gemm, 150, 203, 1100, ab, a_mn=a_mn, b_mn=b_mn, scales=ab == "e5m2",
                           act="silu", r_t="f32", bias_t="bf16")
        if a_mn:
            gemm.set_config(split_k=split, tile_n=48)
            with pytest.raises(G.GemmError):
                _check_forward(gemm, 150, 203, 1100, "f16", a_mn=True)
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("split", [0, 1, 4])
def test_watchdog_ends_a_stalled_layer(gemm, split):
    """The matrix-unit warp waits on a barrier nothing arrives at (an injected stall with a
    100 ms limit): the launch ends by itself, the status names the wait, and the next call
    computes."""
    g = G.Gemm(0)
    try:
        G.gemm_set_timeout_ns(g.handle, 100_000_000)
        g.set_config(inject_stall=1, split_k=split)
        e = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
        d = e(40, 264)
        g.linear(e(40, 512), e(264, 512), d)
        st, detail = g.sync_status()
        assert st == G.GEMM_ERR_DEVICE_TIMEOUT and (detail >> 24) == 0xE0, hex(detail)
        G.gemm_set_timeout_ns(g.handle, 0)
        g.set_config(None)
        g.linear(e(40, 512), e(264, 512), d)
        assert g.sync_status()[0] == G.GEMM_OK and (d == 512).all()
    finally:
        g.close()


@pytest.mark.gpu
def test_forward_refuses_multicast_clusters(gemm):
    gemm.set_config(cluster_m=2)
    try:
        with pytest.raises(G.GemmError) as e:
            _check_forward(gemm, 512, 512, 64)
        assert e.value.status == G.GEMM_ERR_UNSUPPORTED_CONFIG
    finally:
        gemm.set_config(None)


def _check_backward(gemm, M, N, K, t="bf16", act="gelu", da_t=None, db_t=None, dbias_t="f32",
                    accumulate=False, alpha=1.0, pad=16, dz_over=None, give=("dz", "da", "db", "dbias")):
    gen = torch.Generator().manual_seed(M + 3 * N + 5 * K)
    da_t, db_t = da_t or t, db_t or t
    val = lambda *s: torch.randn(*s, generator=gen).to(O.TYPES[t]).double()
    dd, z, a, b = val(M, N), val(M, N) * 2, val(M, K), val(N, K)
    z = z.to(O.TYPES[t]).double()
    dev = lambda v: O.strided(v, t, pad)
    DD, Zd, A, Bd = dev(dd), dev(z), dev(a), dev(b)
    new = lambda r, c, ty: O.strided(torch.full((r, c), float("nan")), ty, pad)
    DZ = {"dd": DD, "z": Zd}[dz_over] if dz_over else new(M, N, t)
    DA = new(M, K, da_t)
    old = torch.randn(N, K, generator=gen).to(O.TYPES[db_t]).double() if accumulate else None
    DB = O.strided(old, db_t, pad) if accumulate else new(N, K, db_t)
    dbias = torch.full((N,), float("nan"), device="cuda").to(O.TYPES[dbias_t])
    outs = dict(dz=DZ[0], da=DA[0], db=DB[0], dbias=dbias)
    gemm.linear_bwd(DD[0], A[0], Bd[0], z=None if act == "none" else Zd[0], activation=act,
                    accumulate=accumulate, alpha=alpha, **{k: outs[k] for k in give})
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    slope = O.act_grad(z, act)
    dz64 = dd * slope
    # the derivative's own evaluation, then the product with dd
    edz = dd.abs() * (0 if act in ("none", "relu") else 2 * EVAL) + dz64.abs() * 2 * O.U32
    if act == "none":
        edz = edz * 0
    if "dz" in give:
        O.within(DZ[0], dz64, edz + O.rounding(dz64.abs() + edz, t), "dz")
        assert O.padding_untouched(*DZ)
    if "dbias" in give:
        size = dz64.abs().sum(0)
        err = edz.sum(0) + size * (M + 40) * O.U32
        O.within(dbias, dz64.sum(0), err + O.rounding(dz64.sum(0).abs() + err, dbias_t), "dbias")
    # what the products read: dz rounded to t
    rz = edz + O.rounding(dz64.abs() + edz, t)
    if "da" in give:
        want = alpha * dz64 @ b
        err = abs(alpha) * (rz @ b.abs() + (dz64.abs() + rz) @ b.abs() * (ACCUM + 4 * O.U32))
        O.within(DA[0], want, err + O.rounding(want.abs() + err, da_t), "da")
        assert O.padding_untouched(*DA)
    if "db" in give:
        want = alpha * dz64.T @ a
        err = abs(alpha) * (rz.T @ a.abs() + (dz64.abs() + rz).T @ a.abs() * (ACCUM + 4 * O.U32))
        if accumulate:
            want = want + old
            err = err + (want.abs() + old.abs()) * O.U32
        O.within(DB[0], want, err + O.rounding(want.abs() + err, db_t), "db")
        assert O.padding_untouched(*DB)
    assert torch.equal(O.f64(A[0]), a) and torch.equal(O.f64(Bd[0]), b)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 40, 24), (3, 77, 130), (9, 264, 65),
                                   (33, 500, 100), (64, 64, 64), (130, 257, 129), (300, 1003, 520),
                                   (1000, 72, 200), (2049, 136, 264)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_backward_sizes(gemm, M, N, K, t):
    _check_backward(gemm, M, N, K, t, ACTS[(M + N) % 5])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(2100, 1003), (2100, 700), (2300, 200), (4000, 1216), (600, 1217)])
def test_backward_narrow_layers(gemm, M, N):
    """Few columns and many rows: the activation gradient's larger blocks, alone."""
    _check_backward(gemm, M, N, 8, "bf16", "gelu", give=("dz", "dbias"))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(gemm, act):
    _check_backward(gemm, 200, 264, 136, "f16", act, da_t="f32", db_t="f32", alpha=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("db_t", ["f32", "bf16"])
@pytest.mark.parametrize("M", [0, 1, 70, 600])
def test_backward_accumulates(gemm, M, db_t):
    _check_backward(gemm, M, 200, 136, "bf16", "silu", db_t=db_t, accumulate=True,
                    give=("dz", "da", "db", "dbias"))


@pytest.mark.gpu
@pytest.mark.parametrize("give", [("dz",), ("dbias",), ("dz", "da"), ("dz", "db"),
                                  ("dz", "da", "db", "dbias")])
def test_backward_any_subset(gemm, give):
    _check_backward(gemm, 150, 200, 72, "f16", "gelu_tanh", give=give, dbias_t="bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("over", ["dd", "z"])
def test_backward_dz_in_place(gemm, over):
    _check_backward(gemm, 150, 203, 72, "bf16", "gelu", dz_over=over)


@pytest.mark.gpu
def test_backward_no_activation_reads_dd_directly(gemm):
    _check_backward(gemm, 150, 200, 72, "bf16", "none", give=("da", "db", "dbias"))
    _check_backward(gemm, 150, 200, 72, "bf16", "none")


@pytest.mark.gpu
def test_backward_empty_extents(gemm):
    """No rows: weight and bias gradients are zero.  No columns: da is zero."""
    _check_backward(gemm, 0, 200, 72, "f16", "gelu")
    e = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    da = torch.full((5, 64), float("nan"), dtype=torch.float16, device="cuda")
    gemm.linear_bwd(e(5, 0), e(5, 64), e(0, 64), activation=None, da=da)
    torch.cuda.synchronize()
    assert (da == 0).all()


@pytest.mark.gpu
def test_large_magnitudes_keep_their_limits(gemm):
    """Pre-activations up to the type's largest: the derivative is 0 or 1 there and no NaN appears."""
    z = torch.tensor([[-3e38, -1e30, -1e4, -90.0, 90.0, 1e4, 1e30, 3e38]], dtype=torch.bfloat16)
    dd = torch.ones_like(z)
    for act in ACTS[1:]:
        dz = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda")
        gemm.linear_bwd(dd.cuda(), torch.zeros(1, 8, dtype=torch.bfloat16).cuda(),
                        torch.zeros(8, 8, dtype=torch.bfloat16).cuda(), z=z.cuda(), activation=act,
                        dz=dz)
        want = torch.tensor([0.0, 0, 0, 0, 1, 1, 1, 1])
        assert float((dz.cpu().float()[0] - want).abs().max()) < 1e-30, act


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 500])
def test_same_bits_on_repeat_another_stream_and_in_a_graph(gemm, M):
    N, K = 712, 520
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen).to("cuda", torch.bfloat16)
    a, b, bias, r, dd = rnd(M, K), rnd(N, K), rnd(N), rnd(M, N), rnd(M, N)

    def outputs():
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        return dict(d=e(M, N), z=e(M, N), dz=e(M, N), da=e(M, K), db=e(N, K), dbias=e(N))

    def both(o, stream):
        gemm.linear(a, b, o["d"], bias=bias, activation="gelu", residual=r, z=o["z"], stream=stream)
        gemm.linear_bwd(dd, a, b, z=o["z"], activation="gelu", dz=o["dz"], da=o["da"], db=o["db"],
                        dbias=o["dbias"], stream=stream)

    o1, o2, o3 = outputs(), outputs(), outputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(o1, None)
    torch.cuda.synchronize()
    both(o2, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(o3, torch.cuda.current_stream())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in o1:
        assert torch.equal(o1[k], o2[k]) and torch.equal(o1[k], o3[k]), k


@pytest.mark.gpu
def test_two_handles_on_two_streams_at_once(gemm):
    """One handle used from two streams without ordering between them."""
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen).to("cuda", torch.float16)
    sets = [(rnd(m, 1024), rnd(776, 1024)) for m in (1, 24, 90, 300)]
    want = []
    for a, b in sets:
        d = torch.empty(a.shape[0], 776, dtype=torch.float16, device="cuda")
        gemm.linear(a, b, d, activation="silu")
        want.append(d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(w) for w in want] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, outs in zip(streams, got):
            for (a, b), d in zip(sets, outs):
                gemm.linear(a, b, d, activation="silu", stream=s)
    torch.cuda.synchronize()
    for outs in got:
        for w, d in zip(want, outs):
            assert torch.equal(w, d)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors(gemm):
    e = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")
    a, b, d = e(4, 64), e(32, 64), e(4, 32)
    for kw in (dict(b=e(32, 72)), dict(d=e(4, 40)), dict(d=e(32, 4).T), dict(bias=e(31)),
               dict(residual=e(5, 32)), dict(z=e(4, 32, dt=torch.int32)),
               dict(row_scale=e(4)), dict(col_scale=e(4, dt=torch.float32)),
               dict(activation="swish"), dict(b=e(32, 64, dt=torch.bfloat16)),
               dict(a=e(8, 128)[::2, ::2])):
        with pytest.raises(G.GemmError):
            gemm.linear(**{**dict(a=a, b=b, d=d), **kw})
    with pytest.raises(G.GemmError):
        gemm.linear_bwd(d, a, b, activation="gelu", dbias=e(32))        # no z
