"""The linear layer over groups of rows and its backward pass: refusals (CPU), the 64-bit
formulas against differences (CPU), and the kernels against them.

Tolerances as in test_linear: a product's fp32 accumulation is off by at most 2^-10 of the
sum of its terms' magnitudes, S below; scales and bias by at most 6 u of S and the bias, u =
2^-24; an activation of slope at most 1.13 carries an error of z on at 1.13 times its
size and its own evaluation is off by at most 2^-21 of max(1, |z|); results are rounded once,
dz before the products read it."""
import ctypes
import itertools

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
import layer_oracle as O

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
SLOPE, EVAL, ACCUM = 1.13, 2.0 ** -21, 2.0 ** -10
NAN, INF = float("nan"), float("inf")


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

P = [(i + 1) << 20 for i in range(14)]     # fake, aligned device addresses
INVALID, DTYPE, ALIGN = (G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE,
                         G.GEMM_ERR_MISALIGNED)


def _fwd(**kw):
    base = dict(M=5, N=96, K=64, groups=3, sets=4, a_type=G.GEMM_E4M3, b_type=G.GEMM_E5M2,
                bias_type=G.GEMM_F32, r_type=G.GEMM_BF16, z_type=G.GEMM_F16, d_type=G.GEMM_BF16,
                activation=G.GEMM_ACT_GELU, alpha=1.0, offsets=P[8], index=P[9], A=P[0], lda=64,
                B=P[1], ldb=64, strideB=96 * 64, row_scale=P[2], col_scale=P[3], bias=P[4], R=P[5],
                ldr=96, Z=P[6], ldz=96, D=P[7], ldd=96)
    base.update(kw)
    return G.gemm_grouped_linear_t(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(M=0, A=None, D=None, offsets=None), 0), (dict(N=0), 0), (dict(groups=0), 0),
    (dict(K=0, A=None, B=None), 0), (dict(sets=0, A=None, B=None), 0),
    (dict(R=None, Z=None, bias=None, row_scale=None, col_scale=None, index=None), 0),
    (dict(R=P[7]), 0), (dict(bias=P[4] + 4), 0), (dict(N=95, K=61, M=1), 0), (dict(sets=2), 0),
    (dict(a_type=G.GEMM_TF32, b_type=G.GEMM_TF32), 0), (dict(sets=1, strideB=3), 0),
    (dict(strideB=0), 0), (dict(offsets=P[8] + 4, index=P[9] + 8), 0), (dict(groups=4096), 0),
    (dict(layoutB=G.GEMM_MN_MAJOR, ldb=96), 0),
    (dict(M=-1), INVALID), (dict(K=1 << 31), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=4097), INVALID), (dict(sets=4097), INVALID), (dict(sets=2, index=None), INVALID),
    (dict(M=(1 << 31) - 8193, N=1 << 16), INVALID), (dict(offsets=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(D=None), INVALID), (dict(lda=48), INVALID), (dict(ldd=88), INVALID),
    (dict(ldz=80), INVALID), (dict(layoutB=2), INVALID), (dict(activation=5), INVALID),
    (dict(activation=-1), INVALID), (dict(R=P[7], ldr=104), INVALID),
    (dict(R=P[7], r_type=G.GEMM_F16), INVALID), (dict(Z=P[7]), INVALID), (dict(Z=P[5]), INVALID),
    (dict(D=P[0]), INVALID), (dict(Z=P[1]), INVALID), (dict(ldb=1 << 40), INVALID),
    (dict(strideB=1 << 40), INVALID), (dict(layoutB=G.GEMM_MN_MAJOR), INVALID),
    (dict(a_type=G.GEMM_F16), DTYPE), (dict(a_type=G.GEMM_F32, b_type=G.GEMM_F32), DTYPE),
    (dict(a_type=G.GEMM_F16, b_type=G.GEMM_BF16), DTYPE), (dict(d_type=G.GEMM_E4M3), DTYPE),
    (dict(r_type=G.GEMM_E4M3), DTYPE), (dict(bias_type=G.GEMM_TF32), DTYPE),
    (dict(z_type=9), DTYPE),
    (dict(a_type=G.GEMM_TF32, b_type=G.GEMM_TF32, layoutB=G.GEMM_MN_MAJOR), DTYPE),
    (dict(A=P[0] + 8), ALIGN), (dict(lda=72), ALIGN), (dict(D=P[7] + 2), ALIGN),
    (dict(ldd=100), ALIGN), (dict(ldr=100), ALIGN), (dict(bias=P[4] + 2), ALIGN),
    (dict(row_scale=P[2] + 2), ALIGN), (dict(col_scale=P[3] + 1), ALIGN),
    (dict(strideB=96 * 64 + 8), ALIGN), (dict(strideB=-16), ALIGN), (dict(offsets=P[8] + 2), ALIGN),
    (dict(index=P[9] + 1), ALIGN),
])
def test_check_grouped(lib, kw, code):
    assert G.gemm_grouped_linear_check(_fwd(**kw)) == code


def _bwd(**kw):
    base = dict(M=5, N=96, K=64, groups=3, type=G.GEMM_F16, da_type=G.GEMM_F16, db_type=G.GEMM_F32,
                dbias_type=G.GEMM_F32, activation=G.GEMM_ACT_SILU, accumulate=1, alpha=1.0,
                offsets=P[8], dd=P[0], lddd=96, z=P[1], ldz=96, a=P[2], lda=64, b=P[3], ldb=64,
                strideb=96 * 64, dz=P[4], lddz=96, da=P[5], ldda=64, db=P[6], lddb=64,
                stridedb=96 * 64, dbias=P[7])
    base.update(kw)
    return G.gemm_grouped_linear_bwd_t(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(da=None, b=None), 0), (dict(db=None, a=None), 0), (dict(dbias=None), 0),
    (dict(M=0, dd=None, z=None, a=None, dz=None, da=None), 0),
    (dict(N=0, dd=None, z=None, b=None, dz=None, db=None, offsets=None), 0),
    (dict(groups=0, offsets=None), 0), (dict(activation=0, z=None, dz=None), 0),
    (dict(da=None, db=None, dz=None), 0), (dict(dz=P[0]), 0), (dict(dz=P[1]), 0),
    (dict(K=0, a=None, b=None, da=None, db=None), 0),
    (dict(groups=1, strideb=1, stridedb=1), 0), (dict(strideb=0), 0),
    (dict(M=-1), INVALID), (dict(dd=None), INVALID), (dict(z=None), INVALID),
    (dict(offsets=None), INVALID), (dict(groups=4097), INVALID),
    (dict(dz=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID),
    (dict(activation=7), INVALID), (dict(lddz=88), INVALID), (dict(dz=P[0], lddz=104), INVALID),
    (dict(dz=P[1], lddz=104), INVALID), (dict(da=P[4]), INVALID), (dict(db=P[4]), INVALID),
    (dict(da=P[2]), INVALID), (dict(db=P[3]), INVALID), (dict(da=P[6]), INVALID),
    (dict(db=P[2]), INVALID), (dict(da=P[3]), INVALID), (dict(stridedb=96 * 64 - 16), INVALID),
    (dict(stridedb=0), INVALID), (dict(da=P[0]), INVALID), (dict(db=P[0]), INVALID),
    (dict(N=1 << 24, groups=4096), INVALID),
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(type=G.GEMM_F32), DTYPE),
    (dict(da_type=G.GEMM_E4M3), DTYPE), (dict(dbias_type=5), DTYPE),
    (dict(dd=P[0] + 8), ALIGN), (dict(lddz=100), ALIGN), (dict(a=P[2] + 2), ALIGN),
    (dict(ldb=68), ALIGN), (dict(dbias=P[7] + 2), ALIGN), (dict(offsets=P[8] + 1), ALIGN),
    (dict(strideb=96 * 64 + 4), ALIGN), (dict(stridedb=96 * 64 + 2), ALIGN),
])
def test_check_grouped_bwd(lib, kw, code):
    assert G.gemm_grouped_linear_bwd_check(_bwd(**kw)) == code


def test_packed_calls_match_the_structures():
    """The tensor calls pack the C structures by format: same size, every field in its place."""
    for fmt, cls in ((G._GROUPED, G.gemm_grouped_linear_t),
                     (G._GROUPED_BWD, G.gemm_grouped_linear_bwd_t)):
        values = [float(i + 1) if t is ctypes.c_float else i + 1
                  for i, (_, t) in enumerate(cls._fields_)]
        assert fmt.size == ctypes.sizeof(cls)
        assert fmt.pack(*values) == bytes(cls(*values)), cls


def test_null_arguments(lib):
    for name in ("gemm_grouped_linear", "gemm_grouped_linear_bwd"):
        assert getattr(lib, name)(None, None, None) == INVALID
        assert getattr(lib, name + "_check")(None) == INVALID


def _rows(bounds, g):
    return slice(bounds[g], max(bounds[g], bounds[g + 1]))


def backward(dd, z, a, b, bounds, act, alpha=1.0, rounded=lambda dz: dz):
    """(dz, da, db, dbias) in 64 bits; rows of no group are NaN in dz and da."""
    n, k = b.shape[1:]
    dz = torch.full_like(dd, NAN)
    da = torch.full((dd.shape[0], k), NAN, dtype=torch.float64)
    db, dbias = torch.zeros_like(b), torch.zeros(b.shape[0], n, dtype=torch.float64)
    for g in range(b.shape[0]):
        rows = _rows(bounds, g)
        dz[rows] = dd[rows] * O.act_grad(z[rows], act)
        r = rounded(dz[rows])
        da[rows] = alpha * r @ b[g]
        db[g] = alpha * r.T @ a[rows]
        dbias[g] = dz[rows].sum(dim=0)
    return dz, da, db, dbias


def test_backward_formula_against_differences():
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    bounds = [0, 2, 2, 5]
    a, b, bias, dd = rnd(5, 4), rnd(3, 2, 4), rnd(3, 2), rnd(5, 2)

    def z_of(a, b, bias):
        return torch.cat([0.5 * a[_rows(bounds, g)] @ b[g].T + bias[g] for g in range(3)])
    loss = lambda *args: float((O.act(z_of(*args), "gelu") * dd).sum())
    _, da, db, dbias = backward(dd, z_of(a, b, bias), a, b, bounds, "gelu", 0.5)
    e = 1e-6
    args = (a, b, bias)
    for i, grad in enumerate((da, db, dbias)):
        for at in itertools.product(*(range(n) for n in args[i].shape)):
            up, down = list(args), list(args)
            up[i], down[i] = args[i].clone(), args[i].clone()
            up[i][at] += e
            down[i][at] -= e
            assert abs((loss(*up) - loss(*down)) / (2 * e) - float(grad[at])) < 1e-8


# ---------------------------------------------------------------- GPU

def _operand(gen, R, K, t, pad=16, scale=1.0):
    """(values in 64 bits, device view [R, K]) of an operand whose padding is NaN."""
    v = torch.randn(R, K, generator=gen) * scale
    if t in O.TOP8:
        v = (v * O.TOP8[t] / 4.5).clamp(-O.TOP8[t], O.TOP8[t])
    if t == "tf32":
        import workloads as W
        v = W.round_to_tf32(v)
        t = "f32"
    v = v.to(O.TYPES[t]).float()
    return v.double(), O.strided(v, t, pad)[0]


def _weights(gen, sets, N, K, t, mn=False, pad=16, scale=1.0):
    """A stack of matrices, rows (or columns: mn) padded, the stack's stride too."""
    v, view = _operand(gen, max(1, sets) * (K if mn else N), N if mn else K, t, pad, scale)
    v, view = (x.unflatten(0, (max(1, sets), -1))[:sets] for x in (v, view))
    return (v.transpose(1, 2), view.transpose(1, 2)) if mn else (v, view)


def _bounds(gen, sizes, before=0):
    b = [before]
    for n in sizes:
        b.append(b[-1] + n)
    return b


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _check_forward(gemm, sizes, N, K, ab="bf16", b_t=None, d_t="bf16", act="none", bias_t=None,
                   r_t=None, z_t=None, scales=False, alpha=1.0, b_mn=False, pad=16, in_place=False,
                   index=None, sets=None, before=0, behind=0, seed=0):
    """sizes: the groups' rows; before, behind: rows of no group."""
    bounds = _bounds(None, sizes, before)
    M, sets = bounds[-1] + behind, len(sizes) if sets is None else sets
    gen = torch.Generator().manual_seed(seed + 7 * M + 13 * N + K)
    b_t = b_t or ab
    a, A = _operand(gen, M, K, ab, pad)
    b, Bd = _weights(gen, sets, N, K, b_t, b_mn, pad, scale=max(K, 1) ** -0.5)
    rs = cs = bias = None
    if scales:
        unit = lambda t: 4.5 / O.TOP8[t] if t in O.TOP8 else 1.0
        rs = ((0.5 + torch.rand(M, generator=gen)) * unit(ab)).float()
        cs = ((0.5 + torch.rand(sets, N, generator=gen)) * unit(b_t)).float()
    if bias_t:
        bias = torch.randn(sets, N, generator=gen).to(O.TYPES[bias_t])
    r = torch.randn(M, N, generator=gen).to(O.TYPES[r_t]).double() if r_t else None
    z64 = torch.full((M, N), NAN, dtype=torch.float64)
    S, eb = torch.zeros_like(z64), torch.zeros_like(z64)
    al = float(torch.tensor(alpha))
    for g in range(len(sizes)):
        rows, e = _rows(bounds, g), g if index is None else index[g]
        if not 0 <= e < sets:
            z64[rows] = 0.0
            continue
        factor = torch.full((rows.stop - rows.start, N), al, dtype=torch.float64)
        if scales:
            factor = factor * torch.outer(rs[rows].double(), cs[e].double())
        z64[rows] = (a[rows] @ b[e].T) * factor + (bias[e].double() if bias_t else 0.0)
        S[rows] = (a[rows].abs() @ b[e].abs().T) * factor.abs()
        if bias_t:
            eb[rows] = bias[e].double().abs()
    R = O.strided(r, r_t, pad) if r_t else None
    nan = torch.full((M, N), NAN)
    D = R if in_place else O.strided(nan, d_t, pad)
    Z = O.strided(nan, z_t, pad) if z_t else None
    cuda = lambda v: None if v is None else v.cuda()
    gemm.grouped_linear(A, Bd, _i32(bounds), D[0], index=None if index is None else _i32(index),
                        bias=cuda(bias), activation=act, residual=R[0] if R else None,
                        z=Z[0] if Z else None, row_scale=cuda(rs), col_scale=cuda(cs), alpha=alpha)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    ez = S * (ACCUM + 6 * O.U32) + eb * O.U32 + z64.abs() * 2 * O.U32
    d64 = O.act(z64, act)
    ed = ez * SLOPE + (0 if act in ("none", "relu") else EVAL * z64.abs().clamp(min=1.0))
    if r_t:
        d64 = d64 + r
        ed = ed + (d64.abs() + r.abs()) * O.U32
    mine = slice(bounds[0], bounds[-1])
    O.within(D[0][mine], d64[mine], (ed + O.rounding(d64.abs() + ed, d_t))[mine], "d")
    others = torch.ones(M, dtype=torch.bool)
    others[mine] = False
    if in_place:
        assert torch.equal(O.f64(D[0])[others], r[others])
    else:
        assert torch.isnan(O.f64(D[0])[others]).all()
    assert O.padding_untouched(*D)
    if z_t:
        O.within(Z[0][mine], z64[mine], (ez + O.rounding(z64.abs() + ez, z_t))[mine], "z")
        assert torch.isnan(O.f64(Z[0])[others]).all() and O.padding_untouched(*Z)
    if r_t and not in_place:
        assert torch.equal(O.f64(R[0]), r) and O.padding_untouched(*R)


SHAPES = [([1], 1, 1), ([1, 0, 2], 8, 16), ([0, 0], 40, 24), ([3, 1, 0, 4], 129, 77),
          ([16, 17, 15], 257, 130), ([0, 65, 63, 1, 0], 136, 520), ([1] * 40, 300, 65),
          ([100, 0, 31, 5], 1003, 260), ([129, 257, 3], 264, 129), ([300, 65, 512], 520, 1000),
          ([700], 771, 129), ([5, 600, 1, 250], 1100, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", SHAPES)
@pytest.mark.parametrize("ab,d_t", [("f16", "f16"), ("bf16", "f32"), ("e4m3", "bf16"),
                                    ("tf32", "f32")])
def test_forward_shapes(gemm, sizes, N, K, ab, d_t):
    i = sum(sizes) + N + K
    _check_forward(gemm, sizes, N, K, ab, d_t=d_t, act=ACTS[i % 5], r_t=[None, "bf16", "f32"][i % 3],
                   z_t=[None, "f16", "f32", "bf16"][i % 4], scales=ab == "e4m3" or i % 7 == 0,
                   bias_t=[None, "f32", "f16", "bf16"][(i // 2) % 4], before=i % 5, behind=i % 3)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=96),
                                 dict(cta_group=1, tile_n=64, stages=2),
                                 dict(cta_group=1, tile_n=128), dict(cta_group=1, tile_n=256),
                                 dict(cta_group=2, tile_n=64), dict(cta_group=2, tile_n=192),
                                 dict(cta_group=2, tile_n=256), dict(cta_group=2, stages=1)])
@pytest.mark.parametrize("ab", ["bf16", "e4m3", "tf32"])
def test_forward_forced_configurations(gemm, cfg, ab):
    gemm.set_config(**cfg)
    try:
        for sizes, N, K in (([40, 0, 1, 129], 1003, 260), ([500, 300, 7, 64], 300, 136)):
            _check_forward(gemm, sizes, N, K, ab, d_t="f16", act="gelu", r_t="bf16", z_t="f32",
                           scales=True, before=3, behind=40)
            c = gemm.last_config()
            assert all(getattr(c, k) == v for k, v in cfg.items())
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cluster_m=2), dict(split_k=2), dict(stream_k=2),
                                 dict(cta_group=2, tile_n=96),
                                 dict(cta_group=2, tile_n=256, stages=12)])
def test_forced_configurations_it_cannot_take(gemm, cfg):
    d, a, b, offsets = (torch.zeros(8, 64, device="cuda").half() for _ in range(4))
    gemm.set_config(**cfg)
    try:
        with pytest.raises(G.GemmError) as e:
            gemm.grouped_linear(a, b.view(1, 8, 64), _i32([0, 8]), d[:, :8])
        assert e.value.status == G.GEMM_ERR_UNSUPPORTED_CONFIG
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("sizes", [[1, 5, 16], [40, 200]])
def test_forward_activations(gemm, sizes, act):
    _check_forward(gemm, sizes, 264, 200, "f16", d_t="f32", act=act, z_t="f32", alpha=2.0,
                   bias_t="f16")


@pytest.mark.gpu
@pytest.mark.parametrize("ab,b_t", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_forward_8bit_pairs(gemm, ab, b_t):
    for sizes in ([1, 3], [12, 50, 150]):
        _check_forward(gemm, sizes, 200, 528, ab, b_t, scales=True, r_t="bf16", act="silu")


@pytest.mark.gpu
@pytest.mark.parametrize("ab", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,N,K", [([1, 2], 40, 24), ([5, 0, 3], 136, 200), ([40, 7], 300, 133),
                                       ([260, 130], 264, 300)])
def test_forward_weights_with_contiguous_features(gemm, sizes, N, K, ab):
    _check_forward(gemm, sizes, N, K, ab, b_mn=True, scales=ab == "e4m3", act="relu", r_t="f16",
                   z_t="bf16", behind=2)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[1, 6], [48, 300]])
@pytest.mark.parametrize("index", [None, [3, -1], [2, 2], [-7, 1 << 30]])
def test_forward_in_place_residual_and_tight_rows(gemm, sizes, index):
    _check_forward(gemm, sizes, 512, 256, "bf16", d_t="bf16", r_t="bf16", in_place=True, pad=0,
                   act="gelu", index=index, sets=4, before=1, behind=5, bias_t="f32")


@pytest.mark.gpu
@pytest.mark.parametrize("index", [[4, 0, 4, -1, 2], [5, 5, -2, 7, 5], [-1] * 5])
@pytest.mark.parametrize("r_t", [None, "f32"])
def test_forward_index(gemm, index, r_t):
    """Groups share weights, or have none: z = 0 and d = r there, whatever bias and scales are."""
    for sizes in ([3, 0, 1, 4, 2], [70, 129, 5, 300, 1]):
        _check_forward(gemm, sizes, 140, 72, "f16", index=index, sets=5, r_t=r_t, act="silu",
                       bias_t="f16", z_t="f32", scales=True, behind=1)


@pytest.mark.gpu
def test_forward_a_group_without_weights_ignores_its_scales(gemm):
    a = torch.randn(4, 64).half().cuda()
    b = torch.randn(1, 32, 64).half().cuda()
    r = torch.randn(4, 32).half().cuda()
    d = torch.zeros(4, 32, device="cuda")
    z = torch.ones(4, 32, device="cuda")
    bad = torch.full((4,), NAN, device="cuda")
    gemm.grouped_linear(a * NAN, b * NAN, _i32([0, 4]), d, index=_i32([1]), residual=r, z=z,
                        row_scale=bad, col_scale=torch.full((1, 32), NAN, device="cuda"),
                        bias=torch.full((1, 32), NAN, device="cuda"), alpha=INF)
    assert torch.equal(d, r.float()) and not z.any()


@pytest.mark.gpu
@pytest.mark.parametrize("b_mn", [False, True])
def test_forward_no_inner_dimension(gemm, b_mn):
    """K = 0: d = act(bias) + residual, z = bias."""
    bias = torch.randn(2, 72).cuda()
    r = torch.randn(9, 72).half()
    a = torch.empty(9, 0, dtype=torch.float16, device="cuda")
    b = torch.empty(2, 72, 0, dtype=torch.float16, device="cuda")
    d, z = (torch.full((9, 72), NAN, device="cuda") for _ in range(2))
    gemm.grouped_linear(a, b.transpose(1, 2).contiguous().transpose(1, 2) if b_mn else b,
                        _i32([0, 4, 9]), d, bias=bias, activation="silu", residual=r.cuda(), z=z)
    zb = O.f64(bias).repeat_interleave(torch.tensor([4, 5]), dim=0)
    want = O.act(zb, "silu") + r.double()
    O.within(z, zb, torch.full((9, 72), 1e-12, dtype=torch.float64), "z")
    O.within(d, want, (want.abs() + r.double().abs()) * 2 * O.U32 + EVAL, "d")


@pytest.mark.gpu
def test_forward_empty_is_a_no_op(gemm):
    e = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    gemm.grouped_linear(e(0, 64), e(2, 32, 64), _i32([0, 0, 0]), e(0, 32))
    gemm.grouped_linear(e(8, 64), e(2, 0, 64), _i32([0, 4, 8]), e(8, 0))
    d = torch.full((8, 32), NAN, device="cuda").half()
    gemm.grouped_linear(e(8, 64), e(0, 32, 64), _i32([0]), d)
    assert torch.isnan(d).all()
    gemm.grouped_linear(e(8, 64), e(0, 32, 64), _i32([0, 3]), d, index=_i32([0]))
    assert not d[:3].any() and torch.isnan(d[3:]).all()
    assert gemm.sync_status()[0] == G.GEMM_OK


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [None, dict(cta_group=1), dict(cta_group=2)])
@pytest.mark.parametrize("offsets", [[-5, 3, 70], [0, 200, 90], [10, 4, 4], [60, 20, 65],
                                     [64, 64, 64], [1 << 30, -(1 << 31), (1 << 31) - 1],
                                     [-9, -5, -1]])
def test_forward_offsets_out_of_range(gemm, cfg, offsets):
    """Offsets are clamped to the rows there are; a group of negative size has none."""
    M, N, K = 65, 72, 64
    gen = torch.Generator().manual_seed(5)
    a, A = _operand(gen, M, K, "f16")
    b, Bd = _weights(gen, 2, N, K, "f16", scale=K ** -0.5)
    d = O.strided(torch.full((M, N), NAN), "f32")
    gemm.set_config(**cfg) if cfg else gemm.set_config(None)
    try:
        gemm.grouped_linear(A, Bd, _i32(offsets), d[0])
        assert gemm.sync_status()[0] == G.GEMM_OK
    finally:
        gemm.set_config(None)
    clamped = [min(max(o, 0), M) for o in offsets]
    got, rest = O.f64(d[0]), torch.ones(M, dtype=torch.bool)
    for g in range(2):
        rows = slice(clamped[g], max(clamped[g], clamped[g + 1]))
        S = a[rows].abs() @ b[g].abs().T
        O.within(got[rows], a[rows] @ b[g].T, S * (ACCUM + 4 * O.U32), g)
        rest[rows] = False
    assert torch.isnan(got[rest]).all() and O.padding_untouched(*d)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1), dict(cta_group=2)])
def test_forward_other_groups_rows_reach_nothing(gemm, cfg):
    """NaN and infinities in one group's rows, weights, bias and scales."""
    sizes, N, K = [20, 37, 9], 136, 200
    bounds = _bounds(None, sizes)
    gen = torch.Generator().manual_seed(1)
    a, A = _operand(gen, 66, K, "f16")
    b, Bd = _weights(gen, 3, N, K, "f16")
    A, Bd = A.clone(), Bd.clone()
    A[20:57] = NAN
    A[30, 5] = INF
    Bd[1] = INF
    d = torch.zeros(66, N, device="cuda")
    gemm.set_config(**cfg)
    try:
        gemm.grouped_linear(A, Bd, _i32(bounds), d)
    finally:
        gemm.set_config(None)
    for g in (0, 2):
        rows = _rows(bounds, g)
        S = a[rows].abs() @ b[g].abs().T
        O.within(d[rows], a[rows] @ b[g].T, S * (ACCUM + 4 * O.U32), g)
    assert torch.isnan(d[20:57]).all()


@pytest.mark.gpu
def test_forward_most_groups(gemm):
    """4096 groups of 0 to 2 rows, by an index into few sets."""
    sizes = [i % 3 for i in range(4096)]
    _check_forward(gemm, sizes, 48, 40, "f16", index=[(7 * i) % 5 - 1 for i in range(4096)], sets=4,
                   r_t="f16", z_t="f32")
    gemm.set_config(cta_group=2)
    try:
        _check_forward(gemm, sizes, 48, 40, "f16", index=[(7 * i) % 5 - 1 for i in range(4096)],
                       sets=4, r_t="f16")
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[3, 0, 9], [200, 70, 900]])
def test_forward_repeats_bit_for_bit(gemm, sizes):
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    M, N, K = sum(sizes), 520, 712
    a, b, off = rnd(M, K), rnd(3, N, K), _i32(_bounds(None, sizes))
    outs = [torch.empty(M, N, device="cuda") for _ in range(4)]
    streams = [None, None, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o, s in zip(outs, streams):
        gemm.grouped_linear(a, b, off, o, activation="gelu", stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.gpu
def test_a_captured_call_follows_the_offsets(gemm):
    """One graph, replayed with other offsets, indices and rows behind the same addresses."""
    M, N, K = 300, 264, 136
    gen = torch.Generator().manual_seed(3)
    a, A = _operand(gen, M, K, "bf16")
    b, Bd = _weights(gen, 4, N, K, "bf16", scale=K ** -0.5)
    d = torch.empty(M, N, device="cuda")
    off, idx = _i32([0, 100, 200, 300]), _i32([0, 1, 2])
    gemm.grouped_linear(A, Bd, off, d, index=idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gemm.grouped_linear(A, Bd, off, d, index=idx, stream=torch.cuda.current_stream())
    for bounds, index in (([0, 1, 1, 300], [3, 0, 1]), ([0, 150, 299, 300], [1, 1, 2])):
        off.copy_(_i32(bounds))
        idx.copy_(_i32(index))
        d.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for g in range(3):
            rows = _rows(bounds, g)
            S = a[rows].abs() @ b[index[g]].abs().T
            O.within(d[rows], a[rows] @ b[index[g]].T, S * (ACCUM + 4 * O.U32), g)


@pytest.mark.gpu
def test_watchdog(gemm):
    a, b = torch.zeros(8, 64, device="cuda").half(), torch.zeros(1, 32, 64, device="cuda").half()
    d = torch.zeros(8, 32, device="cuda")
    for cg in (1, 2):
        gemm.set_config(cta_group=cg, inject_stall=1)
        G.gemm_set_timeout_ns(gemm.handle, 50_000_000)
        try:
            gemm.grouped_linear(a, b, _i32([0, 8]), d)
            st, detail = gemm.sync_status()
            assert st == G.GEMM_ERR_DEVICE_TIMEOUT and detail >> 24 == 0xE0, hex(detail)
        finally:
            G.gemm_set_timeout_ns(gemm.handle, 0)
            gemm.set_config(None)
        gemm.grouped_linear(a, b, _i32([0, 8]), d)
        assert gemm.sync_status()[0] == G.GEMM_OK


# ---------------------------------------------------------------- GPU, gradients

def _check_backward(gemm, sizes, N, K, t="bf16", act="none", da_t="bf16", db_t="bf16",
                    dbias_t="f32", accumulate=False, give=("dz", "da", "db", "dbias"),
                    alpha=1.0, pad=16, before=0, behind=0, in_place=None, fill=None, seed=0):
    """fill: what dd, z and a hold in rows of no group."""
    bounds = _bounds(None, sizes, before)
    M, E = bounds[-1] + behind, len(sizes)
    gen = torch.Generator().manual_seed(seed + 3 * M + 5 * N + K)
    dd, DD = _operand(gen, M, N, t, pad)
    z, Z = _operand(gen, M, N, t, pad)
    a, A = _operand(gen, M, K, t, pad)
    b, Bd = _weights(gen, E, N, K, t, False, pad, scale=max(K, 1) ** -0.5)
    others = torch.ones(M, dtype=torch.bool)
    others[bounds[0]:bounds[-1]] = False
    if fill is not None:
        for x in (DD, Z, A):
            x[others.cuda()] = fill
    rounded = lambda v: v.to(O.TYPES[t]).double()
    dz64, da64, db64, dbias64 = backward(dd, z, a, b, bounds, act, float(torch.tensor(alpha)),
                                         rounded)
    old = torch.randn(E * N, K, generator=gen).to(O.TYPES[db_t])
    nan = lambda *s: torch.full(s, NAN)
    out = {}
    if "dz" in give:
        out["dz"] = {None: None, "dd": (DD, None), "z": (Z, None)}[in_place] or \
            O.strided(nan(M, N), t, pad)
    if "da" in give:
        out["da"] = O.strided(nan(M, K), da_t, pad)
    if "db" in give:
        out["db"] = O.strided(old if accumulate else nan(E * N, K), db_t, pad)
    if "dbias" in give:
        out["dbias"] = (nan(E, N).to(O.TYPES[dbias_t]).cuda(), None)
    keep = O.f64(out["dz"][0]) if in_place else None
    kw = {k: v[0] for k, v in out.items()}
    if "db" in kw:
        kw["db"] = kw["db"].unflatten(0, (E, N))
    gemm.grouped_linear_bwd(DD, A if "db" in give else None, Bd if "da" in give else None,
                            _i32(bounds), z=Z if act != "none" else None, activation=act,
                            accumulate=accumulate, alpha=alpha, **kw)
    st, detail = gemm.sync_status()
    assert st == G.GEMM_OK, (G.gemm_status_string(st), hex(detail))
    mine = slice(bounds[0], bounds[-1])
    # the derivative's evaluation, then the rounding; a dz that rounds the other way differs by
    # one step of its type
    ez = dd.abs() * EVAL * (0 if act in ("none", "relu") else 1) + dz64.abs() * O.U32
    flip = ez + 2 * O.rounding(dz64.abs() + ez, t) if act not in ("none", "relu") else 0 * ez
    if "dz" in out:
        O.within(out["dz"][0][mine], dz64[mine], (ez + O.rounding(dz64.abs() + ez, t))[mine], "dz")
        if in_place:
            assert torch.equal(torch.nan_to_num(O.f64(out["dz"][0])[others], 7.0),
                               torch.nan_to_num(keep[others], 7.0))
        else:
            assert torch.isnan(O.f64(out["dz"][0])[others]).all()
            assert O.padding_untouched(*out["dz"])
    zero = torch.zeros_like(dz64)
    flip = torch.where(torch.isnan(flip), zero, flip)
    mag = torch.where(torch.isnan(dz64), zero, dz64.abs())
    for g in range(E):
        rows = _rows(bounds, g)
        al = abs(float(torch.tensor(alpha)))
        if "da" in out:
            S = al * mag[rows] @ b[g].abs()
            e = S * ACCUM + al * flip[rows] @ b[g].abs() + S * 4 * O.U32
            O.within(out["da"][0][rows], da64[rows], e + O.rounding(da64[rows].abs() + e, da_t), "da")
        if "db" in out:
            S = al * mag[rows].T @ a[rows].abs()
            e = S * ACCUM + al * flip[rows].T @ a[rows].abs() + S * 4 * O.U32
            want = db64[g]
            if accumulate:
                want = want + old.unflatten(0, (E, N))[g].double()
                e = e + (want.abs() + old.unflatten(0, (E, N))[g].double().abs()) * O.U32
            O.within(kw["db"][g], want, e + O.rounding(want.abs() + e, db_t), f"db {g}")
        if "dbias" in out:
            n = rows.stop - rows.start
            e = ez[rows].sum(0) + mag[rows].sum(0) * (n + 8) * O.U32
            O.within(out["dbias"][0][g], dbias64[g], e + O.rounding(dbias64[g].abs() + e, dbias_t),
                     "dbias")
    if "da" in out:
        assert torch.isnan(O.f64(out["da"][0])[others]).all() and O.padding_untouched(*out["da"])
    if "db" in out:
        assert O.padding_untouched(*out["db"])


BWD_SHAPES = [([1], 1, 1), ([1, 0, 2], 8, 16), ([0, 0], 40, 24), ([3, 1, 0, 4], 129, 77),
              ([16, 17, 15, 32], 257, 130), ([0, 65, 63, 1, 0], 136, 520), ([1] * 40, 72, 65),
              ([100, 0, 31, 5], 1003, 260), ([129, 257, 128], 264, 300), ([300, 65, 513], 520, 700),
              ([5, 600, 1, 250], 771, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", BWD_SHAPES)
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_backward_shapes(gemm, sizes, N, K, t):
    i = sum(sizes) + N + K
    _check_backward(gemm, sizes, N, K, t, ACTS[i % 5], da_t=["f16", "bf16", "f32"][i % 3],
                    db_t=["f32", "bf16", "f16"][i % 3], dbias_t=["f32", "bf16"][i % 2],
                    accumulate=i % 2 == 1, alpha=[1.0, 0.5][i % 2], before=i % 4, behind=i % 3)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [dict(cta_group=1, tile_n=64), dict(cta_group=1, tile_n=128),
                                 dict(cta_group=1, tile_n=192, stages=1),
                                 dict(cta_group=2, tile_n=128), dict(cta_group=2, tile_n=256),
                                 dict(cta_group=2, tile_n=256, stages=1)])
def test_backward_forced_configurations(gemm, cfg):
    gemm.set_config(**cfg)
    try:
        for sizes in ([40, 0, 1, 129, 15], [500, 300, 7, 64, 1]):
            _check_backward(gemm, sizes, 300, 203, "f16", "silu", db_t="f32", accumulate=True,
                            before=2, behind=90, fill=INF)
    finally:
        gemm.set_config(None)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", list(range(1, 36)) + [63, 64, 65, 127, 128, 129, 143, 144, 145])
def test_weight_gradient_of_every_remainder(gemm, rows):
    """Infinities in the next group's rows reach no group's weight gradient, nor does what the
    shared memory held before."""
    gen = torch.Generator().manual_seed(rows)
    N, K = 72, 136
    for cg in (1, 2):
        dd = torch.randn(2 * rows + 40, N, generator=gen).half()
        a = torch.randn(2 * rows + 40, K, generator=gen).half()
        bad = slice(rows, rows + 40)
        DD, A = O.strided(dd, "f16")[0], O.strided(a, "f16")[0]
        DD[bad], A[bad] = INF, NAN
        db = torch.empty(3, N, K, device="cuda")
        gemm.set_config(cta_group=cg)
        try:
            gemm.grouped_linear_bwd(DD, A, None, _i32([0, rows, rows + 40, 2 * rows + 40]), db=db)
        finally:
            gemm.set_config(None)
        for g, r in ((0, slice(0, rows)), (2, slice(rows + 40, None))):
            S = dd[r].double().T.abs() @ a[r].double().abs()
            O.within(db[g], dd[r].double().T @ a[r].double(), S * (ACCUM + 4 * O.U32), (cg, g))
        assert not torch.isfinite(db[1]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("give", [("dz",), ("dz", "da"), ("dz", "db"), ("dbias",), ("dz", "dbias"),
                                  ("dz", "da", "db")])
def test_backward_parts(gemm, give):
    for sizes in ([3, 5], [130, 0, 70]):
        _check_backward(gemm, sizes, 136, 72, "bf16", "gelu", give=give, behind=3, fill=NAN)


@pytest.mark.gpu
@pytest.mark.parametrize("give", [("da",), ("db",), ("da", "db", "dbias"), ("dbias",)])
def test_backward_without_activation_reads_dd(gemm, give):
    for sizes in ([3, 5], [130, 0, 70]):
        _check_backward(gemm, sizes, 136, 72, "f16", "none", da_t="f32", give=give, behind=3,
                        fill=NAN)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", ["dd", "z"])
def test_backward_in_place(gemm, in_place):
    for sizes in ([3, 5], [130, 0, 70]):
        _check_backward(gemm, sizes, 136, 72, "f16", "silu", in_place=in_place, before=2, behind=3)


@pytest.mark.gpu
def test_backward_no_rows(gemm):
    """Gradients of no rows are 0, or unchanged where they are added to."""
    e = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    for accumulate in (False, True):
        db, dbias = torch.ones(2, 40, 24, device="cuda"), torch.ones(2, 40, device="cuda")
        gemm.grouped_linear_bwd(e(0, 40), e(0, 24), e(2, 40, 24), _i32([0, 0, 0]), da=e(0, 24),
                                db=db, dbias=dbias, accumulate=accumulate)
        assert gemm.sync_status()[0] == G.GEMM_OK
        assert (db == float(accumulate)).all() and not dbias.any()


@pytest.mark.gpu
def test_backward_refused_configuration_changes_nothing(gemm):
    e = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
    out = dict(dz=e(8, 32), da=e(8, 64), db=e(1, 32, 64), dbias=e(1, 32))
    gemm.set_config(split_k=2)
    try:
        with pytest.raises(G.GemmError) as err:
            gemm.grouped_linear_bwd(e(8, 32) * 0, e(8, 64), e(1, 32, 64), _i32([0, 8]), z=e(8, 32),
                                    activation="silu", **out)
        assert err.value.status == G.GEMM_ERR_UNSUPPORTED_CONFIG
    finally:
        gemm.set_config(None)
    torch.cuda.synchronize()
    assert all((v == 1).all() for v in out.values())


@pytest.mark.gpu
def test_backward_repeats_bit_for_bit(gemm):
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    sizes = [200, 70, 0, 901]
    M, N, K = sum(sizes), 520, 264
    dd, z, a, b, off = rnd(M, N), rnd(M, N), rnd(M, K), rnd(4, N, K), _i32(_bounds(None, sizes))
    outs = []
    for s in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        o = dict(dz=torch.zeros(M, N, device="cuda").bfloat16(), da=torch.zeros(M, K, device="cuda"),
                 db=torch.zeros(4, N, K, device="cuda"), dbias=torch.zeros(4, N, device="cuda"))
        torch.cuda.synchronize()
        gemm.grouped_linear_bwd(dd, a, b, off, z=z, activation="gelu", stream=s, **o)
        outs.append(o)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(outs[0][k], o[k]) for k in o)


@pytest.mark.gpu
@pytest.mark.parametrize("cg", [1, 2])
@pytest.mark.parametrize("give", [("db",), ("da", "db")])
def test_watchdog_of_the_gradients(gemm, cg, give):
    """A stalled launch whose last blocks are zeroed by the warps of both CTAs ends with the error, and
    the next one is right."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()
    dd, a, b = rnd(323, 264), rnd(323, 520), rnd(2, 264, 520)
    out = dict(da=torch.zeros(323, 520, device="cuda").half(), db=torch.zeros(2, 264, 520, device="cuda").half())
    out = {k: out[k] for k in give}
    gemm.set_config(cta_group=cg, tile_n=128 * cg, inject_stall=1)
    G.gemm_set_timeout_ns(gemm.handle, 50_000_000)
    try:
        gemm.grouped_linear_bwd(dd, a, b, _i32([0, 5, 323]), **out)
        assert gemm.sync_status()[0] == G.GEMM_ERR_DEVICE_TIMEOUT
    finally:
        G.gemm_set_timeout_ns(gemm.handle, 0)
        gemm.set_config(cta_group=cg, tile_n=128 * cg)
    gemm.grouped_linear_bwd(dd, a, b, _i32([0, 5, 323]), **out)
    assert gemm.sync_status()[0] == G.GEMM_OK
    gemm.set_config(None)
    for g in range(2):
        rows = slice(0, 5) if g == 0 else slice(5, 323)
        want = O.f64(dd[rows]).T @ O.f64(a[rows])
        mag = O.f64(dd[rows]).abs().T @ O.f64(a[rows]).abs()
        O.within(out["db"][g], want, mag * ACCUM + O.rounding(want.abs() + mag * ACCUM, "f16"), "db")


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[37] + [0] * 14 + [3], [0] * 20 + [16, 17, 0, 1], [100] + [1] * 10, [0, 65, 0, 0, 0, 32, 33]])
@pytest.mark.parametrize("ab", ["bf16", "e4m3", "tf32"])
def test_forward_long_groups_among_short_ones(gemm, sizes, ab):
    """Tiles as narrow as the mean group suggests, and groups of several of them."""
    _check_forward(gemm, sizes, 263, 200, ab, d_t="bf16", act="silu", r_t="f32", z_t="f16", scales=ab == "e4m3",
                   before=2, behind=3)
    _check_forward(gemm, sizes, 264, 300, ab, d_t="f16", r_t="f16")
    if ab != "tf32":
        _check_forward(gemm, sizes, 136, 264, ab, d_t="f32", b_mn=True)
    else:
        _check_forward(gemm, sizes, 136, 264, ab, d_t="f32")
    mean = -(-sum(sizes) // len(sizes))
    assert gemm.last_config().tile_n == (16 if mean <= 4 else 32 if mean <= 16 else 64)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", [([100], 512, 520), ([70, 30], 136, 1032), ([300, 0, 1], 200, 264), ([90], 40, 130),
                                       ([1200], 1000, 512), ([2400], 264, 2056)])
def test_backward_in_one_launch_of_few_items(gemm, sizes, N, K):
    """Both gradients by one launch with the tiles that few items get, and each by itself."""
    for give in (("da", "db"), ("da",), ("db",)):
        _check_backward(gemm, sizes, N, K, "f16", da_t="f16", db_t="f16", give=give, before=3, behind=2)
    _check_backward(gemm, sizes, N, K, "bf16", act="gelu", da_t="bf16", db_t="bf16", accumulate=True)
