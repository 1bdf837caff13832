"""Root-mean-square normalisation and its backward pass: refusals (CPU), the
64-bit implementation against differences (CPU), and the kernels against it.

Tolerances are sums of rounding errors.  With u = 2^-24: the sum of squares of
a row is a chain of at most H/32 + 8 terms per thread, 5 lane adds and 32 warp
adds, its relative error at most (H/32 + 45) u, of which rstd takes half, plus
3 u of its own; h and the two products of y add 3 u; the result is rounded
once to the output's type."""
import itertools

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
import layer_oracle as O

EPS = 1e-6


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

P = [(i + 1) << 20 for i in range(8)]     # fake, aligned device addresses


def _fwd(**kw):
    base = dict(M=4, H=96, type=G.GEMM_BF16, w_type=G.GEMM_BF16, y_type=G.GEMM_E4M3, eps=EPS,
                x=P[0], ldx=96, r=P[1], ldr=96, weight=P[2], h=P[3], ldh=96, y=P[4], ldy=96,
                scale=P[5], rstd=P[6])
    base.update(kw)
    return G.gemm_rmsnorm_t(**base)


def _bwd(**kw):
    base = dict(M=4, H=96, type=G.GEMM_F16, w_type=G.GEMM_F32, dw_type=G.GEMM_F32, dy=P[0], lddy=96,
                h=P[1], ldh=96, weight=P[2], rstd=P[3], dh=P[4], lddh=96, dx=P[5], lddx=96,
                dweight=P[6])
    base.update(kw)
    return G.gemm_rmsnorm_bwd_t(**base)


INVALID, DTYPE, ALIGN = (G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE,
                         G.GEMM_ERR_MISALIGNED)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(M=0, x=None, y=None), 0), (dict(H=0), 0), (dict(r=None, h=None, rstd=None), 0),
    (dict(h=P[1]), 0), (dict(h=P[0]), 0),
    (dict(y_type=G.GEMM_BF16, scale=None), 0), (dict(y_type=G.GEMM_BF16, scale=None, y=P[0]), 0),
    (dict(H=95), 0), (dict(H=1), 0),
    (dict(M=-1), INVALID), (dict(H=-1), INVALID), (dict(M=1 << 31), INVALID),
    (dict(H=(1 << 31) - 1), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(weight=None), INVALID), (dict(ldx=88), INVALID), (dict(scale=None), INVALID),
    (dict(y_type=G.GEMM_BF16), INVALID),                         # a scale without 8 bits
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(h=P[1], ldh=104), INVALID), (dict(h=P[0], ldh=104), INVALID),
    (dict(y=P[0]), INVALID),                                     # 8 bits over 16
    (dict(y=P[3], y_type=G.GEMM_BF16, scale=None), INVALID),     # y over h
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(w_type=G.GEMM_E4M3), DTYPE),
    (dict(y_type=G.GEMM_TF32), DTYPE), (dict(type=9), DTYPE),
    (dict(x=P[0] + 8), ALIGN), (dict(ldx=100), ALIGN), (dict(r=P[1] + 2), ALIGN),
    (dict(ldh=100), ALIGN), (dict(y=P[4] + 8), ALIGN), (dict(ldy=104), ALIGN),
    (dict(weight=P[2] + 4), ALIGN),
])
def test_check_rmsnorm(lib, kw, code):
    assert G.gemm_rmsnorm_check(_fwd(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(M=0, dy=None, h=None, dx=None, rstd=None, weight=None), 0),
    (dict(H=0, dweight=None), 0), (dict(dh=None), 0), (dict(dx=P[4]), 0),
    (dict(M=-1), INVALID), (dict(dy=None), INVALID), (dict(h=None), INVALID),
    (dict(dx=None), INVALID), (dict(rstd=None), INVALID), (dict(weight=None), INVALID),
    (dict(dweight=None), INVALID), (dict(lddx=88), INVALID), (dict(dx=P[0]), INVALID),
    (dict(dx=P[1]), INVALID), (dict(dx=P[4], lddx=104), INVALID),
    (dict(type=G.GEMM_E5M2), DTYPE), (dict(dw_type=G.GEMM_TF32), DTYPE),
    (dict(w_type=-1), DTYPE), (dict(dy=P[0] + 4), ALIGN), (dict(ldh=100), ALIGN),
    (dict(dweight=P[6] + 4), ALIGN), (dict(dh=P[4] + 8), ALIGN),
])
def test_check_rmsnorm_bwd(lib, kw, code):
    assert G.gemm_rmsnorm_bwd_check(_bwd(**kw)) == code


def test_null_arguments(lib):
    assert lib.gemm_rmsnorm(None, None, None) == INVALID
    assert lib.gemm_rmsnorm_check(None) == INVALID
    assert lib.gemm_rmsnorm_bwd(None, None, None, 0, None) == INVALID
    assert lib.gemm_rmsnorm_bwd_check(None) == INVALID
    assert G.gemm_rmsnorm_bwd_workspace(0, 0) >= 0


def test_backward_formula_against_differences():
    """The 64-bit backward pass is the derivative of the 64-bit forward pass: central
    differences of step 1e-5 are off by about 1e-10 of curvature and 1e-11 of rounding."""
    gen = torch.Generator().manual_seed(0)
    M, H = 3, 7
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, w, dy, dh = rnd(M, H), rnd(H), rnd(M, H), rnd(M, H)

    def loss(x, w):
        h, _, y = O.rmsnorm(x, None, w, EPS)
        return float((y * dy).sum() + (h * dh).sum())

    h, rstd, _ = O.rmsnorm(x, None, w, EPS)
    dx, dw = O.rmsnorm_bwd(dy, h, w, rstd, dh)
    e = 1e-5
    for m, c in itertools.product(range(M), range(H)):
        d = torch.zeros_like(x)
        d[m, c] = e
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - float(dx[m, c])) < 1e-8
    for c in range(H):
        d = torch.zeros_like(w)
        d[c] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - float(dw[c])) < 1e-8


# ---------------------------------------------------------------- GPU

def _rel(H):
    """Relative error of y before its rounding."""
    return ((H / 32 + 45) / 2 + 6) * O.U32


def _inputs(M, H, t, seed, residual=True):
    gen = torch.Generator().manual_seed(seed)
    cast = lambda v: v.to(O.TYPES[t]).double()
    x = cast(torch.randn(M, H, generator=gen))
    r = cast(2 * torch.randn(M, H, generator=gen)) if residual else None
    return x, r, cast(0.5 + torch.rand(H, generator=gen))


def _check_forward(gemm, x, r, w, t, y_t, w_t=None, pad=16, alias=None, eps=EPS):
    """One call on padded copies, every output against the 64-bit result."""
    M, H = x.shape
    dev = lambda v: None if v is None else O.strided(v, t, pad)
    X, R = dev(x), dev(r)
    nan = torch.full((M, H), float("nan"))
    Hd = O.strided(nan, t, pad) if alias is None else {"x": X, "r": R}[alias]
    Y = O.strided(nan, y_t, pad)
    fp8 = y_t in O.TOP8
    scale = torch.full((M,), float("nan"), device="cuda") if fp8 else None
    rstd = torch.full((M,), float("nan"), device="cuda")
    gemm.rmsnorm(X[0], w.to("cuda", O.TYPES[w_t or t]), Y[0], residual=None if r is None else R[0],
                 h=Hd[0], scale=scale, rstd=rstd, eps=eps)
    torch.cuda.synchronize()
    h64, rstd64, y64 = O.rmsnorm(x, r, w, eps)
    e = _rel(H)
    O.within(rstd, rstd64, rstd64 * e, "rstd")
    O.within(Hd[0], h64, O.rounding(h64, t) * (1 + 2 * O.U32) + h64.abs() * O.U32, "h")
    if fp8:
        s64 = y64.abs().amax(dim=1).clamp(min=2.0 ** -100) / O.TOP8[y_t]
        O.within(scale, s64, s64 * (e + 2 * O.U32), "scale")
        q64 = y64 / s64[:, None]
        O.within(Y[0], q64, O.rounding(q64, y_t) * (1 + 4 * e) + q64.abs() * 3 * e, "q")
    else:
        O.within(Y[0], y64, O.rounding(y64, y_t) * (1 + 2 * e) + y64.abs() * e, "y")
    for v in (X, Hd, Y) + ((R,) if R else ()):
        assert O.padding_untouched(*v)
    if alias != "x":
        assert torch.equal(O.f64(X[0]), x)
    if R and alias != "r":
        assert torch.equal(O.f64(R[0]), r)


SIZES = [(1, 1), (3, 7), (2, 8), (5, 9), (1, 255), (17, 256), (9, 264), (4, 1000), (3, 1031),
         (2, 2048), (7, 4097), (1, 8192), (5, 8200), (2, 16384), (2, 16391), (1, 40001)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("t,y_t", [("bf16", "e4m3"), ("f16", "f16"), ("f32", "e5m2"),
                                   ("bf16", "f32"), ("f32", "bf16")])
def test_forward(gemm, M, H, t, y_t):
    _check_forward(gemm, *_inputs(M, H, t, M * 100000 + H), t, y_t)


@pytest.mark.gpu
@pytest.mark.parametrize("M,H", [(1, 8), (300, 520), (2000, 1024), (700, 5000)])
@pytest.mark.parametrize("y_t", ["f16", "e4m3"])
def test_forward_many_rows(gemm, M, H, y_t):
    _check_forward(gemm, *_inputs(M, H, "f16", M + H, residual=H % 3 != 0), "f16", y_t)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [40, 4104, 20000])
@pytest.mark.parametrize("w_t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_forward_weight_types_and_no_residual(gemm, H, t, w_t):
    x, _, w = _inputs(6, H, "bf16", H, residual=False)
    _check_forward(gemm, x, None, w, t, "f32", w_t, pad=0)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [24, 3000, 20001])
@pytest.mark.parametrize("alias", ["x", "r"])
def test_forward_in_place_stream(gemm, H, alias):
    """h over x or over the residual."""
    _check_forward(gemm, *_inputs(11, H, "bf16", H), "bf16", "e4m3", alias=alias)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [24, 3000, 20001])
def test_forward_y_in_place(gemm, H):
    x, r, w = _inputs(5, H, "f16", H)
    X, R = O.strided(x, "f16"), O.strided(r, "f16")
    gemm.rmsnorm(X[0], w.to("cuda", torch.float16), X[0], residual=R[0], h=R[0])
    h64, _, y64 = O.rmsnorm(x, r, w, EPS)
    e = _rel(H)
    O.within(X[0], y64, O.rounding(y64, "f16") * (1 + 2 * e) + y64.abs() * e, "y")
    O.within(R[0], h64, O.rounding(h64, "f16") * (1 + 2 * O.U32) + h64.abs() * O.U32, "h")


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 2056, 17000])
def test_forward_special_rows(gemm, H):
    """Rows of zeros, of values so small that their scale is the floor's, of the type's
    largest values, and (last) rows with a NaN or an infinity, which leave the others alone."""
    x = torch.zeros(6, H, dtype=torch.float64)
    x[1] = 2.0 ** -120                                        # squares vanish beside eps
    x[2] = torch.where(torch.arange(H) % 2 == 0, 1.0, -1.0) * 60000.0
    x[3] = torch.linspace(-1, 1, H, dtype=torch.float64)
    w = torch.ones(H, dtype=torch.float64)
    x[3] = x[3].to(torch.float32).double()
    _check_forward(gemm, x[:4], None, w, "f32", "e4m3")
    x[4] = 1.0
    x[4, H // 2] = float("nan")
    x[5] = 1.0
    x[5, 0] = float("inf")
    X, _ = O.strided(x, "f32")
    y, _ = O.strided(torch.zeros(6, H), "e4m3")
    scale, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    gemm.rmsnorm(X, w.to("cuda", torch.float32), y, scale=scale, rstd=rstd)
    assert torch.isnan(scale[4]) and torch.isnan(rstd[4]) and torch.isnan(y[4].float()).all()
    assert rstd[5] == 0 and torch.isnan(scale[5]) and torch.isnan(y[5, 0].float())
    assert (scale[0] == 2.0 ** -100 / 448) and (y[0].float() == 0).all()
    assert torch.isfinite(y[:4].float()).all()


@pytest.mark.gpu
def test_eps_zero_and_large_eps(gemm):
    x, r, w = _inputs(4, 512, "f32", 3)
    for eps in (0.0, 0.5):
        _check_forward(gemm, x, r, w, "f32", "f32", eps=eps)


def _check_backward(gemm, M, H, t, dw_t="f32", with_dh=True, pad=16, alias=False, w_t=None):
    gen = torch.Generator().manual_seed(M * 31 + H)
    cast = lambda v: v.to(O.TYPES[t]).double()
    h = cast(2 * torch.randn(M, H, generator=gen))
    dy = cast(torch.randn(M, H, generator=gen))
    dh = cast(torch.randn(M, H, generator=gen)) if with_dh else None
    w = (0.5 + torch.rand(H, generator=gen)).to(O.TYPES[w_t or t]).double()
    rstd = (1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)).float() if M else torch.empty(0)
    dy_d, h_d = O.strided(dy, t, pad), O.strided(h, t, pad)
    dh_d = O.strided(dh, t, pad) if with_dh else None
    dx_d = dh_d if alias else O.strided(torch.full((M, H), float("nan")), t, pad)
    dw_d = torch.full((H,), float("nan"), device="cuda").to(O.TYPES[dw_t])
    ws = torch.empty(max(1, G.gemm_rmsnorm_bwd_workspace(M, H)), dtype=torch.uint8, device="cuda")
    gemm.rmsnorm_bwd(dy_d[0], h_d[0], w.to("cuda", O.TYPES[w_t or t]), rstd.cuda(), dx_d[0], dw_d,
                     dh=dh_d[0] if with_dh else None, workspace=ws)
    torch.cuda.synchronize()
    dx64, dw64 = O.rmsnorm_bwd(dy, h, w, rstd.double(), dh)
    # the mean is a sum of H terms, chains of at most H/32 + 45, each of 3 roundings
    n, g = h * rstd.double()[:, None], dy * w
    size = rstd.double()[:, None] * (g.abs() + 2 * n.abs() * (g * n).abs().mean(1, keepdim=True))
    err = size * (H / 32 + 53) * O.U32 + (0 if dh is None else dh.abs() * 2 * O.U32)
    O.within(dx_d[0], dx64, O.rounding(dx64.abs() + err, t) + err, "dx")
    # a column's sum: M terms of 2 roundings, at worst one chain
    size = (dy * n).abs().sum(0)
    err = size * (M + 40) * O.U32
    O.within(dw_d, dw64, O.rounding(dw64.abs() + err, dw_t) + err, "dweight")
    assert O.padding_untouched(*dx_d) and torch.equal(O.f64(h_d[0]), h)
    assert torch.equal(O.f64(dy_d[0]), dy)


@pytest.mark.gpu
@pytest.mark.parametrize("M,H", SIZES + [(300, 520), (2000, 1024), (700, 5000), (1, 8), (33, 77)])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_backward(gemm, M, H, t):
    _check_backward(gemm, M, H, t, with_dh=(M + H) % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dw_t,w_t,alias", [("f16", "f32", True), ("bf16", "bf16", False),
                                            ("f32", "f16", True)])
@pytest.mark.parametrize("H", [72, 4096, 20000])
def test_backward_types_and_in_place(gemm, H, dw_t, w_t, alias):
    _check_backward(gemm, 37, H, "bf16", dw_t=dw_t, w_t=w_t, alias=alias, pad=0)


@pytest.mark.gpu
def test_backward_no_rows_gives_zero_weight_gradient(gemm):
    _check_backward(gemm, 0, 1000, "f16")


@pytest.mark.gpu
def test_same_bits_on_repeat_and_on_another_stream(gemm):
    """Both directions on a side stream, twice, and captured into a graph: the same bits."""
    x, r, w = _inputs(517, 3080, "bf16", 1)
    X, R = O.strided(x, "bf16")[0], O.strided(r, "bf16")[0]
    W_ = w.to("cuda", torch.bfloat16)
    ws = torch.empty(max(1, G.gemm_rmsnorm_bwd_workspace(517, 3080)), dtype=torch.uint8,
                     device="cuda")

    def outputs():
        e = lambda dt: torch.zeros(517, 3088, dtype=dt, device="cuda")[:, :3080]
        return dict(y=e(torch.float8_e4m3fn), h=e(torch.bfloat16), dx=e(torch.bfloat16),
                    scale=torch.zeros(517, device="cuda"), rstd=torch.zeros(517, device="cuda"),
                    dw=torch.zeros(3080, device="cuda"))

    def both(o, stream):
        gemm.rmsnorm(X, W_, o["y"], residual=R, h=o["h"], scale=o["scale"], rstd=o["rstd"],
                     stream=stream)
        gemm.rmsnorm_bwd(X, o["h"], W_, o["rstd"], o["dx"], o["dw"], dh=R, workspace=ws,
                         stream=stream)

    a, b, c = outputs(), outputs(), outputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(a, None)
    torch.cuda.synchronize()
    both(b, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(c, torch.cuda.current_stream())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in a:
        raw = lambda t: t.contiguous().view(torch.uint8)
        assert torch.equal(raw(a[k]), raw(b[k])) and torch.equal(raw(a[k]), raw(c[k])), k


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors(gemm):
    e = lambda *s, dt=torch.float16: torch.empty(*s, dtype=dt, device="cuda")
    x, w, y = e(4, 64), e(64), e(4, 64)
    for kw in (dict(x=e(4, 72)[:, :64].t().contiguous().t()), dict(weight=e(63)),
               dict(y=e(3, 64)), dict(residual=e(4, 64, dt=torch.bfloat16)),
               dict(scale=e(4, dt=torch.float32)), dict(rstd=e(4)),
               dict(y=e(4, 64, dt=torch.int8)), dict(weight=e(128)[::2])):
        with pytest.raises(G.GemmError):
            gemm.rmsnorm(**{**dict(x=x, weight=w, y=y), **kw})
    need = G.gemm_rmsnorm_bwd_workspace(4, 64)
    if need:
        with pytest.raises(G.GemmError):
            gemm.rmsnorm_bwd(x, x, w, e(4, dt=torch.float32), y, e(64))
