"""Arguments of the layer operators that no kernel may be given: each is refused on the host
before anything is enqueued.  Those that are somewhere else are tested with a library that
counts its calls."""
import ctypes
import inspect

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G


class Placed:
    """A CPU tensor that says it is on GPU `index`."""

    def __init__(self, t, index):
        self._t, self._index = t, index

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        return getattr(self._t, name)


class Library:
    """A library whose calls succeed and are counted."""
    calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return G.GEMM_OK
        return call


def _handle(lib, device=0):
    g = object.__new__(G.Gemm)
    g.handle, g.device, g._lib = None, device, lib
    return g


def _calls():
    """(method, its tensors by name), every optional one given."""
    e = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    f = lambda n: torch.zeros(n)
    m, n = e(4, 64), e(4, 32)
    return [
        ("rmsnorm", dict(x=m, weight=e(64), y=e(4, 64, dt=torch.float8_e4m3fn), residual=m, h=m,
                         scale=f(4), rstd=f(4))),
        ("rmsnorm_bwd", dict(dy=m, h=m, weight=e(64), rstd=f(4), dx=m, dweight=f(64), dh=m,
                             workspace=e(4096))),
        ("linear", dict(a=m, b=e(32, 64), d=n, bias=f(32), residual=n, z=n, row_scale=f(4),
                        col_scale=f(32))),
        ("linear_bwd", dict(dd=n, a=m, b=e(32, 64), z=n, dz=n, da=m, db=e(32, 64), dbias=f(32))),
    ]


TENSORS = [(name, k) for name, kw in _calls() for k in kw]


@pytest.mark.parametrize("name,wrong", TENSORS)
@pytest.mark.parametrize("where", [-1, 1])
def test_a_tensor_elsewhere_is_refused(name, wrong, where):
    """On the host, or on another GPU than the handle's."""
    kw = {k: Placed(t, where if k == wrong else 0) for k, t in dict(_calls())[name].items()}
    lib = Library()
    with pytest.raises(G.GemmError) as e:
        getattr(_handle(lib), name)(**kw)
    assert e.value.status == G.GEMM_ERR_INVALID_ARG and wrong in str(e.value)
    assert lib.calls == 0


@pytest.mark.parametrize("name", [name for name, _ in _calls()])
@pytest.mark.parametrize("device", [0, 3])
def test_tensors_on_the_handle_s_gpu_are_taken(name, device):
    """... and those that do not say where they are."""
    lib = Library()
    tensors = dict(_calls())[name]
    getattr(_handle(lib, device), name)(**{k: Placed(t, device) for k, t in tensors.items()})

    class Silent:
        def __init__(self, t):
            for attr in ("data_ptr", "dtype", "shape", "stride", "numel", "element_size"):
                setattr(self, attr, getattr(t, attr))

    getattr(_handle(lib, device), name)(**{k: Silent(t) for k, t in tensors.items()})
    assert lib.calls == 2


@pytest.mark.parametrize("workspace", [torch.zeros(1).expand(4096), torch.zeros(8192)[::2],
                                       torch.zeros(64, 64).t()])
def test_a_workspace_whose_bytes_lie_elsewhere_is_refused(workspace):
    """Its size is counted from its elements, which a stride can place on one another or among
    others'."""
    lib = Library()
    kw = {k: Placed(t, 0) for k, t in dict(_calls())["rmsnorm_bwd"].items()}
    with pytest.raises(G.GemmError) as e:
        _handle(lib).rmsnorm_bwd(**{**kw, "workspace": Placed(workspace, 0)})
    assert e.value.status == G.GEMM_ERR_INVALID_ARG and lib.calls == 0


def test_every_tensor_argument_is_covered():
    for name, kw in _calls():
        other = {"self", "eps", "stream", "activation", "alpha", "accumulate"}
        assert set(kw) == set(inspect.signature(getattr(G.Gemm, name)).parameters) - other


@pytest.mark.gpu
def test_host_tensors_are_refused_by_a_real_handle():
    """Each tensor in turn left on the host, pinned or not."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = G.Gemm(0)
    try:
        for name, kw in _calls():
            for wrong in kw:
                for host in (kw[wrong], kw[wrong].pin_memory()):
                    with pytest.raises(G.GemmError) as e:
                        getattr(g, name)(**{k: host if k == wrong else t.cuda()
                                            for k, t in kw.items()})
                    assert e.value.status == G.GEMM_ERR_INVALID_ARG and wrong in str(e.value)
        assert g.sync_status()[0] == G.GEMM_OK
    finally:
        g.close()


# ------------------------------------------------------------------ the C entry points' checks

@pytest.fixture(scope="module")
def lib():
    from dense_gemm_epilogue_persistent_gb300 import build as B
    B.build()
    return G.library()


P = [(i + 1) << 20 for i in range(10)]     # fake, aligned device addresses
LARGEST = (1 << 31) - 8193


def _linear(**kw):
    base = dict(M=4, N=64, K=64, a_type=G.GEMM_F16, b_type=G.GEMM_F16, d_type=G.GEMM_F16,
                activation=G.GEMM_ACT_GELU, alpha=1.0, A=P[0], B=P[1], bias=P[2], D=P[3])
    base.update(kw)
    up = lambda n: (n + 15) // 16 * 16
    return G.gemm_linear_t(lda=up(base["K"]), ldb=up(base["K"]), ldd=up(base["N"]), **base)


def _linear_bwd(**kw):
    base = dict(M=4, N=64, K=64, type=G.GEMM_F16, activation=G.GEMM_ACT_GELU, alpha=1.0,
                dd=P[0], z=P[1], a=P[2], b=P[3], dz=P[4], da=P[5], db=P[6], dbias=P[7])
    base.update(kw)
    up = lambda n: (n + 15) // 16 * 16
    n, k = up(base["N"]), up(base["K"])
    return G.gemm_linear_bwd_t(lddd=n, ldz=n, lda=k, ldb=k, lddz=n, ldda=k, lddb=k, **base)


@pytest.mark.parametrize("size", "MNK")
def test_sizes_end_before_a_32_bit_index_could_wrap(lib, size):
    """Kernels go on to the end of the last tile, whose width need not divide 2^31."""
    for make, check in ((_linear, G.gemm_linear_check), (_linear_bwd, G.gemm_linear_bwd_check)):
        for n, code in ((LARGEST, G.GEMM_OK), (LARGEST + 1, G.GEMM_ERR_INVALID_ARG),
                        ((1 << 31) - 1, G.GEMM_ERR_INVALID_ARG)):
            assert check(make(**{size: n})) == code, (check, n)


@pytest.mark.parametrize("at", [1, 2, 3])
def test_row_factors_off_their_elements_are_refused(lib, at):
    """rstd and scale are read and written as 4-byte elements."""
    fwd = dict(M=4, H=64, type=G.GEMM_BF16, w_type=G.GEMM_BF16, y_type=G.GEMM_E4M3, eps=1e-6, x=P[0],
               ldx=64, weight=P[1], y=P[2], ldy=64, scale=P[3], rstd=P[4])
    bwd = dict(M=4, H=64, type=G.GEMM_BF16, w_type=G.GEMM_BF16, dw_type=G.GEMM_F32, dy=P[0], lddy=64,
               h=P[1], ldh=64, weight=P[2], rstd=P[3], dx=P[4], lddx=64, dweight=P[5])
    for make, check, base, names in (
            (G.gemm_rmsnorm_t, G.gemm_rmsnorm_check, fwd, ("scale", "rstd")),
            (G.gemm_rmsnorm_bwd_t, G.gemm_rmsnorm_bwd_check, bwd, ("rstd",))):
        assert check(make(**base)) == G.GEMM_OK
        for name in names:
            assert check(make(**{**base, name: base[name] + 4})) == G.GEMM_OK
            assert check(make(**{**base, name: base[name] + at})) == G.GEMM_ERR_MISALIGNED


class Checked:
    """The library's host-only check in place of its call."""

    def __init__(self, lib):
        self.lib = lib

    def gemm_linear_bwd(self, handle, packed, stream):
        p = G.gemm_linear_bwd_t.from_buffer_copy(packed)
        return self.lib.gemm_linear_bwd_check(ctypes.byref(p))


@pytest.mark.parametrize("without,give,ok", [
    ("a", ("da",), True), ("b", ("db",), True), ("ab", (), True), ("a", (), True), ("b", (), True),
    ("a", ("db",), False), ("b", ("da",), False), ("a", ("da", "db"), False), ("ab", ("da",), False),
    ("ab", ("db",), False)])
def test_an_operand_no_gradient_reads_may_be_left_out(lib, without, give, ok):
    """a is read for db and b for da."""
    kw = {k: Placed(t, 0) for k, t in dict(_calls())["linear_bwd"].items()
          if k not in ("da", "db") or k in give}
    for k in without:
        kw[k] = None
    g = _handle(Checked(lib))
    if ok:
        g.linear_bwd(**kw, activation="gelu")
    else:
        with pytest.raises(G.GemmError) as e:
            g.linear_bwd(**kw, activation="gelu")
        assert e.value.status == G.GEMM_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 40, 72), (300, 264, 136)])
def test_gradients_without_the_operand_they_do_not_read(M, N, K):
    """The same bits with it and without."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = G.Gemm(0)
    try:
        gen = torch.Generator().manual_seed(M)
        dd, z, a, b = (torch.randn(*s, generator=gen).to("cuda", torch.bfloat16)
                       for s in ((M, N), (M, N), (M, K), (N, K)))
        new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        want, got = ({k: new(*s) for k, s in (("dz", (M, N)), ("da", (M, K)), ("db", (N, K)))}
                     for _ in range(2))
        for k, without in (("da", "a"), ("db", "b")):
            for outs, ab in ((want, dict(a=a, b=b)), (got, {**dict(a=a, b=b), without: None})):
                g.linear_bwd(dd, **ab, z=z, activation="silu", dz=outs["dz"], **{k: outs[k]})
        assert g.sync_status()[0] == G.GEMM_OK
        for k in want:
            assert torch.equal(want[k], got[k]) and (got[k] != 0).any(), k
    finally:
        g.close()


@pytest.mark.gpu
@pytest.mark.parametrize("cfg,give", [
    (cfg, give) for give in (("da", "db"), ("da",), ("db",))
    for cfg in (dict(split_k=1, tile_n=48),      # db's MN-major tokens: whole atoms (da takes it)
                dict(split_k=8),                 # more CTAs than k-blocks
                dict(split_k=2, tile_m=64),      # MN-major features: 128
                dict(cluster_m=2), dict(cta_group=1, tile_n=128, stages=12))
    if give != ("da",) or cfg != dict(split_k=1, tile_n=48)])
@pytest.mark.parametrize("over", [None, "dd", "z"])
def test_a_configuration_the_products_cannot_take_changes_nothing(cfg, give, over):
    """The gradients are planned before any of them is enqueued."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = G.Gemm(0)
    try:
        one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
        t = dict(dd=one(200, 128), z=one(200, 128), a=one(200, 64), b=one(128, 64))
        out = dict(da=one(200, 64), db=one(128, 64), dz=one(200, 128),
                   dbias=torch.ones(128, device="cuda"))
        out["dz"] = t.get(over, out["dz"])
        call = lambda: g.linear_bwd(**t, activation="gelu", dz=out["dz"], dbias=out["dbias"],
                                    **{k: out[k] for k in give})
        g.set_config(**cfg)
        with pytest.raises(G.GemmError) as e:
            call()
        assert e.value.status == G.GEMM_ERR_UNSUPPORTED_CONFIG
        torch.cuda.synchronize()
        assert all((v == 1).all() for v in (*t.values(), *out.values()))
        g.set_config(None)
        call()
        assert g.sync_status()[0] == G.GEMM_OK
        assert all((out[k] != 1).any() for k in ("dz", *give))
    finally:
        g.close()
