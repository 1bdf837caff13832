"""Arguments that no kernel of the operators whose weights change from row to row may be given: each
is refused on the host before anything is enqueued (a library that counts its calls), and by
shape, type and layout."""
import inspect

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from test_layer_arguments import Library, Placed, _handle


def _calls():
    """(method, its tensors by name), every optional one given."""
    e = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    f = lambda *s: torch.zeros(*s)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    m, n, s = e(4, 64), e(4, 32), i(4, 2)
    return [
        ("route", dict(index=torch.zeros(4, 2, dtype=torch.int64), offsets=i(9), slot=s, source=i(8))),
        ("dispatch", dict(x=m, slot=s, y=e(8, 64), scale=f(4), y_scale=f(8))),
        ("combine", dict(ys=e(8, 64), slot=s, y=m, weight=f(4, 2), residual=m)),
        ("combine_bwd", dict(dy=m, slot=s, dys=e(8, 64), weight=f(4, 2), ys=e(8, 64), dweight=f(4, 2))),
        ("grouped_linear", dict(a=m, b=e(3, 32, 64), offsets=i(3), d=n, index=i(2), bias=e(3, 32),
                                residual=n, z=n, row_scale=f(4), col_scale=f(3, 32))),
        ("grouped_linear_bwd", dict(dd=n, a=m, b=e(2, 32, 64), offsets=i(3), z=n, dz=n, da=m,
                                    db=e(2, 32, 64), dbias=f(2, 32))),
        ("adapters", dict(x=m, a=e(3, 8, 64), b=e(3, 32, 8), offsets=i(3), index=i(2), u=e(4, 8), d=n,
                          residual=n, scale=f(3))),
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
            for attr in ("data_ptr", "dtype", "shape", "stride"):
                setattr(self, attr, getattr(t, attr))

    getattr(_handle(lib, device), name)(**{k: Silent(t) for k, t in tensors.items()})
    assert lib.calls == 2


def test_every_tensor_argument_is_covered():
    for name, kw in _calls():
        other = {"self", "stream", "activation", "alpha", "accumulate"}
        assert set(kw) == set(inspect.signature(getattr(G.Gemm, name)).parameters) - other


INVALID, DTYPE = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE
e16 = lambda *s: torch.zeros(*s, dtype=torch.float16)
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)


@pytest.mark.parametrize("name,wrong,status", [
    ("route", dict(index=torch.zeros(4, 2)), DTYPE),
    ("route", dict(index=i32(8)), INVALID), ("route", dict(index=i32(2, 4).t()), INVALID),
    ("route", dict(slot=i32(8)), INVALID), ("route", dict(slot=torch.zeros(4, 2)), DTYPE),
    ("route", dict(slot=i32(4, 3)[:, :2]), INVALID), ("route", dict(source=i32(7)), INVALID),
    ("route", dict(offsets=i32(3, 3)), INVALID), ("route", dict(offsets=i32(0)), INVALID),
    ("route", dict(offsets=torch.zeros(9, dtype=torch.int64)), DTYPE),
    ("dispatch", dict(slot=i32(5, 2)), INVALID), ("dispatch", dict(y=e16(8, 65)), INVALID),
    ("dispatch", dict(y=torch.zeros(8, 64)), DTYPE), ("dispatch", dict(scale=torch.zeros(5)), INVALID),
    ("dispatch", dict(y_scale=e16(8)), DTYPE), ("dispatch", dict(x=e16(64, 4).t()), INVALID),
    ("combine", dict(slot=i32(5, 2)), INVALID), ("combine", dict(ys=e16(8, 63)), INVALID),
    ("combine", dict(weight=torch.zeros(4, 3)[:, :2]), INVALID), ("combine", dict(weight=e16(4, 2)), DTYPE),
    ("combine", dict(weight=torch.zeros(8)), INVALID), ("combine", dict(residual=e16(5, 64)), INVALID),
    ("combine", dict(ys=torch.zeros(8, 64, dtype=torch.int32)), DTYPE),
    ("combine_bwd", dict(dys=e16(9, 64)), INVALID), ("combine_bwd", dict(ys=torch.zeros(8, 64)), DTYPE),
    ("combine_bwd", dict(dweight=torch.zeros(2, 4).t()), INVALID),
    ("combine_bwd", dict(dys=e16(8, 128)[:, ::2]), INVALID),
    ("grouped_linear", dict(b=e16(32, 64)), INVALID), ("grouped_linear", dict(b=e16(3, 32, 63)), INVALID),
    ("grouped_linear", dict(b=e16(3, 32, 128)[:, ::2, ::2]), INVALID),
    ("grouped_linear", dict(index=i32(3)), INVALID), ("grouped_linear", dict(d=e16(4, 31)), INVALID),
    ("grouped_linear", dict(index=torch.zeros(2, dtype=torch.int64)), DTYPE),
    ("grouped_linear", dict(bias=e16(32)), INVALID), ("grouped_linear", dict(bias=e16(32, 3).t()), INVALID),
    ("grouped_linear", dict(col_scale=torch.zeros(3, 31)), INVALID),
    ("grouped_linear", dict(a=e16(64, 4).t()), INVALID), ("grouped_linear", dict(activation="swish"), INVALID),
    ("grouped_linear", dict(d=i32(4, 32)), DTYPE),
    ("grouped_linear_bwd", dict(b=e16(3, 32, 64)), INVALID),
    ("grouped_linear_bwd", dict(b=e16(2, 64, 32).transpose(1, 2)), INVALID),
    ("grouped_linear_bwd", dict(db=e16(2, 64, 32).transpose(1, 2)), INVALID),
    ("grouped_linear_bwd", dict(dbias=torch.zeros(32)), INVALID),
    ("grouped_linear_bwd", dict(z=torch.zeros(4, 32)), DTYPE),
    ("adapters", dict(a=e16(3, 8, 63)), INVALID), ("adapters", dict(b=e16(3, 8, 32).transpose(1, 2)), INVALID),
    ("adapters", dict(b=e16(2, 32, 8)), INVALID), ("adapters", dict(u=e16(4, 9)), INVALID),
    ("adapters", dict(u=torch.zeros(4, 8)), DTYPE), ("adapters", dict(scale=torch.zeros(2)), INVALID),
    ("adapters", dict(index=i32(3)), INVALID), ("adapters", dict(a=e16(8, 64)), INVALID),
])
def test_shapes_types_and_layouts(name, wrong, status):
    lib = Library()
    with pytest.raises(G.GemmError) as e:
        getattr(_handle(lib), name)(**{**{k: Placed(t, 0) for k, t in dict(_calls())[name].items()},
                                       **{k: Placed(t, 0) if isinstance(t, torch.Tensor) else t
                                          for k, t in wrong.items()}})
    assert e.value.status == status and lib.calls == 0


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
                        getattr(g, name)(**{k: host if k == wrong else t.cuda() for k, t in kw.items()})
                    assert e.value.status == G.GEMM_ERR_INVALID_ARG and wrong in str(e.value)
    finally:
        g.close()


@pytest.mark.gpu
def test_two_handles_on_two_streams_at_once():
    """Every operator by two handles, interleaved, gives what one alone gives."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, k, E, H, N = 300, 2, 5, 136, 264

    def problem(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
        R, i = T * k, torch.int32
        p = dict(x=rnd(T, H), index=torch.randint(0, E, (T, k), generator=gen, device="cuda"),
                 w=rnd(E, N, H), weight=torch.rand(T, k, generator=gen, device="cuda"), dy=rnd(T, N),
                 la=rnd(3, 8, H), lb=rnd(3, N, 8),
                 bounds=torch.tensor([0, 100, 101, T], dtype=i, device="cuda"),
                 which=torch.tensor([2, -1, 0], dtype=i, device="cuda"))
        o = dict(offsets=z(E + 1, dt=i), slot=z(T, k, dt=i), xs=z(R, H), ys=z(R, N), z=z(R, N), y=z(T, N),
                 dys=z(R, N), dw=z(T, k, dt=torch.float32), dz=z(R, N), da=z(R, H), db=z(E, N, H),
                 dbias=z(E, N), u=z(T, 8), d=z(T, N))
        return p, o

    def run(g, p, o, s):
        g.route(p["index"], o["offsets"], o["slot"], stream=s)
        g.dispatch(p["x"], o["slot"], o["xs"], stream=s)
        g.grouped_linear(o["xs"], p["w"], o["offsets"], o["ys"], activation="silu", z=o["z"], stream=s)
        g.combine(o["ys"], o["slot"], o["y"], weight=p["weight"], stream=s)
        g.combine_bwd(p["dy"], o["slot"], o["dys"], weight=p["weight"], ys=o["ys"], dweight=o["dw"],
                      stream=s)
        g.grouped_linear_bwd(o["dys"], o["xs"], p["w"], o["offsets"], z=o["z"], activation="silu",
                             dz=o["dz"], da=o["da"], db=o["db"], dbias=o["dbias"], stream=s)
        g.adapters(p["x"], p["la"], p["lb"], p["bounds"], p["which"], o["u"], o["d"], residual=o["y"],
                   stream=s)

    handles = [G.Gemm(0), G.Gemm(0)]
    try:
        alone = []
        for seed in (1, 2):
            p, o = problem(seed)
            run(handles[0], p, o, None)
            torch.cuda.synchronize()
            alone.append(o)
        both = [problem(1), problem(2)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(8):
            for h, (p, o), s in zip(handles, both, streams):
                run(h, p, o, s)
        torch.cuda.synchronize()
        for h, (_, o), want in zip(handles, both, alone):
            assert h.sync_status()[0] == G.GEMM_OK
            for name in want:
                assert torch.equal(o[name], want[name]), name
    finally:
        for h in handles:
            h.close()
