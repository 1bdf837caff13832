"""Where the tensors of the operators whose weights change from row to row may lie: rows and matrices so
far apart that their elements' offsets pass 2^31, sets of weights that are one matrix or lie
row by row beside one another.  Each call gives bit for bit what it gives for tensors that lie
close together (test_grouped, test_routing and test_adapters hold those against 64 bits)."""
import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G

pytestmark = pytest.mark.gpu
FAR = (1 << 23) + 16         # elements between rows: 300 rows of them are 2.5e9 elements
FAR_SETS = (1 << 30) + 16    # ... between three matrices


@pytest.fixture(scope="module")
def gemm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = G.Gemm(0)
    yield h
    h.close()


def _far(t):
    """t's values, its outermost rows (or matrices) far apart."""
    step = FAR_SETS if t.dim() == 3 else FAR
    room = torch.empty((t.shape[0] - 1) * step + t[0].numel() + 64, dtype=t.dtype, device="cuda")
    out = room.as_strided(t.shape, (step, *t[0].contiguous().stride()))
    return out.copy_(t)


def _both(gemm, call, given, outputs):
    """call(**tensors) for tensors close together and far apart."""
    near = {k: v.clone() for k, v in outputs.items()}
    call(**given, **near)
    assert gemm.sync_status()[0] == G.GEMM_OK
    spread = lambda v: _far(v) if v.dim() > 1 and v.dtype != torch.int32 else v.clone()
    far = {k: spread(v) for k, v in outputs.items()}
    call(**{k: spread(v) for k, v in given.items()}, **far)
    assert gemm.sync_status()[0] == G.GEMM_OK
    for k in near:
        assert not torch.equal(near[k], outputs[k]), k
        assert torch.equal(near[k], far[k]), k


T, K_, E, H, N = 300, 2, 3, 136, 264


def _tensors(seed, *shapes, t=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*s, generator=gen, device="cuda").to(t) for s in shapes]


def _slots(n):
    gen = torch.Generator(device="cuda").manual_seed(n)
    return torch.randperm(n, generator=gen, device="cuda").int()


def _zeros(*s, t=torch.bfloat16):
    return torch.zeros(*s, dtype=t, device="cuda")


def test_route(gemm):
    gen = torch.Generator(device="cuda").manual_seed(0)
    index = torch.randint(0, E, (T, K_), generator=gen, device="cuda", dtype=torch.int32)
    room = torch.empty((T - 1) * FAR + K_, dtype=torch.int32, device="cuda")
    far = room.as_strided((T, K_), (FAR, 1)).copy_(index)
    got = []
    for i in (index, far):
        offsets, slot = _zeros(E + 1, t=torch.int32), _zeros(T, K_, t=torch.int32)
        gemm.route(i, offsets, slot)
        got += [offsets, slot]
    assert gemm.sync_status()[0] == G.GEMM_OK
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float8_e4m3fn])
def test_dispatch(gemm, t):
    x, = _tensors(1, (T, 144), t=t)
    slot = _slots(2 * T)[:T].reshape(T, 1)           # (half of y's rows)
    _both(gemm, lambda x, y: gemm.dispatch(x.view(t), slot, y.view(t)),
          dict(x=x.view(torch.uint8)), dict(y=_zeros(2 * T, 144, t=t).view(torch.uint8)))


@pytest.mark.parametrize("width", [H, 2064])
def test_combine_and_its_gradients(gemm, width):
    """(Both kernels: 4 KB a row and 32 MB of choices' rows need many choices of the same rows.)"""
    k = 32 if width > H else 2
    ys, r, dy = _tensors(2, (T, width), (T, width), (T, width))
    weight = torch.rand(T, k, device="cuda")
    slot = torch.randint(-1, T, (T, k), device="cuda", dtype=torch.int32)
    _both(gemm, lambda ys, r, y: gemm.combine(ys, slot, y, weight=weight, residual=r),
          dict(ys=ys, r=r), dict(y=_zeros(T, width)))
    one = _slots(T).reshape(T, 1)
    dweight = _zeros(T, 1, t=torch.float32)
    _both(gemm, lambda dy, ys, dys: gemm.combine_bwd(dy, one, dys, weight=weight[:, :1].contiguous(),
                                                     ys=ys, dweight=dweight),
          dict(dy=dy, ys=ys), dict(dys=_zeros(T, width)))


@pytest.mark.parametrize("sizes", [[100, 0, 200], [3, 5, 292], [20, 30, 40]])
@pytest.mark.parametrize("whole", [True, False])
def test_grouped_linear(gemm, sizes, whole):
    a, b, r = _tensors(3, (T, H), (E, N, H), (T, N))
    bounds = torch.tensor([0, *sizes], device="cuda").cumsum(0).int()
    if whole:
        _both(gemm, lambda a, b, r, z, d: gemm.grouped_linear(a, b, bounds, d, activation="silu", z=z,
                                                              residual=r),
              dict(a=a, b=b, r=r), dict(z=_zeros(T, N), d=_zeros(T, N)))
    else:
        _both(gemm, lambda a, b, r, d: gemm.grouped_linear(a, b, bounds, d, residual=r),
              dict(a=a, b=b, r=r), dict(d=_zeros(T, N)))


@pytest.mark.parametrize("sizes", [[100, 0, 200], [3, 5, 292]])
def test_grouped_linear_bwd(gemm, sizes):
    dd, z, a, b = _tensors(4, (T, N), (T, N), (T, H), (E, N, H))
    bounds = torch.tensor([0, *sizes], device="cuda").cumsum(0).int()
    for accumulate in (False, True):
        _both(gemm, lambda dd, z, a, b, dz, da, db: gemm.grouped_linear_bwd(
            dd, a, b, bounds, z=z, activation="gelu", dz=dz, da=da, db=db, accumulate=accumulate),
            dict(dd=dd, z=z, a=a, b=b), dict(dz=_zeros(T, N), da=_zeros(T, H), db=_zeros(E, N, H)))


@pytest.mark.parametrize("sizes", [[100, 0, 200], [1, 299, 0], [1, 1, 1]])
def test_adapters(gemm, sizes):
    rows = max(3, sum(sizes))
    x, a, b, r = _tensors(5, (rows, H), (E, 16, H), (E, N, 16), (rows, N))
    bounds = torch.tensor([0, *sizes], device="cuda").cumsum(0).int()
    index = torch.tensor([2, 1, 0], dtype=torch.int32, device="cuda")
    _both(gemm, lambda x, a, b, r, u, d: gemm.adapters(x, a, b, bounds, index, u, d, residual=r),
          dict(x=x, a=a, b=b, r=r, u=_zeros(rows, 16)), dict(d=_zeros(rows, N)))


@pytest.mark.parametrize("sizes", [[1, 2, 1], [100, 0, 200]])
@pytest.mark.parametrize("layout", ["one matrix", "row by row", "features contiguous"])
def test_sets_of_weights(gemm, sizes, layout):
    """Sets that are one matrix, rows of the sets in turn, and matrices of contiguous features, as
    the forward pass, its gradient and the adapters read them."""
    M = sum(sizes)
    a, b, dd, x = _tensors(6, (M, H), (E, N, H), (M, N), (M, N))
    la, lb = _tensors(7, (E, 16, N), (E, H, 16))
    bounds = torch.tensor([0, *sizes], device="cuda").cumsum(0).int()
    index = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")

    def lie(w):
        if layout == "one matrix":
            return w[:1].expand(E, -1, -1)
        if layout == "row by row":
            return w.transpose(0, 1).contiguous().transpose(0, 1)
        return w.transpose(1, 2).contiguous().transpose(1, 2)

    def run(w, la, lb):
        d, da, u, e = _zeros(M, N), _zeros(M, H), _zeros(M, 16), _zeros(M, H)
        gemm.grouped_linear(a, w, bounds, d, index=index)
        if w.stride(2) == 1:
            gemm.grouped_linear_bwd(dd, a, w, bounds, da=da)
            gemm.adapters(x, la, lb, bounds, index, u, e)
        assert gemm.sync_status()[0] == G.GEMM_OK
        return d, da, e
    got = run(lie(b), lie(la), lie(lb))
    want = run(*(lie(w).contiguous() for w in (b, la, lb)))
    if layout == "features contiguous":              # another layout of the matrix units' operand:
        # each result is off by at most 2^-10 of its terms' magnitudes (below H), and rounded
        torch.testing.assert_close(got[0].float(), want[0].float(), rtol=2 ** -7, atol=2 ** -9 * H)
    else:
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_calls_of_one_graph_share_nothing(gemm):
    """Two captured graphs of the same calls, replayed at once on two streams with tensors of their
    own, and one of them twice in a row."""
    bounds = torch.tensor([0, 40, 100, 300], dtype=torch.int32, device="cuda")
    sets = [_tensors(10 + i, (T, H), (E, N, H), (T, N)) for i in range(2)]
    outs = [[_zeros(T, N), _zeros(T, H), _zeros(E, N, H), _zeros(E, N, t=torch.float32), _zeros(T, N)]
            for _ in sets]

    def step(s, o):
        stream = torch.cuda.current_stream()
        gemm.grouped_linear(s[0], s[1], bounds, o[0], stream=stream)
        gemm.grouped_linear_bwd(s[2], s[0], s[1], bounds, z=o[0], activation="gelu", dz=o[4], da=o[1],
                                db=o[2], dbias=o[3], stream=stream)
    for s, o in zip(sets, outs):
        with torch.cuda.stream(torch.cuda.Stream()):
            step(s, o)
        torch.cuda.synchronize()
    want = [[t.clone() for t in o] for o in outs]
    graphs = []
    for s, o in zip(sets, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s, o)
        graphs.append(graph)
        for t in o:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for graph, stream in zip(graphs + graphs[:1], streams + streams[:1]):
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    assert gemm.sync_status()[0] == G.GEMM_OK
    for o, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(o, w))
