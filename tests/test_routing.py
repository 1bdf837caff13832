"""Tokens sorted by expert and back: refusals (CPU), the 64-bit formulas against differences
(CPU), and the kernels against plain torch.

Tolerances: the sort and the copy are exact.  A sum of k weighted rows and a residual in fp32 is off
by at most (k + 1) u of its terms' magnitudes, u = 2^-24; a weighted row by u; a sum of H products
by at most (H / 16 + 40) u of its terms' magnitudes (a thread adds up to H / 256 vectors of 8 products
each in turn, rows shorter than that fewer, then lanes and warps); results are rounded once."""
import ctypes
import itertools

import pytest
import torch

import dense_gemm_epilogue_persistent_gb300 as G
from dense_gemm_epilogue_persistent_gb300 import build as B
import layer_oracle as O

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

P = [(i + 1) << 20 for i in range(10)]     # fake, aligned device addresses
OK, INVALID, DTYPE, ALIGN = (0, G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED_DTYPE,
                             G.GEMM_ERR_MISALIGNED)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(T=0, index=None, slot=None), OK), (dict(k=0, index=None, slot=None), OK),
    (dict(source=None), OK), (dict(E=0), OK), (dict(E=4096, k=128, ldi=128), OK), (dict(ldi=9), OK),
    (dict(index=P[0] + 4), OK), (dict(index_bytes=8), OK),
    (dict(T=-1), INVALID), (dict(k=129, ldi=200), INVALID), (dict(E=4097), INVALID),
    (dict(E=-1), INVALID), (dict(T=1 << 30, k=4), INVALID), (dict(ldi=2), INVALID),
    (dict(index=None), INVALID), (dict(slot=None), INVALID), (dict(offsets=None), INVALID),
    (dict(T=0, offsets=None), INVALID), (dict(slot=P[1]), INVALID), (dict(source=P[2]), INVALID),
    (dict(source=P[1]), INVALID), (dict(index=P[2]), INVALID), (dict(index=P[3]), INVALID),
    (dict(index=P[1]), INVALID), (dict(index_bytes=2), DTYPE), (dict(index_bytes=0), DTYPE),
    (dict(index=P[0] + 2), ALIGN), (dict(index_bytes=8, index=P[0] + 4), ALIGN),
    (dict(offsets=P[1] + 2), ALIGN), (dict(slot=P[2] + 1), ALIGN), (dict(source=P[3] + 3), ALIGN),
])
def test_check_route(lib, kw, code):
    base = dict(T=5, k=3, E=7, index_bytes=4, index=P[0], ldi=3, offsets=P[1], slot=P[2],
                source=P[3])
    assert G.gemm_route_check(G.gemm_route_t(**{**base, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(T=0, x=None, slot=None), OK), (dict(k=0, slot=None), OK), (dict(H=0), OK),
    (dict(R=0, y=None), OK), (dict(type=G.GEMM_F32), OK), (dict(scale=None, y_scale=None), OK),
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(H=1 << 31), INVALID), (dict(k=129), INVALID),
    (dict(slot=None), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(scale=None), INVALID), (dict(y_scale=None), INVALID), (dict(y_scale=P[3]), INVALID),
    (dict(y=P[0]), INVALID), (dict(ldx=16), INVALID), (dict(ldy=16), INVALID),
    (dict(type=G.GEMM_TF32), DTYPE), (dict(type=9), DTYPE),
    (dict(x=P[0] + 8), ALIGN), (dict(ldx=40), ALIGN), (dict(ldy=40), ALIGN),
    (dict(y=P[2] + 1), ALIGN), (dict(scale=P[3] + 2), ALIGN), (dict(slot=P[1] + 2), ALIGN),
])
def test_check_dispatch(lib, kw, code):
    base = dict(T=5, k=3, H=30, R=9, type=G.GEMM_E4M3, x=P[0], ldx=32, slot=P[1], y=P[2], ldy=32,
                scale=P[3], y_scale=P[4])
    assert G.gemm_dispatch_check(G.gemm_dispatch_t(**{**base, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(T=0, ys=None, slot=None, y=None), OK), (dict(k=0, slot=None, ys=None), OK),
    (dict(R=0, ys=None), OK), (dict(H=0), OK), (dict(weight=None, r=None), OK), (dict(r=P[4]), OK),
    (dict(T=-1), INVALID), (dict(slot=None), INVALID), (dict(ys=None), INVALID),
    (dict(y=None), INVALID), (dict(ldys=16), INVALID), (dict(ldr=16), INVALID),
    (dict(ldy=16), INVALID), (dict(y=P[0]), INVALID), (dict(r=P[4], ldr=40), INVALID),
    (dict(r=P[4], r_type=G.GEMM_F16), INVALID), (dict(k=200), INVALID),
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(y_type=G.GEMM_E5M2), DTYPE), (dict(r_type=5), DTYPE),
    (dict(ys=P[0] + 2), ALIGN), (dict(ldys=36), ALIGN), (dict(weight=P[2] + 2), ALIGN),
    (dict(slot=P[1] + 1), ALIGN), (dict(r=P[3] + 8), ALIGN),
])
def test_check_combine(lib, kw, code):
    base = dict(T=5, k=3, H=30, R=9, type=G.GEMM_F16, r_type=G.GEMM_BF16, y_type=G.GEMM_BF16,
                ys=P[0], ldys=32, slot=P[1], weight=P[2], r=P[3], ldr=32, y=P[4], ldy=32)
    assert G.gemm_combine_check(G.gemm_combine_t(**{**base, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(T=0, dy=None, slot=None), OK), (dict(k=0, slot=None), OK), (dict(H=0), OK),
    (dict(R=0, ys=None, dys=None), OK), (dict(weight=None), OK), (dict(dys=None), OK),
    (dict(dweight=None, ys=None), OK), (dict(dys=P[3]), OK),
    (dict(T=-1), INVALID), (dict(slot=None), INVALID), (dict(dy=None), INVALID),
    (dict(ys=None), INVALID), (dict(lddy=16), INVALID), (dict(ldys=16), INVALID),
    (dict(lddys=16), INVALID), (dict(dys=P[0]), INVALID), (dict(dys=P[3], lddys=40), INVALID),
    (dict(dweight=P[2]), INVALID), (dict(k=129), INVALID),
    (dict(type=G.GEMM_E4M3), DTYPE), (dict(type=5), DTYPE),
    (dict(dy=P[0] + 2), ALIGN), (dict(lddys=36), ALIGN), (dict(weight=P[2] + 2), ALIGN),
    (dict(dweight=P[5] + 1), ALIGN), (dict(slot=P[1] + 1), ALIGN),
])
def test_check_combine_bwd(lib, kw, code):
    base = dict(T=5, k=3, H=30, R=9, type=G.GEMM_F16, dy=P[0], lddy=32, slot=P[1], weight=P[2],
                ys=P[3], ldys=32, dys=P[4], lddys=32, dweight=P[5])
    assert G.gemm_combine_bwd_check(G.gemm_combine_bwd_t(**{**base, **kw})) == code


def test_packed_calls_match_the_structures():
    """The tensor calls pack the C structures by format: same size, every field in its place."""
    for fmt, cls in ((G._ROUTE, G.gemm_route_t), (G._DISPATCH, G.gemm_dispatch_t),
                     (G._COMBINE, G.gemm_combine_t), (G._COMBINE_BWD, G.gemm_combine_bwd_t)):
        values = [float(i + 1) if t is ctypes.c_float else i + 1
                  for i, (_, t) in enumerate(cls._fields_)]
        assert fmt.size == ctypes.sizeof(cls)
        assert fmt.pack(*values) == bytes(cls(*values)), cls


def test_null_arguments(lib):
    for name in ("gemm_route", "gemm_dispatch", "gemm_combine", "gemm_combine_bwd"):
        assert getattr(lib, name)(None, None, None) == INVALID
        assert getattr(lib, name + "_check")(None) == INVALID


def combine(ys, slot, weight, r):
    """In 64 bits; places outside ys add nothing."""
    y = torch.zeros(slot.shape[0], ys.shape[1], dtype=torch.float64) if r is None else r.clone()
    for t, j in itertools.product(*(range(n) for n in slot.shape)):
        if 0 <= slot[t, j] < ys.shape[0]:
            y[t] += (1.0 if weight is None else weight[t, j]) * ys[slot[t, j]]
    return y


def combine_bwd(dy, slot, weight, ys):
    """(dys, dweight) in 64 bits; rows that no choice has are NaN."""
    dys = torch.full_like(ys, NAN)
    dweight = torch.zeros(slot.shape, dtype=torch.float64)
    for t, j in itertools.product(*(range(n) for n in slot.shape)):
        if 0 <= slot[t, j] < ys.shape[0]:
            dys[slot[t, j]] = (1.0 if weight is None else weight[t, j]) * dy[t]
            dweight[t, j] = (dy[t] * ys[slot[t, j]]).sum()
    return dys, dweight


def test_combine_s_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    slot = torch.tensor([[2, 0, -1], [1, 4, 3]])
    ys, weight, dy = rnd(5, 4), rnd(2, 3), rnd(2, 4)
    loss = lambda ys, weight: float((combine(ys, slot, weight, None) * dy).sum())
    grads = combine_bwd(dy, slot, weight, ys)
    e = 1e-6
    for i, grad in enumerate(grads):
        for at in itertools.product(*(range(n) for n in (ys, weight)[i].shape)):
            up, down = [ys, weight], [ys, weight]
            up[i], down[i] = up[i].clone(), down[i].clone()
            up[i][at] += e
            down[i][at] -= e
            assert abs((loss(*up) - loss(*down)) / (2 * e) - float(grad[at])) < 1e-8
    # dispatch copies a row to its choices' places: its gradient is their unweighted sum
    x = rnd(2, 4)
    g = rnd(5, 4)
    copied = lambda x: combine_bwd(x, slot, None, ys)[0]
    d = combine(g, slot, None, None)
    for at in itertools.product(range(2), range(4)):
        up, down = x.clone(), x.clone()
        up[at] += e
        down[at] -= e
        diff = (copied(up) - copied(down)).nan_to_num(0.0) / (2 * e)
        assert abs(float((diff * g).sum()) - float(d[at])) < 1e-8


# ---------------------------------------------------------------- GPU

def sort(index, E):
    """(offsets, slot, source) with Python's stable sort."""
    flat = index.reshape(-1).tolist()
    order = sorted((i for i, e in enumerate(flat) if 0 <= e < E), key=lambda i: flat[i])
    slot = [-1] * len(flat)
    for place, i in enumerate(order):
        slot[i] = place
    offsets = [sum(1 for i in order if flat[i] < e) for e in range(E)] if E < 50 else None
    if offsets is None:
        counts = [0] * E
        for i in order:
            counts[flat[i]] += 1
        offsets = [sum(counts[:e]) for e in range(E)] if E < 300 else \
            [0] + list(itertools.accumulate(counts))[:-1]
    return offsets + [len(order)], slot, order


def _check_route(gemm, index, E, wide=False, ld=None, source=True, stream=None):
    T, k = index.shape
    dtype = torch.int64 if wide else torch.int32
    dev = torch.full((max(T, 1), ld or max(k, 1)), 0, dtype=dtype, device="cuda")[:T, :k]
    dev.copy_(index)
    offsets = torch.full((E + 3,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full((T * k + 2,), -7, dtype=torch.int32, device="cuda")
    src = torch.full((T * k + 2,), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    gemm.route(dev, offsets[1:E + 2], slot[1:T * k + 1].view(T, k),
               source=src[1:T * k + 1] if source else None, stream=stream)
    assert gemm.sync_status(stream)[0] == G.GEMM_OK
    want = sort(index, E)
    assert offsets.tolist() == [-7] + want[0] + [-7]
    assert slot.tolist() == [-7] + want[1] + [-7]
    left = T * k - len(want[2])
    assert src.tolist() == ([-7] + want[2] + [-7] * (left + 1) if source else [-7] * (T * k + 2))


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (31, 1, 2), (33, 3, 7),
                                   (100, 8, 64), (1000, 2, 8), (1024, 2, 300), (1025, 2, 9),
                                   (2048, 1, 4096), (777, 8, 60), (4099, 4, 128), (8192, 8, 64),
                                   (5, 128, 256), (9000, 1, 1), (3000, 3, 4096), (70000, 2, 17)])
@pytest.mark.parametrize("wide", [False, True])
def test_route(gemm, T, k, E, wide):
    gen = torch.Generator().manual_seed(T + k + E)
    index = torch.randint(0, E, (T, k), generator=gen)
    _check_route(gemm, index, E, wide)
    # few experts, and choices of none
    index = (index % max(1, E // 5)) * torch.randint(-1, 2, (T, k), generator=gen).clamp(-1, 1)
    index[0, 0] = E
    index[-1, -1] = (1 << 40) + 1 if wide else (1 << 31) - 1
    _check_route(gemm, index, E, wide, ld=k + 3, source=T % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 5000])
def test_route_all_or_none(gemm, T):
    for value, E in ((0, 4), (3, 4), (-1, 4), (4, 4), (0, 0)):
        _check_route(gemm, torch.full((T, 2), value), E)
    _check_route(gemm, torch.zeros(0, 2, dtype=torch.int64), 3)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f32", "f16", "bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("T,k,H", [(1, 8, 4096), (3, 1, 1), (5, 3, 7), (64, 2, 130), (33, 8, 1031),
                                   (9, 4, 512), (2, 2, 20001), (300, 5, 264), (1, 128, 48)])
def test_dispatch(gemm, t, T, k, H):
    gen = torch.Generator().manual_seed(T + H)
    R = T * k + 2
    slot = torch.randperm(R, generator=gen)[:T * k].view(T, k)
    drop = torch.rand(T, k, generator=gen) < 0.2
    slot[drop] = torch.tensor([-1, R, -5, (1 << 31) - 1])[torch.arange(int(drop.sum())) % 4]
    x = torch.randn(T, H, generator=gen).to(O.TYPES[t])
    X = O.strided(x.float(), t)
    Y = O.strided(torch.full((R, H), NAN), t)
    scaled = t in O.TOP8
    scale = torch.rand(T, generator=gen)
    y_scale = torch.full((R,), NAN, device="cuda")
    gemm.dispatch(X[0], slot.int().cuda(), Y[0], scale=scale.cuda() if scaled else None,
                  y_scale=y_scale if scaled else None)
    assert gemm.sync_status()[0] == G.GEMM_OK
    want, ws = torch.full((R, H), NAN), torch.full((R,), NAN)
    for i, j in itertools.product(range(T), range(k)):
        if 0 <= slot[i, j] < R:
            want[slot[i, j]] = x[i].float()
            ws[slot[i, j]] = scale[i]
    assert torch.equal(torch.nan_to_num(Y[0].cpu().float(), 1e9), torch.nan_to_num(want, 1e9))
    assert O.padding_untouched(*Y)
    if scaled:
        assert torch.equal(torch.nan_to_num(y_scale.cpu(), 9.0), torch.nan_to_num(ws, 9.0))


@pytest.mark.gpu
def test_dispatch_keeps_bits(gemm):
    """Whatever the bits are: NaN payloads, infinities, negative zeros."""
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(256, 256).cuda()
    y = torch.zeros(256, 256, dtype=torch.int16, device="cuda")
    slot = torch.arange(255, -1, -1, dtype=torch.int32, device="cuda").view(256, 1)
    gemm.dispatch(x.view(torch.bfloat16), slot, y.view(torch.bfloat16))
    torch.cuda.synchronize()
    assert torch.equal(y, x.flip(0))


def _places(gen, T, k, R):
    slot = torch.randperm(max(R, T * k), generator=gen)[:T * k].view(T, k)
    drop = torch.rand(T, k, generator=gen) < 0.15
    slot[drop] = torch.tensor([-1, R, -(1 << 31), (1 << 31) - 1])[torch.arange(int(drop.sum())) % 4]
    return slot


SIZES = [(1, 8, 4096), (3, 1, 1), (5, 3, 7), (64, 2, 130), (33, 8, 1031), (9, 4, 520), (2, 2, 20001),
         (100, 5, 264), (1, 128, 48), (40, 7, 2048)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", SIZES)
@pytest.mark.parametrize("t,r_t,y_t,weighted", [("bf16", "bf16", "bf16", True),
                                                ("f16", None, "f32", True), ("f32", "f16", "f32", False),
                                                ("f16", "f32", "bf16", True), ("bf16", None, "f16", False)])
def test_combine(gemm, T, k, H, t, r_t, y_t, weighted):
    gen = torch.Generator().manual_seed(T + k + H)
    R = T * k + 1
    slot = _places(gen, T, k, R)
    ys = torch.randn(R, H, generator=gen).to(O.TYPES[t])
    r = torch.randn(T, H, generator=gen).to(O.TYPES[r_t]) if r_t else None
    weight = torch.randn(T, k, generator=gen) if weighted else None
    if weighted:
        weight[(slot < 0) | (slot >= R)] = NAN            # (of no choice)
    YS, Y = O.strided(ys.float(), t), O.strided(torch.full((T, H), NAN), y_t)
    gemm.combine(YS[0], slot.int().cuda(), Y[0], weight=weight.cuda() if weighted else None,
                 residual=O.strided(r.float(), r_t)[0] if r_t else None)
    assert gemm.sync_status()[0] == G.GEMM_OK
    w64 = weight.double() if weighted else None
    want = combine(ys.double(), slot, w64, r.double() if r_t else None)
    mag = combine(ys.double().abs(), slot, w64.abs() if weighted else None,
                  r.double().abs() if r_t else None)
    e = mag * (k + 1) * O.U32
    O.within(Y[0], want, e + O.rounding(want.abs() + e, y_t), "y")
    assert O.padding_untouched(*Y)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,t,r_t,y_t,weighted", [
    (1500, 3, 5003, "f16", "f16", "f16", True), (2100, 4, 2048, "bf16", "bf16", "f32", True),
    (2000, 1, 9001, "bf16", None, "bf16", False), (600, 40, 1025, "f32", "f32", "f32", True),
    (700, 6, 4100, "f16", "f32", "bf16", True), (410, 2, 20011, "bf16", "f16", "f16", False),
    (301, 33, 2051, "f16", "f16", "f16", True)])
def test_combine_of_large_batches(gemm, T, k, H, t, r_t, y_t, weighted):
    """Those whose rows come through a ring: rows ending inside 16 bytes, the last row of each matrix
    among the choices, tokens without any, more choices than lanes."""
    gen = torch.Generator().manual_seed(T + k + H)
    R = T * k + 1 - T // 3
    slot = _places(gen, T, k, T * k).clamp(max=T * k)
    slot[slot >= R] = R + 3
    slot[1] = -1
    slot[0, 0] = R - 1
    ys = torch.randn(R, H, generator=gen).to(O.TYPES[t])
    r = torch.randn(T, H, generator=gen).to(O.TYPES[r_t]) if r_t else None
    weight = torch.randn(T, k, generator=gen) if weighted else None
    there = (slot >= 0) & (slot < R)
    if weighted:
        weight[~there] = NAN
    # no padding behind the last row: the buffer ends with it
    tight = lambda v, n: torch.empty((n - 1) * ((H + 15) // 16 * 16) + H, dtype=v.dtype, device="cuda") \
        .as_strided((n, H), ((H + 15) // 16 * 16, 1)).copy_(v)
    Y = O.strided(torch.full((T, H), NAN), y_t)
    gemm.combine(tight(ys, R), slot.int().cuda(), Y[0], weight=weight.cuda() if weighted else None,
                 residual=tight(r, T) if r_t else None)
    assert gemm.sync_status()[0] == G.GEMM_OK
    want = r.double() if r_t else torch.zeros(T, H, dtype=torch.float64)
    mag = want.abs()
    for j in range(k):
        w = (weight[:, j].double() if weighted else torch.ones(T, dtype=torch.float64))
        w = torch.where(there[:, j], w, torch.zeros_like(w))[:, None]
        rows = ys[slot[:, j].clamp(0, R - 1)].double()
        want, mag = want + w * rows, mag + w.abs() * rows.abs()
    e = mag * (k + 1) * O.U32
    O.within(Y[0], want, e + O.rounding(want.abs() + e, y_t), "y")
    assert O.padding_untouched(*Y)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", [(1, 8, 4096), (30, 3, 1001)])
def test_combine_in_place_residual(gemm, T, k, H):
    gen = torch.Generator().manual_seed(1)
    ys, r = torch.randn(T * k, H, generator=gen).half(), torch.randn(T, H, generator=gen).half()
    slot = torch.randperm(T * k, generator=gen).view(T, k)
    Y = O.strided(r.float(), "f16")
    gemm.combine(O.strided(ys.float(), "f16")[0], slot.int().cuda(), Y[0], residual=Y[0])
    want = combine(ys.double(), slot, None, r.double())
    e = combine(ys.double().abs(), slot, None, r.double().abs()) * (k + 1) * O.U32
    O.within(Y[0], want, e + O.rounding(want.abs() + e, "f16"), "y")
    assert O.padding_untouched(*Y)


@pytest.mark.gpu
def test_combine_of_nothing(gemm):
    """No choices, no rows, or only choices of none: the residual, or 0."""
    r = torch.randn(6, 40, device="cuda")
    y = torch.full((6, 40), NAN, device="cuda")
    e = lambda *s: torch.zeros(*s, device="cuda")
    none = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    for ys, slot in ((e(4, 40), none), (e(0, 40), none.abs()), (e(4, 40), none[:, :0])):
        gemm.combine(ys, slot, y, residual=r)
        torch.cuda.synchronize()
        assert torch.equal(y, r)
        gemm.combine(ys, slot, y.fill_(NAN))
        torch.cuda.synchronize()
        assert not y.any()
    dys, dw = torch.full((4, 40), NAN, device="cuda"), torch.full((6, 2), NAN, device="cuda")
    gemm.combine_bwd(r, none, dys, ys=e(4, 40), dweight=dw)
    assert gemm.sync_status()[0] == G.GEMM_OK
    assert torch.isnan(dys).all() and not dw.any()
    gemm.combine_bwd(r, none.abs(), ys=e(0, 40), dweight=dw.fill_(NAN))
    gemm.combine_bwd(r[:, :0], none.abs(), ys=e(4, 0), dweight=dw)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", SIZES)
@pytest.mark.parametrize("t,weighted", [("bf16", True), ("f16", True), ("f32", True), ("bf16", False)])
def test_combine_bwd(gemm, T, k, H, t, weighted):
    gen = torch.Generator().manual_seed(T + k + H)
    R = T * k + 1
    slot = _places(gen, T, k, R)
    dy, ys = (torch.randn(n, H, generator=gen).to(O.TYPES[t]) for n in (T, R))
    weight = torch.randn(T, k, generator=gen) if weighted else None
    want, dw = combine_bwd(dy.double(), slot, weight.double() if weighted else None, ys.double())
    mag = combine_bwd(dy.double().abs(), slot, None, ys.double().abs())[1]
    DY, YS = O.strided(dy.float(), t)[0], O.strided(ys.float(), t)[0]
    W = weight.cuda() if weighted else None
    for give in (("dys", "dweight"), ("dys",), ("dweight",)):
        DYS = O.strided(torch.full((R, H), NAN), t)
        dweight = torch.full((T, k), NAN, device="cuda")
        gemm.combine_bwd(DY, slot.int().cuda(), DYS[0] if "dys" in give else None, weight=W,
                         ys=YS if "dweight" in give else None,
                         dweight=dweight if "dweight" in give else None)
        assert gemm.sync_status()[0] == G.GEMM_OK
        if "dys" in give:
            has = ~torch.isnan(want[:, 0])
            e = want[has].abs() * O.U32
            O.within(DYS[0].cpu()[has], want[has], e + O.rounding(want[has].abs() + e, t), "dys")
            assert torch.isnan(DYS[0].cpu().float()[~has]).all() and O.padding_untouched(*DYS)
        if "dweight" in give:
            O.within(dweight, dw, mag * (H / 16 + 40) * O.U32, "dweight")


@pytest.mark.gpu
def test_combine_bwd_in_place(gemm):
    gen = torch.Generator().manual_seed(1)
    T, k, H = 30, 3, 1001
    dy, ys = (torch.randn(n, H, generator=gen).half() for n in (T, T * k))
    weight = torch.randn(T, k, generator=gen)
    slot = torch.randperm(T * k, generator=gen).view(T, k)
    want, dw = combine_bwd(dy.double(), slot, weight.double(), ys.double())
    Y = O.strided(ys.float(), "f16")
    dweight = torch.empty(T, k, device="cuda")
    gemm.combine_bwd(O.strided(dy.float(), "f16")[0], slot.int().cuda(), Y[0], weight=weight.cuda(),
                     ys=Y[0], dweight=dweight)
    O.within(Y[0], want, want.abs() * O.U32 + O.rounding(want, "f16"), "dys")
    mag = combine_bwd(dy.double().abs(), slot, None, ys.double().abs())[1]
    O.within(dweight, dw, mag * (H / 16 + 40) * O.U32, "dweight")


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_rows(gemm):
    ys = torch.ones(8, 72, device="cuda")
    ys[3], ys[5, 7] = INF, NAN
    slot = torch.tensor([[0, 1], [3, 2], [5, 4], [6, 7]], dtype=torch.int32, device="cuda")
    y, dw = torch.zeros(4, 72, device="cuda"), torch.zeros(4, 2, device="cuda")
    gemm.combine(ys, slot, y)
    dys = torch.zeros_like(ys)
    dy = torch.ones(4, 72, device="cuda")
    dy[3, 1] = INF
    gemm.combine_bwd(dy, slot, dys, ys=ys, dweight=dw)
    torch.cuda.synchronize()
    assert (y[0] == 2).all() and (y[3] == 2).all() and (y[1] == INF).all()
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 2).all() and (y[2, 8:] == 2).all()
    assert (dw[0] == 72).all() and dw[1, 0] == INF and dw[1, 1] == 72 and torch.isnan(dw[2, 0])
    assert dw[2, 1] == 72 and (dw[3] == INF).all()
    assert (dys[:6] == 1).all() and (dys[6:, 1] == INF).all() and (dys[6:, 2:] == 1).all()


@pytest.mark.gpu
def test_large_batches_repeat_bit_for_bit(gemm):
    """The same sums by the ring and without it (a smaller batch of the same rows), and in place."""
    T, k, H = 2000, 4, 2200
    gen = torch.Generator(device="cuda").manual_seed(3)
    ys = torch.randn(T * k, H, generator=gen, device="cuda").bfloat16()
    r = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    w = torch.randn(T, k, generator=gen, device="cuda")
    slot = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
    outs = [torch.zeros_like(r) for _ in range(3)]
    gemm.combine(ys, slot, outs[0], weight=w, residual=r)
    for t in range(0, T, 500):
        gemm.combine(ys, slot[t:t + 500], outs[1][t:t + 500], weight=w[t:t + 500],
                     residual=r[t:t + 500])
    outs[2].copy_(r)
    gemm.combine(ys, slot, outs[2], weight=w, residual=outs[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.gpu
def test_repeats_bit_for_bit_on_any_stream_and_in_a_graph(gemm):
    T, k, E, H = 700, 4, 24, 520
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy = rnd(T, H).bfloat16(), rnd(T, H).bfloat16()
    index, weight = torch.randint(0, E, (T, k), generator=gen, device="cuda"), rnd(T, k)

    def chain(stream):
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        o = dict(offsets=i32(E + 1), slot=i32(T, k), source=i32(T * k),
                 ys=torch.zeros(T * k, H, device="cuda").bfloat16(), y=torch.zeros(T, H, device="cuda"),
                 dys=torch.zeros(T * k, H, device="cuda").bfloat16(),
                 dw=torch.zeros(T, k, device="cuda"))
        torch.cuda.synchronize()

        def run(s):
            gemm.route(index, o["offsets"], o["slot"], source=o["source"], stream=s)
            gemm.dispatch(x, o["slot"], o["ys"], stream=s)
            gemm.combine(o["ys"], o["slot"], o["y"], weight=weight, residual=x, stream=s)
            gemm.combine_bwd(dy, o["slot"], o["dys"], weight=weight, ys=o["ys"], dweight=o["dw"],
                             stream=s)
        return o, run
    outs = []
    for s in (None, torch.cuda.Stream()):
        o, run = chain(s)
        run(s)
        outs.append(o)
    torch.cuda.synchronize()
    o, run = chain(None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(outs[0][k], o[k]) for k in o)
    # the graph follows what lies behind its addresses
    index.copy_(index.flip(0) % 5)
    graph.replay()
    torch.cuda.synchronize()
    assert o["slot"].view(-1).tolist() == sort(index.cpu(), E)[1]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,t,weighted,parts", [
    (5001, 3, 5003, "f16", True, "both"), (2100, 4, 2048, "bf16", True, "both"),
    (2000, 1, 9001, "bf16", False, "both"), (300, 32, 2051, "f32", True, "both"),
    (410, 9, 4999, "f16", True, "dweight"), (301, 31, 2064, "bf16", True, "both"),
    (300, 33, 2051, "f16", True, "both")])
def test_combine_bwd_of_large_batches(gemm, T, k, H, t, weighted, parts):
    """Rows of several passes ending inside 16 bytes, the last row of each matrix among the choices,
    tokens without any, infinities and NaN in rows of no choice and behind rows."""
    gen = torch.Generator().manual_seed(T + k + H)
    R = T * k + 1 - T // 3
    slot = torch.randperm(T * k, generator=gen).view(T, k)
    slot[T // 2] = -1
    slot[-1, -1], slot[slot == R - 1] = R - 1, -1
    dy = torch.randn(T, H, generator=gen).to(O.TYPES[t])
    ys = torch.randn(R, H, generator=gen).to(O.TYPES[t])
    chosen = torch.zeros(R, dtype=torch.bool)
    chosen[slot[(slot >= 0) & (slot < R)]] = True
    ys[~chosen] = torch.tensor([NAN, float("inf")])[torch.arange(int((~chosen).sum())) % 2][:, None].to(ys.dtype)
    weight = torch.randn(T, k, generator=gen) if weighted else None
    DY, YS, DYS = O.strided(dy.float(), t), O.strided(ys.float(), t), O.strided(torch.full((R, H), NAN), t)
    dweight = torch.full((T, k), NAN, device="cuda")
    gemm.combine_bwd(DY[0], slot.int().cuda(), DYS[0] if parts == "both" else None,
                     weight=weight.cuda() if weighted else None, ys=YS[0], dweight=dweight)
    assert gemm.sync_status()[0] == G.GEMM_OK
    safe = ys.double().masked_fill(~chosen[:, None], 0.0)
    there = (slot >= 0) & (slot < R)
    at = slot.clamp(0, R - 1)
    for j in range(k):
        terms = dy.double() * safe[at[:, j]] * there[:, j, None]
        # a sum of H terms in fp32, in threads' and lanes' parts: each partial sum rounds once
        O.within(dweight[:, j], terms.sum(1), terms.abs().sum(1) * 200 * O.U32 + 1e-30, "dweight")
    if parts == "both":
        want = torch.full((R, H), NAN, dtype=torch.float64)
        w = weight.double() if weighted else torch.ones(T, k, dtype=torch.float64)
        for j in range(k):
            want[at[there[:, j], j]] = (w[:, j, None] * dy.double())[there[:, j]]
        got = O.f64(DYS[0])
        assert torch.isnan(got[~chosen]).all() and O.padding_untouched(*DYS)
        O.within(got[chosen], want[chosen], O.rounding(want[chosen].abs() * (1 + O.U32), t) +
                 want[chosen].abs() * O.U32, "dys")


@pytest.mark.gpu
def test_combine_bwd_of_large_batches_in_place_and_again(gemm):
    T, k, H = 4000, 2, 2056
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    dy, ys, weight = rnd(T, H), rnd(T * k, H), torch.rand(T, k, generator=gen, device="cuda")
    slot = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
    first = None
    for in_place in (False, True, False):
        rows = ys.clone()
        dys, dweight = rows if in_place else torch.empty_like(ys), torch.empty(T, k, device="cuda")
        gemm.combine_bwd(dy, slot, dys, weight=weight, ys=rows, dweight=dweight)
        assert gemm.sync_status()[0] == G.GEMM_OK
        first = first or (dys.clone(), dweight.clone())
        assert torch.equal(first[0], dys) and torch.equal(first[1], dweight)
