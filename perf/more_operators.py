"""Cases and plain forms of the operators whose weights change from row to row.

Six operators, each as a case of this file names it in "op":

  dispatch     a token's choices of experts sorted by expert (route), its row copied to the place
               of each (8-bit rows with their scales)
  combine      y[t] = residual[t] + sum_j weight[t, j] * ys[slot[t, j]]; without weights it is
               the gradient of dispatch
  combine_bwd  gradients of ys and of the weights
  grouped      the linear layer with weights of its own for each group of rows:
               z = alpha * (a b[g]^T) * row_scale * col_scale[g] + bias[g],  d = act(z) + residual
  grouped_bwd  dz = dd * act'(z),  dbias[g],  da = dz b[g],  db[g] = dz^T a over the group's rows
  adapters     d = r + scale[e] * (x A[e]^T) B[e]^T, e the adapter of the row's request (-1: none)

Where `own` is false, run() computes them with elementary torch operations in
32 bits, rounded once at the end; where it is true, with the package's kernels.
"""
import functools
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}     # largest finite value of the 8-bit types
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token on its way to its experts
        dict(name="dispatch_token", op="dispatch", tokens=1, top=8, experts=64, cols=4096,
             dtype="bf16"),
        # a training batch, 8 experts a token
        dict(name="dispatch_train", op="dispatch", tokens=8192, top=8, experts=64, cols=4096,
             dtype="bf16"),
        # a decode batch coming back into the residual stream
        dict(name="combine_decode", op="combine", tokens=48, top=8, experts=64, cols=4096,
             dtype="bf16", weighted=True, residual=True),
        # the training batch coming back
        dict(name="combine_train", op="combine", tokens=8192, top=8, experts=64, cols=4096,
             dtype="bf16", weighted=True, residual=True),
        # the way back's gradient at an odd size
        dict(name="combine_bwd_odd", op="combine_bwd", tokens=5001, top=3, experts=24, cols=5003,
             dtype="f16"),
        # a decode batch through the experts' first product: few rows each
        dict(name="experts_decode", op="grouped", tokens=16, top=8, experts=64, cols=2048,
             inner=4096, dtype="bf16", out="bf16", act="silu", bias=False, keep=False),
        # a ragged 8-bit prompt through the experts, with scales
        dict(name="experts_fp8_ragged", op="grouped", tokens=1001, top=4, experts=32, cols=5000,
             inner=2048, dtype="e4m3", out="bf16", act="none", bias=False, keep=False),
        # the training forward of large experts, the pre-activation kept
        dict(name="experts_train", op="grouped", tokens=8192, top=2, experts=8, cols=8192,
             inner=4096, dtype="bf16", out="bf16", act="gelu", bias=True, keep=True),
        # the backward pass of experts at a training size
        dict(name="experts_bwd", op="grouped_bwd", tokens=4096, top=2, experts=16, cols=4096,
             inner=4096, dtype="bf16", act="silu", bias=False),
        # odd sizes, the bias's gradient too
        dict(name="experts_bwd_odd", op="grouped_bwd", tokens=1001, top=2, experts=6, cols=2003,
             inner=1501, dtype="f16", act="gelu", bias=True),
        # one token each of many requests, some without an adapter
        dict(name="adapters_decode", op="adapters", requests=64, rows=64, adapters=48, rank=16,
             cols=4096, inner=4096, dtype="bf16"),
        # a few long prompts
        dict(name="adapters_prompts", op="adapters", requests=7, rows=8191, adapters=16, rank=64,
             cols=8192, inner=4096, dtype="bf16"),
    ]


def _size(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm, a multiple of `step`."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return (n + step - 1) // step * step


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_bwd", "grouped", "grouped", "grouped_bwd",
                     "adapters"])
    dtype = rng.choice(["f16", "bf16"])
    step = rng.choice([1, 64])
    while True:
        top = rng.randint(1, 8)
        experts = _size(rng, 8, 256)
        tokens = _size(rng, 1, 8192)
        cols = _size(rng, 256, 8192, step)
        inner = _size(rng, 256, 8192, step)
        if op in ("dispatch", "combine", "combine_bwd"):
            if tokens * top * cols > 8192 * 8 * 4096:
                continue
            case = dict(op=op, tokens=tokens, top=top, experts=experts, cols=cols, dtype=dtype)
            if op == "dispatch":
                case["dtype"] = rng.choice([dtype, "e4m3"])
            if op == "combine":
                case["weighted"] = rng.random() < 0.7
                case["residual"] = rng.random() < 0.7
            return case
        if op == "adapters":
            requests = _size(rng, 1, 256)
            rows = requests if rng.random() < 0.4 else _size(rng, requests, 8192)
            return dict(op=op, requests=requests, rows=rows, adapters=_size(rng, 1, 64),
                        rank=rng.choice([8, 12, 16, 32, 64, 128]), cols=cols, inner=inner,
                        dtype=dtype)
        # (weights of 2 GB in fp32 at most, and no more products than the largest)
        if experts * cols * inner > 64 * 2048 * 4096 or \
                tokens * top * cols * inner > 8192 * 2 * 4096 * 4096:
            continue
        case = dict(op=op, tokens=tokens, top=min(top, experts), experts=experts, cols=cols,
                    inner=inner, dtype=dtype, act=rng.choice(ACTIVATIONS),
                    bias=rng.random() < 0.4)
        if op == "grouped":
            case["out"] = dtype
            if rng.random() < 0.4:
                case["dtype"] = rng.choice(["e4m3", "e4m3", "e5m2"])
            case["keep"] = rng.random() < 0.25
        return case


# ------------------------------------------------------------------ inputs

def _empty(rows, cols, dtype):
    """A rows x cols matrix whose rows start on 16-byte boundaries."""
    return torch.empty(rows, (cols + 15) // 16 * 16, dtype=DTYPES[dtype], device="cuda")[:, :cols]


def _matrix(gen, rows, cols, dtype, scale=1.0):
    m = _empty(rows, cols, dtype)
    m.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)
    return m


def _codes(gen, rows, cols, dtype):
    """Values as a row-wise quantisation leaves them: each row reaches near the type's end."""
    top = LARGEST[dtype]
    m = _empty(rows, cols, dtype)
    v = torch.randn(rows, cols, generator=gen, device="cuda").mul_(top / 4.5)
    m.copy_(v.clamp_(-top, top))
    return m


def _stack(m, n):
    """A matrix of n stacked ones as n matrices."""
    return m.unflatten(0, (n, m.shape[0] // n))


def _choices(gen, case):
    """Experts and weights of each token as a router leaves them: some experts are in demand."""
    t, e = case["tokens"], case["experts"]
    logits = torch.randn(t, e, generator=gen, device="cuda") + \
        0.5 * torch.randn(e, generator=gen, device="cuda")
    best, index = torch.topk(logits, case["top"], dim=1)
    return index.int(), torch.softmax(best, dim=1)


def _sorted(index, experts):
    """(offsets, slot, source) of the choices in order of expert and place."""
    flat = index.reshape(-1).long()
    source = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(source)
    slot[source] = torch.arange(flat.numel(), device="cuda")
    counts = (flat[:, None] == torch.arange(experts, device="cuda")).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets.int(), slot.int().view(index.shape), source.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, cols, dtype = case["op"], case["cols"], case["dtype"]
    s = dict(case)
    vector = lambda *n, lo=-0.5, hi=0.5: lo + (hi - lo) * torch.rand(*n, generator=gen,
                                                                     device="cuda")
    if op == "adapters":
        n, rows, rank, inner = case["requests"], case["rows"], case["rank"], case["inner"]
        # every request has a row; the others are dealt out unevenly
        share = torch.rand(n, generator=gen, device="cuda") ** 3 + 1e-3
        ends = (share.cumsum(0) / share.sum() * (rows - n)).long().clamp(max=rows - n)
        ends[-1] = rows - n
        ends = ends + torch.arange(1, n + 1, device="cuda")
        s["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        index = torch.randint(0, case["adapters"], (n,), generator=gen, device="cuda")
        none = torch.rand(n, generator=gen, device="cuda") < (0.1 if n > 1 else 0.0)
        s["index"] = index.masked_fill(none, -1).int()
        s["x"] = _matrix(gen, rows, inner, dtype)
        s["a"] = _stack(_matrix(gen, case["adapters"] * rank, inner, dtype, inner ** -0.5),
                        case["adapters"])
        s["b"] = _stack(_matrix(gen, case["adapters"] * cols, rank, dtype, rank ** -0.5),
                        case["adapters"])
        s["scale"] = vector(case["adapters"], lo=0.25, hi=1.0)
        s["r"] = _matrix(gen, rows, cols, dtype)
        s["u"] = _empty(rows, rank, dtype)
        s["d"] = _empty(rows, cols, dtype)
        return s
    index, weight = _choices(gen, case)
    tokens, experts, rows = case["tokens"], case["experts"], case["tokens"] * case["top"]
    if op == "dispatch":
        s["index"] = index
        s["x"] = _matrix(gen, tokens, cols, dtype) if dtype not in LARGEST else \
            _codes(gen, tokens, cols, dtype)
        if dtype in LARGEST:
            s["scale"] = vector(tokens, lo=0.5, hi=1.5) * (4.5 / LARGEST[dtype])
            s["y_scale"] = torch.empty(rows, device="cuda")
        s["y"] = _empty(rows, cols, dtype)
        s["offsets"] = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        s["slot"] = torch.empty(tokens, case["top"], dtype=torch.int32, device="cuda")
        s["source"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        return s
    offsets, slot, source = _sorted(index, experts)
    if op == "combine":
        s["slot"] = slot
        s["ys"] = _matrix(gen, rows, cols, dtype)
        if case["weighted"]:
            s["weight"] = weight
        if case["residual"]:
            s["r"] = _matrix(gen, tokens, cols, dtype)
        s["y"] = _empty(tokens, cols, dtype)
        return s
    if op == "combine_bwd":
        s["slot"], s["weight"] = slot, weight
        s["dy"] = _matrix(gen, tokens, cols, dtype, 0.1)
        s["ys"] = _matrix(gen, rows, cols, dtype)
        s["dys"] = _empty(rows, cols, dtype)
        s["dweight"] = torch.empty(tokens, case["top"], device="cuda")
        return s
    inner = case["inner"]
    s["offsets"] = offsets
    s["longest"] = int((offsets[1:] - offsets[:-1]).max())
    if op == "grouped":
        out = case["out"]
        if dtype in LARGEST:
            unit = 4.5 / LARGEST[dtype]
            s["a"] = _codes(gen, rows, inner, dtype)
            s["b"] = _stack(_codes(gen, experts * cols, inner, dtype), experts)
            s["row_scale"] = vector(rows, lo=0.5, hi=1.5) * unit
            s["col_scale"] = vector(experts, cols, lo=0.5, hi=1.5) * (unit / math.sqrt(inner))
        else:
            s["a"] = _matrix(gen, rows, inner, dtype)
            s["b"] = _stack(_matrix(gen, experts * cols, inner, dtype, inner ** -0.5), experts)
        if case["bias"]:
            s["bias"] = vector(experts, cols).to(DTYPES[out])
        s["d"] = _empty(rows, cols, out)
        if case["keep"]:
            s["z"] = _empty(rows, cols, out)
        return s
    s["a"] = _matrix(gen, rows, inner, dtype)
    s["b"] = _stack(_matrix(gen, experts * cols, inner, dtype, inner ** -0.5), experts)
    s["z"] = _matrix(gen, rows, cols, dtype)
    s["dd"] = _matrix(gen, rows, cols, dtype, 0.1)
    s["dz"] = _empty(rows, cols, dtype)
    s["da"] = _empty(rows, inner, dtype)
    s["db"] = _stack(_empty(experts * cols, inner, dtype), experts)
    if case["bias"]:
        s["dbias"] = torch.empty(experts, cols, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + \
            v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * v * v)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    return torch.ones_like(v)


def _plain_dispatch(s):
    offsets, slot, source = _sorted(s["index"], s["experts"])
    token = source.long() // s["top"]
    out = {"offsets": offsets, "slot": slot, "source": source}
    if s["dtype"] in LARGEST:
        out["y"] = s["x"].view(torch.uint8)[token].view(DTYPES[s["dtype"]])
        out["y_scale"] = s["scale"][token]
    else:
        out["y"] = s["x"][token]
    return out


def _plain_combine(s):
    rows = s["ys"].float()[s["slot"].long()]
    if s["weighted"]:
        rows = rows * s["weight"][:, :, None]
    y = rows.sum(dim=1)
    if s["residual"]:
        y = y + s["r"].float()
    return {"y": y.to(DTYPES[s["dtype"]])}


def _plain_combine_bwd(s):
    dy, slot = s["dy"].float(), s["slot"].long()
    dys = torch.empty(s["ys"].shape, dtype=DTYPES[s["dtype"]], device="cuda")
    dys[slot] = (s["weight"][:, :, None] * dy[:, None, :]).to(dys.dtype)
    return {"dys": dys, "dweight": (dy[:, None, :] * s["ys"].float()[slot]).sum(dim=2)}


def _places(s, rows):
    """Each row's group and its place in the group."""
    at = torch.arange(rows, device="cuda")
    group = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return group, at - s["offsets"].long()[group]


def _padded(m, group, place, groups, longest):
    """The rows of each group as a matrix, filled up with zeros to the longest group's."""
    p = torch.zeros(groups, longest, m.shape[1], device="cuda")
    p[group, place] = m.float()
    return p


def _plain_grouped(s):
    group, place = _places(s, s["a"].shape[0])
    a = _padded(s["a"], group, place, s["experts"], s["longest"])
    z = torch.bmm(a, s["b"].float().transpose(1, 2))[group, place]
    if s["dtype"] in LARGEST:
        z = z * s["row_scale"][:, None] * s["col_scale"][group]
    if s["bias"] is not False:
        z = z + s["bias"].float()[group]
    out = {"d": _act(z, s["act"]).to(DTYPES[s["out"]])}
    if s["keep"]:
        out["z"] = z.to(DTYPES[s["out"]])
    return out


def _plain_grouped_bwd(s):
    t = DTYPES[s["dtype"]]
    group, place = _places(s, s["a"].shape[0])
    dz = s["dd"].float() * _act_grad(s["z"].float(), s["act"])
    a = _padded(s["a"], group, place, s["experts"], s["longest"])
    g = _padded(dz, group, place, s["experts"], s["longest"])
    out = {"dz": dz.to(t), "da": torch.bmm(g, s["b"].float())[group, place].to(t),
           "db": torch.bmm(g.transpose(1, 2), a).to(t)}
    if s["bias"] is not False:
        out["dbias"] = g.sum(dim=1)
    return out


def _plain_adapters(s):
    group, place = _places(s, s["x"].shape[0])
    e = s["index"].long().clamp(min=0)
    scale = torch.where(s["index"] >= 0, s["scale"][e], torch.zeros_like(s["scale"][e]))
    x = _padded(s["x"], group, place, s["requests"], s["longest"])
    u = torch.bmm(x, s["a"][e].float().transpose(1, 2)) * scale[:, None, None]
    v = torch.bmm(u, s["b"][e].float().transpose(1, 2))
    return {"d": (s["r"].float() + v[group, place]).to(DTYPES[s["dtype"]])}


_plain = {"dispatch": _plain_dispatch, "combine": _plain_combine,
          "combine_bwd": _plain_combine_bwd, "grouped": _plain_grouped,
          "grouped_bwd": _plain_grouped_bwd, "adapters": _plain_adapters}


@functools.lru_cache(maxsize=None)
def _gemm():
    """The library handle, created once, as a program keeps it."""
    import dense_gemm_epilogue_persistent_gb300 as G
    return G.Gemm(torch.cuda.current_device())


def _own_dispatch(s):
    g = _gemm()
    g.route(s["index"], s["offsets"], s["slot"], source=s["source"])
    g.dispatch(s["x"], s["slot"], s["y"], scale=s.get("scale"), y_scale=s.get("y_scale"))
    return {k: s[k] for k in ("offsets", "slot", "source", "y", "y_scale") if k in s}


def _own_combine(s):
    _gemm().combine(s["ys"], s["slot"], s["y"], weight=s.get("weight"), residual=s.get("r"))
    return {"y": s["y"]}


def _own_combine_bwd(s):
    _gemm().combine_bwd(s["dy"], s["slot"], s["dys"], weight=s["weight"], ys=s["ys"],
                        dweight=s["dweight"])
    return {"dys": s["dys"], "dweight": s["dweight"]}


def _own_grouped(s):
    _gemm().grouped_linear(s["a"], s["b"], s["offsets"], s["d"],
                           bias=s["bias"] if s["bias"] is not False else None,
                           activation=s["act"], z=s.get("z"), row_scale=s.get("row_scale"),
                           col_scale=s.get("col_scale"))
    return {k: s[k] for k in ("d", "z") if k in s}


def _own_grouped_bwd(s):
    _gemm().grouped_linear_bwd(s["dd"], s["a"], s["b"], s["offsets"], z=s["z"],
                               activation=s["act"], dz=s["dz"], da=s["da"], db=s["db"],
                               dbias=s.get("dbias"))
    return {k: s[k] for k in ("dz", "da", "db", "dbias") if k in s}


def _own_adapters(s):
    _gemm().adapters(s["x"], s["a"], s["b"], s["offsets"], s["index"], s["u"], s["d"],
                     residual=s["r"], scale=s["scale"])
    return {"d": s["d"]}


_own = {"dispatch": _own_dispatch, "combine": _own_combine, "combine_bwd": _own_combine_bwd,
        "grouped": _own_grouped, "grouped_bwd": _own_grouped_bwd, "adapters": _own_adapters}


# ------------------------------------------------------------------ work

def _met(groups, chance, times):
    """How many of `groups` are met when each has that chance each time."""
    return groups * (1.0 - (1.0 - min(1.0, chance)) ** times)


def work(case):
    op, n, es = case["op"], case["cols"], BYTES[case["dtype"]]
    if op == "adapters":
        m, k, r = case["rows"], case["inner"], case["rank"]
        used = _met(case["adapters"], 1.0 / case["adapters"], case["requests"])
        return {"bytes": es * (m * k + 2 * m * n + used * r * (k + n)),
                "flops": 2 * m * r * (k + n)}
    t, top, e = case["tokens"], case["top"], case["experts"]
    m = t * top
    if op == "dispatch":
        scales = 4 * (t + m) if case["dtype"] in LARGEST else 0
        return {"bytes": es * (t + m) * n + scales + 12 * m + 4 * e, "flops": 0}
    if op == "combine":
        return {"bytes": es * n * (m + t * (1 + case["residual"])) +
                4 * m * (1 + case["weighted"]), "flops": 2 * m * n}
    if op == "combine_bwd":
        return {"bytes": es * n * (t + 2 * m) + 12 * m, "flops": 3 * m * n}
    k = case["inner"]
    used = _met(e, top / e, t)
    if op == "grouped":
        eo = BYTES[case["out"]]
        nbytes = es * (m * k + used * n * k) + eo * m * n * (1 + case["keep"]) + \
            eo * used * n * case["bias"]
        if case["dtype"] in LARGEST:
            nbytes += 4 * (m + used * n)
        return {"bytes": nbytes, "flops": 2 * m * n * k}
    # every input (dd, z, a, the experts' b) once, every output (dz, da, db, dbias) once
    return {"bytes": es * (3 * m * n + 2 * m * k + (used + e) * n * k) + 4 * e * n * case["bias"],
            "flops": 4 * m * n * k}


# ------------------------------------------------------------------ in 64 bits

def _exact_act(v, act):
    """(act(v), act'(v)) in 64 bits."""
    zero, one = torch.zeros_like(v), torch.ones_like(v)
    if act == "relu":
        return torch.maximum(v, zero), torch.where(v > 0, one, zero)
    if act == "gelu":
        cdf = torch.special.erfc(v * -math.sqrt(0.5)) / 2
        return v * cdf, cdf + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        p = torch.special.expit(2 * u)
        return v * p, p + 2 * v * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 0.134145 * v ** 2)
    if act == "silu":
        p = torch.special.expit(v)
        return v * p, p + v * p * (1 - p)
    return v, one


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "dispatch":               # copies; the whole numbers have no such value
        place = torch.argsort(torch.argsort(s["index"].flatten().long(), stable=True))
        out = {"y": torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")}
        out["y"].index_copy_(0, place, s["x"].double().repeat_interleave(case["top"], dim=0))
        if case["dtype"] in LARGEST:
            out["y_scale"] = torch.empty(s["y"].shape[0], dtype=torch.float64, device="cuda")
            out["y_scale"].index_copy_(0, place, s["scale"].double().repeat_interleave(case["top"]))
        return {**out, "offsets": None, "slot": None, "source": None}
    if op == "combine":
        y = s["r"].double() if case["residual"] else \
            torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            rows = s["ys"].index_select(0, s["slot"][:, j].long()).double()
            y = y + (torch.einsum("tn,t->tn", rows, s["weight"][:, j].double())
                     if case["weighted"] else rows)
        return {"y": y}
    if op == "combine_bwd":
        dy = s["dy"].double()
        dys = torch.empty(s["ys"].shape, dtype=torch.float64, device="cuda")
        dweight = torch.empty(s["weight"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            at, w = s["slot"][:, j].long(), s["weight"][:, j].double()
            dys.index_copy_(0, at, torch.einsum("tn,t->tn", dy, w))
            dweight[:, j] = torch.einsum("tn,tn->t", dy, s["ys"].index_select(0, at).double())
        return {"dys": dys, "dweight": dweight}
    bounds = s["offsets"].tolist()
    f64 = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    if op == "adapters":
        d = s["r"].double()
        for g, e in enumerate(s["index"].tolist()):
            rows = slice(bounds[g], bounds[g + 1])
            if e >= 0:
                u = torch.mm(s["x"][rows].double(), s["a"][e].double().T)
                d[rows] += float(s["scale"][e]) * torch.mm(u, s["b"][e].double().T)
        return {"d": d}
    n, k = case["cols"], case["inner"]
    if op == "grouped":
        z = f64(s["a"].shape[0], n)
        for g in range(case["experts"]):
            rows = slice(bounds[g], bounds[g + 1])
            v = torch.mm(s["a"][rows].double(), s["b"][g].double().T)
            if case["dtype"] in LARGEST:
                v *= torch.outer(s["row_scale"][rows].double(), s["col_scale"][g].double())
            z[rows] = v + s["bias"][g].double() if case["bias"] else v
        d = _exact_act(z, case["act"])[0]
        return {"d": d, "z": z} if case["keep"] else {"d": d}
    dz = s["dd"].double() * _exact_act(s["z"].double(), case["act"])[1]
    out = {"dz": dz, "da": f64(s["a"].shape[0], k), "db": f64(case["experts"], n, k)}
    if case["bias"]:
        out["dbias"] = f64(case["experts"], n)
    for g in range(case["experts"]):
        rows = slice(bounds[g], bounds[g + 1])
        out["da"][rows] = torch.mm(dz[rows], s["b"][g].double())
        out["db"][g] = torch.mm(dz[rows].T, s["a"][rows].double())
        if case["bias"]:
            out["dbias"][g] = torch.einsum("mn->n", dz[rows])
    return out
