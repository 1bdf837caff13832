"""Cases and plain forms of the normalisation and linear-layer operators.

Four operators, each as a case of this file names it in "op":

  rmsnorm       h = x + residual,  y = h * rstd * weight,  rstd = 1 / sqrt(mean(h^2) + eps);
                y in 16 bits, or in 8 bits (E4M3, E5M2) with one fp32 scale per row
  rmsnorm_bwd   gradients of x (= of the residual) and of weight
  linear        z = alpha * (a b^T) * row_scale * col_scale + bias,  d = act(z) + residual
  linear_bwd    dz = dd * act'(z),  dbias,  da = dz b,  db = dz^T a

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
AMAX_FLOOR = 2.0 ** -100                       # a row's largest magnitude counts as at least this
EPS = 1e-6
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token entering a block: x joins the residual stream, fp8 out
        dict(name="norm_token", op="rmsnorm", rows=1, cols=8192, dtype="bf16", out="e4m3",
             residual=True),
        # a long prompt, the same step
        dict(name="norm_prefill", op="rmsnorm", rows=8192, cols=8192, dtype="bf16", out="e4m3",
             residual=True),
        # the training forward of a ragged size: 16-bit output
        dict(name="norm_train_ragged", op="rmsnorm", rows=3000, cols=5000, dtype="f16",
             out="f16", residual=True),
        # its backward pass at an ordinary training size, the residual's gradient added
        dict(name="norm_bwd", op="rmsnorm_bwd", rows=8192, cols=4096, dtype="bf16",
             residual=True),
        # odd sizes, no residual
        dict(name="norm_bwd_odd", op="rmsnorm_bwd", rows=1001, cols=5003, dtype="f16",
             residual=False),
        # one decoded token through a layer
        dict(name="linear_token", op="linear", rows=1, cols=8192, inner=8192, dtype="bf16",
             out="bf16", act="silu", residual=False, keep=False),
        # a decode batch through an 8-bit layer with scales, back into the residual stream
        dict(name="linear_decode_fp8", op="linear", rows=48, cols=5000, inner=4096,
             dtype="e4m3", out="bf16", act="none", residual=True, keep=False),
        # a short prompt through a small layer
        dict(name="linear_short", op="linear", rows=300, cols=1024, inner=1024, dtype="f16",
             out="f16", act="gelu_tanh", residual=True, keep=False),
        # a ragged 8-bit prefill with scales
        dict(name="linear_fp8_ragged", op="linear", rows=3000, cols=5000, inner=4096,
             dtype="e4m3", out="f16", act="silu", residual=True, keep=False),
        # the training forward of a large layer, its pre-activation kept
        dict(name="linear_train", op="linear", rows=8192, cols=8192, inner=8192, dtype="bf16",
             out="bf16", act="gelu", residual=False, keep=True),
        # the backward pass of a layer at a training size
        dict(name="linear_bwd", op="linear_bwd", rows=4096, cols=8192, inner=4096, dtype="bf16",
             act="gelu"),
        # odd sizes
        dict(name="linear_bwd_odd", op="linear_bwd", rows=1001, cols=2003, inner=1501,
             dtype="f16", act="silu"),
    ]


def _size(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm, a multiple of `step`.
    (3072 is left out: no workload of this repository has it.)"""
    n = 3072
    while n == 3072:
        n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        n = (n + step - 1) // step * step
    return n


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm", "rmsnorm_bwd", "linear", "linear", "linear",
                     "linear_bwd", "linear_bwd"])
    dtype = rng.choice(["f16", "bf16"])
    step = rng.choice([1, 64])
    if op.startswith("rmsnorm"):
        rows = _size(rng, 1 if op == "rmsnorm" else 16, 16384)
        cols = _size(rng, 256, 16384, step)
        while rows * cols > 8192 * 8192:
            rows = _size(rng, 16, 16384)
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6)
        if op == "rmsnorm":
            case["out"] = rng.choice([dtype, "e4m3", "e4m3", "e5m2"])
        return case
    case = dict(op=op, rows=_size(rng, 1 if op == "linear" else 64, 8192),
                cols=_size(rng, 256, 8192, step), inner=_size(rng, 256, 8192, step),
                dtype=dtype, act=rng.choice(ACTIVATIONS))
    if op == "linear":
        case["out"] = dtype
        if rng.random() < 0.4:
            case["dtype"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        case["residual"] = rng.random() < 0.5
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, dtype = case["rows"], case["cols"], case["dtype"]
    s = dict(case)
    vector = lambda n, lo, hi: lo + (hi - lo) * torch.rand(n, generator=gen, device="cuda")
    if case["op"] in ("rmsnorm", "rmsnorm_bwd"):
        s["weight"] = vector(cols, 0.5, 1.5).to(DTYPES[dtype])
    if case["op"] == "rmsnorm":
        s["x"] = _matrix(gen, rows, cols, dtype)
        s["y"] = _empty(rows, cols, case["out"])
        s["rstd"] = torch.empty(rows, device="cuda")
        if case["residual"]:
            s["r"] = _matrix(gen, rows, cols, dtype, 2.0)
            s["h"] = _empty(rows, cols, dtype)
        if case["out"] in LARGEST:
            s["scale"] = torch.empty(rows, device="cuda")
    elif case["op"] == "rmsnorm_bwd":
        s["h"] = _matrix(gen, rows, cols, dtype, 2.0)
        s["dy"] = _matrix(gen, rows, cols, dtype, 0.1)
        # what the forward pass left
        s["rstd"] = (s["h"].float().square().mean(dim=1) + EPS).rsqrt()
        s["dx"] = _empty(rows, cols, dtype)
        s["dweight"] = torch.empty(cols, device="cuda")
        if case["residual"]:
            s["dh"] = _matrix(gen, rows, cols, dtype, 0.1)
        if own:
            import dense_gemm_epilogue_persistent_gb300 as G
            s["workspace"] = torch.empty(G.gemm_rmsnorm_bwd_workspace(rows, cols),
                                         dtype=torch.uint8, device="cuda")
    elif case["op"] == "linear":
        inner = case["inner"]
        s["bias"] = vector(cols, -0.5, 0.5).to(DTYPES[case["out"]])
        if dtype in LARGEST:
            unit = 4.5 / LARGEST[dtype]
            s["a"] = _codes(gen, rows, inner, dtype)
            s["b"] = _codes(gen, cols, inner, dtype)
            s["row_scale"] = vector(rows, 0.5, 1.5) * unit
            s["col_scale"] = vector(cols, 0.5, 1.5) * (unit / math.sqrt(inner))
        else:
            s["a"] = _matrix(gen, rows, inner, dtype)
            s["b"] = _matrix(gen, cols, inner, dtype, 1.0 / math.sqrt(inner))
        if case["residual"]:
            s["r"] = _matrix(gen, rows, cols, case["out"])
        s["d"] = _empty(rows, cols, case["out"])
        if case["keep"]:
            s["z"] = _empty(rows, cols, case["out"])
    else:
        inner = case["inner"]
        s["a"] = _matrix(gen, rows, inner, dtype)
        s["b"] = _matrix(gen, cols, inner, dtype, 1.0 / math.sqrt(inner))
        s["z"] = _matrix(gen, rows, cols, dtype)
        s["dd"] = _matrix(gen, rows, cols, dtype, 0.1)
        s["dz"] = _empty(rows, cols, dtype)
        s["da"] = _empty(rows, inner, dtype)
        s["db"] = _empty(cols, inner, dtype)
        s["dbias"] = torch.empty(cols, device="cuda")
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


def _plain_rmsnorm(s):
    h = s["x"].float()
    if s["residual"]:
        h = h + s["r"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)
    y = h * rstd[:, None] * s["weight"].float()
    out = {"rstd": rstd}
    if s["residual"]:
        out["h"] = h.to(DTYPES[s["dtype"]])
    if s["out"] in LARGEST:
        scale = y.abs().amax(dim=1).clamp(min=AMAX_FLOOR) / LARGEST[s["out"]]
        out["scale"] = scale
        y = (y / scale[:, None]).clamp(-LARGEST[s["out"]], LARGEST[s["out"]])
    out["y"] = y.to(DTYPES[s["out"]])
    return out


def _plain_rmsnorm_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    if s["residual"]:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(DTYPES[s["dtype"]]), "dweight": (dy * n).sum(dim=0)}


def _plain_linear(s):
    z = s["a"].float() @ s["b"].float().t()
    if s["dtype"] in LARGEST:
        z = z * s["row_scale"][:, None] * s["col_scale"]
    z = z + s["bias"].float()
    d = _act(z, s["act"])
    if s["residual"]:
        d = d + s["r"].float()
    out = {"d": d.to(DTYPES[s["out"]])}
    if s["keep"]:
        out["z"] = z.to(DTYPES[s["out"]])
    return out


def _plain_linear_bwd(s):
    t = DTYPES[s["dtype"]]
    dz = s["dd"].float() * _act_grad(s["z"].float(), s["act"])
    return {"dz": dz.to(t), "dbias": dz.sum(dim=0), "da": (dz @ s["b"].float()).to(t),
            "db": (dz.t() @ s["a"].float()).to(t)}


_plain = {"rmsnorm": _plain_rmsnorm, "rmsnorm_bwd": _plain_rmsnorm_bwd,
          "linear": _plain_linear, "linear_bwd": _plain_linear_bwd}


@functools.lru_cache(maxsize=None)
def _gemm():
    """The library handle, created once, as a program keeps it."""
    import dense_gemm_epilogue_persistent_gb300 as G
    return G.Gemm(torch.cuda.current_device())


def _own_rmsnorm(s):
    _gemm().rmsnorm(s["x"], s["weight"], s["y"], residual=s.get("r"), h=s.get("h"),
                    scale=s.get("scale"), rstd=s["rstd"], eps=EPS)
    return {k: s[k] for k in ("rstd", "h", "scale", "y") if k in s}


def _own_rmsnorm_bwd(s):
    _gemm().rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"],
                        dh=s.get("dh"), workspace=s["workspace"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_linear(s):
    _gemm().linear(s["a"], s["b"], s["d"], bias=s["bias"], activation=s["act"],
                   residual=s.get("r"), z=s.get("z"), row_scale=s.get("row_scale"),
                   col_scale=s.get("col_scale"))
    return {k: s[k] for k in ("d", "z") if k in s}


def _own_linear_bwd(s):
    _gemm().linear_bwd(s["dd"], s["a"], s["b"], z=s["z"], activation=s["act"], dz=s["dz"],
                       da=s["da"], db=s["db"], dbias=s["dbias"])
    return {k: s[k] for k in ("dz", "dbias", "da", "db")}


_own = {"rmsnorm": _own_rmsnorm, "rmsnorm_bwd": _own_rmsnorm_bwd, "linear": _own_linear,
        "linear_bwd": _own_linear_bwd}


# ------------------------------------------------------------------ work

def work(case):
    m, n, es = case["rows"], case["cols"], BYTES[case["dtype"]]
    if case["op"] == "rmsnorm":
        fp8 = case["out"] in LARGEST
        nbytes = m * n * (es * (3 if case["residual"] else 1) + BYTES[case["out"]]) + n * es + \
            4 * m * (2 if fp8 else 1)
        return {"bytes": nbytes, "flops": m * n * (5 + (3 if fp8 else 0))}
    if case["op"] == "rmsnorm_bwd":
        return {"bytes": m * n * es * (4 if case["residual"] else 3) + n * (es + 4) + 4 * m,
                "flops": m * n * 11}
    k = case["inner"]
    if case["op"] == "linear":
        eo = BYTES[case["out"]]
        nbytes = (m + n) * k * es + n * eo + \
            m * n * eo * (1 + bool(case["residual"]) + bool(case["keep"]))
        if case["dtype"] in LARGEST:
            nbytes += 4 * (m + n)
        return {"bytes": nbytes, "flops": 2 * m * n * k}
    # every input (dd, z, a, b) once, every output (dz, da, db, dbias) once
    return {"bytes": es * (3 * m * n + 2 * m * k + 2 * n * k) + 4 * n, "flops": 4 * m * n * k}


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
    s = prepare(case, seed)
    w = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)
         and k not in ("y", "dx", "d", "dz", "da", "db", "workspace")}
    if case["op"] == "rmsnorm":
        h = w["x"] + w["r"] if case["residual"] else w["x"]
        rstd = torch.pow(torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + EPS, -0.5)
        y = torch.einsum("mn,m,n->mn", h, rstd, w["weight"])
        out = {"rstd": rstd, "y": y}
        if case["residual"]:
            out["h"] = h
        if case["out"] in LARGEST:
            scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / LARGEST[case["out"]]
            out["scale"] = torch.clamp(scale, min=AMAX_FLOOR / LARGEST[case["out"]])
            out["y"] = y / out["scale"][:, None]
        return out
    if case["op"] == "rmsnorm_bwd":
        g = w["dy"] * w["weight"]
        inner = torch.einsum("mn,mn->m", g, w["h"]) * w["rstd"] ** 3 / case["cols"]
        dx = torch.einsum("mn,m->mn", g, w["rstd"]) - torch.einsum("mn,m->mn", w["h"], inner)
        if case["residual"]:
            dx += w["dh"]
        return {"dx": dx, "dweight": torch.einsum("mn,mn,m->n", w["dy"], w["h"], w["rstd"])}
    if case["op"] == "linear":
        z = torch.mm(w["a"], w["b"].T)
        if case["dtype"] in LARGEST:
            z *= torch.outer(w["row_scale"], w["col_scale"])
        z += w["bias"]
        d = _exact_act(z, case["act"])[0]
        if case["residual"]:
            d = d + w["r"]
        return {"d": d, "z": z} if case["keep"] else {"d": d}
    dz = w["dd"] * _exact_act(w["z"], case["act"])[1]
    return {"dz": dz, "dbias": torch.einsum("mn->n", dz), "da": torch.mm(dz, w["b"]),
            "db": torch.mm(dz.T, w["a"])}
