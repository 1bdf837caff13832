"""The layer operators (normalisation, linear layer and their gradients) written
from their formulas in 64 bits on the CPU, the helpers that lay tensors out for
the GPU calls, and the rounding units their tolerances are made of."""
import math

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
U32 = 2.0 ** -24
# largest relative error of one rounding to nearest
ROUND = {"f32": U32, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
# half the distance between a type's smallest neighbours
SMALL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10,
         "e5m2": 2.0 ** -17}
TOP8 = {"e4m3": 448.0, "e5m2": 57344.0}


def rounding(ref, t):
    """Largest error of rounding `ref` to type t."""
    return ref.abs() * ROUND[t] + SMALL[t]


def strided(values, t, pad=16, device="cuda", fill=float("nan")):
    """`values` (2-D) as type t with rows `pad` elements wider than the next multiple of 16,
    the rest of each row filled with `fill`: (view, whole buffer)."""
    rows, cols = values.shape
    buf = torch.full((max(rows, 1), (cols + 15) // 16 * 16 + pad), fill, device=device).to(TYPES[t])
    buf[:rows, :cols] = values.to(device=device, dtype=torch.float32).to(TYPES[t])
    return buf[:rows, :cols], buf


def padding_untouched(view, buf):
    """Whether everything outside the view still holds its NaN fill."""
    b = buf.float().clone()
    b[:view.shape[0], :view.shape[1]] = float("nan")
    return bool(torch.isnan(b).all())


def f64(t):
    return t.detach().cpu().to(torch.float64)


def within(got, want, bound, what=""):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                           f"{float(((got - want).abs() / bound).nan_to_num(math.inf).max()):.3g} "
                           f"of the bound")


# ------------------------------------------------------------------ normalisation

def rmsnorm(x, r, w, eps):
    h = x if r is None else x + r
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + eps)
    return h, rstd, h * rstd[:, None] * w


def rmsnorm_bwd(dy, h, w, rstd, dh):
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(dim=1, keepdim=True))
    return (dx if dh is None else dx + dh), (dy * n).sum(dim=0)


# ------------------------------------------------------------------ activations

def act(v, name):
    if name == "relu":
        return v.clamp(min=0.0)
    if name == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def act_grad(v, name):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) + \
            v * torch.exp(-v * v / 2.0) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (v + 0.044715 * v ** 3))
        return s + v * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * v * v)
    if name == "silu":
        s = torch.sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    return torch.ones_like(v)
