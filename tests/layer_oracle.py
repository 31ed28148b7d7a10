"""fp64 oracle of the fully connected layer and its gradient, with elementwise error bounds.

The bounds count roundings: a sum of k fp32 products is off by at most (k + 4) 2^-23 times the sum of
the products' magnitudes (every addition of the matrix unit off by a whole step, in any order); an
activation or slope by its own evaluation (ACT_REL, ACT_ABS, SLOPE_ABS below); a stored 16-bit value by
half a step, eps / 2 relative, or half the smallest subnormal."""
import math

import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LIPSCHITZ = 1.13  # largest |act'| of any activation (gelu: 1.129)
# 16-bit results: the fitted erfc is off by 2.2e-5 relative, exponentials and reciprocals by a few
# 2^-23 each; fp32 results: the library functions' few 2^-23, and the rounding of an exponent's or
# erfc's argument (at most 2 a^2 2^-24 relative for the |z| <= 8 of these tests).
ACT_REL = {"f32": 8e-6, "bf16": 4e-5, "f16": 4e-5}
ACT_ABS = {"f32": 1e-6, "bf16": 5e-6, "f16": 5e-6}
SLOPE_ABS = {"f32": 8e-6, "bf16": 5e-5, "f16": 5e-5}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * cdf(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("gelu_tanh", "silu"):
        r = 2 * math.sqrt(2 / math.pi)
        u, du = (z, 1.0) if act == "silu" else (r * (z + 0.044715 * z ** 3), r * (1 + 3 * 0.044715 * z ** 2))
        q = torch.sigmoid(u)
        return q + z * q * (1 - q) * du
    return torch.ones_like(z)


def forward(X, W, bias, residual, act):
    """(out, bound of out, pre, bound of pre) in fp64 for inputs of one type."""
    t = {v: k for k, v in DTYPES.items()}[X.dtype]
    k = X.shape[1]
    x, w = X.double(), W.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = (k + 4) * 2.0 ** -23 * mag
    y = act64(z, act)
    ey = ez * LIPSCHITZ
    if act not in ("none", "relu"):
        ey = ey + ACT_REL[t] * y.abs() + ACT_ABS[t]
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * (y.abs() + residual.double().abs())
    h, s = half_step(X.dtype), smallest(X.dtype)
    return y, ey * (1 + h) + h * y.abs() + s, z, ez * (1 + h) + h * z.abs() + s


def backward(G, X, W, pre, act):
    """{name: (value, bound)} of dX, dW and db in fp64."""
    t = {v: k for k, v in DTYPES.items()}[X.dtype]
    m, k = X.shape
    n = W.shape[0]
    g, x, w = G.double(), X.double(), W.double()
    d = g if act == "none" else g * slope64(pre.double(), act)
    ed = torch.zeros_like(d) if act in ("none", "relu") else SLOPE_ABS[t] * g.abs() + 2.0 ** -23 * d.abs()
    db, edb = d.sum(0), ed.sum(0) + (m + 4) * 2.0 ** -23 * (d.abs() + ed).sum(0)
    h, s = half_step(X.dtype), smallest(X.dtype)
    er = ed if act == "none" or t == "f32" else ed * (1 + h) + h * d.abs() + s  # d as the products take it
    dX, dW = d @ w, d.T @ x
    eX = er @ w.abs() + (n + 4) * 2.0 ** -23 * ((d.abs() + er) @ w.abs())
    eW = er.T @ x.abs() + (m + 4) * 2.0 ** -23 * ((d.abs() + er).T @ x.abs())
    return {"dX": (dX, eX * (1 + h) + h * dX.abs() + s), "dW": (dW, eW * (1 + h) + h * dW.abs() + s),
            "db": (db, edb + 2.0 ** -24 * db.abs() + 1e-40)}


def check(got, ref, bound, what):
    got = got.double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, what
    fine = torch.isfinite(ref)
    assert torch.isfinite(got[fine]).all(), "%s: non-finite results" % what
    if fine.any():
        over = ((got - ref).abs()[fine] / bound[fine]).max().item()
        assert over <= 1.0, "%s: error %.3g times its bound" % (what, over)
