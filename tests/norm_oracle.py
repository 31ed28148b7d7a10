"""fp64 oracle of layer norm and its gradient, with elementwise error bounds that count roundings: a sum over a
row passes through at most n / 64 + 40 additions on its way (a thread's share, the wavefront, the wavefronts), each
off by half a step of fp32 relative to the sum of magnitudes; a column's sum through m / 256 + 40."""
import torch

from layer_oracle import half_step, smallest

U = 2.0 ** -24


def forward(X, weight, bias, eps):
    """(out, bound), (mean, bound), (rstd, bound) in fp64."""
    x = X.double()
    m, n = x.shape
    w = torch.ones(n, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(n, dtype=torch.float64) if bias is None else bias.double()
    depth = n / 64 + 40
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    e_mean = depth * U * x.abs().mean(1, keepdim=True)
    e_d = e_mean + U * d.abs()
    e_var = depth * U * var + (2 * d.abs() * e_d + e_d * e_d).mean(1, keepdim=True)
    # a square root, a division, the sum with eps: a step of fp32 each at most
    rel = 0.5 * e_var / (var + eps) + 8 * U
    y = d * rstd * w + b
    e = w.abs() * rstd * (e_d + d.abs() * rel) * (1 + rel) + 4 * U * ((d * rstd * w).abs() + b.abs())
    h, s = half_step(X.dtype), smallest(X.dtype)
    return (y, e * (1 + h) + h * y.abs() + s), (mean[:, 0], e_mean[:, 0] + 1e-40), (rstd[:, 0], (rel * rstd)[:, 0])


def backward(G, X, mean, rstd, weight):
    """{name: (value, bound)}; mean and rstd as the call gets them."""
    g, x = G.double(), X.double()
    m, n = x.shape
    w = torch.ones(n, dtype=torch.float64) if weight is None else weight.double()
    r = rstd.double()[:, None]
    xhat, h = (x - mean.double()[:, None]) * r, g * w
    ex, eh = 2 * U * xhat.abs(), U * h.abs()
    depth = n / 64 + 40
    s, q = h.mean(1, keepdim=True), (h * xhat).mean(1, keepdim=True)
    es = depth * U * h.abs().mean(1, keepdim=True)
    eq = (depth + 4) * U * (h * xhat).abs().mean(1, keepdim=True)
    dX = r * (h - s - xhat * q)
    e = r * (eh + es + eq * xhat.abs() + q.abs() * ex + 5 * U * (h.abs() + s.abs() + (xhat * q).abs()))
    hs, sm = half_step(X.dtype), smallest(X.dtype)
    rows = m / 256 + 40
    dw, db = (g * xhat).sum(0), g.sum(0)
    return {"dX": (dX, e * (1 + hs) + hs * dX.abs() + sm),
            "dweight": (dw, (rows + 4) * U * (g * xhat).abs().sum(0) + 1e-40),
            "dbias": (db, rows * U * g.abs().sum(0) + 1e-40)}
