"""fp64 oracle of the losses over an output layer and their gradients, with elementwise error bounds that count roundings.

Logits: sums of k fp32 products, as in the layer's oracle. exp(x) is off by 2 |x| 2^-24 + 2^-23 relative (the product with
log2 e, that constant, the hardware's exponential). A sum of exponentials passes through at most 32 additions in a lane, 2
between lanes, and one for each part of the vocabulary that a thread joins, and is taken relative to up to three
largest logits on its way (of the half tile, of the parts, of the pieces), each a product with an exponential."""
import torch

from layer_oracle import half_step, smallest

U = 2.0 ** -24


def _logits(X, W, bias, temperature):
    k = X.shape[1]
    x, w = X.double(), W.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + torch.where(torch.isinf(bias), 0.0, bias.double().abs())
    ez = (k + 4) * 2 * U * mag
    t = z / temperature
    return t, ez / temperature + 2 * U * torch.where(torch.isinf(t), 0.0, t.abs())


def _exp_error(x):
    return (2 * x.abs() + 2) * U


def _lse(t, et):
    n = t.shape[1]
    top = t.max(1, keepdim=True)[0]
    lse = torch.logsumexp(t, 1, keepdim=True)
    p = torch.exp(t - lse)
    far = torch.where(p > 0, t - top, 0.0)
    e = (p * (et + 3 * _exp_error(far))).sum(1, keepdim=True)
    return lse, e * 1.01 + (60 + n / 512) * U + 4 * U * (top.abs() + lse.abs()), p


def targets(classes, teacher, n, temperature):
    """(P, bound), m x s, from a teacher's logits."""
    t = teacher.double() / temperature
    t = t.masked_fill(classes < 0, float("-inf"))
    P = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)
    top = t.max(1, keepdim=True)[0]
    s = classes.shape[1]
    far = torch.where(P > 0, t - top, 0.0)
    size = torch.where(P > 0, t, 0.0).abs() + torch.where(torch.isinf(top), 0.0, top).abs()
    rel = 4 * U * size + 2 * _exp_error(far) + (s + 16) * U
    rel = rel + (P * rel).sum(1, keepdim=True)
    merged, bound = torch.zeros_like(P), torch.zeros_like(P)
    for e in range(s):  # equal classes in the first place
        same = (classes == classes[:, e:e + 1]) & (classes >= 0)
        first = ~same[:, :e].any(1) & (classes[:, e] >= 0)
        merged[:, e] = torch.where(first, (P * same).sum(1), 0.0)
        bound[:, e] = torch.where(first, (P * rel * same).sum(1) + s * U * (P * same).sum(1), 0.0)
    return merged, bound


def _losses(X, W, bias, classes, P, eP, temperature):
    t, et = _logits(X, W, bias, temperature)
    lse, e_lse, p = _lse(t, et)
    at = classes.long().clamp_min(0)
    ts, es = t.gather(1, at), et.gather(1, at)
    on = P > 0
    logP = torch.where(on, torch.log(P.clamp_min(1e-300)), 0.0)
    inner = torch.where(on, logP - ts + lse, 0.0)
    size = torch.where(on, logP.abs() + ts.abs() + lse.abs(), 0.0)
    loss = (P * inner).sum(1)
    e = (P * (es + e_lse) * on + eP * (inner.abs() + 1) + 4 * U * P * size).sum(1) + (P.shape[1] + 20) * U * (P * inner.abs()).sum(1)
    return t, et, lse, e_lse, p, loss, e + U * loss.abs()


def forward(X, W, bias, classes, P, eP, temperature=1.0):
    """((loss, bound), (lse, bound)); labels: classes m x 1 and P one where they count."""
    _, _, lse, e_lse, _, loss, e = _losses(X, W, bias, classes, P, eP, temperature)
    return (loss, e + 1e-30), (lse[:, 0], e_lse[:, 0])


def backward(grad, X, W, bias, classes, P, eP, temperature=1.0, lse=None):
    """{name: (value, bound)} of dX, dW and db; lse as the call gets it (float32)."""
    m, k = X.shape
    n = W.shape[0]
    t, et = _logits(X, W, bias, temperature)
    l = lse.double()[:, None]
    p = torch.exp(t - l)
    g = torch.where((P > 0).any(1), grad.double(), 0.0)[:, None] / temperature
    at = classes.long().clamp_min(0)
    d = p.clone().scatter_add_(1, at, -P) * g
    far = torch.where(p > 0, t - l, 0.0)
    ed = p * (et + _exp_error(far) + 2 * U) + 4 * U * p
    ed = (ed.scatter_add_(1, at, eP + 8 * U * P)) * g.abs() + 2 * U * d.abs()
    x, w = X.double(), W.double()
    db, edb = d.sum(0), ed.sum(0) + (m + 4) * 2 * U * (d.abs() + ed).sum(0)
    h, s = half_step(X.dtype), smallest(X.dtype)
    if X.dtype == torch.float32:
        er = ed
    else:  # d as the products take it; fp16 scaled so that the largest factor is at least 2^13
        least = s if X.dtype == torch.bfloat16 else s * 2.0 ** -13 * g.abs().max()
        er = ed * (1 + h) + h * d.abs() + least
    dX, dW = d @ w, d.T @ x
    eX = er @ w.abs() + (n + 4) * 2 * U * ((d.abs() + er) @ w.abs())
    eW = er.T @ x.abs() + (m + 4) * 2 * U * ((d.abs() + er).T @ x.abs())
    return {"dX": (dX, eX * (1 + h) + h * dX.abs() + s), "dW": (dW, eW * (1 + h) + h * dW.abs() + s),
            "db": (db, edb + U * db.abs() + 1e-40)}


def of_labels(labels):
    """(classes m x 1, P, bound) of labels."""
    return labels[:, None], (labels[:, None] >= 0).double(), torch.zeros(len(labels), 1, dtype=torch.float64, device=labels.device)
