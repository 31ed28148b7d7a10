"""The bounds that the GPU tests compare with tell lost rows from rounding."""
import torch

import layer_oracle as L


def test_bound_of_a_weight_gradient_tells_lost_rows():
    """1200 rows that are not zero among millions: without the last 300, or 16 of them, nearly every entry of dW is
    outside its bound, on the diagonal and off it."""
    g = torch.Generator().manual_seed(1)
    X = torch.randn((1200, 96), generator=g).bfloat16()
    W = torch.zeros(96, 96).bfloat16()
    dW, bound = L.backward(X, X, W, None, "none")["dW"]
    for lost in (300, 16):
        without, _ = L.backward(X[:-lost], X[:-lost], W, None, "none")["dW"]
        off = (without - dW).abs() > bound
        assert off.double().mean() > 0.8 and off.diagonal().all()
