"""GPU parity of the fully connected layer and its gradient at sizes next to the limits of a launch and of the
kernels' rows. Oracle and bounds are those of the small sizes, evaluated in fp64 on the GPU."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev()) * scale).to(dtype)


@pytest.mark.parametrize("m,k", [(1, 8), (3, 7)])
def test_few_rows_of_more_outputs_than_their_kernel_can_launch(m, k):
    n = (1 << 28) + 1000
    X, W, b = rand((m, k), 1, torch.bfloat16), rand((n, k), 2, torch.bfloat16, 0.5), rand((n,), 3, torch.float32)
    note("linear %d x %d x %d" % (m, k, n))
    out = xt.linear(X, W, b, act="relu")
    torch.cuda.synchronize()
    for at in (0, (1 << 27) - 500, (1 << 28) - 500, n - 1000):
        y, ey, _, _ = L.forward(X, W[at:at + 1000], b[at:at + 1000], None, "relu")
        L.check(out[:, at:at + 1000], y, ey, "outputs from %d on" % at)
    # every output, to fp32: the products are exact there, their sum is off by a few units
    for at in range(0, n, 1 << 25):
        w = W[at:at + (1 << 25)].float()
        z = b[at:at + (1 << 25)] + sum(X[:, i:i + 1].float() * w[:, i] for i in range(k))
        big = b[at:at + (1 << 25)].abs() + sum(X[:, i:i + 1].float().abs() * w[:, i].abs() for i in range(k))
        assert ((out[:, at:at + (1 << 25)].float() - z.clamp_min(0)).abs()
                <= L.half_step(torch.bfloat16) * z.abs() + 2 * (k + 4) * 2.0 ** -23 * big).all()


ROWS, FEATURES, OUTPUTS = (1 << 22) + 300, 520, 520  # 2^31 elements lie before row 4129776
BORDER = (1 << 31) // FEATURES
LIVE = torch.cat([torch.arange(0, 300), torch.arange(BORDER - 300, BORDER + 300), torch.arange(ROWS - 300, ROWS)])


def test_weight_gradient_over_offsets_beyond_32_bits():
    """dW sums rows on both sides of element 2^31 of G and X, and the last ones. Its bound is that of the rows that
    are not zero: adding an exact zero rounds nothing. The slope is one, so d is G, unrounded."""
    rows = LIVE.to(dev())
    X = torch.zeros(ROWS, FEATURES, dtype=torch.bfloat16, device=dev())
    X[rows] = rand((len(rows), FEATURES), 1, torch.bfloat16)
    W = rand((OUTPUTS, FEATURES), 2, torch.bfloat16, FEATURES ** -0.5)
    pre = torch.ones(ROWS, OUTPUTS, dtype=torch.bfloat16, device=dev())
    note("linear_backward beyond 2^31 elements: dW")
    _, dW, _ = xt.linear_backward(X, X, W, pre, "relu", need_dX=False)  # G is X
    torch.cuda.synchronize()
    L.check(dW, *L.backward(X[rows], X[rows], W, None, "none")["dW"], what="dW")
