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


def check(got, ref, bound, what):
    """layer_oracle.check() of finite references, without copies to the host."""
    assert got.shape == ref.shape, what
    assert ((got.double() - ref).abs() <= bound).all(), what


LONG = (1 << 21) + 9  # rows of more than 4 MiB in every type
SOME = torch.cat([torch.arange(0, 130), torch.arange(LONG // 2 - 130, LONG // 2 + 130), torch.arange(LONG - 130, LONG)])


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("m", [5, 40, 130])
def test_forward_over_long_rows(m, dtype):
    """A contraction of over 2^21 features, which only the kernels for rows of any length take; zeros in all but some
    of them, so that the bound is theirs."""
    n, cols = 24, SOME.to(dev())
    X, W = torch.zeros(m, LONG, dtype=L.DTYPES[dtype], device=dev()), rand((n, LONG), 2, L.DTYPES[dtype], 0.05)
    X[:, cols] = rand((m, len(cols)), 1, X.dtype)
    b, R = rand((n,), 3, torch.float32), rand((m, n), 4, X.dtype)
    note("linear over long rows %s m=%d" % (dtype, m))
    out, pre = xt.linear(X, W, b, R, "gelu", save_pre=True)
    torch.cuda.synchronize()
    y, ey, z, ez = L.forward(X[:, cols], W[:, cols], b, R, "gelu")
    L.check(out, y, ey, "out")
    L.check(pre, z, ez, "pre")


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("size", [(40, LONG, 24), (70, LONG, 9), (130, LONG - 1, 33)], ids=lambda s: "%dx%dx%d" % s)
def test_backward_over_long_rows(size, act, dtype):
    """Rows of X and W too long for the ring kernel: the tile kernel forms d itself, in 16 bits too."""
    m, k, n = size
    X, W = rand((m, k), 1, L.DTYPES[dtype]), rand((n, k), 2, L.DTYPES[dtype])
    G, pre = rand((m, n), 3, X.dtype), rand((m, n), 4, X.dtype)
    for need in ((True, True, True), (True, False, True), (False, True, False)):
        note("linear_backward over long rows %s %s %s %s" % (size, act, dtype, need))
        got = xt.linear_backward(G, X, W, None if act == "none" else pre, act, need_dX=need[0], need_dW=need[1],
                                 need_db=need[2])
        torch.cuda.synchronize()
        ref = L.backward(G, X, W, pre, act)
        for t, name, wanted in zip(got, ("dX", "dW", "db"), need):
            assert (t is not None) == wanted
            if wanted:
                check(t, *ref[name], what=name)
        del got, ref


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_backward_over_many_outputs(act, dtype):
    """Rows of G and pre too long for the ring kernel, zeros in all but some of G's columns."""
    m, k, n = 70, 33, LONG
    cols = SOME.to(dev())
    X, W, pre = rand((m, k), 1, L.DTYPES[dtype]), rand((n, k), 2, L.DTYPES[dtype]), rand((m, n), 4, L.DTYPES[dtype])
    G = torch.zeros(m, n, dtype=X.dtype, device=dev())
    G[:, cols] = rand((m, len(cols)), 3, X.dtype)
    note("linear_backward over many outputs %s %s" % (act, dtype))
    dX, dW, db = xt.linear_backward(G, X, W, None if act == "none" else pre, act)
    torch.cuda.synchronize()
    ref = L.backward(G[:, cols], X, W[cols], pre[:, cols], act)
    check(dX, *ref["dX"], what="dX")
    check(dW[cols], *ref["dW"], what="dW")
    check(db[cols], *ref["db"], what="db")
    others = torch.ones(n, dtype=torch.bool, device=dev())
    others[cols] = False
    assert not dW[others].any() and not db[others].any()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("m", [3, 40, 300])
def test_no_features(m, dtype):
    """k = 0: the layer is act(bias) + residual, the gradient db alone."""
    n, dt = 264, L.DTYPES[dtype]
    X, W = torch.empty(m, 0, dtype=dt, device=dev()), torch.empty(n, 0, dtype=dt, device=dev())
    b, R, pre = rand((n,), 3, torch.float32), rand((m, n), 4, dt), rand((m, n), 5, dt)
    note("no features %s m=%d" % (dtype, m))
    out, z = xt.linear(X, W, b, R, "silu", save_pre=True)
    dX, dW, db = xt.linear_backward(R, X, W, pre, "silu")
    torch.cuda.synchronize()
    y, ey, z64, ez = L.forward(X, W, b, R, "silu")
    check(out, y, ey, "out")
    check(z, z64, ez, "pre")
    assert dX.shape == (m, 0) and dW.shape == (n, 0)
    check(db, *L.backward(R, X, W, pre, "silu")["db"], what="db")
