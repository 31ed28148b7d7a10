"""GPU parity of the fully connected layer and its gradient where they run in large tiles, whole rounds
of them and split rest ones, on rows of odd length and on rows beyond 2^31 elements. Oracle and bounds
are those of the small sizes, evaluated in fp64 on the GPU."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev()) * scale).to(dtype)


def inputs(m, k, n, dtype, seed):
    return (rand((m, k), seed, dtype), rand((n, k), seed + 1, dtype, k ** -0.5), rand((n,), seed + 2, torch.float32, 0.5),
            rand((m, n), seed + 3, dtype), rand((m, n), seed + 4, dtype))


FORWARD = [("bf16", (2308, 1288, 6800)), ("f16", (4100, 520, 4104)), ("bf16", (2307, 333, 6801)), ("f16", (256, 4096, 256)),
           ("f32", (1030, 524, 2056)), ("f32", (1500, 1000, 3001)), ("bf16", (1856, 1512, 3200)), ("f16", (900, 6000, 1801)),
           ("bf16", (23, 11392, 2528)), ("f32", (6, 7297, 9958)), ("f16", (9, 2000, 8200))]


@pytest.mark.parametrize("dtype,size", FORWARD, ids=lambda v: v if isinstance(v, str) else "%dx%dx%d" % v)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_forward(dtype, size, act):
    m, k, n = size
    X, W, b, R, _ = inputs(m, k, n, L.DTYPES[dtype], 3)
    note("large linear %s %s %s" % (size, dtype, act))
    out, pre = xt.linear(X, W, b, R, act, save_pre=True)
    torch.cuda.synchronize()
    y, ey, z, ez = L.forward(X, W, b, R, act)
    L.check(out, y, ey, "out")
    L.check(pre, z, ez, "pre")
    note("large linear in place %s %s %s" % (size, dtype, act))
    xt.linear(X, W, b, R, act, out=R)
    torch.cuda.synchronize()
    assert torch.equal(R, out)


BACKWARD = [("bf16", (2308, 1288, 3400)), ("f16", (5000, 1288, 2310)), ("bf16", (3001, 1111, 2222)), ("f16", (1100, 2049, 1208)),
            ("f32", (1030, 524, 2056)), ("f32", (3000, 827, 555))]


@pytest.mark.parametrize("dtype,size", BACKWARD, ids=lambda v: v if isinstance(v, str) else "%dx%dx%d" % v)
def test_backward(dtype, size):
    m, k, n = size
    X, W, _, G, pre = inputs(m, k, n, L.DTYPES[dtype], 5)
    for act in ("none", "gelu_tanh"):
        note("large linear_backward %s %s %s" % (size, dtype, act))
        got = xt.linear_backward(G, X, W, None if act == "none" else pre, act)
        torch.cuda.synchronize()
        ref = L.backward(G, X, W, pre, act)
        for t, name in zip(got, ("dX", "dW", "db")):
            L.check(t, *ref[name], what="%s %s" % (act, name))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(60, 50, 70), (700, 320, 904), (2000, 136, 264), (96, 4000, 33), (1100, 2049, 1208)],
                         ids=lambda s: "%dx%dx%d" % s)
def test_each_output_alone(size, dtype):
    """Any subset of dX, dW and db: a product alone may be split otherwise than the two together."""
    m, k, n = size
    X, W, _, G, pre = inputs(m, k, n, L.DTYPES[dtype], 11)
    ref = L.backward(G, X, W, pre, "silu")
    for want in range(1, 8):
        need = dict(need_dX=bool(want & 1), need_dW=bool(want & 2), need_db=bool(want & 4))
        note("linear_backward alone %s %s %s" % (size, dtype, need))
        got = xt.linear_backward(G, X, W, pre, "silu", **need)
        torch.cuda.synchronize()
        for t, name in zip(got, ("dX", "dW", "db")):
            assert (t is not None) == need["need_" + name]
            if t is not None:
                L.check(t, *ref[name], what=name)


def test_offsets_beyond_32_bits():
    """X, out and pre of more than 2^31 elements; the rows on both sides of that border and the last ones."""
    m, k, n = (1 << 22) + 300, 520, 520  # 2^31 elements lie before row 4129776 of 520
    X, W = torch.zeros(m, k, dtype=torch.bfloat16, device=dev()), rand((n, k), 2, torch.bfloat16, k ** -0.5)
    border = (1 << 31) // k
    rows = torch.cat([torch.arange(0, 300), torch.arange(border - 300, border + 300), torch.arange(m - 300, m)]).to(dev())
    X[rows] = rand((len(rows), k), 1, torch.bfloat16)
    note("linear beyond 2^31 elements")
    out, pre = xt.linear(X, W, act="relu", save_pre=True)
    torch.cuda.synchronize()
    y, ey, z, ez = L.forward(X[rows], W, None, None, "relu")
    L.check(out[rows], y, ey, "out")
    L.check(pre[rows], z, ez, "pre")
    assert not out[1000].any() and not out[border - 1000].any()
    note("linear_backward beyond 2^31 elements")
    pre.fill_(1.0)
    dX, dW, db = xt.linear_backward(X, X, W, pre, "relu")  # G is X, zero but in those rows
    torch.cuda.synchronize()
    ref = L.backward(X[rows], X[rows], W, pre[rows], "relu")
    L.check(dX[rows], *ref["dX"], what="dX")
    assert not dX[1000].any() and not dX[border - 1000].any()
    # all m rows count as terms of dW and db
    w, ew = ref["dW"]
    L.check(dW, w, ew + (m + 4) * 2.0 ** -23 * (X[rows].double().abs().T @ X[rows].double().abs()), what="dW")
    d, ed = ref["db"]
    L.check(db, d, ed, what="db")
