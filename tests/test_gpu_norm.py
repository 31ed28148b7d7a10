"""GPU parity of layer norm and its gradient against the fp64 oracle: sizes from one element up, odd ones, every type
and kernel, offsets that would cancel, views, streams, graphs."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
import norm_oracle as N
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype=torch.float32, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).to(dtype)


def cuda(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


# one element; rows shorter than 16 bytes; one wavefront, four and sixteen a row, each with every number of chunks a
# thread; rows beyond the registers; odd widths at each
# (threads a row since then: forward 16, 64, 256 or 1024, gradient every power of two from 16 to 1024; IN_TURNS_16 and
# IN_TURNS_32 below reach each of them with rows enough for several turns)
SIZES = [(1, 1), (3, 2), (7, 5), (1, 8), (5, 9), (4, 64), (9, 100), (1, 511), (70, 512), (13, 777), (33, 1024), (6, 1111),
         (1100, 1030), (5, 2048), (3, 2049), (1, 4096), (300, 4096), (4, 5001), (2, 8192), (3, 10007), (2, 16384), (3, 16385),
         (2, 20001), (2, 33000), (5000, 96), (4099, 260)]


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_forward_and_backward(size, dtype):
    m, n = size
    dt = L.DTYPES[dtype]
    X, G = rand((m, n), m + n, dt, 2.0, 0.7), rand((m, n), m + n + 1, dt)
    w, b = rand(n, 3, offset=1.0), rand(n, 4)
    w, b = (w if m % 3 else None), (b if n % 2 else None)
    gX, gG, gw, gb = cuda(X, G, w, b)
    note("layer_norm %s %s" % (size, dtype))
    out, mean, rstd = xt.layer_norm(gX, gw, gb, 1e-5, save_stats=True)
    plain = xt.layer_norm(gX, gw, gb, 1e-5)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    refs = N.forward(X, w, b, 1e-5)
    for got, (ref, bound), what in zip((out, mean, rstd), refs, ("out", "mean", "rstd")):
        L.check(got, ref, bound, "%s %s %s" % (size, dtype, what))
    note("layer_norm_backward %s %s" % (size, dtype))
    got = xt.layer_norm_backward(gG, gX, mean, rstd, gw)
    again = xt.layer_norm_backward(gG, gX, mean, rstd, gw)
    torch.cuda.synchronize()
    ref = N.backward(G, X, mean.cpu(), rstd.cpu(), w)
    for t, u, name in zip(got, again, ("dX", "dweight", "dbias")):
        L.check(t, *ref[name], what="%s %s %s" % (size, dtype, name))
        assert torch.equal(t, u), name


def test_gradient_against_differences():
    """The gradient of sum(out C) against differences of the fp64 formula."""
    X, w, b, C = rand((6, 50), 1), rand(50, 2, offset=1.0), rand(50, 3), rand((6, 50), 4)
    _, mean, rstd = xt.layer_norm(*cuda(X, w, b), save_stats=True)
    dX, dw, db = xt.layer_norm_backward(*cuda(C, X), mean, rstd, w.to(dev()))
    torch.cuda.synchronize()

    def f(x, v, c):
        d = x - x.mean(1, keepdim=True)
        return ((d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * v + c) * C.double()).sum()

    args, eps = [X.double(), w.double(), b.double()], 1e-5
    for which, got in ((0, dX), (1, dw), (2, db)):
        for at in (0, 7, 49):
            def moved(by):
                a = [t.clone() for t in args]
                a[which].view(-1)[at] += by
                return f(*a)
            slope = (moved(eps) - moved(-eps)) / (2 * eps)  # off by eps^2 f''' / 6 ~ 1e-10
            assert abs(got.view(-1)[at].item() - slope.item()) <= 2e-5 * max(1.0, abs(slope.item()))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_large_offset(dtype):
    """Rows far from zero: squares are of distances from the mean, not differences of squares."""
    dt = L.DTYPES[dtype]
    X = rand((17, 1000), 5, dt, 1.0, 300.0)
    note("layer_norm offset %s" % dtype)
    out, mean, rstd = xt.layer_norm(X.to(dev()), save_stats=True)
    torch.cuda.synchronize()
    for got, (ref, bound), what in zip((out, mean, rstd), N.forward(X, None, None, 1e-5), ("out", "mean", "rstd")):
        L.check(got, ref, bound, what)


def test_constant_rows_and_non_finite_ones():
    X = torch.zeros(5, 640)
    X[1] = 3.25
    X[2, 5] = float("nan")
    X[3, 639] = float("inf")
    X[4] = rand(640, 6)
    w, b = rand(640, 7), rand(640, 8)
    out, mean, rstd = xt.layer_norm(*cuda(X, w, b), save_stats=True)
    torch.cuda.synchronize()
    assert torch.equal(out[:2].cpu(), b.expand(2, 640)) and mean[1] == 3.25
    assert torch.isnan(out[2:4]).all() and torch.isfinite(out[4]).all()
    assert torch.allclose(rstd[:2].cpu(), torch.full((2,), 1e-5 ** -0.5))


def test_zero_sizes():
    d = dev()
    assert xt.layer_norm(torch.empty(0, 5, device=d)).shape == (0, 5)
    assert xt.layer_norm(torch.empty(4, 0, device=d)).shape == (4, 0)
    e = torch.empty(0, device=d)
    dX, dw, db = xt.layer_norm_backward(torch.empty(0, 5, device=d), torch.empty(0, 5, device=d), e, e)
    torch.cuda.synchronize()
    assert dX.shape == (0, 5) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("n", [64, 1111, 5003])
def test_views_of_wider_buffers_and_single_outputs(n, dtype):
    """Rows at odd offsets inside wider buffers, whose surroundings stay untouched; one output at a time."""
    dt, m = L.DTYPES[dtype], 21
    X, G, w = rand((m, n), 11, dt), rand((m, n), 12, dt), rand(n, 13)

    def view(t=None):
        buf = torch.full((m, n + 12), 7.0, dtype=dt, device=dev())
        v = buf[:, 3:3 + n]
        if t is not None:
            v.copy_(t)
        return buf, v

    (_, vX), (_, vG), (ob, vO), (xb, vD) = view(X), view(G), view(), view()
    gw = w.to(dev())
    note("layer_norm views %d %s" % (n, dtype))
    out, mean, rstd = xt.layer_norm(vX, gw, save_stats=True, out=vO)
    dX, dw, db = xt.layer_norm_backward(vG, vX, mean, rstd, gw, dX=vD)
    one = [xt.layer_norm_backward(vG, vX, mean, rstd, gw, need_dX=i == 0, need_dweight=i == 1, need_dbias=i == 2)[i] for i in range(3)]
    torch.cuda.synchronize()
    assert out is vO and dX is vD
    L.check(out, *N.forward(X, w, None, 1e-5)[0], what="out")
    ref = N.backward(G, X, mean.cpu(), rstd.cpu(), w)
    for t, u, name in zip((dX, dw, db), one, ("dX", "dweight", "dbias")):
        L.check(t, *ref[name], what=name)
        assert torch.equal(t, u)
    for buf in (ob, xb):
        assert (buf[:, :3] == 7.0).all() and (buf[:, 3 + n:] == 7.0).all()


def test_rows_beyond_two_to_the_31_elements():
    m, n = 530_000, 4100  # 2.17e9 elements; the last rows are looked at
    X = torch.zeros(m, n, dtype=torch.bfloat16, device=dev())
    tail = rand((3, n), 21, torch.bfloat16)
    X[-3:] = tail.to(dev())
    note("layer_norm of 2^31 elements")
    out, mean, rstd = xt.layer_norm(X, save_stats=True)
    dX, dw, _ = xt.layer_norm_backward(X, X, mean, rstd)
    torch.cuda.synchronize()
    L.check(out[-3:], *[v for v in N.forward(tail, None, None, 1e-5)[0]], what="out")
    ref = N.backward(tail, tail, mean[-3:].cpu(), rstd[-3:].cpu(), None)
    L.check(dX[-3:], *ref["dX"], what="dX")
    L.check(dw, *ref["dweight"], what="dweight")  # the other rows are zero
    assert not out[:1000].any()


def test_streams_and_graph():
    """On a side stream, and captured: replays follow changed inputs and equal eager calls."""
    d = dev()
    X, G, w, b = cuda(rand((500, 1000), 31), rand((500, 1000), 32), rand(1000, 33), rand(1000, 34))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    note("layer_norm on a stream")
    out, mean, rstd = xt.layer_norm(X, w, b, save_stats=True, stream=side)
    grads = xt.layer_norm_backward(G, X, mean, rstd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = xt.layer_norm(X, w, b)
    ref = xt.layer_norm_backward(G, X, mean, rstd, w)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, c) for a, c in zip(grads, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, mn, rs = xt.layer_norm(X, w, b, save_stats=True)
        gr = xt.layer_norm_backward(G, X, mn, rs, w)
    for seed in range(3):
        X.copy_(rand((500, 1000), 40 + seed))
        note("layer_norm replay %d" % seed)
        graph.replay()
        torch.cuda.synchronize()
        eo, em, er = xt.layer_norm(X, w, b, save_stats=True)
        eg = xt.layer_norm_backward(G, X, em, er, w)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and all(torch.equal(a, c) for a, c in zip(gr, eg))
    assert d.type == "cuda"


# Rows in turns: so many that every workgroup takes three turns, the last one of a part of them. Gradient: 256 workgroups,
# each of 1024 / lanes rows a turn with the fewest lanes (16 to 1024) that have two 16-byte chunks of a row each, one (the
# first) or four (fp32 9152). Forward: 16 lanes up to 64 chunks, 64 up to 256, 256 up to 1024, 1024 up to 4096, 1024
# workgroups of 256 / lanes rows a turn or 512 of one. The last in 16 bits: the forward's registers, the gradient's kernels
# for any length.
IN_TURNS_16 = [(33000, 100), (33001, 250), (33000, 500), (8300, 1001), (4201, 1999), (2200, 4096), (1100, 5117), (700, 12000), (1100, 20001)]
IN_TURNS_32 = [(33000, 61), (33001, 125), (33000, 250), (8300, 501), (4201, 1000), (2200, 2047), (1100, 4090), (1050, 6001), (700, 9152), (1050, 16384)]


@pytest.mark.parametrize("dtype, size", [(t, s) for t in L.DTYPES for s in (IN_TURNS_32 if t == "f32" else IN_TURNS_16)],
                         ids=lambda v: v if isinstance(v, str) else "%dx%d" % v)
def test_rows_in_turns(dtype, size):
    """Every row of many turns against the oracle, on the GPU. G is whole numbers: their sums in fp32 are exact, so that dbias
    tells a row that is lost or counted twice."""
    m, n = size
    dt = L.DTYPES[dtype]
    g = torch.Generator(dev()).manual_seed(m + n)
    X = (torch.randn(m, n, generator=g, device=dev()) * 2.0 + 0.7).to(dt)
    G = torch.randint(-3, 4, (m, n), generator=g, device=dev()).to(dt)
    w, b = (torch.randn(n, generator=g, device=dev()) + 1.0 for _ in range(2))
    note("layer_norm in turns %s %s" % (size, dtype))
    out, mean, rstd = xt.layer_norm(X, w, b, save_stats=True)
    got = xt.layer_norm_backward(G, X, mean, rstd, w)
    torch.cuda.synchronize()
    for t, (ref, bound), what in zip((out, mean, rstd), N.forward(X, w, b, 1e-5), ("out", "mean", "rstd")):
        L.check(t, ref, bound, "%s %s %s" % (size, dtype, what))
    ref = N.backward(G, X, mean, rstd, w)
    for t, name in zip(got, ("dX", "dweight", "dbias")):
        L.check(t, *ref[name], what="%s %s %s" % (size, dtype, name))
    assert torch.equal(got[2].double(), G.double().sum(0))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("n", [33_000, 100_003, 40_000_003])
def test_long_constant_rows(n, dtype):
    """The mean of a constant row is that constant at any length: sums that drift would leave distances, which 1 / sqrt(eps)
    blows up."""
    dt = L.DTYPES[dtype]
    X = torch.full((2, n), 1.1, dtype=dt, device=dev())
    X[1] = -300.7
    note("layer_norm constant %d %s" % (n, dtype))
    out, mean, rstd = xt.layer_norm(X, save_stats=True)
    torch.cuda.synchronize()
    assert torch.equal(mean, X[:, 0].float()) and not out.any()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


def test_longest_rows():
    """A row of 2^27 - 1 columns, the most. The row's sums are fp64 of four terms at a time in fp32; what is left are the roundings
    of xhat (2), h (1), the means of h (3 additions, stored) and h xhat (the same, and 4 of its terms) and of the formula
    (5), each 2^-24 of what it rounds."""
    n, U = 2 ** 27 - 1, N.U
    g = torch.Generator(dev()).manual_seed(1)
    X = torch.randn(1, n, generator=g, device=dev()) + 100.0
    G, w = torch.full((1, n), 0.1, device=dev()), torch.rand(n, generator=g, device=dev()) * 0.01 + 1.0
    note("layer_norm of 2^27 - 1 columns")
    out, mean, rstd = xt.layer_norm(X, w, save_stats=True)
    got = xt.layer_norm_backward(G, X, mean, rstd, w)
    torch.cuda.synchronize()
    x = X.double()
    ref = x.mean()
    var = ((x - ref) ** 2).mean()
    assert abs(mean.double() - ref) <= 2 * U * ref and abs(rstd.double() * torch.sqrt(var + 1e-5) - 1) <= 8 * U
    d = x - ref
    # mean off by 2 U of itself, the distance from it, rstd and two products
    assert ((out.double() - d * rstd.double() * w).abs() <= rstd * w * (2 * U * ref + 4 * U * d.abs()) * 1.01).all()
    xhat, h = (x - mean.double()) * rstd.double(), G.double() * w
    s, q, qa = h.mean(), (h * xhat).mean(), (h * xhat).abs().mean()
    want = rstd.double() * (h - s - xhat * q)
    bound = rstd * U * (h + 4 * s + 8 * qa * xhat.abs() + 2 * xhat.abs() * q.abs() + 5 * (h + s.abs() + (xhat * q).abs())) * 1.01
    assert ((got[0].double() - want).abs() <= bound).all()
    assert ((got[1].double() - (G * xhat)[0]).abs() <= 4 * U * (G * xhat)[0].abs()).all() and torch.equal(got[2], G[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 8, 100, 1000, 1030, 4096, 5003, 12000, 20001, 40000])
def test_rows_whose_squares_leave_fp32(n, dtype):
    """Distances whose squares are beyond fp32's largest or below its smallest numbers, next to ordinary rows."""
    dt = L.DTYPES[dtype]
    X = rand((23, n), n)
    X *= torch.tensor([1.0, 1e20, 1e-25, 3e37, 1e-30, 1e10, 1e-15, 1e19])[torch.arange(23) % 8][:, None]
    X[8] = 0.0
    X[9] += 1e25  # the mean is far, the distances as those of row 1
    X = X.to(dt)
    w, b = rand(n, 1, offset=1.0), rand(n, 2)
    for eps in (0.0, 1e-38, 1e-5, 1e30):
        note("layer_norm scaled rows %d %s %g" % (n, dtype, eps))
        out, mean, rstd = xt.layer_norm(*cuda(X, w, b), eps, save_stats=True)
        torch.cuda.synchronize()
        # a row without distances has no 1 / 0
        rows = [i for i in range(23) if eps > 0 or (X[i] != X[i, 0]).any()]
        for t, (ref, bound), what in zip((out, mean, rstd), N.forward(X, w, b, eps), ("out", "mean", "rstd")):
            L.check(t[rows], ref[rows], bound[rows], "%s eps %g" % (what, eps))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(33000, 100), (8300, 1001), (2200, 4096), (1100, 12000)], ids=lambda s: "%dx%d" % s)
def test_rows_next_to_those_that_leave_fp32(size, dtype):
    """Rows of any turn of a workgroup, and what they leave of the others: every bit."""
    m, n = size
    dt = L.DTYPES[dtype]
    X, w, b = cuda(rand((m, n), 1, dt), rand(n, 2, offset=1.0), rand(n, 3))
    plain = xt.layer_norm(X, w, b, 0.0, save_stats=True)
    rows = torch.tensor([0, 5, m // 3, m // 2 + 1, m - 2, m - 1], device=dev())
    scales = torch.tensor([1e25, 1e-24, 1e30, 1e-30, 1e-23, 1e20], device=dev())
    X[rows] = (X[rows].float() * scales[:, None]).to(dt)
    note("layer_norm next to far rows %s %s" % (size, dtype))
    got = xt.layer_norm(X, w, b, 0.0, save_stats=True)
    torch.cuda.synchronize()
    for t, (ref, bound), what in zip(got, N.forward(X[rows], w, b, 0.0), ("out", "mean", "rstd")):
        L.check(t[rows], ref, bound, what)
    others = torch.ones(m, dtype=torch.bool, device=dev())
    others[rows] = False
    assert all(torch.equal(t[others], u[others]) for t, u in zip(got, plain))
