"""GPU parity of the fully connected layer and its gradient against the fp64 oracle, within bounds that
count roundings: sizes from one element up, odd ones, every type, activation and operand layout."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def inputs(m, k, n, dtype, seed=1):
    X = rand((m, k), seed, dtype)
    W = rand((n, k), seed + 1, dtype, max(k, 1) ** -0.5)
    return X, W, rand((n,), seed + 2, torch.float32, 0.5), rand((m, n), seed + 3, dtype), rand((m, n), seed + 4, dtype)


def on_gpu(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


SIZES = [(1, 1, 1), (1, 64, 8), (3, 5, 7), (2, 300, 2000), (17, 33, 65), (64, 64, 64), (65, 129, 70), (1, 4096, 513),
         (33, 1024, 130), (300, 40, 1000), (255, 1111, 77), (128, 256, 512), (256, 512, 264), (513, 768, 520),
         (31, 72, 96), (16, 2048, 2056), (61, 1000, 333), (700, 320, 904)]


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%dx%d" % s)
def test_forward(size, dtype):
    m, k, n = size
    dt = L.DTYPES[dtype]
    X, W, b, R, _ = inputs(m, k, n, dt)
    gX, gW, gb, gR = on_gpu(X, W, b, R)
    for c, act in enumerate(L.ACTS):
        bias, res, pre = (c + m) % 2 == 0, (c + n) % 3 != 1, (c + k) % 2 == 1
        note("linear %s %s %s bias=%d residual=%d pre=%d" % (size, dtype, act, bias, res, pre))
        got = xt.linear(gX, gW, gb if bias else None, gR if res else None, act, save_pre=pre)
        torch.cuda.synchronize()
        y, ey, z, ez = L.forward(X, W, b if bias else None, R if res else None, act)
        L.check(got[0] if pre else got, y, ey, "%s %s %s out" % (size, dtype, act))
        if pre:
            L.check(got[1], z, ez, "%s %s %s pre" % (size, dtype, act))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%dx%d" % s)
def test_backward(size, dtype):
    m, k, n = size
    dt = L.DTYPES[dtype]
    X, W, _, G, pre = inputs(m, k, n, dt, seed=7)
    gX, gW, gG, gP = on_gpu(X, W, G, pre)
    for act in (L.ACTS[(m + n) % 5], L.ACTS[(m + n + 2) % 5], "none"):
        note("linear_backward %s %s %s" % (size, dtype, act))
        got = xt.linear_backward(gG, gX, gW, None if act == "none" else gP, act)
        torch.cuda.synchronize()
        ref = L.backward(G, X, W, pre, act)
        for t, name in zip(got, ("dX", "dW", "db")):
            L.check(t, *ref[name], what="%s %s %s %s" % (size, dtype, act, name))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_zero_sizes(dtype):
    dt = L.DTYPES[dtype]
    d = dev()
    b = rand((6,), 3, torch.float32)
    note("zero sizes %s" % dtype)
    out = xt.linear(torch.empty(4, 0, dtype=dt, device=d), torch.empty(6, 0, dtype=dt, device=d), b.to(d))
    torch.cuda.synchronize()
    L.check(out, b.double().expand(4, 6), L.half_step(dt) * b.double().abs().expand(4, 6), "k = 0")
    assert xt.linear(torch.empty(0, 5, dtype=dt, device=d), torch.empty(6, 5, dtype=dt, device=d)).shape == (0, 6)
    assert xt.linear(torch.empty(4, 5, dtype=dt, device=d), torch.empty(0, 5, dtype=dt, device=d)).shape == (4, 0)
    dX, dW, db = xt.linear_backward(torch.empty(0, 6, dtype=dt, device=d), torch.empty(0, 5, dtype=dt, device=d),
                                    torch.ones(6, 5, dtype=dt, device=d))
    torch.cuda.synchronize()
    assert dX.shape == (0, 5) and not dW.any() and dW.shape == (6, 5) and not db.any() and db.shape == (6,)
    dX, dW, db = xt.linear_backward(torch.empty(4, 0, dtype=dt, device=d), torch.ones(4, 5, dtype=dt, device=d),
                                    torch.empty(0, 5, dtype=dt, device=d))
    torch.cuda.synchronize()
    assert not dX.any() and dX.shape == (4, 5) and dW.shape == (0, 5) and db.shape == (0,)


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(70, 96, 130), (300, 520, 260)], ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_views_of_wider_buffers(size, dtype, offset):
    """Rows inside wider buffers, whose surroundings stay untouched; out in place of the residual."""
    m, k, n = size
    dt = L.DTYPES[dtype]
    X, W, b, R, P = inputs(m, k, n, dt, seed=20)

    def view(t, fill=float("nan")):
        buf = torch.full((t.shape[0], t.shape[1] + offset + 8), fill, dtype=t.dtype, device=dev())
        v = buf[:, offset:offset + t.shape[1]]
        v.copy_(t)
        return buf, v

    (_, gX), (_, gW), (rb, gR), (pb, gP) = view(X), view(W), view(R, 7.0), view(P, 7.0)
    note("linear views %s %s offset %d" % (size, dtype, offset))
    out, pre = xt.linear(gX, gW, b.to(dev()), gR, "silu", out=gR, pre=gP)
    torch.cuda.synchronize()
    y, ey, z, ez = L.forward(X, W, b, R, "silu")
    L.check(out, y, ey, "out")
    L.check(pre, z, ez, "pre")
    for buf in (rb, pb):
        assert (buf[:, :offset] == 7.0).all() and (buf[:, offset + n:] == 7.0).all()
    (_, gG), (_, gP), (xb, dX), (wb, dW) = view(R), view(P), view(X, 7.0), view(W, 7.0)
    note("linear_backward views %s %s offset %d" % (size, dtype, offset))
    _, _, db = xt.linear_backward(gG, gX, gW, gP, "gelu", dX=dX, dW=dW)
    torch.cuda.synchronize()
    ref = L.backward(R, X, W, P, "gelu")
    for t, name in ((dX, "dX"), (dW, "dW"), (db, "db")):
        L.check(t, *ref[name], what=name)
    for buf, w in ((xb, k), (wb, k)):
        assert (buf[:, :offset] == 7.0).all() and (buf[:, offset + w:] == 7.0).all()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("m", [2, 40, 520])
def test_infinities_and_nan_reach_the_outputs_they_belong_to(dtype, m):
    k, n = 136, 264
    dt = L.DTYPES[dtype]
    X, W, _, _, _ = inputs(m, k, n, dt, seed=5)
    X[0, 3], X[1, 100] = float("inf"), float("nan")
    W[5] = W[5].abs() + 0.01
    note("linear inf/nan %s m=%d" % (dtype, m))
    out = xt.linear(X.to(dev()), W.to(dev())).cpu().double()
    ref = X.double() @ W.double().T
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    assert torch.equal(out[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert torch.isinf(ref[0]).all() and torch.isnan(ref[1]).all()


@pytest.mark.parametrize("act", [a for a in L.ACTS if a != "none"])
@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_activations_and_slopes_at_far_arguments(dtype, act):
    """One feature, weight 1: z runs over the type's whole range, so that exponentials overflow."""
    dt = L.DTYPES[dtype]
    big = 6e4 if dtype == "f16" else 1e30
    z = torch.cat([torch.linspace(-12, 12, 241), torch.tensor([-big, -1e4, -100.0, -30.0, 0.0, 30.0, 100.0, 1e4, big])]).to(dt)[:, None]
    one = torch.ones(1, 1, dtype=dt)
    note("far arguments %s %s" % (dtype, act))
    y = xt.linear(z.to(dev()), one.to(dev()), act=act).cpu().double()
    ref = L.act64(z.double(), act)
    # relative to the result, with exp's argument rounded (|x| 2^-23); nothing below 1e-30 is compared
    tol = (L.ACT_REL[dtype] + L.half_step(dt) + 100 * 2.0 ** -23) * ref.abs() + L.ACT_ABS[dtype] + L.smallest(dt)
    assert ((y - ref).abs() <= tol).all()
    dX, _, _ = xt.linear_backward(one.expand(z.shape[0], 1).contiguous().to(dev()), z.to(dev()), one.to(dev()),
                                  z.to(dev()), act)
    s = torch.nan_to_num(L.slope64(z.double().clamp(-100, 100), act))
    assert ((dX.cpu().double() - s).abs() <= L.SLOPE_ABS[dtype] + 2 * L.half_step(dt) * s.abs() + L.smallest(dt)).all()


def test_gradient_against_differences():
    """The fp32 gradient against central differences of the fp64 loss sum(C * out)."""
    m, k, n = 9, 14, 11
    X, W, b, C, _ = inputs(m, k, n, torch.float32, seed=31)
    for act in L.ACTS:
        if act == "relu":
            continue  # not differentiable where a difference straddles zero

        def loss(x, w, bb):
            return (C.double() * L.act64(x @ w.T + bb, act)).sum().item()

        note("gradient differences %s" % act)
        _, pre = xt.linear(X.to(dev()), W.to(dev()), b.to(dev()), act=act, save_pre=True)
        dX, dW, db = [t.cpu().double() for t in
                      xt.linear_backward(C.to(dev()), X.to(dev()), W.to(dev()), pre, act)]
        h = 1e-5
        args = [X.double(), W.double(), b.double()]
        for which, g in ((0, dX), (1, dW), (2, db)):
            flat = args[which].view(-1)
            for at in range(0, flat.numel(), 13):
                keep = flat[at].item()
                flat[at] = keep + h
                up = loss(*args)
                flat[at] = keep - h
                down = loss(*args)
                flat[at] = keep
                diff = (up - down) / (2 * h)
                assert abs(diff - g.view(-1)[at].item()) <= 2e-4 * max(1.0, abs(diff)), (act, which, at)


def test_other_stream_workspace_and_repeats():
    """On a stream of its own with the caller's workspace, and the same bits on every call."""
    m, k, n = 40, 4096, 96
    X, W, b, R, P = inputs(m, k, n, torch.bfloat16, seed=9)
    gX, gW, gb, gR, gP = on_gpu(X, W, b, R, P)
    first = xt.linear(gX, gW, gb, gR, "gelu").clone()
    grads = [t.clone() for t in xt.linear_backward(gR, gX, gW, gP, "silu")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=dev())
    s.wait_stream(torch.cuda.current_stream())
    note("linear on another stream")
    for _ in range(3):
        got = xt.linear(gX, gW, gb, gR, "gelu", stream=s, workspace=ws)
        back = xt.linear_backward(gR, gX, gW, gP, "silu", stream=s, workspace=ws)
        s.synchronize()
        assert torch.equal(got, first)
        assert all(torch.equal(a, b) for a, b in zip(back, grads))


@pytest.mark.parametrize("dtype,size", [("bf16", (300, 520, 260)), ("f32", (64, 2048, 48)), ("f16", (8, 4096, 128)),
                                        ("f16", (77, 333, 131)), ("f32", (1100, 264, 320))])
def test_graph_replays(dtype, size):
    """A captured step (layer and gradient) replayed with new inputs in the same tensors."""
    m, k, n = size
    dt = L.DTYPES[dtype]
    gX, gW, gb, gR, gP = on_gpu(*inputs(m, k, n, dt, seed=40))

    def step():
        out, pre = xt.linear(gX, gW, gb, None, "gelu_tanh", save_pre=True)
        return (out, pre) + xt.linear_backward(gR, gX, gW, pre, "gelu_tanh")

    note("graph %s %s" % (dtype, size))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (50, 60, 70):
        for t, v in zip((gX, gW, gb, gR), inputs(m, k, n, dt, seed=seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
