"""GPU parity of the losses over an output layer and their gradients against the fp64 oracle, within bounds that count
roundings: sizes from one class up, odd ones, several pieces of the vocabulary, rows that do not count, classes taken out
by the bias, lists with empty and equal places, views, streams, graphs."""
import math

import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
import loss_oracle as O
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def whole(n, shape, seed):
    return torch.randint(0, n, shape, generator=torch.Generator().manual_seed(seed))


def inputs(m, k, n, dt, seed, bias=True):
    X, W = rand((m, k), seed, dt), rand((n, k), seed + 1, dt, 2.0 * max(k, 1) ** -0.5)
    labels = whole(n, (m,), seed + 2)
    if m > 1:
        labels = torch.where(torch.rand(m, generator=torch.Generator().manual_seed(seed + 3)) < 0.2, -100, labels)
    grad = rand(m, seed + 4).abs() + 0.1
    return X, W, rand(n, seed + 5) if bias else None, labels, grad / m


def lists(m, n, s, seed):
    """Classes with empty and equal places and rows without any, and a teacher's logits."""
    classes = whole(n, (m, s), seed)
    empty = torch.rand((m, s), generator=torch.Generator().manual_seed(seed + 1)) < 0.2
    classes = torch.where(empty, -1, classes)
    if m > 3:
        classes[3] = -1
    return classes, rand((m, s), seed + 2, scale=2.0)


def cuda(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


def check_all(got, ref, what):
    for t, name in zip(got, ("dX", "dW", "db")):
        L.check(t, *ref[name], what="%s %s" % (what, name))


SIZES = [(1, 1, 1), (3, 5, 2), (2, 8, 1), (17, 33, 65), (64, 64, 64), (65, 129, 70), (1, 256, 1000), (33, 100, 513), (300, 40, 1000),
         (130, 264, 5000), (257, 96, 8200), (5, 1031, 300), (1000, 64, 10), (513, 520, 264), (700, 256, 2500),
         (1, 4096, 300), (32, 77, 9000), (16, 8200, 200), (33, 96, 17000), (20, 9, 4097),
         (93, 1415, 105), (200, 4072, 144), (48, 3776, 110), (40, 9000, 600)]


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%dx%d" % s)
def test_cross_entropy(size, dtype):
    m, k, n = size
    dt = L.DTYPES[dtype]
    X, W, b, labels, grad = inputs(m, k, n, dt, m + k + n, (m + n) % 3 != 0)
    labels = labels.to(torch.int32 if k % 2 else torch.int64)
    gX, gW, gb, gl, gg = cuda(X, W, b, labels, grad)
    note("linear_cross_entropy %s %s" % (size, dtype))
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    torch.cuda.synchronize()
    target = O.of_labels(labels)
    for got, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, *target), ("loss", "lse")):
        L.check(got, ref, bound, "%s %s %s" % (size, dtype, what))
    note("linear_cross_entropy_backward %s %s" % (size, dtype))
    got = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
    again = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
    torch.cuda.synchronize()
    check_all(got, O.backward(grad, X, W, b, *target, lse=lse.cpu()), "%s %s" % (size, dtype))
    assert all(torch.equal(a, c) for a, c in zip(got, again))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(1, 8, 3, 1), (17, 33, 65, 2), (65, 129, 700, 8), (300, 64, 2500, 32), (130, 264, 900, 70), (5, 16, 5000, 1024), (40, 16, 600, 200), (31, 8192, 100, 20), (100, 4072, 144, 30), (50, 6000, 5, 4)],
                         ids=lambda s: "%dx%dx%dx%d" % s)
def test_distillation(size, dtype):
    m, k, n, s = size
    dt = L.DTYPES[dtype]
    X, W, b, _, grad = inputs(m, k, n, dt, m + k + n, n % 2 == 0)
    classes, teacher = lists(m, n, s, s)
    classes = classes.to(torch.int32 if k % 2 else torch.int64)
    teacher = teacher.to((dt, torch.float32)[s % 2])
    T = (1.0, 2.0, 0.7)[m % 3]
    gX, gW, gb, gc, gt, gg = cuda(X, W, b, classes, teacher, grad)
    note("linear_distillation %s %s" % (size, dtype))
    loss, lse, weights = xt.linear_distillation(gX, gW, gc, gt, gb, T)
    torch.cuda.synchronize()
    P, eP = O.targets(classes, teacher, n, T)
    L.check(weights, P, eP + 1e-40, "%s %s weights" % (size, dtype))
    for got, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, classes, P, eP, T), ("loss", "lse")):
        L.check(got, ref, bound, "%s %s %s" % (size, dtype, what))
    note("linear_distillation_backward %s %s" % (size, dtype))
    got = xt.linear_distillation_backward(gg, gX, gW, gc, weights, lse, gb, T)
    torch.cuda.synchronize()
    check_all(got, O.backward(grad, X, W, b, classes, weights.cpu().double(), torch.zeros_like(P), T, lse=lse.cpu()), "%s %s" % (size, dtype))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(64, 32, 1, 900), (7, 512, 65, 65), (300, 64, 50, 300), (40, 4000, 300, 250), (33, 16, 1000, 1024),
                                  (500, 2048, 1100, 129), (20, 8, 40000, 513)], ids=lambda s: "%dx%dx%dx%d" % s)
def test_long_lists(size, dtype):
    """More places than lanes, most classes listed several times; logits in tiles and in memory."""
    m, k, n, s = size
    X, W, b, _, grad = inputs(m, k, n, L.DTYPES[dtype], m + s)
    classes, teacher = lists(m, n, s, s + 1)
    classes[-1] = classes[-1, 0]
    gX, gW, gb, gc, gt, gg = cuda(X, W, b, classes, teacher, grad)
    note("long lists %s %s" % (size, dtype))
    loss, lse, weights = xt.linear_distillation(gX, gW, gc, gt, gb, 1.5)
    got = xt.linear_distillation_backward(gg, gX, gW, gc, weights, lse, gb, 1.5)
    again = xt.linear_distillation_backward(gg, gX, gW, gc, weights, lse, gb, 1.5)
    torch.cuda.synchronize()
    P, eP = O.targets(classes, teacher, n, 1.5)
    L.check(weights, P, eP + 1e-40, "%s %s weights" % (size, dtype))
    for t, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, classes, P, eP, 1.5), ("loss", "lse")):
        L.check(t, ref, bound, "%s %s %s" % (size, dtype, what))
    check_all(got, O.backward(grad, X, W, b, classes, weights.cpu().double(), torch.zeros_like(P), 1.5, lse=lse.cpu()), "%s %s" % (size, dtype))
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [566, 1150, 9000])
def test_rounding_of_a_mean(m, dtype):
    """1 / m in 16 bits is off by up to half a step, alike in all rows. d is scaled so that it is a power of two, and what is
    left is the rounding of its softmax, as that of d / grad here, and the outputs' own: independent, so that their squares
    add; a tenth more for what is left of their product. The oracle runs on the GPU."""
    k, n = 96, 3000
    dt = L.DTYPES[dtype]
    X, W, _, labels, _ = cuda(*inputs(m, k, n, dt, m, bias=False))
    grad = torch.full((m,), 1.0 / m, device=dev())
    note("rounding of a mean %s %d" % (dtype, m))
    _, lse = xt.linear_cross_entropy(X, W, labels)
    dX, dW, _ = xt.linear_cross_entropy_backward(grad, X, W, labels, lse)
    torch.cuda.synchronize()
    x, w, on = X.double(), W.double(), labels >= 0
    d = torch.softmax(x @ w.T, 1)
    d[on, labels[on]] -= 1.0
    d *= on[:, None]
    rounded = (d * 2.0 ** 13).to(dt).double() * 2.0 ** -13
    for got, ref, near, what in ((dX, d @ w, rounded @ w, "dX"), (dW, d.T @ x, rounded.T @ x, "dW")):
        ref, near = ref / m, near / m
        off = float((got.double() - ref).norm() / ref.norm())
        inside = float((near - ref).norm() / ref.norm())
        # the output's own, scaled so that no fp16 output is below the smallest numbers
        own = float(((ref * 2.0 ** 12).to(dt).double() * 2.0 ** -12 - ref).norm() / ref.norm())
        least = L.smallest(dt) / 2 * ref.numel() ** 0.5 / float(ref.norm())
        assert off < 1.1 * (inside ** 2 + own ** 2 + least ** 2) ** 0.5, (what, off, inside, own, least)


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("k", [32, 35])
def test_several_pieces_of_the_vocabulary(dtype, k):
    """So many rows that d is formed in pieces; k = 35: copies of the weights' pieces too. The oracle runs on the GPU."""
    m, n = (10000, 13001) if dtype == "f32" else (20000, 13001)
    dt = L.DTYPES[dtype]
    X, W, b, labels, grad = cuda(*inputs(m, k, n, dt, 7))
    note("pieces %s %d" % (dtype, k))
    loss, lse = xt.linear_cross_entropy(X, W, labels, b)
    got = xt.linear_cross_entropy_backward(grad, X, W, labels, lse, b)
    only = [xt.linear_cross_entropy_backward(grad, X, W, labels, lse, b, need_dX=i == 0, need_dW=i == 1, need_db=i == 2)[i] for i in range(3)]
    torch.cuda.synchronize()
    target = O.of_labels(labels)
    for t, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, *target), ("loss", "lse")):
        L.check(t, ref, bound, what)
    ref = O.backward(grad, X, W, b, *target, lse=lse)
    check_all(got, ref, dtype)
    check_all(only, ref, dtype + " alone")


@pytest.mark.parametrize("size", [(1118, 912, 12800), (924, 4072, 144), (600, 2000, 1000), (1500, 700, 9000)], ids=lambda s: "%dx%dx%d" % s)
def test_tiles_that_no_round_is_full_of(size):
    """fp32 products whose last round of tiles would be split: all tiles are, with the logits in memory, or none. The
    oracle runs on the GPU."""
    m, k, n = size
    X, W, b, _, grad = cuda(*inputs(m, k, n, torch.float32, 19))
    classes, teacher = cuda(*lists(m, n, 13, 20))
    note("last rounds %s" % (size,))
    loss, lse, weights = xt.linear_distillation(X, W, classes, teacher, b)
    got = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, b)
    torch.cuda.synchronize()
    P, eP = O.targets(classes, teacher, n, 1.0)
    for t, (ref, bound) in zip((loss, lse), O.forward(X, W, b, classes, P, eP)):
        L.check(t, ref, bound, "loss")
    check_all(got, O.backward(grad, X, W, b, classes, weights.double(), torch.zeros_like(P), lse=lse), "%s" % (size,))


def test_parts_of_dx_joined_on_the_way():
    """More pieces of the vocabulary than there is room for their parts of dX."""
    m, k, n = 65536, 1024, 13_000
    X, W, b, labels, grad = cuda(*inputs(m, k, n, torch.bfloat16, 15))
    note("parts of dX")
    # four pieces, each a part of 268 MB at least, and d of one
    assert xt.xtvxy_linear_cross_entropy_backward_bf16_workspace_size(m, k, n) < 4 * m * k * 4
    _, lse = xt.linear_cross_entropy(X, W, labels, b)
    dX, _, _ = xt.linear_cross_entropy_backward(grad, X, W, labels, lse, b)
    torch.cuda.synchronize()
    rows = torch.arange(0, m, 131, device=dev())
    ref = O.backward(grad[rows], X[rows], W, b, *O.of_labels(labels[rows]), lse=lse[rows])
    L.check(dX[rows], *ref["dX"], what="dX")


def test_many_rows_in_the_forward_pass():
    """Statistics in pieces of the vocabulary: rows x classes beyond what is kept at once."""
    m, k, n = 300_000, 8, 10_000
    X, W, b, labels, _ = cuda(*inputs(m, k, n, torch.bfloat16, 9))
    note("statistics in pieces")
    assert xt.xtvxy_linear_cross_entropy_bf16_workspace_size(m, k, n) < m * (n // 32) * 8
    loss, lse = xt.linear_cross_entropy(X, W, labels, b)
    torch.cuda.synchronize()
    rows = torch.arange(0, m, 3001, device=dev())
    for t, (ref, bound) in zip((loss, lse), O.forward(X[rows], W, b, *O.of_labels(labels[rows]))):
        L.check(t[rows], ref, bound, "rows")


def test_gradient_against_differences():
    X, W, b, labels, grad = inputs(6, 10, 17, torch.float32, 11)
    classes, teacher = lists(6, 17, 4, 12)
    gX, gW, gb, gl, gg, gc, gt = cuda(X, W, b, labels, grad, classes, teacher)
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    hard = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
    _, lse, weights = xt.linear_distillation(gX, gW, gc, gt, gb, 2.0)
    soft = xt.linear_distillation_backward(gg, gX, gW, gc, weights, lse, gb, 2.0)
    torch.cuda.synchronize()
    P = O.targets(classes, teacher, 17, 2.0)[0]

    def total(x, w, c, which):
        z = x @ w.T + c
        if which == "hard":
            on = labels >= 0
            l = torch.where(on, torch.logsumexp(z, 1) - z.gather(1, labels.clamp_min(0)[:, None])[:, 0], 0.0)
        else:
            logp = torch.log_softmax(z / 2.0, 1).gather(1, classes.clamp_min(0))
            l = (P * (torch.log(P.clamp_min(1e-30)) - logp)).sum(1)
        return (l * grad.double()).sum()

    args, eps = [X.double(), W.double(), b.double()], 1e-5
    for which, got in (("hard", hard), ("soft", soft)):
        for i in range(3):
            for at in (0, 5, args[i].numel() - 1):
                def moved(by):
                    a = [t.clone() for t in args]
                    a[i].view(-1)[at] += by
                    return total(*a, which)
                slope = (moved(eps) - moved(-eps)) / (2 * eps)  # off by eps^2 f''' / 6 ~ 1e-10
                assert abs(got[i].view(-1)[at].item() - slope.item()) <= 1e-6, (which, i, at)


def test_rows_that_do_not_count_and_bad_ones():
    m, k, n = 70, 40, 200
    X, W, b, _, grad = inputs(m, k, n, torch.float32, 21)
    labels = whole(n, (m,), 3)
    labels[5], labels[6], labels[7] = -1, -100, -2 ** 40
    X[6] = float("nan")  # what padding holds does not reach the loss
    gX, gW, gb, gl, gg = cuda(X, W, b, labels, grad)
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    torch.cuda.synchronize()
    assert (loss[5:8] == 0).all() and torch.isfinite(loss).all() and torch.isnan(lse[6])
    dX, _, db = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb, need_dW=False)
    torch.cuda.synchronize()
    assert not dX[5:8].any() and torch.isfinite(dX).all() and torch.isfinite(db).all()
    for bad in (n, 2 ** 40):
        gl[9] = bad
        gX[6] = 0.0
        loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
        dX, _, _ = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
        torch.cuda.synchronize()
        assert torch.isnan(loss[9]) and torch.isfinite(lse).all() and loss.isnan().sum() == 1
        assert torch.isnan(dX[9]).all() and torch.isfinite(dX[:9]).all() and torch.isfinite(dX[10:]).all()
    # a grad of zero takes a row out, too
    gl[9], gg[11] = 0, 0.0
    dX, _, _ = xt.linear_cross_entropy_backward(gg, gX, gW, gl, xt.linear_cross_entropy(gX, gW, gl, gb)[1], gb)
    torch.cuda.synchronize()
    assert not dX[11].any() and dX[12].any()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_classes_taken_out(dtype):
    """A bias of -infinity: whole tiles of the vocabulary, single classes, all classes; the lowest value of the type."""
    m, k, n = 40, 64, 1500
    dt = L.DTYPES[dtype]
    X, W, b, labels, grad = inputs(m, k, n, dt, 31)
    labels = labels.clamp_max(99)
    b[100:900] = float("-inf")
    b[1200::7] = torch.finfo(torch.float32).min
    gX, gW, gb, gl, gg = cuda(X, W, b, labels, grad)
    note("classes taken out %s" % dtype)
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    dX, dW, db = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
    torch.cuda.synchronize()
    keep = torch.isfinite(b) & (b > -1e30)
    few, where = b[keep], torch.cumsum(keep, 0) - 1
    there = torch.where(labels >= 0, where[labels.clamp_min(0)], labels)
    target = O.of_labels(there)
    for t, (ref, bound) in zip((loss, lse), O.forward(X, W[keep], few, *target)):
        L.check(t, ref, bound * 1.1, "loss")
    ref = O.backward(grad, X, W[keep], few, *target, lse=lse.cpu())
    check_all((dX, dW[keep.to(dev())], db[keep.to(dev())]), ref, dtype)
    assert not dW[~keep.to(dev())].any() and not db[~keep.to(dev())].any()
    gl[:] = 150  # taken out itself
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    gb[:] = float("-inf")
    none, empty = xt.linear_cross_entropy(gX, gW, gl, gb)
    torch.cuda.synchronize()
    assert (loss == float("inf")).all() and torch.isnan(none).all() and (empty == float("-inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_logits_and_small_gradients(dtype):
    """Logits up to about 1000, and gradients that fp16 does not hold unscaled."""
    m, k, n = 100, 128, 3000
    dt = L.DTYPES[dtype]
    X, W, b, labels, _ = inputs(m, k, n, dt, 41)
    X = (X.float() * 40).to(dt)
    grad = torch.full((m,), 1e-4)
    gX, gW, gb, gl, gg = cuda(X, W, b, labels, grad)
    note("large logits %s" % dtype)
    loss, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    got = xt.linear_cross_entropy_backward(gg, gX, gW, gl, lse, gb)
    torch.cuda.synchronize()
    target = O.of_labels(labels)
    for t, (ref, bound) in zip((loss, lse), O.forward(X, W, b, *target)):
        L.check(t, ref, bound, "loss")
    check_all(got, O.backward(grad, X, W, b, *target, lse=lse.cpu()), dtype)
    X = (X.float() / 40).to(dt)
    gX = X.to(dev())
    _, lse = xt.linear_cross_entropy(gX, gW, gl, gb)
    for size in (1e-9, 1e-5, 300.0):
        grad = torch.full((m,), size)
        dX, dW, db = xt.linear_cross_entropy_backward(grad.to(dev()), gX, gW, gl, lse, gb)
        torch.cuda.synchronize()
        check_all((dX, dW, db), O.backward(grad, X, W, b, *target, lse=lse.cpu()), "%s %g" % (dtype, size))


def test_teacher_rows_without_a_distribution():
    m, k, n, s = 6, 16, 50, 4
    X, W, b, _, grad = inputs(m, k, n, torch.float32, 51)
    classes = whole(n, (m, s), 52)
    for i in range(m):
        classes[i] = torch.arange(s) + i
    teacher = rand((m, s), 53)
    classes[0] = -1
    teacher[1] = float("-inf")
    classes[2, 1] = n
    teacher[3, 2] = float("nan")
    teacher[4, :3] = float("-inf")
    gX, gW, gb, gc, gt, gg = cuda(X, W, b, classes, teacher, grad)
    loss, lse, w = xt.linear_distillation(gX, gW, gc, gt, gb)
    dX, _, _ = xt.linear_distillation_backward(gg, gX, gW, gc, w, lse, gb)
    torch.cuda.synchronize()
    assert (loss[:2] == 0).all() and not w[:2].any() and not dX[:2].any()
    assert torch.isnan(loss[2:4]).all() and torch.isnan(w[2:4]).all() and torch.isnan(dX[2:4]).all()
    assert torch.equal(w[4].cpu(), torch.tensor([0.0, 0.0, 0.0, 1.0]))
    # one class with all the probability is a label
    hard, _ = xt.linear_cross_entropy(gX[4:], gW, gc[4:, 3].contiguous(), gb)
    torch.cuda.synchronize()
    assert hard[0] == loss[4] and torch.isfinite(loss[4:]).all()
    none, l0, w0 = xt.linear_distillation(gX, gW, gc[:, :0].contiguous(), gt[:, :0], gb)
    d0, _, _ = xt.linear_distillation_backward(gg, gX, gW, gc[:, :0].contiguous(), w0, l0, gb)
    torch.cuda.synchronize()
    assert not none.any() and torch.equal(l0, lse) and w0.shape == (m, 0) and not d0.any()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_zero_sizes(dtype):
    d, dt = dev(), L.DTYPES[dtype]
    e = lambda *s: torch.empty(*s, dtype=dt, device=d)  # noqa: E731
    labels = torch.tensor([0, -1, 2], device=d)
    b = torch.arange(3.0, device=d)
    note("zero sizes %s" % dtype)
    loss, lse = xt.linear_cross_entropy(e(3, 0), e(3, 0), labels, b)
    dX, dW, db = xt.linear_cross_entropy_backward(torch.ones(3, device=d), e(3, 0), e(3, 0), labels, lse, b)
    torch.cuda.synchronize()
    want = torch.logsumexp(b.double(), 0)
    assert torch.allclose(lse.double(), want.expand(3), atol=1e-6) and dX.shape == (3, 0) and dW.shape == (3, 0)
    assert torch.allclose(loss.double(), torch.stack([want, want * 0, want - 2]), atol=1e-6)
    p = torch.softmax(b, 0) * 2
    assert torch.allclose(db, p - torch.tensor([1.0, 0.0, 1.0], device=d), atol=1e-6)
    loss, lse = xt.linear_cross_entropy(e(3, 5), e(0, 5), labels)
    dX, dW, db = xt.linear_cross_entropy_backward(torch.ones(3, device=d), e(3, 5), e(0, 5), labels, lse)
    torch.cuda.synchronize()
    assert torch.isnan(loss[[0, 2]]).all() and loss[1] == 0 and (lse == float("-inf")).all()
    assert not dX.any() and dW.shape == (0, 5) and db.shape == (0,)
    none = torch.empty(0, dtype=torch.int64, device=d)
    loss, lse = xt.linear_cross_entropy(e(0, 5), e(4, 5), none)
    dX, dW, db = xt.linear_cross_entropy_backward(lse, e(0, 5), e(4, 5), none, lse)
    torch.cuda.synchronize()
    assert loss.shape == (0,) and dX.shape == (0, 5) and not dW.any() and not db.any()


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(70, 96, 130), (300, 100, 1000)], ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("offset", [1, 8])
def test_views_of_wider_buffers(size, dtype, offset):
    m, k, n = size
    dt = L.DTYPES[dtype]
    X, W, b, labels, grad = inputs(m, k, n, dt, 61)

    def view(t, fill=float("nan")):
        buf = torch.full((t.shape[0], t.shape[1] + offset + 8), fill, dtype=t.dtype, device=dev())
        v = buf[:, offset:offset + t.shape[1]]
        v.copy_(t)
        return buf, v

    (_, vX), (_, vW), (xb, dX), (wb, dW) = view(X), view(W), view(X, 7.0), view(W, 7.0)
    gb, gl, gg = cuda(b, labels, grad)
    note("loss views %s %s offset %d" % (size, dtype, offset))
    loss, lse = xt.linear_cross_entropy(vX, vW, gl, gb)
    got = xt.linear_cross_entropy_backward(gg, vX, vW, gl, lse, gb, dX=dX, dW=dW)
    torch.cuda.synchronize()
    target = O.of_labels(labels)
    for t, (ref, bound) in zip((loss, lse), O.forward(X, W, b, *target)):
        L.check(t, ref, bound, "loss")
    check_all(got, O.backward(grad, X, W, b, *target, lse=lse.cpu()), dtype)
    for buf, w in ((xb, k), (wb, k)):
        assert (buf[:, :offset] == 7.0).all() and (buf[:, offset + w:] == 7.0).all()


def test_weights_beyond_two_to_the_31_elements():
    m, k, n = 5, 4096, 530_000
    W = torch.zeros(n, k, dtype=torch.float16, device=dev())
    X, tail = rand((m, k), 71, torch.float16), rand((2, k), 72, torch.float16, 0.05)
    W[-2:] = tail.to(dev())
    labels = torch.tensor([n - 1, 0, n - 2, n - 1, 5])
    gX, gl = cuda(X, labels)
    note("weights of 2^31 elements")
    loss, lse = xt.linear_cross_entropy(gX, W, gl)
    dX, dW, _ = xt.linear_cross_entropy_backward(torch.ones(m, device=dev()), gX, W, gl, lse)
    torch.cuda.synchronize()
    z = X.double() @ tail.double().T
    want = torch.logsumexp(torch.cat([z, torch.full((m, 1), float(n - 2), dtype=torch.float64).log()], 1), 1)
    at = torch.tensor([1, -1, 0, 1, -1])
    zl = torch.where(at >= 0, z.gather(1, at.clamp_min(0)[:, None])[:, 0], 0.0)
    # 1e-4: sums of 4096 products of magnitude below 0.2, (4096 + 4) 2^-23 of their 160
    assert (lse.cpu().double() - want).abs().max() <= 1e-4 and (loss.cpu().double() - (want - zl)).abs().max() <= 2e-4
    d = torch.exp(z - want[:, None])
    d[0, 1] -= 1
    d[3, 1] -= 1
    d[2, 0] -= 1
    assert (dW[-2:].cpu().double() - d.T @ X.double()).abs().max() <= 2e-2 and dW[0].any() and not dW[6:-2:1000].abs().gt(1e-4).any()
    assert (dX.cpu().double() - d @ tail.double()).abs().max() <= 1e-3


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_streams_and_graph(dtype):
    m, k, n, s = 200, 128, 3000, 8
    dt = L.DTYPES[dtype]
    X, W, b, labels, grad = cuda(*inputs(m, k, n, dt, 81))
    classes, teacher = cuda(*lists(m, n, s, 82))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        kw = {} if stream is None else {"stream": stream}
        loss, lse = xt.linear_cross_entropy(X, W, labels, b, **kw)
        soft, lse2, w = xt.linear_distillation(X, W, classes, teacher, b, 2.0, **kw)
        return (loss, lse, soft, lse2, w) + xt.linear_cross_entropy_backward(grad, X, W, labels, lse, b, **kw) \
            + xt.linear_distillation_backward(grad, X, W, classes, w, lse2, b, 2.0, **kw)

    note("losses on a stream %s" % dtype)
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        X.copy_(rand((m, k), 90 + seed))
        labels.copy_(whole(n, (m,), 93 + seed))
        note("losses replay %d" % seed)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))


def test_calls_at_once():
    """Four host threads, each with its sizes and its stream, against the same calls one after the other."""
    import threading

    sizes = [(300, 64, 1000, "bf16"), (7, 512, 5000, "f16"), (93, 1415, 105, "f32"), (1000, 96, 3000, "bf16")]
    given = [cuda(*inputs(m, k, n, L.DTYPES[t], m)) for m, k, n, t in sizes]

    def calls(X, W, b, labels, grad):
        out = []
        for _ in range(5):
            loss, lse = xt.linear_cross_entropy(X, W, labels, b)
            out.append((loss, lse) + xt.linear_cross_entropy_backward(grad, X, W, labels, lse, b))
        return out

    note("calls at once")
    expected = [calls(*g) for g in given]
    torch.cuda.synchronize()
    results, errors = [None] * len(given), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                results[i] = calls(*given[i])
        except Exception as e:  # shown by the test
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(given))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for got, ref in zip(results, expected):
        assert all(torch.equal(a, b) for x, y in zip(got, ref) for a, b in zip(x, y))


def fresh(m, k, n, dt, seed, s, edges):
    """Inputs made on the GPU; lists that hold classes on both sides of each edge, empty and equal places and rows without any."""
    g = torch.Generator(dev()).manual_seed(seed)
    X, W = (torch.randn(r, k, generator=g, device=dev()).to(dt) for r in (m, n))
    W *= 2.0 * k ** -0.5
    b, grad = torch.randn(n, generator=g, device=dev()), torch.rand(m, generator=g, device=dev()) + 0.1
    classes = torch.randint(0, n, (m, s), generator=g, device=dev())
    near = torch.tensor([0, n - 1] + [e + by for e in edges for by in (-1, 0)], device=dev())
    at = torch.rand(m, s, generator=g, device=dev()) < 0.5
    classes = torch.where(at, near[torch.randint(0, len(near), (m, s), generator=g, device=dev())], classes)
    classes[torch.rand(m, s, generator=g, device=dev()) < 0.2] = -1
    classes[3] = -1
    return X, W, b, grad / m, classes, torch.randn(m, s, generator=g, device=dev()) * 2.0


def inside(got, ref, bound, what):
    over = ((got.double() - ref).abs() / bound).max().item()
    assert over <= 1.0, "%s: error %.3g times its bound" % (what, over)


# 300 x 66001: copies of W, whose pieces hold 4096 classes of 12001 in both directions. 20000 x 35: pieces of the gradient's d, of
# a multiple of 256 classes (10000 rows of fp32). Lists of 8 are searched, of 48 and 100 put in order; the weights of 100 are
# formed in a launch of their own, of the others with the last piece.
@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("s", [8, 48, 100])
@pytest.mark.parametrize("many", [False, True])
def test_lists_over_several_pieces(many, s, dtype):
    """Distillation over a vocabulary that is processed in pieces. The oracle runs on the GPU."""
    dt = L.DTYPES[dtype]
    es = torch.finfo(dt).bits // 8
    m, k, n = (40000 // es, 35, 13001) if many else (300, 132000 // es + 1, 12001)
    X, W, b, grad, classes, teacher = fresh(m, k, n, dt, s, s, range(256, n, 256) if many else (4096, 8192))
    T = 1.5
    size = getattr(xt, "xtvxy_linear_distillation_backward_%s_workspace_size" % dtype)
    assert size(m, k, n, s, 0) < (m * n * es if many else n * k * es)  # neither all of d nor a copy of all of W
    note("lists over pieces %d %d %s" % (many, s, dtype))
    loss, lse, weights = xt.linear_distillation(X, W, classes, teacher, b, T)
    got = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, b, T)
    again = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, b, T)
    torch.cuda.synchronize()
    P, eP = O.targets(classes, teacher, n, T)
    inside(weights, P, eP + 1e-40, "weights")
    assert loss[3] == 0 and not weights[3].any()
    for t, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, classes, P, eP, T), ("loss", "lse")):
        inside(t, ref, bound, what)
    ref = O.backward(grad, X, W, b, classes, weights.double(), torch.zeros_like(P), T, lse=lse)
    for t, u, name in zip(got, again, ("dX", "dW", "db")):
        inside(t, *ref[name], what=name)
        assert torch.equal(t, u)


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("s", [5, 40, 70])
def test_few_rows_over_several_pieces(s, dtype):
    """So many classes that few rows' logits, which pass through the workspace, are taken in two pieces. The oracle runs on
    the GPU."""
    m, k, n, edge = (32, 8, 1_500_001, 750_080) if dtype == "f32" else (16, 8, 3_000_001, 1_500_160)
    T = 2.0
    X, W, b, grad, classes, teacher = fresh(m, k, n, L.DTYPES[dtype], s, s, [edge])
    assert getattr(xt, "xtvxy_linear_distillation_%s_workspace_size" % dtype)(m, k, n, s) < m * n * 4
    note("few rows over pieces %d %s" % (s, dtype))
    loss, lse, weights = xt.linear_distillation(X, W, classes, teacher, b, T)
    dX, dW, db = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, b, T)
    torch.cuda.synchronize()
    P, eP = O.targets(classes, teacher, n, T)
    inside(weights, P, eP + 1e-40, "weights")
    for t, (ref, bound), what in zip((loss, lse), O.forward(X, W, b, classes, P, eP, T), ("loss", "lse")):
        inside(t, ref, bound, what)
    ref = O.backward(grad, X, W, b, classes, weights.double(), torch.zeros_like(P), T, lse=lse)
    for t, name in zip((dX, dW, db), ("dX", "dW", "db")):
        inside(t, *ref[name], what=name)


@pytest.mark.parametrize("offset", [0, 400, -3000])
@pytest.mark.parametrize("size", [(64, 5120), (200, 20480), (130, 5000)], ids=lambda s: "%dx%d" % s)
def test_far_logits_keep_their_distances(size, offset):
    """fp32 logits that are whole numbers, exact: an exponential is off by its distance's roundings, however far from zero
    all of them are. Features that are one for one row and weigh nothing make dW hold d itself."""
    m, n = size
    g = torch.Generator(dev()).manual_seed(n)
    X = torch.cat([torch.ones(m, 1, device=dev()), torch.randint(-2, 3, (m, 15), generator=g, device=dev()).float(), torch.eye(m, device=dev())], 1)
    W = torch.zeros(n, 16 + m, device=dev())
    W[:, 0], W[:, 1:16] = offset, torch.randint(-1, 2, (n, 15), generator=g, device=dev()).float()
    labels = torch.randint(0, n, (m,), generator=g, device=dev())
    grad = torch.rand(m, generator=g, device=dev()) + 0.5
    note("far logits %s %d" % (size, offset))
    loss, lse = xt.linear_cross_entropy(X, W, labels)
    _, dW, _ = xt.linear_cross_entropy_backward(grad, X, W, labels, lse)
    torch.cuda.synchronize()
    t = X.double() @ W.double().T
    ref, e, p = O._lse(t, torch.zeros_like(t))
    inside(lse, ref[:, 0], e[:, 0], "lse")
    inside(loss, ref[:, 0] - t.gather(1, labels[:, None])[:, 0], e[:, 0] + 2 * O.U * ref[:, 0].abs(), "loss")
    far = t - lse.double()[:, None]  # rounded once, then as every exponential
    p, on = torch.exp(far), torch.zeros_like(t).scatter_(1, labels[:, None], 1.0)
    d = grad.double()[:, None] * (p - on)
    bound = grad.double()[:, None] * (p * (O._exp_error(far) + O.U * far.abs() + 4 * O.U) + 2 * O.U * on) + 2 * O.U * d.abs()
    inside(dW[:, 16:].T, d, bound + 1e-40, "d")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("temperature", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("offset", [0, 400, -3008])
@pytest.mark.parametrize("size", [(64, 8192), (300, 20480), (130, 5000)], ids=lambda s: "%dx%d" % s)
def test_far_logits_of_16_bits(size, offset, temperature, dtype):
    """The same of 16-bit features: their losses and db are fp32, and only dX and dW see d rounded."""
    m, n = size
    dt = L.DTYPES[dtype]
    g = torch.Generator(dev()).manual_seed(n)
    X = torch.cat([torch.ones(m, 1, device=dev()), torch.randint(-2, 3, (m, 15), generator=g, device=dev()).float()], 1).to(dt)
    W = torch.zeros(n, 16, device=dev())
    W[:, 0], W[:, 1:] = offset, torch.randint(-1, 2, (n, 15), generator=g, device=dev()).float()
    W = W.to(dt)
    classes = torch.randint(0, n, (m, 3), generator=g, device=dev())
    teacher = torch.randn(m, 3, generator=g, device=dev())
    grad = torch.rand(m, generator=g, device=dev()) + 0.5
    note("far logits of 16 bits %s %d %g %s" % (size, offset, temperature, dtype))
    loss, lse, weights = xt.linear_distillation(X, W, classes, teacher, None, temperature)
    _, _, db = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, None, temperature)
    torch.cuda.synchronize()
    inv = float(torch.tensor(1.0) / torch.tensor(temperature))  # in fp32, as the call has it
    t = (X.double() @ W.double().T) * inv
    et = t.abs() * (0.0 if temperature in (1.0, 2.0) else O.U)  # each t is rounded once, or exact
    ref, e, _ = O._lse(t, et)
    inside(lse, ref[:, 0], e[:, 0], "lse")
    P = weights.double()
    ts = t.gather(1, classes)
    inner = torch.where(P > 0, torch.log(P.clamp_min(1e-300)) - ts + ref, 0.0)
    size_of = torch.where(P > 0, torch.log(P.clamp_min(1e-300)).abs() + ts.abs() + ref.abs(), 0.0)
    inside(loss, (P * inner).sum(1), e[:, 0] + 6 * O.U * (P * size_of).sum(1) + 1e-30, "loss")
    far = t - lse.double()[:, None]
    p = torch.exp(far)
    T = torch.zeros_like(t).scatter_add_(1, classes, P)
    d = grad.double()[:, None] * inv * (p - T)
    bound = grad.double()[:, None] * inv * (p * (O._exp_error(far) + et + O.U * far.abs() + 6 * O.U) + 4 * O.U * T) + 2 * O.U * d.abs()
    inside(db, d.sum(0), bound.sum(0) + (m + 4) * 2 * O.U * d.abs().sum(0) + 1e-40, "db")


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_logits_beyond_what_their_exponents_resolve(dtype):
    """Logits of 2^36 and more (2^30 in fp16): finite, a few equal largest ones, everything else infinitely far below."""
    m, k, n = 70, 8, 4096
    dt = L.DTYPES[dtype]
    big = 2.0 ** 15 if dtype == "f16" else 2.0 ** 18
    X, W = torch.zeros(m, k, device=dev()), torch.zeros(n, k, device=dev())
    X[:, 0], W[:, 0] = big, big
    X[:, 0] *= torch.tensor([1.0, 1.25, 1.5, 1.375], device=dev())[torch.arange(m, device=dev()) % 4]
    W[[5, 1000, 4000], 0] = big * 1.75
    labels = torch.tensor([5, 1000, 4000], device=dev())[torch.arange(m, device=dev()) % 3]
    X, W = X.to(dt), W.to(dt)
    grad = torch.ones(m, device=dev())
    note("huge logits %s" % dtype)
    loss, lse = xt.linear_cross_entropy(X, W, labels)
    dX, dW, db = xt.linear_cross_entropy_backward(grad, X, W, labels, lse)
    torch.cuda.synchronize()
    top = X[:, 0].double() * big * 1.75  # log 3 is below half of its step
    assert torch.equal(lse.double(), top) and not loss.any()
    d = torch.zeros(m, n, dtype=torch.float64, device=dev())  # exp(0) of each, less the label
    d[:, [5, 1000, 4000]] = 1.0
    d[torch.arange(m), labels] = 0.0
    assert torch.equal(db.double(), d.sum(0))
    # sums of a few multiples of 2^12 and 2^16, exact; beyond fp16's largest they round to infinity
    assert torch.equal(dX, (d @ W.double()).to(dt)) and torch.equal(dW, (d.T @ X.double()).to(dt))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_smallest_temperature(dtype):
    """1 / temperature is finite, its product with log2 e is not: logits of zero stay zero."""
    m, k, n, T = 70, 16, 8192, 3e-39
    dt = L.DTYPES[dtype]
    X, W = torch.zeros(m, k, dtype=dt, device=dev()), rand((n, k), 1, dt).to(dev())
    classes, teacher = torch.full((m, 2), 7, device=dev()), torch.zeros(m, 2, device=dev())
    classes[:, 1] = n - 1
    grad = torch.full((m,), 2.0 ** -130, device=dev())
    note("smallest temperature %s" % dtype)
    loss, lse, weights = xt.linear_distillation(X, W, classes, teacher, None, T)
    _, _, db = xt.linear_distillation_backward(grad, X, W, classes, weights, lse, None, T)
    torch.cuda.synchronize()
    assert (weights == 0.5).all()
    assert ((lse.double() - math.log(n)).abs() <= 4 * O.U * math.log(n)).all()
    assert ((loss.double() - math.log(n / 2)).abs() <= 8 * O.U * math.log(n)).all()
    d = torch.full((n,), 1.0 / n, dtype=torch.float64, device=dev())
    d[[7, n - 1]] -= 0.5
    want = m * 2.0 ** -130 * float(torch.tensor(1.0) / torch.tensor(T)) * d
    # lse off by 4 steps of log n, the factor and sums of m equal terms
    assert ((db.double() - want).abs() <= want.abs() * (4 * math.log(n) + m + 8) * O.U).all()
