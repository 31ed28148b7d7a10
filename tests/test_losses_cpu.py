"""Refusals of the losses over an output layer without a GPU: every call returns before a kernel is launched."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from dense_linear_algebra_alpha_amd import _abi, build

A = 1 << 40  # never dereferenced
MB = 1 << 20
SUFFIXES = ("f32", "bf16", "f16")
BAD, NULL, ALIAS = _abi.XTVXY_ERROR_INVALID_VALUE, _abi.XTVXY_ERROR_NULL_POINTER, _abi.XTVXY_ERROR_ALIASING
WORKSPACE, UNSUPPORTED = _abi.XTVXY_ERROR_WORKSPACE, _abi.XTVXY_ERROR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    if build.sources_newer_than_library():
        build.build()
    return _abi.load()


def entropy(s, m=8, k=8, n=8, X=A, ldx=8, W=A + MB, ldw=8, bias=A + 2 * MB, labels=A + 3 * MB, bits=64, loss=A + 4 * MB,
            lse=A + 5 * MB, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_cross_entropy_" + s)(m, k, n, X, ldx, W, ldw, bias, labels, bits, loss, lse, ws,
                                                                   wsb, None)


def entropy_backward(s, m=8, k=8, n=8, grad=A + 9 * MB, X=A, ldx=8, W=A + MB, ldw=8, bias=A + 2 * MB, labels=A + 3 * MB, bits=64,
                     lse=A + 5 * MB, dX=A + 6 * MB, lddx=8, dW=A + 7 * MB, lddw=8, db=A + 8 * MB, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_cross_entropy_backward_" + s)(m, k, n, grad, X, ldx, W, ldw, bias, labels, bits, lse,
                                                                            dX, lddx, dW, lddw, db, ws, wsb, None)


def distil(s, m=8, k=8, n=8, X=A, ldx=8, W=A + MB, ldw=8, bias=A + 2 * MB, per_row=4, classes=A + 3 * MB, ldc=4, bits=64,
           teacher=A + 10 * MB, ldt=4, tt=1, T=2.0, loss=A + 4 * MB, lse=A + 5 * MB, weights=A + 11 * MB, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_distillation_" + s)(m, k, n, X, ldx, W, ldw, bias, per_row, classes, ldc, bits,
                                                                  teacher, ldt, tt, T, loss, lse, weights, ws, wsb, None)


def distil_backward(s, m=8, k=8, n=8, grad=A + 9 * MB, X=A, ldx=8, W=A + MB, ldw=8, bias=A + 2 * MB, per_row=4, classes=A + 3 * MB,
                    ldc=4, bits=64, weights=A + 11 * MB, T=2.0, lse=A + 5 * MB, dX=A + 6 * MB, lddx=8, dW=A + 7 * MB, lddw=8,
                    db=A + 8 * MB, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_distillation_backward_" + s)(m, k, n, grad, X, ldx, W, ldw, bias, per_row, classes,
                                                                           ldc, bits, weights, T, lse, dX, lddx, dW, lddw, db, ws,
                                                                           wsb, None)


SHAPE = ({"m": -1}, {"k": -1}, {"n": -1}, {"ldx": 7}, {"ldw": 7}, {"bits": 16}, {"m": 1 << 60}, {"n": 1 << 60})


@pytest.mark.parametrize("s", SUFFIXES)
def test_cross_entropy_errors(s):
    for kw in SHAPE:
        assert entropy(s, **kw) == BAD, kw
    for kw in ({"X": None}, {"W": None}, {"labels": None}, {"loss": None}, {"lse": None}):
        assert entropy(s, **kw) == NULL, kw
    for kw in ({"loss": A + 8}, {"lse": A + MB + 4}, {"loss": A + 2 * MB}, {"lse": A + 3 * MB + 60}, {"lse": A + 4 * MB + 28}):
        assert entropy(s, **kw) == ALIAS, kw
    need = getattr(xt, "xtvxy_linear_cross_entropy_%s_workspace_size" % s)(8, 8, 8)
    for ws, b in ((None, 0), (A << 1, need - 1), ((A << 1) + 4, need)):
        assert entropy(s, ws=ws, wsb=b) == WORKSPACE
    assert entropy(s, m=0, X=None, loss=None) == 0
    for kw in ({"k": 1 << 22, "ldx": 1 << 22, "ldw": 1 << 22, "W": A << 1, "bias": None, "labels": A << 2, "loss": A << 3, "lse": A << 4},
               {"n": 1 << 31, "W": A << 1, "bias": None, "labels": A << 2, "loss": A << 3, "lse": A << 4}, {"m": 1 << 25, "n": 100}):
        assert entropy(s, **kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("s", SUFFIXES)
def test_cross_entropy_backward_errors(s):
    for kw in SHAPE + ({"lddx": 7}, {"lddw": 7}):
        assert entropy_backward(s, **kw) == BAD, kw
    for kw in ({"grad": None}, {"X": None}, {"W": None}, {"labels": None}, {"lse": None}):
        assert entropy_backward(s, **kw) == NULL, kw
    for kw in ({"dX": A}, {"dW": A + MB + 16}, {"db": A + 2 * MB}, {"db": A + 5 * MB + 28}, {"dX": A + 9 * MB}, {"dW": A + 6 * MB + 16},
               {"db": A + 7 * MB + 4}):
        assert entropy_backward(s, **kw) == ALIAS, kw
    need = getattr(xt, "xtvxy_linear_cross_entropy_backward_%s_workspace_size" % s)(8, 8, 8)
    for ws, b in ((None, 0), (A << 1, need - 1), ((A << 1) + 4, need)):
        assert entropy_backward(s, ws=ws, wsb=b) == WORKSPACE
    assert entropy_backward(s, dX=None, dW=None, db=None) == 0


@pytest.mark.parametrize("s", SUFFIXES)
def test_distillation_errors(s):
    for kw in SHAPE + ({"per_row": -1}, {"ldc": 3}, {"ldt": 3}, {"tt": 0}, {"tt": 9}, {"T": 0.0}, {"T": -1.0}, {"T": float("nan")},
                       {"T": float("inf")}, {"T": 1e-44}):
        assert distil(s, **kw) == BAD, kw
    for kw in ({"X": None}, {"classes": None}, {"teacher": None}, {"weights": None}, {"loss": None}):
        assert distil(s, **kw) == NULL, kw
    for kw in ({"weights": A + 10 * MB}, {"weights": A + 4 * MB}, {"loss": A + 10 * MB}, {"weights": A + 3 * MB + 16}):
        assert distil(s, **kw) == ALIAS, kw
    assert distil(s) == WORKSPACE and distil(s, per_row=1025, ldc=1025, ldt=1025, X=A << 1, W=A << 2, teacher=A << 3) == UNSUPPORTED
    assert distil(s, m=0) == 0


@pytest.mark.parametrize("s", SUFFIXES)
def test_distillation_backward_errors(s):
    for kw in SHAPE + ({"per_row": -1}, {"ldc": 3}, {"T": 0.0}, {"lddx": 7}):
        assert distil_backward(s, **kw) == BAD, kw
    for kw in ({"grad": None}, {"classes": None}, {"weights": None}, {"lse": None}):
        assert distil_backward(s, **kw) == NULL, kw
    for kw in ({"dX": A + 11 * MB}, {"db": A + 3 * MB}, {"dW": A + 6 * MB + 4}):
        assert distil_backward(s, **kw) == ALIAS, kw
    assert distil_backward(s) == WORKSPACE


@pytest.mark.parametrize("s", SUFFIXES)
def test_workspaces(s):
    """They grow with what they hold and stay bounded in the vocabulary."""
    forward = getattr(xt, "xtvxy_linear_cross_entropy_%s_workspace_size" % s)
    backward = getattr(xt, "xtvxy_linear_cross_entropy_backward_%s_workspace_size" % s)
    es = 4 if s == "f32" else 2
    assert forward(0, 8, 8) == 0 and backward(8, 8, 0) == 0 and forward(1000, 64, 5000) > 0
    assert forward(1000, 63, 5000, 0) >= forward(1000, 64, 5000)  # copies
    # without the logits: of 8192 rows and a million classes less than an eighth of them
    for size in (forward, backward):
        assert size(8192, 512, 1_000_000) < 8192 * 1_000_000 * es // 8
    for args in ((-1, 8, 8), (8, 1 << 23, 8), (1 << 26, 8, 5000), (8, 8, 1 << 32)):
        for size in (forward, backward):
            with pytest.raises(xt.XtvxyError):
                size(*args)
    lists = getattr(xt, "xtvxy_linear_distillation_%s_workspace_size" % s)
    assert lists(1000, 64, 5000, 32) > lists(1000, 64, 5000, 1)
    with pytest.raises(xt.XtvxyError):
        lists(1000, 64, 5000, 1025)


def test_helpers_refuse_host_tensors():
    X, W, v = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(4)
    y, c, t = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    for call in (lambda: xt.linear_cross_entropy(X, W, y), lambda: xt.linear_cross_entropy_backward(v, X, W, y, v),
                 lambda: xt.linear_distillation(X, W, c, t), lambda: xt.linear_distillation_backward(v, X, W, c, t, v)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_helpers_refuse_what_the_kernels_cannot_take():
    d = "cuda"
    X, W, v, b = torch.zeros(4, 8, device=d), torch.zeros(6, 8, device=d), torch.zeros(4, device=d), torch.zeros(6, device=d)
    y, c, t = torch.zeros(4, dtype=torch.int64, device=d), torch.zeros(4, 2, dtype=torch.int64, device=d), torch.zeros(4, 2, device=d)
    E, B, D, F = xt.linear_cross_entropy, xt.linear_cross_entropy_backward, xt.linear_distillation, xt.linear_distillation_backward
    for call in (lambda: E(X.double(), W.double(), y), lambda: E(X, W.half(), y), lambda: E(X, W[:, :7], y), lambda: E(X, W, y[:3]),
                 lambda: E(X, W, y.float()), lambda: E(X, W, y.cpu()), lambda: E(X, W, y[None]), lambda: E(X, W, y, v),
                 lambda: E(X, W, y, b.half()), lambda: E(X, W, y, loss=b), lambda: E(X, W, torch.zeros(8, dtype=torch.int64, device=d)[::2]),
                 lambda: B(b, X, W, y, v), lambda: B(v, X, W, y, b), lambda: B(v[:1].expand(4), X, W, y, v), lambda: B(v, X, W, y, v, dX=W),
                 lambda: B(v, X, W, y, v, db=v), lambda: D(X, W, y, t), lambda: D(X, W, c, t[:, :1]), lambda: D(X, W, c, t.double()),
                 lambda: D(X, W, c.t(), t), lambda: D(X, W, c, t, weights=v), lambda: F(v, X, W, c, t[:, :1], v),
                 lambda: F(v, X, W, c, t.half(), v), lambda: F(v, X, W, y, t, v)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: E(X, W, y, loss=v, lse=v), lambda: D(X, W, c, t, temperature=0.0), lambda: B(v, X, W, y, v, dX=X),
                 lambda: E(X, W, y, workspace=torch.zeros(16, dtype=torch.uint8, device=d)[1:])):
        with pytest.raises(xt.XtvxyError):
            call()


@pytest.mark.gpu
def test_without_the_extension(monkeypatch):
    """The helpers' Python path gives what the compiled one gives."""
    from dense_linear_algebra_alpha_amd import layers
    d = "cuda"
    g = torch.Generator(device=d).manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device=d)  # noqa: E731
    X, W, b, grad, w = new(50, 40), new(90, 40), new(90), new(50), new(40)
    y = torch.randint(-1, 90, (50,), generator=g, device=d)
    c = torch.randint(-1, 90, (50, 5), generator=g, device=d).int()
    t = new(50, 5).half()

    def every():
        out, mean, rstd = xt.layer_norm(X, w, None, save_stats=True)
        loss, lse = xt.linear_cross_entropy(X, W, y, b)
        soft, lse2, P = xt.linear_distillation(X, W, c, t, b, 2.0)
        r = [out, mean, rstd, xt.layer_norm(X), loss, lse, soft, lse2, P, xt.embedding(y, W, 2.0), xt.embedding_backward(X, y, 90)]
        r += xt.layer_norm_backward(X, out, mean, rstd, w) + xt.layer_norm_backward(X, out, mean, rstd, need_dX=False, need_dbias=False)
        r += xt.linear_cross_entropy_backward(grad, X, W, y, lse, b) + xt.linear_cross_entropy_backward(grad, X, W, y, lse, need_dW=False)
        return r + list(xt.linear_distillation_backward(grad, X, W, c, P, lse2, b, 2.0, need_db=False))

    fast = every()
    assert layers._extension() is not None
    monkeypatch.setattr(layers, "_extension", lambda: None)
    slow = every()
    torch.cuda.synchronize()
    assert len(fast) == len(slow)
    for a, e in zip(fast, slow):
        assert (a is None and e is None) or torch.equal(a.nan_to_num(7.0), e.nan_to_num(7.0))
