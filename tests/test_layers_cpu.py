"""Refusals of the fully connected layer and its gradient without a GPU: every call returns before a
kernel is launched."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from dense_linear_algebra_alpha_amd import _abi, build

A = 1 << 40  # never dereferenced
MB = 1 << 20
SUFFIXES = ("f32", "bf16", "f16")


@pytest.fixture(scope="module")
def lib():
    if build.sources_newer_than_library():
        build.build()
    return _abi.load()


def linear_status(s, m=8, k=8, n=8, X=A, ldx=8, W=A + MB, ldw=8, bias=None, residual=None, ldr=8, act=0, out=A + 2 * MB,
                  ldo=8, pre=None, ldp=8, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_" + s)(m, k, n, X, ldx, W, ldw, bias, residual, ldr, act, out, ldo, pre,
                                                     ldp, ws, wsb, None)


@pytest.mark.parametrize("s", SUFFIXES)
def test_linear_argument_errors(lib, s):
    bad, null, alias = _abi.XTVXY_ERROR_INVALID_VALUE, _abi.XTVXY_ERROR_NULL_POINTER, _abi.XTVXY_ERROR_ALIASING
    for kw in ({"m": -1}, {"k": -1}, {"n": -3}, {"ldx": 7}, {"ldw": 7}, {"ldo": 7}, {"act": -1}, {"act": 5},
               {"residual": A + 3 * MB, "ldr": 7}, {"pre": A + 3 * MB, "ldp": 7}, {"m": 1 << 60}, {"k": 0, "ldx": 0}):
        assert linear_status(s, **kw) == bad, kw
    for kw in ({"X": None}, {"W": None}, {"out": None}):
        assert linear_status(s, **kw) == null, kw
    for kw in ({"out": A + 16}, {"out": A + MB + 16}, {"bias": A + 2 * MB + 4}, {"pre": A + 2 * MB + 8}, {"pre": A + 8},
               {"residual": A + 2 * MB + 8}, {"residual": A + 2 * MB, "ldr": 9}, {"pre": A + 3 * MB, "residual": A + 3 * MB},
               {"pre": A + 3 * MB, "bias": A + 3 * MB}):
        assert linear_status(s, **kw) == alias, kw
    assert linear_status(s, m=0) == 0 and linear_status(s, n=0) == 0  # nothing to compute
    assert linear_status(s, m=1 << 28, n=1 << 28, ldo=1 << 28, k=1, ldx=1, ldw=1, X=A, W=A << 2, out=A << 4) \
        == _abi.XTVXY_ERROR_UNSUPPORTED


@pytest.mark.parametrize("s", SUFFIXES)
def test_linear_workspace(lib, s):
    size = getattr(xt, "xtvxy_linear_%s_workspace_size" % s)
    k = 65537  # rows that need copies
    need = size(400, k, 100)
    assert need > 0
    # a missing, short or misaligned workspace is refused
    for ws, b in ((None, 0), (A + 8 * MB, need - 1), (A + 8 * MB + 4, need)):
        assert linear_status(s, m=400, k=k, n=100, X=A << 1, ldx=k, W=A << 2, ldw=k, out=A << 3, ldo=100, ws=ws,
                             wsb=b) == _abi.XTVXY_ERROR_WORKSPACE
    assert size(0, 5, 5) == 0 and size(5, 5, 0) == 0
    for args in ((-1, 5, 5), (1 << 40, 5, 1 << 40)):
        with pytest.raises(xt.XtvxyError):
            size(*args)


def backward_status(s, m=8, k=8, n=8, G=A, ldg=8, X=A + MB, ldx=8, W=A + 2 * MB, ldw=8, pre=A + 3 * MB, ldp=8, act=1,
                    dX=A + 4 * MB, lddx=8, dW=A + 5 * MB, lddw=8, db=A + 6 * MB, ws=None, wsb=0):
    return getattr(_abi.load(), "xtvxy_linear_backward_" + s)(m, k, n, G, ldg, X, ldx, W, ldw, pre, ldp, act, dX, lddx,
                                                              dW, lddw, db, ws, wsb, None)


@pytest.mark.parametrize("s", SUFFIXES)
def test_backward_argument_errors(lib, s):
    bad, null, alias = _abi.XTVXY_ERROR_INVALID_VALUE, _abi.XTVXY_ERROR_NULL_POINTER, _abi.XTVXY_ERROR_ALIASING
    for kw in ({"m": -1}, {"k": -1}, {"n": -3}, {"ldg": 7}, {"ldx": 7}, {"ldw": 7}, {"ldp": 7}, {"lddx": 7}, {"lddw": 7},
               {"act": 9}, {"m": 1 << 60}):
        assert backward_status(s, **kw) == bad, kw
    for kw in ({"G": None}, {"X": None}, {"W": None}, {"pre": None}):
        assert backward_status(s, **kw) == null, kw
    for kw in ({"dX": A + 8}, {"dX": A + MB + 8}, {"dW": A + 2 * MB}, {"db": A + 3 * MB}, {"dW": A + 4 * MB + 16},
               {"db": A + 5 * MB}, {"db": A + 4 * MB + 4}):
        assert backward_status(s, **kw) == alias, kw
    assert backward_status(s) == _abi.XTVXY_ERROR_WORKSPACE
    assert backward_status(s, m=0, n=0) == 0
    size = getattr(xt, "xtvxy_linear_backward_%s_workspace_size" % s)
    assert size(1000, 640, 960, xt.ACTIVATIONS["gelu"]) > size(1000, 640, 960, xt.ACTIVATIONS["none"])
    with pytest.raises(xt.XtvxyError):
        size(8, 8, 8, 77)


def test_helpers_refuse_host_tensors(lib):
    X, W = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="GPU"):
        xt.linear(X, W)
    with pytest.raises(ValueError, match="GPU"):
        xt.linear_backward(torch.zeros(4, 6), X, W)


@pytest.mark.gpu
def test_helpers_refuse_what_the_kernels_cannot_take():
    d = "cuda"
    X, W = torch.zeros(4, 8, device=d), torch.zeros(6, 8, device=d)
    for args, kw in (((X.double(), W.double()), {}), ((X, W.half()), {}), ((X, W.t()), {}), ((X, W[:, :7]), {}),
                     ((X[0], W), {}), ((X.t(), W), {}), ((X, W), {"act": "tanh"}), ((X, W, torch.zeros(5, device=d)), {}),
                     ((X, W, torch.zeros(6, device=d).half()), {}), ((X, W, torch.zeros(6)), {}),
                     ((X, W, None, torch.zeros(4, 5, device=d)), {}), ((X, W, None, torch.zeros(1, 6, device=d).expand(4, 6)), {}),
                     ((X, W), {"out": torch.zeros(4, 6, device=d).half()})):
        with pytest.raises(ValueError):
            xt.linear(*args, **kw)
    G = torch.zeros(4, 6, device=d)
    with pytest.raises(ValueError, match="pre"):
        xt.linear_backward(G, X, W, None, "gelu")
    with pytest.raises(ValueError):
        xt.linear_backward(G[:, :5], X, W)


def test_adamw_argument_errors(lib):
    import ctypes
    ptrs = lambda *a: (ctypes.c_void_p * len(a))(*a)  # noqa: E731
    h = ctypes.c_void_p()

    def create(n=1, numel=(64,), p=(A,), bits=32, m=(A + MB,), v=(A + 2 * MB,), me=None, ve=None, ct=0, c=None):
        return lib.xtvxy_adamw_create(n, numel and (ctypes.c_int64 * len(numel))(*numel), p and ptrs(*p), bits, m and ptrs(*m),
                                      v and ptrs(*v), me and ptrs(*me), ve and ptrs(*ve), ct, c and ptrs(*c), ctypes.byref(h))

    bad, null, alias = _abi.XTVXY_ERROR_INVALID_VALUE, _abi.XTVXY_ERROR_NULL_POINTER, _abi.XTVXY_ERROR_ALIASING
    for kw in ({"n": -1}, {"bits": 16}, {"numel": (-1,)}, {"p": (A + 2,)}, {"m": (A + MB + 1,)}, {"ct": 1}, {"ct": 9}):
        assert create(**kw) == bad, kw
    for kw in ({"numel": None}, {"p": None}, {"m": None}, {"v": (None,)}, {"p": (None,)}, {"bits": 8}, {"ct": 2},
               {"ct": 2, "c": (None,)}):
        assert create(**kw) == null, kw
    for kw in ({"m": (A + 128,)}, {"v": (A + MB + 4,)}, {"ct": 2, "c": (A + 252,)},
               {"bits": 8, "me": (A + 3 * MB,), "ve": (A + 3 * MB,)}):
        assert create(**kw) == alias, kw
    assert h.value is None
    assert lib.xtvxy_adamw_create(0, None, None, 32, None, None, None, None, 0, None, None) == null
    assert create(n=0, numel=None, p=None, m=None, v=None) in (_abi.XTVXY_SUCCESS, _abi.XTVXY_ERROR_LAUNCH)
    assert lib.xtvxy_adamw_step(None, None, 1, 1, 0.1, 0.9, 0.9, 1e-8, 0.0, 0, None) == null
    assert lib.xtvxy_adamw_state_values(None, None, None, 1, None) == null


def test_adamw_oracle_formats():
    """The 8-bit formats' tables, ends included, and the oracle's rounding at its extremes."""
    import numpy as np

    import adamw_oracle as O
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.m_value(np.arange(256)), t, equal_nan=True)
    v = O.v_value(np.arange(256))
    assert v[0] == 0 and v[1] == 2.0 ** -18 and v[15] == 15 * 2.0 ** -18 and v[16] == 2.0 ** -14 and v[255] == 1.9375
    assert (np.diff(v) > 0).all()
    # every value is its own code
    for value, n, bits, least in ((O.m_value, 127, 3, -6), (O.v_value, 256, 4, -14)):
        code, frac = O.codes_and_fractions(value(np.arange(n)), bits, least)
        assert np.array_equal(code, np.arange(n)) and not frac.any()
