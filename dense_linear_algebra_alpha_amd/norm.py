"""Layer norm and its gradient: the C names of include/xtvxy.h and the torch tensor helpers on them (argument
marshalling only, as in the package's other helpers)."""
from __future__ import annotations

import functools

from . import _abi
from .layers import _check, _check_bias, _entry, _fast, _new, _pitch, _scratch, _size, _stream_of, _suffix, _torch


# ---------------------------------------------------------------------------
# C names
# ---------------------------------------------------------------------------

def xtvxy_layer_norm_backward_workspace_size(m, n) -> int:
    return _size("xtvxy_layer_norm_backward_workspace_size", m, n)


def xtvxy_layer_norm_f32(m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream):
    return _abi.call("xtvxy_layer_norm_f32", m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream)


def xtvxy_layer_norm_bf16(m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream):
    return _abi.call("xtvxy_layer_norm_bf16", m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream)


def xtvxy_layer_norm_f16(m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream):
    return _abi.call("xtvxy_layer_norm_f16", m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream)


def xtvxy_layer_norm_backward_f32(m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight, dbias, workspace,
                                  workspace_bytes, stream):
    return _abi.call("xtvxy_layer_norm_backward_f32", m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight,
                     dbias, workspace, workspace_bytes, stream)


def xtvxy_layer_norm_backward_bf16(m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight, dbias, workspace,
                                   workspace_bytes, stream):
    return _abi.call("xtvxy_layer_norm_backward_bf16", m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight,
                     dbias, workspace, workspace_bytes, stream)


def xtvxy_layer_norm_backward_f16(m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight, dbias, workspace,
                                  workspace_bytes, stream):
    return _abi.call("xtvxy_layer_norm_backward_f16", m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight,
                     dbias, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# torch tensor helpers
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _backward_bytes(m, n) -> int:
    return xtvxy_layer_norm_backward_workspace_size(m, n)


def _rows(X):
    """(device index, type, suffix, m, n, row stride) of a matrix, checked."""
    dev = X.get_device()
    if dev < 0:
        raise ValueError("X must be on the GPU, not on %s" % X.device)
    if dev != _torch()._C._cuda_getDevice():
        raise ValueError("X must be on the current GPU, not on %s" % X.device)
    suffix = _suffix(X.dtype)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    m, n = X.shape
    return dev, X.dtype, suffix, m, n, _pitch("X", X, m, n, X.dtype, dev)


def _vector(name, t, n, dev):
    """Address of an optional float32 vector, checked."""
    if t is None:
        return None
    _check_bias(name, t, n, dev)
    return t.data_ptr()


def layer_norm(X, weight=None, bias=None, eps=1e-5, *, save_stats=False, out=None, mean=None, rstd=None, stream=None):
    """out = (X - mean) rstd weight + bias over each row (xtvxy_layer_norm_f32, _bf16, _f16).

    X and out (m x n) are 2-D tensors with unit column stride, of one type: float32, bfloat16 or
    float16; weight and bias (None: ones, zeros) are float32 (n). With ``save_stats`` the call also stores
    each row's mean and 1 / sqrt(variance + eps) in float32 (m), which layer_norm_backward takes, and
    returns (out, mean, rstd); so it does with ``mean`` and ``rstd`` given. Autograd records nothing, as in
    linear."""
    if stream is None:  # the usual call in compiled code, as in linear
        got = _fast("layer_norm", "xtvxy_layer_norm", X, X, weight, bias, eps, save_stats, out, mean, rstd)
        if got is not None:
            return got
    dev, dtype, suffix, m, n, ldx = _rows(X)
    wp, bp = _vector("weight", weight, n, dev), _vector("bias", bias, n, dev)
    if out is None:
        out = _new(X, (m, n), stream)
        ldo = n or 1
    else:
        ldo = _pitch("out", out, m, n, dtype, dev)
    stats = save_stats or mean is not None or rstd is not None
    if stats:
        f32 = _torch().float32
        mean = _new(X, m, stream, f32) if mean is None else mean
        rstd = _new(X, m, stream, f32) if rstd is None else rstd
    mp, rp = _vector("mean", mean, m, dev), _vector("rstd", rstd, m, dev)
    name = "xtvxy_layer_norm_" + suffix
    _check(_entry(name)(m, n, X.data_ptr(), ldx, wp, bp, float(eps), out.data_ptr(), ldo, mp, rp, _stream_of(stream, dev)),
           name)
    return (out, mean, rstd) if stats else out


def layer_norm_backward(G, X, mean, rstd, weight=None, *, need_dX=True, need_dweight=True, need_dbias=True, dX=None,
                        dweight=None, dbias=None, workspace=None, stream=None):
    """The gradient of layer_norm: (dX, dweight, dbias) for G = d loss / d out, from the forward call's mean and
    rstd. dX has the tensors' type, dweight and dbias are float32 (n). Outputs that are not needed are not
    computed and come back as None."""
    if stream is None:
        got = _fast("layer_norm_backward", "xtvxy_layer_norm_backward", X, G, X, mean, rstd, weight, need_dX, need_dweight,
                    need_dbias, dX, dweight, dbias, workspace)
        if got is not None:
            return got
    dev, dtype, suffix, m, n, ldx = _rows(X)
    ldg = _pitch("G", G, m, n, dtype, dev)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            raise ValueError("%s is required" % name)
    mp, rp, wp = _vector("mean", mean, m, dev), _vector("rstd", rstd, m, dev), _vector("weight", weight, n, dev)
    f32 = _torch().float32
    lddx = n or 1
    if not need_dX:
        dX = None
    elif dX is None:
        dX = _new(X, (m, n), stream)
    else:
        lddx = _pitch("dX", dX, m, n, dtype, dev)
    if not need_dweight:
        dweight = None
    elif dweight is None:
        dweight = _new(X, n, stream, f32)
    if not need_dbias:
        dbias = None
    elif dbias is None:
        dbias = _new(X, n, stream, f32)
    dwp, dbp = _vector("dweight", dweight, n, dev), _vector("dbias", dbias, n, dev)
    need = _backward_bytes(m, n) if need_dweight or need_dbias else 0
    ws, ws_ptr, ws_bytes = _scratch(need, workspace, X, stream)
    name = "xtvxy_layer_norm_backward_" + suffix
    _check(_entry(name)(m, n, G.data_ptr(), ldg, X.data_ptr(), ldx, mp, rp, wp, None if dX is None else dX.data_ptr(),
                        lddx, dwp, dbp, ws_ptr, ws_bytes, _stream_of(stream, dev)), name)
    return dX, dweight, dbias
