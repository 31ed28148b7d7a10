"""Losses over an output layer and their gradients, without the logits in memory: softmax cross entropy and
distillation from a teacher's top logits. The C names of include/xtvxy.h and the torch tensor helpers on them
(argument marshalling only, as in the package's other helpers)."""
from __future__ import annotations

import functools

from . import _abi
from .embeddings import _index_bits
from .layers import _MAX_PITCH, _check, _check_bias, _entry, _fast, _features, _new, _pitch, _scratch, _size, _stream_of, _torch
from .norm import _vector
from .optimiser import _type_code


# ---------------------------------------------------------------------------
# C names
# ---------------------------------------------------------------------------

def xtvxy_linear_cross_entropy_f32_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_f32_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_bf16_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_bf16_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_f16_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_f16_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_f32(m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse, workspace,
                                   workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_f32", m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse,
                     workspace, workspace_bytes, stream)


def xtvxy_linear_cross_entropy_bf16(m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse, workspace,
                                    workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_bf16", m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse,
                     workspace, workspace_bytes, stream)


def xtvxy_linear_cross_entropy_f16(m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse, workspace,
                                   workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_f16", m, k, n, X, ldx, W, ldw, bias, labels, index_bits, loss, lse,
                     workspace, workspace_bytes, stream)


def xtvxy_linear_cross_entropy_backward_f32_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_backward_f32_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_backward_bf16_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_backward_bf16_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_backward_f16_workspace_size(m, k, n, aligned16=1) -> int:
    return _size("xtvxy_linear_cross_entropy_backward_f16_workspace_size", m, k, n, int(aligned16))


def xtvxy_linear_cross_entropy_backward_f32(m, k, n, grad, X, ldx, W, ldw, bias, labels, index_bits, lse, dX, lddx,
                                            dW, lddw, db, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_backward_f32", m, k, n, grad, X, ldx, W, ldw, bias, labels,
                     index_bits, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes, stream)


def xtvxy_linear_cross_entropy_backward_bf16(m, k, n, grad, X, ldx, W, ldw, bias, labels, index_bits, lse, dX, lddx,
                                             dW, lddw, db, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_backward_bf16", m, k, n, grad, X, ldx, W, ldw, bias, labels,
                     index_bits, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes, stream)


def xtvxy_linear_cross_entropy_backward_f16(m, k, n, grad, X, ldx, W, ldw, bias, labels, index_bits, lse, dX, lddx,
                                            dW, lddw, db, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_cross_entropy_backward_f16", m, k, n, grad, X, ldx, W, ldw, bias, labels,
                     index_bits, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes, stream)


def xtvxy_linear_distillation_f32_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_f32_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_bf16_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_bf16_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_f16_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_f16_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_f32(m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, teacher, ldt,
                                  teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_distillation_f32", m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits,
                     teacher, ldt, teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream)


def xtvxy_linear_distillation_bf16(m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, teacher, ldt,
                                   teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_distillation_bf16", m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits,
                     teacher, ldt, teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream)


def xtvxy_linear_distillation_f16(m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, teacher, ldt,
                                  teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream):
    return _abi.call("xtvxy_linear_distillation_f16", m, k, n, X, ldx, W, ldw, bias, s, classes, ldc, index_bits,
                     teacher, ldt, teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream)


def xtvxy_linear_distillation_backward_f32_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_backward_f32_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_backward_bf16_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_backward_bf16_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_backward_f16_workspace_size(m, k, n, s, aligned16=1) -> int:
    return _size("xtvxy_linear_distillation_backward_f16_workspace_size", m, k, n, s, int(aligned16))


def xtvxy_linear_distillation_backward_f32(m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, weights,
                                           temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                                           stream):
    return _abi.call("xtvxy_linear_distillation_backward_f32", m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc,
                     index_bits, weights, temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                     stream)


def xtvxy_linear_distillation_backward_bf16(m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, weights,
                                            temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                                            stream):
    return _abi.call("xtvxy_linear_distillation_backward_bf16", m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc,
                     index_bits, weights, temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                     stream)


def xtvxy_linear_distillation_backward_f16(m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc, index_bits, weights,
                                           temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                                           stream):
    return _abi.call("xtvxy_linear_distillation_backward_f16", m, k, n, grad, X, ldx, W, ldw, bias, s, classes, ldc,
                     index_bits, weights, temperature, lse, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                     stream)


# ---------------------------------------------------------------------------
# torch tensor helpers
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _bytes(name, *shape) -> int:
    return _size(name + "_workspace_size", *shape)


def _aligned(X, ldx, W, ldw) -> int:
    es = X.element_size()
    ld = max(ldx, ldw) * es
    return 0 if (X.data_ptr() | W.data_ptr() | ldx * es | ldw * es) & 15 or ld > _MAX_PITCH else 1


def _per_row(name, t, like, m, stream, dev):
    """A float32 vector of the rows that the call writes: the caller's, or a new one."""
    if t is None:
        return _new(like, m, stream, _torch().float32)
    _check_bias(name, t, m, dev)
    return t


def _outputs(X, W, need_dX, need_dW, need_db, dX, dW, db, m, k, n, dtype, dev, stream):
    """The gradients' tensors, made here where the caller gives none, and their row strides."""
    lddx, lddw = k or 1, k or 1
    if not need_dX:
        dX = None
    elif dX is None:
        dX = _new(X, (m, k), stream)
    else:
        lddx = _pitch("dX", dX, m, k, dtype, dev)
    if not need_dW:
        dW = None
    elif dW is None:
        dW = _new(X, (n, k), stream)
    else:
        lddw = _pitch("dW", dW, n, k, dtype, dev)
    if not need_db:
        db = None
    elif db is None:
        db = _new(X, n, stream, _torch().float32)
    else:
        _check_bias("db", db, n, dev)
    return dX, lddx, dW, lddw, db


def _ptr(t):
    return None if t is None else t.data_ptr()


def linear_cross_entropy(X, W, labels, bias=None, *, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse): loss[i] = lse[i] - z[i, labels[i]] with the logits z = X W^T + bias, which are not kept, and
    lse[i] = log sum_j exp(z[i, j]) (xtvxy_linear_cross_entropy_f32, _bf16, _f16).

    X (m x k) and W (n x k, one row per class) are as in linear, bias is float32 (n), labels is a contiguous int32 or
    int64 vector (m). Rows with a negative label do not count: their loss is zero. A label beyond the classes gives
    NaN (a check would wait for the GPU). loss and lse are float32 (m); linear_cross_entropy_backward takes lse.
    Autograd records nothing, as in linear."""
    if stream is None:  # the usual call in compiled code, as in linear
        got = _fast("cross_entropy", "xtvxy_linear_cross_entropy", X, X, W, labels, bias, loss, lse, workspace)
        if got is not None:
            return got
    dev, _, suffix, m, k, n, ldx, ldw = _features(X, W)
    bp = _vector("bias", bias, n, dev)
    bits = _index_bits("labels", labels, (m,), dev)
    loss, lse = _per_row("loss", loss, X, m, stream, dev), _per_row("lse", lse, X, m, stream, dev)
    name = "xtvxy_linear_cross_entropy_" + suffix
    ws, ws_ptr, ws_bytes = _scratch(_bytes(name, m, k, n, _aligned(X, ldx, W, ldw)), workspace, X, stream)
    _check(_entry(name)(m, k, n, X.data_ptr(), ldx, W.data_ptr(), ldw, bp, labels.data_ptr(), bits, loss.data_ptr(),
                        lse.data_ptr(), ws_ptr, ws_bytes, _stream_of(stream, dev)), name)
    return loss, lse


def linear_cross_entropy_backward(grad, X, W, labels, lse, bias=None, *, need_dX=True, need_dW=True, need_db=True, dX=None,
                                  dW=None, db=None, workspace=None, stream=None):
    """The gradient of linear_cross_entropy: (dX, dW, db) for grad[i] = d total / d loss[i] (float32, m) from the
    forward call's lse. With d[i, j] = grad[i] (softmax(z)[i, j] - [j == labels[i]]): dX = d W, dW = d^T X, and db the
    column sums of d (float32). A mean over the rows that count has grad = 1 / their number. The products take d in the
    features' type: 16-bit dX and dW are off by up to 1.41 times their own rounding.

    Outputs that are not needed are not computed and come back as None."""
    if stream is None:
        got = _fast("cross_entropy_backward", "xtvxy_linear_cross_entropy_backward", X, grad, X, W, labels, lse, bias, need_dX,
                    need_dW, need_db, dX, dW, db, workspace)
        if got is not None:
            return got
    dev, dtype, suffix, m, k, n, ldx, ldw = _features(X, W)
    bp = _vector("bias", bias, n, dev)
    bits = _index_bits("labels", labels, (m,), dev)
    _check_bias("grad", grad, m, dev)
    _check_bias("lse", lse, m, dev)
    dX, lddx, dW, lddw, db = _outputs(X, W, need_dX, need_dW, need_db, dX, dW, db, m, k, n, dtype, dev, stream)
    name = "xtvxy_linear_cross_entropy_backward_" + suffix
    ws, ws_ptr, ws_bytes = _scratch(_bytes(name, m, k, n, _aligned(X, ldx, W, ldw)), workspace, X, stream)
    _check(_entry(name)(m, k, n, grad.data_ptr(), X.data_ptr(), ldx, W.data_ptr(), ldw, bp, labels.data_ptr(), bits,
                        lse.data_ptr(), _ptr(dX), lddx, _ptr(dW), lddw, _ptr(db), ws_ptr, ws_bytes,
                        _stream_of(stream, dev)), name)
    return dX, dW, db


def linear_distillation(X, W, classes, teacher, bias=None, temperature=1.0, *, loss=None, lse=None, weights=None,
                        workspace=None, stream=None):
    """(loss, lse, weights): the Kullback-Leibler distance of softmax(t), t = (X W^T + bias) / temperature, from the
    teacher's P = softmax(teacher / temperature) over the classes that a row lists (xtvxy_linear_distillation_f32, _bf16,
    _f16): loss[i] = sum_c P[i, c] (log P[i, c] - t[i, c] + lse[i]), lse[i] = log sum_j exp(t[i, j]). The logits are not
    kept.

    classes (m x s) is a contiguous int32 or int64 tensor, teacher (m x s) a float32, bfloat16 or float16 one with unit
    column stride; weights (m x s, float32) gets P. Negative classes are empty places; a class that a row lists
    twice gets both probabilities in its first place; rows without classes do not count. X, W and bias are as in
    linear_cross_entropy. linear_distillation_backward takes lse and weights."""
    if stream is None:
        got = _fast("distillation", "xtvxy_linear_distillation", X, X, W, classes, teacher, bias, temperature, loss, lse,
                    weights, workspace)
        if got is not None:
            return got
    dev, _, suffix, m, k, n, ldx, ldw = _features(X, W)
    bp = _vector("bias", bias, n, dev)
    if classes.dim() != 2:
        raise ValueError("classes must be 2-D")
    s = classes.shape[1]
    bits = _index_bits("classes", classes, (m, s), dev)
    ldt = _pitch("teacher", teacher, m, s, teacher.dtype, dev)
    code = _type_code(teacher.dtype)
    loss, lse = _per_row("loss", loss, X, m, stream, dev), _per_row("lse", lse, X, m, stream, dev)
    if weights is None:
        weights = _new(X, (m, s), stream, _torch().float32)
    _check_weights(weights, m, s, dev)
    name = "xtvxy_linear_distillation_" + suffix
    ws, ws_ptr, ws_bytes = _scratch(_bytes(name, m, k, n, s, _aligned(X, ldx, W, ldw)), workspace, X, stream)
    _check(_entry(name)(m, k, n, X.data_ptr(), ldx, W.data_ptr(), ldw, bp, s, classes.data_ptr(), s or 1, bits,
                        teacher.data_ptr(), ldt, code, float(temperature), loss.data_ptr(), lse.data_ptr(),
                        weights.data_ptr(), ws_ptr, ws_bytes, _stream_of(stream, dev)), name)
    return loss, lse, weights


def _check_weights(t, m, s, dev):
    if t.dtype is not _torch().float32 or t.get_device() != dev or tuple(t.shape) != (m, s) or not t.is_contiguous():
        raise ValueError("weights must be a contiguous float32 tensor of %d x %d on GPU %d" % (m, s, dev))


def linear_distillation_backward(grad, X, W, classes, weights, lse, bias=None, temperature=1.0, *, need_dX=True,
                                 need_dW=True, need_db=True, dX=None, dW=None, db=None, workspace=None, stream=None):
    """The gradient of linear_distillation: (dX, dW, db) for grad[i] = d total / d loss[i] (float32, m) from the forward
    call's weights and lse, with d[i, j] = grad[i] / temperature (softmax(t)[i, j] - P[i, j]); otherwise as
    linear_cross_entropy_backward. The gradient of a hard loss on the same layer is added to it by the caller."""
    if stream is None:
        got = _fast("distillation_backward", "xtvxy_linear_distillation_backward", X, grad, X, W, classes, weights, lse, bias,
                    temperature, need_dX, need_dW, need_db, dX, dW, db, workspace)
        if got is not None:
            return got
    dev, dtype, suffix, m, k, n, ldx, ldw = _features(X, W)
    bp = _vector("bias", bias, n, dev)
    if classes.dim() != 2:
        raise ValueError("classes must be 2-D")
    s = classes.shape[1]
    bits = _index_bits("classes", classes, (m, s), dev)
    _check_weights(weights, m, s, dev)
    _check_bias("grad", grad, m, dev)
    _check_bias("lse", lse, m, dev)
    dX, lddx, dW, lddw, db = _outputs(X, W, need_dX, need_dW, need_db, dX, dW, db, m, k, n, dtype, dev, stream)
    name = "xtvxy_linear_distillation_backward_" + suffix
    ws, ws_ptr, ws_bytes = _scratch(_bytes(name, m, k, n, s, _aligned(X, ldx, W, ldw)), workspace, X, stream)
    _check(_entry(name)(m, k, n, grad.data_ptr(), X.data_ptr(), ldx, W.data_ptr(), ldw, bp, s, classes.data_ptr(), s or 1,
                        bits, weights.data_ptr(), float(temperature), lse.data_ptr(), _ptr(dX), lddx, _ptr(dW), lddw,
                        _ptr(db), ws_ptr, ws_bytes, _stream_of(stream, dev)), name)
    return dX, dW, db
