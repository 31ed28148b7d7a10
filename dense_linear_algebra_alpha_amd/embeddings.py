"""Embedding lookup and its gradient: the C names of include/xtvxy.h and the torch tensor helpers on them
(argument marshalling only, as in the package's other helpers)."""
from __future__ import annotations

import functools

from . import _abi
from .layers import _check, _entry, _fast, _new, _pitch, _scratch, _size, _stream_of, _suffix, _torch


# ---------------------------------------------------------------------------
# C names
# ---------------------------------------------------------------------------

def xtvxy_embedding_f32(count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream):
    return _abi.call("xtvxy_embedding_f32", count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream)


def xtvxy_embedding_bf16(count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream):
    return _abi.call("xtvxy_embedding_bf16", count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream)


def xtvxy_embedding_f16(count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream):
    return _abi.call("xtvxy_embedding_f16", count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream)


def xtvxy_embedding_backward_f32_workspace_size(count, k, rows) -> int:
    return _size("xtvxy_embedding_backward_f32_workspace_size", count, k, rows)


def xtvxy_embedding_backward_bf16_workspace_size(count, k, rows) -> int:
    return _size("xtvxy_embedding_backward_bf16_workspace_size", count, k, rows)


def xtvxy_embedding_backward_f16_workspace_size(count, k, rows) -> int:
    return _size("xtvxy_embedding_backward_f16_workspace_size", count, k, rows)


def xtvxy_embedding_backward_f32(count, k, rows, G, ldg, ids, index_bits, scale, accumulate, dtable, lddt, workspace,
                                 workspace_bytes, stream):
    return _abi.call("xtvxy_embedding_backward_f32", count, k, rows, G, ldg, ids, index_bits, scale, accumulate,
                     dtable, lddt, workspace, workspace_bytes, stream)


def xtvxy_embedding_backward_bf16(count, k, rows, G, ldg, ids, index_bits, scale, accumulate, dtable, lddt, workspace,
                                  workspace_bytes, stream):
    return _abi.call("xtvxy_embedding_backward_bf16", count, k, rows, G, ldg, ids, index_bits, scale, accumulate,
                     dtable, lddt, workspace, workspace_bytes, stream)


def xtvxy_embedding_backward_f16(count, k, rows, G, ldg, ids, index_bits, scale, accumulate, dtable, lddt, workspace,
                                 workspace_bytes, stream):
    return _abi.call("xtvxy_embedding_backward_f16", count, k, rows, G, ldg, ids, index_bits, scale, accumulate,
                     dtable, lddt, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# torch tensor helpers
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _backward_bytes(suffix, count, k, rows) -> int:
    return _size("xtvxy_embedding_backward_%s_workspace_size" % suffix, count, k, rows)


def _index_bits(name, t, shape, dev) -> int:
    """Bits of an index tensor's elements, checked: contiguous, of that shape."""
    torch = _torch()
    bits = 64 if t.dtype is torch.int64 else 32 if t.dtype is torch.int32 else 0
    if not bits or t.get_device() != dev or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 or int64 tensor of shape %s on GPU %d" % (name, tuple(shape), dev))
    return bits


def _on_current_gpu(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be on the GPU, not on %s" % (name, t.device))
    if dev != _torch()._C._cuda_getDevice():
        raise ValueError("%s must be on the current GPU, not on %s" % (name, t.device))
    return dev


def embedding(ids, table, scale=1.0, *, out=None, stream=None):
    """out[i] = scale table[ids[i]] (xtvxy_embedding_f32, _bf16, _f16).

    ids is a contiguous int32 or int64 vector, table (rows x k) and out (len(ids) x k) are 2-D tensors with unit
    column stride, of one type: float32, bfloat16 or float16. Negative ids are padding and give zeros; ids beyond
    the table give NaN (a check would wait for the GPU). Autograd records nothing; the gradient is
    embedding_backward's."""
    if stream is None:  # the usual call in compiled code, as in linear
        got = _fast("embedding", "xtvxy_embedding", table, ids, table, scale, out)
        if got is not None:
            return got
    dev = _on_current_gpu("table", table)
    dtype = table.dtype
    suffix = _suffix(dtype)
    if table.dim() != 2 or ids.dim() != 1:
        raise ValueError("table must be 2-D and ids 1-D")
    rows, k = table.shape
    count = ids.shape[0]
    ldt = _pitch("table", table, rows, k, dtype, dev)
    bits = _index_bits("ids", ids, (count,), dev)
    if out is None:
        out = _new(table, (count, k), stream)
        ldo = k or 1
    else:
        ldo = _pitch("out", out, count, k, dtype, dev)
    name = "xtvxy_embedding_" + suffix
    _check(_entry(name)(count, k, rows, ids.data_ptr(), bits, table.data_ptr(), ldt, float(scale), out.data_ptr(), ldo,
                        _stream_of(stream, dev)), name)
    return out


def embedding_backward(G, ids, rows, scale=1.0, *, dtable=None, accumulate=False, workspace=None, stream=None):
    """The gradient of embedding: dtable (rows x k) with dtable[r] = scale times the sum of the G[i] of which
    ids[i] == r, summed in float32 in the order of the tokens. G (len(ids) x k) has the table's type.

    With ``accumulate`` it is added to ``dtable``, of which only the rows that occur are touched (a table that is also
    an output layer's weight: dtable is that layer's dW); else every element is written. Negative ids and ids
    beyond the table take no part."""
    if stream is None:
        got = _fast("embedding_backward", "xtvxy_embedding_backward", G, G, ids, rows, scale, dtable, accumulate, workspace)
        if got is not None:
            return got
    dev = _on_current_gpu("G", G)
    dtype = G.dtype
    suffix = _suffix(dtype)
    if G.dim() != 2 or ids.dim() != 1:
        raise ValueError("G must be 2-D and ids 1-D")
    count, k = G.shape
    ldg = _pitch("G", G, count, k, dtype, dev)
    bits = _index_bits("ids", ids, (count,), dev)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs dtable")
        if rows < 0:
            raise ValueError("rows must not be negative")
        dtable = _new(G, (rows, k), stream)
        lddt = k or 1
    else:
        lddt = _pitch("dtable", dtable, rows, k, dtype, dev)
    ws, ws_ptr, ws_bytes = _scratch(_backward_bytes(suffix, count, k, rows), workspace, G, stream)
    name = "xtvxy_embedding_backward_" + suffix
    _check(_entry(name)(count, k, rows, G.data_ptr(), ldg, ids.data_ptr(), bits, float(scale), int(bool(accumulate)),
                        dtable.data_ptr(), lddt, ws_ptr, ws_bytes, _stream_of(stream, dev)), name)
    return dtable
