"""The AdamW step over many tensors with 32-bit or 8-bit states: the C names of include/xtvxy.h and the
optimiser object on torch tensors (argument marshalling only)."""
from __future__ import annotations

import ctypes
import functools

from . import _abi
from .layers import _extension, _stream_of, _torch
from ._abi import XTVXY_TYPE_BF16, XTVXY_TYPE_F16, XTVXY_TYPE_F32, XTVXY_TYPE_NONE

ADAMW_BLOCK = 128  # elements that share an exponent in 8-bit states


# ---------------------------------------------------------------------------
# C names
# ---------------------------------------------------------------------------

def xtvxy_adamw_create(tensors, numel, params, state_bits, m, v, m_exp, v_exp, copy_type, copies) -> int:
    h = ctypes.c_void_p()
    _abi.call("xtvxy_adamw_create", tensors, numel, params, state_bits, m, v, m_exp, v_exp, copy_type, copies,
              ctypes.byref(h))
    return h.value or 0


def xtvxy_adamw_destroy(optimiser):
    return _abi.call("xtvxy_adamw_destroy", optimiser)


def xtvxy_adamw_step(optimiser, grads, grad_type, step, lr, beta1, beta2, eps, weight_decay, seed, stream):
    return _abi.call("xtvxy_adamw_step", optimiser, grads, grad_type, step, lr, beta1, beta2, eps, weight_decay, seed,
                     stream)


def xtvxy_adamw_state_values(optimiser, m_out, v_out, type, stream):
    return _abi.call("xtvxy_adamw_state_values", optimiser, m_out, v_out, type, stream)


# ---------------------------------------------------------------------------
# the optimiser object
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _type_code(dtype) -> int:
    import torch
    code = {torch.float32: XTVXY_TYPE_F32, torch.bfloat16: XTVXY_TYPE_BF16, torch.float16: XTVXY_TYPE_F16}.get(dtype)
    if code is None:
        raise ValueError("element type must be float32, bfloat16 or float16, not %s" % dtype)
    return code


class AdamW:
    """AdamW (Adam with decoupled weight decay) over a list of contiguous float32 tensors on one GPU.

    ``copies`` are bfloat16 or float16 tensors of the parameters' sizes that every step rewrites with
    the rounded parameters (what a mixed-precision model computes with). ``state_bits`` 32 keeps both
    moments in float32; 8 keeps them as one byte per element with an exponent byte per 128 elements and
    rounds them at random from ``seed`` (formats in include/xtvxy.h). ``state`` resumes from (m, v), or
    (m, v, m_exp, v_exp) for 8 bits, lists of tensors that the object goes on using (uint8 for 8 bits);
    None starts from zeros. ``steps`` is the number of steps taken before. The object keeps its tensors:
    they must not be resized or moved, and their GPU has to be the current one in every call. To autograd a
    step is a write in place: a backward pass through what it saved of params or copies before raises. lr,
    betas, eps, weight_decay and seed are plain attributes."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, *, copies=None, state_bits=32,
                 state=None, steps=0, seed=0):
        import torch
        self.handle = 0
        params = list(params)
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if int(steps) < 0:
            raise ValueError("steps must not be negative")
        for i, p in enumerate(params):
            if p.dtype != torch.float32 or p.device.type != "cuda" or p.device != params[0].device or not p.is_contiguous():
                raise ValueError("params[%d] must be a contiguous float32 tensor on the GPU of the others" % i)
        self.device = params[0].device if params else torch.device("cuda", torch.cuda.current_device())
        self._check_device()
        numel = [p.numel() for p in params]
        blocks = [(n + ADAMW_BLOCK - 1) // ADAMW_BLOCK for n in numel]
        st = torch.float32 if state_bits == 32 else torch.uint8
        lengths = (numel, numel) if state_bits == 32 else (numel, numel, blocks, blocks)
        if state is None:
            state = tuple([torch.zeros(n, dtype=st, device=self.device) for n in ls] for ls in lengths)
            torch.cuda.current_stream().synchronize()  # the first step may run on any stream
        if len(state) != len(lengths):
            raise ValueError("state of %d-bit states has %d lists" % (state_bits, len(lengths)))
        state = tuple(list(s) for s in state)
        for name, s, ls in zip(("m", "v", "m_exp", "v_exp"), state, lengths):
            self._check_list("state " + name, s, ls, st)
        copy_type = XTVXY_TYPE_NONE
        if copies is not None:
            copies = list(copies)
            dtype = copies[0].dtype if copies else torch.bfloat16
            if dtype not in (torch.bfloat16, torch.float16):
                raise ValueError("copies must be bfloat16 or float16")
            copy_type = _type_code(dtype)
            self._check_list("copies", copies, numel, dtype)
        self.params, self.copies, self.state, self.state_bits, self.steps = params, copies, state, state_bits, int(steps)
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, tuple(betas), eps, weight_decay, seed
        n = len(params)
        self._numel = numel
        self._written = params + (copies or [])
        self._pointers = ctypes.c_void_p * n
        self._count = count = (ctypes.c_int64 * n)(*numel)
        self._numel_address = ctypes.addressof(count)
        exps = (self._array(state[2]), self._array(state[3])) if state_bits == 8 else (None, None)
        # the caller's tensors may still be in the making: steps are ordered after that by the streams that the
        # caller runs them on
        self.handle = xtvxy_adamw_create(n, count, self._array(params), state_bits, self._array(state[0]),
                                         self._array(state[1]), *exps, copy_type,
                                         None if copies is None else self._array(copies))

    def _check_device(self):
        current = _torch()._C._cuda_getDevice()
        if self.device.index != current:
            raise ValueError("the optimiser's tensors are on %s, which must be the current GPU, not cuda:%d"
                             % (self.device, current))

    def _check_list(self, name, tensors, lengths, dtype):
        if len(tensors) != len(lengths):
            raise ValueError("%s has %d tensors, the parameters are %d" % (name, len(tensors), len(lengths)))
        for i, (t, n) in enumerate(zip(tensors, lengths)):
            if t.dtype != dtype or t.device != self.device or t.numel() != n or not t.is_contiguous():
                raise ValueError("%s[%d] must be a contiguous %s tensor of %d elements on %s"
                                 % (name, i, dtype, n, self.device))

    def _array(self, tensors):
        return self._pointers(*[t.data_ptr() for t in tensors])

    def _like_params(self, name, tensors):
        """(pointers, type code) of a list of contiguous tensors of one type and the parameters' sizes."""
        tensors = list(tensors)
        n = len(self._numel)
        if len(tensors) != n:
            raise ValueError("%s has %d tensors, the parameters are %d" % (name, len(tensors), n))
        pointers = self._pointers()
        if not n:
            return pointers, XTVXY_TYPE_F32
        e = _extension()
        bad = (e.addresses(tensors, self._numel_address, ctypes.addressof(pointers), n, self.device.index) if e else
               self._addresses(tensors, pointers))
        if bad >= 0:
            raise ValueError("%s[%d] must be a contiguous tensor of %d elements on %s, of the list's one type"
                             % (name, bad, self._numel[bad], self.device))
        return pointers, _type_code(tensors[0].dtype)

    def _addresses(self, tensors, pointers) -> int:
        """What the extension's addresses() does."""
        strided = _torch().strided
        for i, (t, n) in enumerate(zip(tensors, self._numel)):
            if (getattr(t, "layout", None) is not strided or t.get_device() != self.device.index
                    or t.dtype is not tensors[0].dtype or t.numel() != n or not t.is_contiguous()):
                return i
            pointers[i] = t.data_ptr()
        return -1

    def step(self, grads, *, stream=None):
        """One step with the gradients of the parameters, in their order: contiguous tensors of one type
        (float32, bfloat16 or float16)."""
        self._check_device()
        pointers, code = self._like_params("grads", grads)
        xtvxy_adamw_step(self.handle, pointers, code, self.steps + 1, self.lr, self.betas[0], self.betas[1], self.eps,
                         self.weight_decay, self.seed & 0xffffffff, _stream_of(stream, self.device.index))
        self.steps += 1
        e = _extension()
        if e:
            e.written(self._written)
        else:
            _torch().autograd.graph.increment_version([t for t in self._written if not t.is_inference()])

    def state_values(self, m_out, v_out, *, stream=None):
        """Writes the values that the moments stand for into tensors of the parameters' sizes."""
        self._check_device()
        m_pointers, code = self._like_params("m_out", m_out)
        v_pointers, v_code = self._like_params("v_out", v_out)
        if v_code != code:
            raise ValueError("m_out and v_out must have one type")
        xtvxy_adamw_state_values(self.handle, m_pointers, v_pointers, code, _stream_of(stream, self.device.index))

    def close(self):
        if getattr(self, "handle", 0):
            xtvxy_adamw_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
