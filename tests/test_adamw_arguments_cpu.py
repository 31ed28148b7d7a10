"""Refusals of the AdamW object beyond the plain ones, without a GPU."""
import ctypes

import pytest

from dense_linear_algebra_alpha_amd import _abi, build

A, MB = 1 << 40, 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if build.sources_newer_than_library():
        build.build()
    return _abi.load()


@pytest.mark.parametrize("copy_type", [_abi.XTVXY_TYPE_BF16, _abi.XTVXY_TYPE_F16])
def test_copies_are_aligned_to_their_type(lib, copy_type):
    """As parameters, 32-bit states and gradients are."""
    def create(copy):
        h = ctypes.c_void_p()
        p, m, v, c = [(ctypes.c_void_p * 1)(a) for a in (A, A + MB, A + 2 * MB, copy)]
        return lib.xtvxy_adamw_create(1, (ctypes.c_int64 * 1)(64), p, 32, m, v, None, None, copy_type, c, ctypes.byref(h))

    assert create(A + 3 * MB + 1) == _abi.XTVXY_ERROR_INVALID_VALUE
    assert create(A + 64 * 4 - 1) == _abi.XTVXY_ERROR_INVALID_VALUE
