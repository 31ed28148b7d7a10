"""Sizes next to the limits of a launch and of 64-bit sizes, on the host: no call here reaches the GPU."""
import pytest

import dense_linear_algebra_alpha_amd as xt
from dense_linear_algebra_alpha_amd import _abi, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    if build.sources_newer_than_library():
        build.build()
    return _abi.load()


@pytest.mark.parametrize("s", ["f32", "bf16", "f16"])
def test_few_rows_of_many_outputs_go_to_a_kernel_that_can_launch(s):
    """The kernel for few rows takes 16 or 32 outputs a workgroup and never copies X and W; the others do,
    where rows are no whole 16-byte chunks. A launch holds less than 2^32 threads, 256 a workgroup."""
    size = getattr(xt, "xtvxy_linear_%s_workspace_size" % s)
    k = 9  # 2^33 multiplications and more
    for m, n in ((32, 1 << 29), (32, (1 << 29) + 1), (32, (1 << 30) - 64), (16, 1 << 29)):
        assert size(m, k, n) >= n * k * (4 if s == "f32" else 2), (m, n)
    for m, n in ((32, (1 << 29) - 64), (32, 1 << 27), (16, 1 << 27)):
        assert size(m, k, n) == 0, (m, n)
    # up to 4 rows always take 16 outputs
    assert size(4, 65, 1 << 28) >= (1 << 28) * 65 and size(4, 65, (1 << 28) - 64) == 0


HUGE = (1 << 63) - 1


@pytest.mark.parametrize("s", ["f32", "bf16", "f16"])
def test_sizes_next_to_the_end_of_64_bits_are_refused(s):
    """A size query of a matrix that no address space holds is an error, whichever of its sizes is large."""
    for off in (0, 3, 7, 8, 31, 64):
        big = HUGE - off
        for m, k, n in ((4, big, 4), (4, 4, big), (big, 4, 4), (big, big, big), (1, big, 1), (1, 1, big), (big, 1, 1)):
            for size, args in (("xtvxy_linear_%s_workspace_size", ()), ("xtvxy_linear_backward_%s_workspace_size", (1,))):
                for aligned in (0, 1):
                    with pytest.raises(xt.XtvxyError, match="INVALID_VALUE"):
                        getattr(xt, size % s)(m, k, n, *args, aligned)
