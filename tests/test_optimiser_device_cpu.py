"""An optimiser whose tensors are not on the current GPU is refused before anything is enqueued. Host only: the
tensors are stand-ins that claim to be on a GPU."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt

DEVICE = torch.device("cuda", 1)


class OnAnotherGpu:
    def __init__(self, n, dtype=torch.float32):
        self.n, self.dtype, self.device = n, dtype, DEVICE

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("an address was taken")


@pytest.fixture(autouse=True)
def current_gpu_is_the_first(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def test_making_one():
    state = ([OnAnotherGpu(4)], [OnAnotherGpu(4)])
    with pytest.raises(ValueError, match="current GPU"):
        xt.AdamW([OnAnotherGpu(4)], state=state)
    with pytest.raises(ValueError, match="current GPU"):  # nor are fresh states made first
        xt.AdamW([OnAnotherGpu(4)])


def test_calls_of_one():
    opt = xt.AdamW.__new__(xt.AdamW)  # as made while its GPU was the current one
    opt.handle, opt.device, opt._numel, opt.steps = 0, DEVICE, [4], 0
    for call in (lambda: opt.step([OnAnotherGpu(4)]), lambda: opt.state_values([OnAnotherGpu(4)], [OnAnotherGpu(4)])):
        with pytest.raises(ValueError, match="current GPU"):
            call()
    assert opt.steps == 0
