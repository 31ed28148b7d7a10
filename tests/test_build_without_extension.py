"""The library without the host extension of the torch helpers: it builds where torch or a host compiler is missing,
and the helpers then work through their Python path. Host only."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from dense_linear_algebra_alpha_amd import build, layers, optimiser


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Everything is built in a folder of its own; compiling and linking only leave their outputs."""
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libxtvxy.so"))
    monkeypatch.setattr(build, "TENSORS_PATH", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build, "_compile", lambda src: str(tmp_path / src))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd[0])
        if cmd[0] == "g++" and not shutil.which("g++"):
            raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_with_both(elsewhere):
    build.build()
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.TENSORS_PATH) and "g++" in elsewhere


def test_without_torch(elsewhere, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert os.path.exists(build.build()) and not os.path.exists(build.TENSORS_PATH)
    assert "_tensors.so" in capsys.readouterr().err
    assert not build.sources_newer_than_library()  # what cannot be built is not waited for


def test_without_a_host_compiler(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None)
    assert os.path.exists(build.build()) and not os.path.exists(build.TENSORS_PATH)
    assert "_tensors.so" in capsys.readouterr().err
    assert not build.sources_newer_than_library()


def test_a_compile_error_of_the_extension_is_an_error_after_the_library(elsewhere, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_build_tensors", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and build.sources_newer_than_library()


def test_helpers_without_the_extension(monkeypatch):
    """Arguments are still checked and refused, now by the Python path."""
    class Tensor:
        def __init__(self, *shape, dtype=torch.float32):
            self.shape, self.dtype, self.layout = shape, dtype, torch.strided
            self.is_cuda, self.device = True, torch.device("cuda", 0)

        def get_device(self):
            return 0

        def dim(self):
            return len(self.shape)

        def stride(self, i=None):
            return (self.shape[1], 1) if i is None else (self.shape[1], 1)[i]

        def numel(self):
            return self.shape[0]

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 1 << 40

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setitem(sys.modules, "dense_linear_algebra_alpha_amd._tensors", None)
    layers._extension.cache_clear()
    try:
        with pytest.warns(RuntimeWarning, match="_tensors.so"):
            assert layers._extension() is None
        with pytest.raises(ValueError, match="W must be 6 x 8"):
            xt.linear(Tensor(4, 8), Tensor(6, 7))
        with pytest.raises(ValueError, match="W must be 6 x 8"):
            xt.linear_backward(Tensor(4, 6), Tensor(4, 8), Tensor(6, 7))
        opt = optimiser.AdamW.__new__(optimiser.AdamW)
        opt.handle, opt.device, opt._numel, opt._numel_address = 0, torch.device("cuda", 0), [4, 6], 0
        opt._pointers = optimiser.ctypes.c_void_p * 2
        pointers, code = opt._like_params("grads", [Tensor(4), Tensor(6)])
        assert list(pointers) == [1 << 40] * 2 and code == optimiser.XTVXY_TYPE_F32
        for bad in ([Tensor(4), Tensor(5)], [Tensor(4), Tensor(6, dtype=torch.float16)], [Tensor(4), torch.zeros(6)], [Tensor(4), None]):
            with pytest.raises(ValueError, match=r"grads\[1\]"):
                opt._like_params("grads", bad)
    finally:
        layers._extension.cache_clear()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_same_results_without_the_extension(monkeypatch, bits):
    d = torch.device("cuda", 0)
    g = torch.Generator(device=d).manual_seed(1)
    X, W, G = [torch.randn(s, generator=g, device=d).half() for s in ((70, 96), (40, 96), (70, 40))]
    b = torch.randn(40, generator=g, device=d)

    def results():
        out, pre = xt.linear(X, W, b, G, "silu", save_pre=True)
        grads = xt.linear_backward(G, X, W, pre, "silu")
        p = [torch.ones(40, 96, device=d), torch.ones(5, device=d)]
        opt = xt.AdamW(p, state_bits=bits, seed=3)
        opt.step([grads[1].float(), b[:5]])
        values = [[torch.empty_like(t) for t in p] for _ in range(2)]
        opt.state_values(*values)
        torch.cuda.synchronize()
        return [out, pre, *grads, *p, *values[0], *values[1]]

    print("[gpu] layer and optimiser without the extension", flush=True)
    want = results()
    for module in (layers, optimiser):
        monkeypatch.setattr(module, "_extension", lambda: None)
    assert all(torch.equal(a, c) for a, c in zip(want, results()))
