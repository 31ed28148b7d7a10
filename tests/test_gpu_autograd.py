"""What autograd learns of the helpers: the layer's results carry no graph, and the optimiser's step is a write in
place to whatever autograd saved of the parameters and their copies."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from dense_linear_algebra_alpha_amd import optimiser
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def test_layer_is_detached():
    X = torch.ones(8, 16, device=dev(), requires_grad=True)
    W = torch.nn.Parameter(torch.ones(4, 16, device=dev()))
    note("layer of tensors that require gradients")
    out, pre = xt.linear(X, W, act="relu", save_pre=True)
    assert not out.requires_grad and not pre.requires_grad and (out == 16).all()
    assert not any(t.requires_grad for t in xt.linear_backward(out, X, W, pre, "relu"))


@pytest.mark.parametrize("extension", [True, False])
def test_step_is_seen_by_saved_tensors(monkeypatch, extension):
    if not extension:
        monkeypatch.setattr(optimiser, "_extension", lambda: None)
    p, c = torch.nn.Parameter(torch.ones(300, device=dev())), torch.ones(300, device=dev(), dtype=torch.bfloat16)
    x, z = p * p, c.clone().requires_grad_() * c  # products keep their factors
    g = torch.ones(300, device=dev())
    note("autograd around a step, extension %s" % extension)
    opt = xt.AdamW([p], copies=[c])
    opt.step([g])
    for saved in (x, z):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()
    (p * p).sum().backward()  # what is formed after the step is differentiated
    torch.cuda.synchronize()
    assert torch.equal(p.grad, 2 * p.detach())
    with pytest.raises(xt.XtvxyError):
        opt.step([p])  # refused: nothing was written
    before = p._version
    with pytest.raises(xt.XtvxyError):
        opt.step([p])
    assert p._version == before


def test_tensors_of_inference_mode():
    with torch.inference_mode():
        p = torch.ones(5, device=dev())
    note("step on tensors of inference mode")
    xt.AdamW([p]).step([torch.ones(5, device=dev())])
    torch.cuda.synchronize()
    assert (p < 1).all()
