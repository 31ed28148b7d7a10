"""The training example runs: its loss falls, a row alone gets the answer it gets among others, and its
gradients are those of the same network in fp64."""
import importlib.util
import os

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_mlp.py")
    spec = importlib.util.spec_from_file_location("train_mlp", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_example(dtype, state_bits):
    note("training example %s, %d-bit states" % (dtype, state_bits))
    _, losses, accuracy, single = example().train(60, batch=1024, width=256, dtype=dtype, state_bits=state_bits)
    # ten classes: chance is 10% and log 10 = 2.3
    assert sum(losses[-5:]) / 5 < 0.6 * losses[0] and accuracy > 0.5
    # logits of a few units, summed in another order and rounded through three layers: some steps of 2^-8
    assert single <= 0.125


def test_gradients_of_the_example():
    m = example()
    model = m.Mlp(72, 136, 10, torch.float16, 3, 32)
    g = torch.Generator(device="cuda").manual_seed(9)
    X = torch.randn((333, 72), generator=g, device="cuda").half()
    labels = torch.randint(0, 10, (333,), generator=g, device="cuda")
    note("gradients of the example")
    logits, kept = model.forward(X)
    _, G = m.cross_entropy(logits, labels)
    G = (G.float() * 1024).half()  # away from fp16's subnormals
    got = [t.double().cpu() for ts in model.gradient(G, kept) for t in ts]
    W = [w.double().cpu().requires_grad_() for w in model.weights]
    b = [v.double().cpu().requires_grad_() for v in model.biases]
    gelu = lambda z: z * 0.5 * (1 + torch.erf(z / 2 ** 0.5))  # noqa: E731
    h1 = gelu(X.double().cpu() @ W[0].T + b[0])
    h2 = gelu(h1 @ W[1].T + b[1]) + h1
    out = h2 @ W[2].T + b[2]
    ref = torch.autograd.grad((out * G.double().cpu()).sum(), W + b)
    # every stored fp16 value is off by 2^-11 of itself; about ten of them lie on a gradient's longest path
    for a, r in zip(got, ref):
        assert (a - r).norm() <= 10 * 2.0 ** -11 * r.norm()
