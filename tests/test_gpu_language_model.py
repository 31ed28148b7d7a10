"""The language model of examples/train_language_model.py: it runs in every type, and its gradients (embedding, layer norm,
layer, cross entropy or distillation, with a tied table) are those of the fp64 formula."""
import importlib.util
import math
import os

import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_language_model.py")
    spec = importlib.util.spec_from_file_location("train_language_model", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_runs(example, dtype):
    note("language model %s" % dtype)
    teacher, student, losses, distances = example.train(steps=3, vocabulary=1001, batch=500, width=64, hidden=96, dtype=dtype)
    assert len(losses) == len(distances) == 3 and all(math.isfinite(v) for v in losses + distances)
    for model in (teacher, student):
        assert all(torch.isfinite(t).all() for t in model.masters + model.vectors)


def reference(model, tokens, loss_of):
    """Loss and gradients in fp64 by automatic differentiation of the formula."""
    leaves = [t.detach().double().cpu().requires_grad_() for t in model.matrices + model.vectors]
    (table, W1, W2), (b1, b2, n1, c1, n2, c2, bias) = leaves[:3], leaves[3:]

    def norm(x, w, c):
        d = x - x.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * w + c

    x = table[tokens.cpu()] * model.scale
    h = norm(x, n1, c1) @ W1.T + b1
    h = 0.5 * h * torch.special.erfc(-h / math.sqrt(2.0))
    loss = loss_of(norm(x + h @ W2.T + b2, n2, c2) @ table.T + bias)
    loss.backward()
    return loss.item(), [t.grad for t in leaves]


@pytest.mark.parametrize("soft", [False, True], ids=["labels", "teacher"])
def test_gradients(example, soft):
    model = example.Model(301, 64, 96, torch.float32, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    for v in model.vectors:
        v += 0.1 * torch.randn(v.shape, generator=g, device="cuda")
    tokens = torch.randint(0, 301, (200,), generator=g, device="cuda")
    note("language model's gradients %s" % soft)
    if soft:
        classes = torch.rand((200, 301), generator=g, device="cuda").argsort(1)[:, :8].contiguous()
        logits = torch.randn((200, 8), generator=g, device="cuda")
        loss, grads = model.distillation_gradient(tokens, classes, logits, 2.0)
        P = torch.softmax(logits.double().cpu() / 2.0, 1)

        def of(z):
            logp = torch.log_softmax(z / 2.0, 1).gather(1, classes.cpu())
            return 4.0 * (P * (torch.log(P) - logp)).sum(1).mean()
    else:
        labels = torch.randint(0, 301, (200,), generator=g, device="cuda")
        labels[::7] = -100
        loss, grads = model.loss_gradient(tokens, labels)

        def of(z):
            on = labels.cpu() >= 0
            return torch.nn.functional.cross_entropy(z[on], labels.cpu()[on])
    torch.cuda.synchronize()
    want, ref = reference(model, tokens, of)
    want = want / 4.0 if soft else want
    # Seven operators one after the other and back; each of their sums of at most 301 products is off by (301 + 4) 2^-23
    # = 3.6e-5 of its products' magnitudes at most, which exceed the sum's by sqrt(301) = 17 where signs are random:
    # 7 x 2 x 3.6e-5 x 17 = 9e-3.
    assert abs(loss.item() - want) <= 9e-3 * abs(want)
    for got, r in zip(grads[0] + grads[1], ref):
        assert got.shape == r.shape
        assert (got.double().cpu() - r).norm() <= 9e-3 * r.norm()


def test_a_step_in_a_graph(example):
    """Losses, gradients and their sum into the tied table, captured: replays with other tokens equal eager calls."""
    model = example.Model(500, 64, 96, torch.bfloat16, 7)
    g = torch.Generator(device="cuda").manual_seed(8)
    new = lambda: torch.randint(0, 500, (300,), generator=g, device="cuda")  # noqa: E731
    tokens, labels = new(), new()

    def step():
        f, kept = model.forward(tokens)
        loss, lse = xt.linear_cross_entropy(f, model.matrices[0], labels, model.vectors[-1])
        df, dtable, db = xt.linear_cross_entropy_backward(weight, f, model.matrices[0], labels, lse, model.vectors[-1])
        m, v = model.gradient(df, dtable, db, kept)
        return [loss] + m + v

    weight = torch.full((300,), 1 / 300, device="cuda")
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        tokens.copy_(new())
        labels.copy_(new())
        note("language model replay %d" % i)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
