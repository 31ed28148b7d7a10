"""Trains a small multi-layer perceptron in mixed precision and answers with it, row by row: the fully
connected layer, its gradient and the AdamW step together, as a training program uses them.

    python examples/train_mlp.py [--steps 200] [--state-bits 8] [--dtype bf16]

Two hidden layers with gelu, the second added to its input, and a linear output. fp32 master weights;
the layers compute with 16-bit copies that every step rewrites. The task is synthetic: the label of a row
is the largest of ten fixed random projections of tanh(row).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_linear_algebra_alpha_amd as xt  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Mlp:
    """Weights W (outputs x features, 16-bit, and fp32 masters) and biases (fp32)."""

    def __init__(self, features, width, classes, dtype, seed, state_bits):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = [(width, features), (width, width), (classes, width)]
        self.masters = [torch.randn(s, generator=g, device="cuda") * s[1] ** -0.5 for s in shapes]
        self.weights = [w.to(dtype) for w in self.masters]
        self.biases = [torch.zeros(s[0], device="cuda") for s in shapes]
        # gradients come in two types, so weights and biases have an optimiser each
        self.optimisers = [xt.AdamW(self.masters, lr=2e-3, copies=self.weights, state_bits=state_bits, seed=seed),
                           xt.AdamW(self.biases, lr=2e-3, weight_decay=0.0, state_bits=state_bits, seed=seed + 1)]

    def forward(self, X):
        """(logits, what the gradient needs)."""
        (W1, W2, W3), (b1, b2, b3) = self.weights, self.biases
        h1, z1 = xt.linear(X, W1, b1, act="gelu", save_pre=True)
        h2, z2 = xt.linear(h1, W2, b2, h1, "gelu", save_pre=True)
        return xt.linear(h2, W3, b3), (X, h1, z1, h2, z2)

    def gradient(self, G, kept):
        """Gradients of the weights and biases from that of the logits."""
        X, h1, z1, h2, z2 = kept
        W2, W3 = self.weights[1:]
        d2, dW3, db3 = xt.linear_backward(G, h2, W3)
        d1, dW2, db2 = xt.linear_backward(d2, h1, W2, z2, "gelu")
        d1 += d2  # of the residual
        _, dW1, db1 = xt.linear_backward(d1, X, self.weights[0], z1, "gelu", need_dX=False)
        return [dW1, dW2, dW3], [db1, db2, db3]

    def step(self, weight_grads, bias_grads):
        for optimiser, grads in zip(self.optimisers, (weight_grads, bias_grads)):
            optimiser.step(grads)


def cross_entropy(logits, labels):
    """(mean loss, its gradient in the logits' type)."""
    p = torch.softmax(logits.float(), 1)
    rows = torch.arange(len(labels), device=labels.device)
    loss = -torch.log(p[rows, labels].clamp_min(1e-30)).mean()
    p[rows, labels] -= 1.0
    return loss, (p / len(labels)).to(logits.dtype)


def train(steps=200, batch=2048, features=128, width=512, classes=10, dtype="bf16", state_bits=32, seed=0, report=None):
    """(model, losses, accuracy on fresh rows, largest difference of rows answered one by one)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    truth = torch.randn((features, classes), generator=g, device="cuda")

    def rows(n):
        X = torch.randn((n, features), generator=g, device="cuda").to(TYPES[dtype])
        return X, (torch.tanh(X.float()) @ truth).argmax(1)

    model, losses = Mlp(features, width, classes, TYPES[dtype], seed, state_bits), []
    for i in range(steps):
        X, labels = rows(batch)
        logits, kept = model.forward(X)
        loss, G = cross_entropy(logits, labels)
        model.step(*model.gradient(G, kept))
        losses.append(loss)
        if report and i % 20 == 19:
            report("step %d: loss %.4f" % (i + 1, loss.item()))
    X, labels = rows(1000)
    logits = model.forward(X)[0]
    single = torch.cat([model.forward(X[i:i + 1])[0] for i in range(16)])
    accuracy = (logits.argmax(1) == labels).float().mean().item()
    return model, [v.item() for v in losses], accuracy, (single - logits[:16]).abs().max().item()


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    p.add_argument("--dtype", default="bf16", choices=sorted(TYPES))
    a = p.parse_args()
    _, losses, accuracy, single = train(a.steps, dtype=a.dtype, state_bits=a.state_bits, report=lambda s: print(s, flush=True))
    print("loss %.4f -> %.4f, accuracy on fresh rows %.1f%%, rows one by one differ by at most %.2g"
          % (losses[0], losses[-1], 100 * accuracy, single))


if __name__ == "__main__":
    main()
