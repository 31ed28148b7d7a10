"""Trains a small next-token model in mixed precision, then a smaller one from its answers: embedding, layer norm, the
fully connected layer, the cross entropy over the vocabulary, distillation and AdamW together, as a training program uses
them.

    python examples/train_language_model.py [--steps 200] [--dtype bf16]

A token's row of the table, a residual block (layer norm, a wide layer with gelu, a layer back), a last layer norm, and
logits by the same table (tied). fp32 master weights; the operators compute with 16-bit copies that every step
rewrites. The task is synthetic: the next token is one of four that a fixed random map gives, the first most often.
The student has a table of its own and learns from the teacher's eight largest logits of each token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_linear_algebra_alpha_amd as xt  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Model:
    """Matrices (16-bit, with fp32 masters): table (vocabulary x width), W1 (hidden x width), W2 (width x hidden).
    Vectors (fp32): the layers' biases, the norms' weights and biases."""

    def __init__(self, vocabulary, width, hidden, dtype, seed, lr=2e-3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.masters = [torch.randn(s, generator=g, device="cuda") * by for s, by in
                        (((vocabulary, width), width ** -0.5), ((hidden, width), width ** -0.5), ((width, hidden), hidden ** -0.5))]
        copies = dtype != torch.float32
        self.matrices = [w.to(dtype) for w in self.masters] if copies else self.masters
        zeros, ones = (lambda n: torch.zeros(n, device="cuda")), (lambda n: torch.ones(n, device="cuda"))
        # b1, b2, the first norm's weight and bias, the last one's, the bias of the logits
        self.vectors = [zeros(hidden), zeros(width), ones(width), zeros(width), ones(width), zeros(width), zeros(vocabulary)]
        self.scale = width ** 0.5
        self.optimisers = [xt.AdamW(self.masters, lr=lr, weight_decay=0.0, copies=self.matrices if copies else None),
                           xt.AdamW(self.vectors, lr=lr, weight_decay=0.0)]

    def forward(self, tokens):
        """(features before the logits, what the gradient needs)."""
        (table, W1, W2), (b1, b2, n1, c1, n2, c2, _) = self.matrices, self.vectors
        x = xt.embedding(tokens, table, self.scale)
        y, mean1, rstd1 = xt.layer_norm(x, n1, c1, save_stats=True)
        h, pre = xt.linear(y, W1, b1, act="gelu", save_pre=True)
        z = xt.linear(h, W2, b2, x)
        f, mean2, rstd2 = xt.layer_norm(z, n2, c2, save_stats=True)
        return f, (tokens, x, mean1, rstd1, y, pre, h, z, mean2, rstd2)

    def gradient(self, df, dtable, dlogit_bias, kept):
        """Gradients of matrices and vectors from those of the features and, by the logits, of the table."""
        tokens, x, mean1, rstd1, y, pre, h, z, mean2, rstd2 = kept
        (table, W1, W2), (_, _, n1, _, n2, _, _) = self.matrices, self.vectors
        dz, dn2, dc2 = xt.layer_norm_backward(df, z, mean2, rstd2, n2)
        dh, dW2, db2 = xt.linear_backward(dz, h, W2)
        dy, dW1, db1 = xt.linear_backward(dh, y, W1, pre, "gelu")
        dx, dn1, dc1 = xt.layer_norm_backward(dy, x, mean1, rstd1, n1)
        dx += dz  # of the residual
        xt.embedding_backward(dx, tokens, len(table), self.scale, dtable=dtable, accumulate=True)  # the table is tied
        return [dtable, dW1, dW2], [db1, db2, dn1, dc1, dn2, dc2, dlogit_bias]

    def loss_gradient(self, tokens, labels, scale=1.0):
        """(mean loss over the labels that count, the gradients of scale times it)."""
        f, kept = self.forward(tokens)
        loss, lse = xt.linear_cross_entropy(f, self.matrices[0], labels, self.vectors[-1])
        counts = (labels >= 0).sum()
        grad = (scale / counts).float().expand(len(labels)).contiguous()
        df, dtable, db = xt.linear_cross_entropy_backward(grad, f, self.matrices[0], labels, lse, self.vectors[-1])
        return loss.sum() / counts, self.gradient(df, dtable, db, kept)

    def distillation_gradient(self, tokens, classes, teacher, temperature):
        f, kept = self.forward(tokens)
        loss, lse, weights = xt.linear_distillation(f, self.matrices[0], classes, teacher, self.vectors[-1], temperature)
        grad = torch.full((len(tokens),), temperature ** 2 / len(tokens), device="cuda")
        df, dtable, db = xt.linear_distillation_backward(grad, f, self.matrices[0], classes, weights, lse, self.vectors[-1],
                                                         temperature)
        return loss.mean(), self.gradient(df, dtable, db, kept)

    def step(self, gradients):
        for optimiser, grads in zip(self.optimisers, gradients):
            optimiser.step(grads)

    def logits(self, tokens):
        f, _ = self.forward(tokens)
        return xt.linear(f, self.matrices[0], self.vectors[-1])


def batches(vocabulary, batch, seed):
    """Tokens and what follows them; a tenth of the labels does not count."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    follows = torch.randint(0, vocabulary, (vocabulary, 4), generator=g, device="cuda")
    odds = torch.tensor([0.55, 0.25, 0.15, 0.05], device="cuda")
    while True:
        tokens = torch.randint(0, vocabulary, (batch,), generator=g, device="cuda")
        which = torch.multinomial(odds, batch, replacement=True, generator=g)
        labels = follows[tokens, which]
        yield tokens, torch.where(torch.rand(batch, generator=g, device="cuda") < 0.1, -100, labels)


def train(steps=200, vocabulary=4000, batch=4096, width=256, hidden=1024, dtype="bf16", seed=0, report=None):
    """(teacher, student, the teacher's losses, the student's)."""
    data = batches(vocabulary, batch, seed)
    teacher = Model(vocabulary, width, hidden, TYPES[dtype], seed + 1)
    student = Model(vocabulary, width // 2, hidden // 4, TYPES[dtype], seed + 2)
    losses, distances = [], []
    for i in range(steps):
        tokens, labels = next(data)
        loss, gradients = teacher.loss_gradient(tokens, labels)
        teacher.step(gradients)
        losses.append(loss)
        if report and i % 20 == 19:
            report("teacher, step %d: loss %.4f" % (i + 1, loss.item()))
    for i in range(steps):
        tokens, _ = next(data)
        top, classes = torch.topk(teacher.logits(tokens).float(), 8)
        loss, gradients = student.distillation_gradient(tokens, classes, top, 2.0)
        student.step(gradients)
        distances.append(loss)
        if report and i % 20 == 19:
            report("student, step %d: distance %.4f" % (i + 1, loss.item()))
    return teacher, student, [v.item() for v in losses], [v.item() for v in distances]


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--dtype", default="bf16", choices=sorted(TYPES))
    a = p.parse_args()
    _, _, losses, distances = train(a.steps, dtype=a.dtype, report=lambda s: print(s, flush=True))
    print("teacher's loss %.4f -> %.4f, student's distance %.4f -> %.4f" % (losses[0], losses[-1], distances[0], distances[-1]))


if __name__ == "__main__":
    main()
