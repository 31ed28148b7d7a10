"""The AdamW step at the ends of its range."""
import numpy as np
import pytest
import torch

import adamw_oracle as O
import dense_linear_algebra_alpha_amd as xt
from gpu_util import dev, note

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LR, BETAS = 3e-3, (0.9, 0.99)


def gradients(big, grad):
    """Two steps' gradients of 384 elements, element 5's first one `big`, and the same without it."""
    g = [torch.randn(384, generator=torch.Generator().manual_seed(s)).mul(1e-3).to(DT[grad]) for s in (1, 2)]
    clean = [x.clone() for x in g]
    g[0][5] = big
    return g, clean


@pytest.mark.parametrize("grad", list(DT))
@pytest.mark.parametrize("big", [1e19, -1e20, 1.5e20, 1e21, -1e30, 3.3e38])
@pytest.mark.parametrize("bits", [8, 32])
def test_one_large_finite_gradient(bits, big, grad):
    """(1 - beta2) g^2 is formed without g^2, which leaves fp32 from 1.9e19 on; where it leaves fp32 itself
    (1.9e20) p is left alone, by the next step too."""
    g, clean = gradients(big, grad)
    p0 = torch.randn(384, generator=torch.Generator().manual_seed(3))
    note("adamw %d bits, one gradient of %g in %s" % (bits, big, grad))
    runs = []
    for gs in (g, clean):
        p = p0.to(dev())
        opt = xt.AdamW([p], lr=LR, betas=BETAS, weight_decay=0.0, state_bits=bits)
        steps = [p0.double()]
        m, v = torch.zeros(384, device=dev()), torch.zeros(384, device=dev())
        for i, x in enumerate(gs):
            opt.step([x.to(dev())])
            if i == 0:
                opt.state_values([m], [v])
                first = (m.double().cpu(), v.double().cpu())
            steps.append(p.double().cpu())
        runs.append((steps, first))
    (steps, (m1, v1)), (clean_steps, _) = runs
    assert all(torch.isfinite(s).all() for s in steps)
    x = g[0][5].double().item()
    true_v = (1 - BETAS[1]) * x * x
    # a step's size is at most (1 - b1) / sqrt(1 - b2) once both moments are corrected; twice that with codes
    # off by 2^-3 (m) and 2^-4 (v), or v cut off at its largest value (half of fp32's end)
    for a, b in zip(steps[:-1], steps[1:]):
        assert abs(b[5] - a[5]) <= 4 * LR
    if true_v < 1.6e38:
        assert abs(m1[5] / (0.1 * x) - 1) <= (2.0 ** -3 if bits == 8 else 1e-6)
        assert abs(v1[5] / true_v - 1) <= (2.0 ** -4 if bits == 8 else 1e-6)
        assert abs((steps[0][5] - steps[1][5]) / (LR * np.sign(x)) - 1) <= 1e-3  # the first step's size is lr
    else:
        if true_v > 3.5e38:
            assert steps[1][5] == steps[0][5]
        # the others keep their steps
        keep = torch.arange(384) != 5
        if true_v > 3.5e38 or bits == 32:
            assert all(torch.equal(a[keep], b[keep]) for a, b in zip(steps, clean_steps))


def test_first_moments_next_to_the_end_of_fp32():
    """8-bit first moments of up to 2^128 keep their sign and size; only NaN and infinity become NaN."""
    codes = np.arange(256, dtype=np.int64)
    codes = codes[(codes & 127) < 127]
    n = 254
    for exponent, beta1 in ((245, 0.999), (246, 0.999), (246, 0.9), (247, 0.5)):
        exps = np.full(2, exponent, np.int64)
        m0 = O.decode(codes, exps, O.m_value)
        fits = np.abs(m0) < 2.0 ** 127 * (2 - 2.0 ** -23)
        held = np.where(fits, codes, 0)
        m0 = np.where(fits, m0, 0.0)
        state = [torch.from_numpy(x.astype(np.uint8)).to(dev()) for x in (held, np.zeros(n), exps, np.ones(2))]
        note("adamw first moments with exponent %d, beta1 %g" % (exponent, beta1))
        opt = xt.AdamW([torch.zeros(n, device=dev())], lr=0.0, betas=(beta1, 0.99), weight_decay=0.0, state_bits=8,
                       state=tuple([s] for s in state), steps=3)
        opt.step([torch.zeros(n, device=dev())])
        m, v = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
        opt.state_values([m], [v])
        got, want = m.double().cpu().numpy(), beta1 * m0
        # a code's step is 2^-3 of its value, or 2^-9 of the block's unit (448 units at most)
        top = np.repeat([np.abs(want[:128]).max(), np.abs(want[128:]).max()], 128)[:n]
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= np.maximum(2.0 ** -3 * np.abs(want), 2.0 ** -9 * top / 224)).all()
        assert (np.sign(got) * np.sign(want) >= 0).all()
