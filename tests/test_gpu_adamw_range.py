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


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("lr", [2e-6, 1e-5])
def test_weight_decay_below_the_spacing_of_fp32(lr, bits):
    """lr weight_decay of 2e-8 and 1e-7: the mean decay over many elements, whose updates of many units of p
    spread the rounding of the sum evenly."""
    n, wd, b1, b2, t = 1 << 20, 0.01, 0.9, 0.99, 7
    gen = torch.Generator().manual_seed(8)
    p0 = 1.0 + torch.rand(n, generator=gen)
    g = torch.randn(n, generator=gen)
    p = p0.to(dev())
    note("adamw %d bits, lr %g and weight decay %g" % (bits, lr, wd))
    if bits == 32:
        m0, v0 = torch.randn(n, generator=gen) * 0.3, torch.rand(n, generator=gen) + 0.5
        state = ([m0.to(dev())], [v0.to(dev())])
        md, vd = m0.double(), v0.double()
    else:
        qm = (torch.randint(0, 0x60, (n,), generator=gen) + 128 * torch.randint(0, 2, (n,), generator=gen)).numpy()
        qv = torch.randint(0xa0, 0x100, (n,), generator=gen).numpy()
        em, ev = np.full(n // 128, 122), np.full(n // 128, 127)
        state = tuple([torch.from_numpy(x.astype(np.uint8)).to(dev())] for x in (qm, qv, em, ev))
        md, vd = torch.from_numpy(O.decode(qm, em, O.m_value)), torch.from_numpy(O.decode(qv, ev, O.v_value))
    opt = xt.AdamW([p], lr=lr, betas=(b1, b2), weight_decay=wd, state_bits=bits, state=state, steps=t - 1)
    opt.step([g.to(dev())])
    m1, v1 = b1 * md + (1 - b1) * g.double(), b2 * vd + (1 - b2) * g.double() ** 2
    update = lr / (1 - b1 ** t) * m1 / (v1.sqrt() / (1 - b2 ** t) ** 0.5 + opt.eps)
    assert update.std() > 2.0 ** -23  # of several units: the sum is rounded evenly to 1e-8 of a unit
    decay = (p0.double() - update - p.double().cpu()).mean().item()
    want = lr * wd * p0.double().mean().item()
    # the sum's rounding is off by at most half of 2^-23, evenly; five standard deviations of its mean, and the
    # update's own few units
    assert abs(decay - want) <= 5 * 2.0 ** -23 / 12 ** 0.5 / n ** 0.5 + 16 * 2.0 ** -24 * update.abs().mean().item()


def test_infinite_parameters_stay():
    p = torch.tensor([float("inf"), -float("inf"), 1.0], device=dev())
    for wd in (0.0, 0.01):
        note("adamw infinite parameters, weight decay %g" % wd)
        xt.AdamW([p], lr=1e-3, weight_decay=wd).step([torch.ones(3, device=dev())])
        assert p[0] == float("inf") and p[1] == -float("inf") and torch.isfinite(p[2])


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("beta2,eps", [(0.999999, 1e-12), (0.999, 1e-12), (0.99, 1e-13), (0.999999, 1e-8)])
def test_second_moments_below_fp32s_normal_range(beta2, eps, bits):
    """Gradients whose v is subnormal: its root counts next to eps, as the formula says."""
    n = 512
    # from 2^-140 to 2^-126: 2^-9 of the value at the least, halved by the root
    v = 2.0 ** torch.linspace(-140, -126, n, dtype=torch.float64)
    g = (v / (1 - beta2)).sqrt().float()
    p = torch.zeros(n, device=dev())
    note("adamw %d bits, subnormal second moments, beta2 %g, eps %g" % (bits, beta2, eps))
    xt.AdamW([p], lr=1e-2, betas=(0.9, beta2), eps=eps, weight_decay=0.0, state_bits=bits).step([g.to(dev())])
    want = -1e-2 * g.double() / (g.double().abs() + eps)
    root = g.double() / (g.double() + eps)  # share of the root in the denominator
    # v is kept to 2^-149; 32 units for the rest
    tol = 32 * 2.0 ** -24 + root * 2.0 ** -149 / v
    assert ((p.double().cpu() / want - 1).abs() <= tol).all()


def test_values_of_states_do_not_share_memory():
    p, x = torch.ones(300, device=dev()), torch.zeros(700, device=dev())
    for bits in (8, 32):
        note("adamw %d bits, values into overlapping tensors" % bits)
        opt = xt.AdamW([p, p.clone()], state_bits=bits)
        opt.step([p.clone(), p.clone()])
        a, b, c, d = [torch.zeros(300, device=dev()) for _ in range(4)]
        opt.state_values([a, b], [c, d])
        for m, v in (([a, b], [a, d]), ([a, a], [c, d]), ([a, b], [c, c]), ([x[:300], b], [c, x[299:599]])):
            with pytest.raises(xt.XtvxyError, match="ALIASING"):
                opt.state_values(m, v)
        opt.state_values([x[:300], b], [c, x[300:600]])
        torch.cuda.synchronize()
        assert torch.equal(x[:300], a) and torch.equal(x[300:600], d)
