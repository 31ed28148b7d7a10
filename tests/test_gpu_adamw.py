"""GPU parity of the AdamW step against the fp64 oracle (32-bit states) and, code by code, against the
integer oracle (8-bit states)."""
import numpy as np
import pytest
import torch

import adamw_oracle as O
import dense_linear_algebra_alpha_amd as xt
from gpu_util import dev, note

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def placed(x, offset):
    """x on the GPU, `offset` elements into a larger buffer whose ends are watched."""
    buf = torch.full((x.numel() + offset + 9,), 7, dtype=x.dtype, device=dev())
    v = buf[offset:offset + x.numel()]
    v.copy_(x)
    return buf, v


def untouched(buf, offset, n):
    return bool((buf[:offset] == 7).all() and (buf[offset + n:] == 7).all())


def make(sizes, grad, seed):
    g = torch.Generator().manual_seed(seed)
    ps = [torch.randn(n, generator=g) for n in sizes]
    gs = [(torch.randn(n, generator=g) * 10.0 ** (-(i % 5))).to(DT[grad]) for i, n in enumerate(sizes)]
    ms = [torch.randn(n, generator=g) * 10.0 ** (-(i % 5)) * 0.3 for i, n in enumerate(sizes)]
    vs = [torch.rand(n, generator=g) * 10.0 ** (-2 * (i % 5)) for i, n in enumerate(sizes)]
    return ps, gs, ms, vs


def within(got, ref, bound, what):
    got = got.double().cpu().numpy()
    over = np.max(np.abs(got - ref) / bound) if len(ref) else 0.0
    assert over <= 1.0, "%s: error %.3g times its bound" % (what, over)


SIZES = [[1], [127, 0, 128, 129], [5, 2048, 2049, 4095, 1], [100003], [64] * 450 + [3]]


@pytest.mark.parametrize("grad", list(DT))
@pytest.mark.parametrize("copy", ["none", "bf16", "f16"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), sum(s)))
@pytest.mark.parametrize("offset", [0, 1])
def test_step_32(sizes, copy, grad, offset):
    ps, gs, ms, vs = make(sizes, grad, 11)
    P, G, M, V = [[placed(x, offset) for x in xs] for xs in (ps, gs, ms, vs)]
    C = None if copy == "none" else [placed(x.to(DT[copy]), offset) for x in ps]
    note("adamw 32 bits %d tensors grad %s copy %s offset %d" % (len(sizes), grad, copy, offset))
    opt = xt.AdamW([v for _, v in P], copies=C and [v for _, v in C], state=([v for _, v in M], [v for _, v in V]),
                   steps=6, **HYPER)
    opt.step([v for _, v in G])
    torch.cuda.synchronize()
    assert opt.steps == 7
    for i, n in enumerate(sizes):
        p, m, v, ep, em, ev = O.update(*[x.double().numpy() for x in (ps[i], gs[i], ms[i], vs[i])], 7, HYPER["lr"],
                                       *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        for (buf, t), ref, e, w in ((P[i], p, ep, "p"), (M[i], m, em, "m"), (V[i], v, ev, "v")):
            within(t, ref, e, "%s of tensor %d" % (w, i))
            assert untouched(buf, offset, n)
        if C:
            buf, c = C[i]
            assert torch.equal(c, P[i][1].to(DT[copy])) and untouched(buf, offset, n)


@pytest.mark.parametrize("grad", list(DT))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), sum(s)))
@pytest.mark.parametrize("offset", [0, 3])
def test_step_8(sizes, grad, offset):
    ps, gs, ms, vs = make(sizes, grad, 12)
    seed, t = 0x9ABCDEF1, 5
    first, states = 0, []
    for n, m, v in zip(sizes, ms, vs):  # codes of earlier steps
        states.append(O.encode(m.double().numpy(), v.double().numpy(), first, seed, t - 1)[:4])
        first += (n + 127) // 128 * 128
    P, G = [[placed(x, offset) for x in xs] for xs in (ps, gs)]
    S = [[placed(torch.from_numpy(s[k].astype(np.uint8)), offset) for s in states] for k in range(4)]
    note("adamw 8 bits %d tensors grad %s offset %d" % (len(sizes), grad, offset))
    opt = xt.AdamW([v for _, v in P], state_bits=8, state=tuple([v for _, v in s] for s in S), steps=t - 1, seed=seed,
                   copies=[torch.zeros(n, dtype=torch.bfloat16, device=dev()) for n in sizes], **HYPER)
    opt.step([v for _, v in G])
    mv = [[torch.zeros(n, device=dev()) for n in sizes] for _ in range(2)]
    opt.state_values(*mv)
    torch.cuda.synchronize()
    first = 0
    for i, n in enumerate(sizes):
        qm, qv, me, ve = states[i]
        m0, v0 = O.decode(qm, me, O.m_value), O.decode(qv, ve, O.v_value)
        p, m, v, ep, em, ev = O.update(ps[i].double().numpy(), gs[i].double().numpy(), m0, v0, t, HYPER["lr"],
                                       *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        within(P[i][1], p, ep, "p of tensor %d" % i)
        assert torch.equal(opt.copies[i], P[i][1].bfloat16())
        got = [s[i][1].cpu().numpy().astype(np.int64) for s in S]
        assert all(untouched(s[i][0], offset, len(g)) for s, g in zip(S, got))
        cm, cv, xm, xv, near_m, near_v = O.encode(m, v, first, seed, t)
        # exponents: equal unless the block's top is within fp32's rounding of the border
        assert max(np.sum(got[2] != xm), np.sum(got[3] != xv)) <= 1e-3 * len(xm)
        same = np.repeat((got[2] == xm) & (got[3] == xv), 128)[:n]
        # codes: equal unless the remainder is within fp32's rounding of the random threshold
        # (a step is 2^-3 or 2^-4 of the value: 2^-20 of a step is more than the update's roundings)
        rel = lambda e, x: e / np.maximum(np.abs(x), 1e-300)  # noqa: E731
        sure_m = same & (near_m > 16 * rel(em, m) + 2.0 ** -20)
        sure_v = same & (near_v > 32 * rel(ev, v) + 2.0 ** -18)
        assert np.array_equal(got[0][sure_m], cm[sure_m]) and np.array_equal(got[1][sure_v], cv[sure_v])
        assert n < 1000 or (sure_m.mean() > 0.98 and sure_v.mean() > 0.98)
        # what the states stand for
        for k, value in ((0, O.m_value), (1, O.v_value)):
            want = O.decode(got[k], got[k + 2], value)
            assert np.array_equal(mv[k][i].double().cpu().numpy(), want)
        first += (n + 127) // 128 * 128


def test_random_rounding_has_no_bias():
    """The stored values' mean over many elements of one value is that value."""
    n = 1 << 18
    p, g = torch.zeros(n, device=dev()), torch.full((n,), 0.37, device=dev())
    g[::128] = 1.0  # the blocks' top
    note("adamw 8 bits bias")
    opt = xt.AdamW([p], betas=(0.9, 0.99), state_bits=8, seed=5)
    opt.step([g])
    m, v = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    opt.state_values([m], [v])
    keep = torch.arange(n, device=dev()) % 128 != 0
    m, v = m[keep].double(), v[keep].double()
    # a step is at most 2^-3 (m) or 2^-4 (v) of the value; five standard deviations of the mean
    for got, want, step in ((m, 0.1 * 0.37, 2.0 ** -3), (v, 0.01 * 0.37 ** 2, 2.0 ** -4)):
        assert got.min() <= want <= got.max()
        assert abs(got.mean().item() / want - 1) <= 5 * 0.5 * step / len(got) ** 0.5 + 2.0 ** -13


@pytest.mark.parametrize("bits", [8, 32])
def test_training_runs_and_resumes(bits):
    """Several steps equal the oracle's (32 bits) and a resumed optimiser continues bit for bit."""
    sizes = [300, 7, 1024]
    ps, _, _, _ = make(sizes, "f32", 3)
    grads = [[x.to(dev()) for x in make(sizes, "f32", 100 + t)[1]] for t in range(6)]
    P = [x.to(dev()) for x in ps]
    note("adamw %d bits several steps" % bits)
    opt = xt.AdamW(P, state_bits=bits, seed=77, **HYPER)
    for g in grads[:3]:
        opt.step(g)
    Q = [p.clone() for p in P]
    again = xt.AdamW(Q, state_bits=bits, seed=77, steps=opt.steps,
                     state=tuple([t.clone() for t in s] for s in opt.state), **HYPER)
    for g in grads[3:]:
        opt.step(g)
        again.step(g)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(P, Q))
    assert all(torch.equal(a, b) for x, y in zip(opt.state, again.state) for a, b in zip(x, y))
    if bits == 32:
        for i in range(3):
            p, m, v, e = ps[i].double().numpy(), 0.0, 0.0, 0.0
            for t in range(6):
                p, m, v, ep, _, _ = O.update(p, grads[t][i].double().cpu().numpy(), m, v, t + 1, HYPER["lr"],
                                             *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
                e = e + 2 * ep
            within(P[i], p, e, "p after six steps")


@pytest.mark.parametrize("bits", [8, 32])
def test_infinities_nan_and_zero_gradients(bits):
    n = 384
    g = torch.randn(n, generator=torch.Generator().manual_seed(1))
    bad = [5, 130]
    g[5], g[130] = float("nan"), float("inf")
    g[256:] = 0.0
    p0 = torch.randn(n, generator=torch.Generator().manual_seed(2))
    p, q = p0.to(dev()), p0.to(dev())
    clean = g.clone()
    clean[bad] = 0.0
    note("adamw %d bits inf/nan" % bits)
    a, b = xt.AdamW([p], state_bits=bits, **HYPER), xt.AdamW([q], state_bits=bits, **HYPER)
    for _ in range(2):
        a.step([g.to(dev())])
        b.step([clean.to(dev())])
    torch.cuda.synchronize()
    keep = torch.ones(n, dtype=torch.bool)
    keep[bad] = False
    assert torch.isnan(p.cpu()[bad]).all() and torch.equal(p.cpu()[keep], q.cpu()[keep])
    # no gradient: decay alone
    want = p0[256:].double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) ** 2
    assert ((p.cpu()[256:].double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("eps", [0.0, 1e-15, 1e-8])
def test_small_eps(eps):
    g = torch.tensor([1e-25, 1e-21, -1e-15, 1e-3, 2.0])
    p = torch.zeros(5)
    note("adamw eps %g" % eps)
    P = p.to(dev())
    opt = xt.AdamW([P], lr=1e-2, betas=(0.9, 0.99), eps=eps, weight_decay=0.0)
    opt.step([g.to(dev())])
    got = P.cpu().double().numpy()
    gd = g.double().numpy()
    # fp32 squares below 2^-149 vanish: the first two elements have v = 0 (or a few subnormal steps)
    want = -1e-2 * gd / (np.abs(gd) + eps)
    assert np.allclose(got[2:], want[2:], rtol=1e-5, atol=0)
    assert eps == 0.0 or np.isfinite(got).all()


def test_graph_and_stream():
    sizes = [1000, 33]
    ps, gs, _, _ = make(sizes, "bf16", 9)
    P, Q, G = [[x.to(dev()) for x in xs] for xs in (ps, ps, gs)]
    a, b = xt.AdamW(P, state_bits=8, seed=1, **HYPER), xt.AdamW(Q, state_bits=8, seed=1, **HYPER)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    note("adamw stream and graph")
    a.step(G, stream=s)
    s.synchronize()
    b.step(G)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(P, Q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(G)  # captured as step 2: every replay takes step 2's rates and random bits
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        b.steps = 1
        b.step(G)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(P + list(a.state[0]), Q + list(b.state[0])))


def test_refusals():
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device=dev())  # noqa: E731
    with pytest.raises(ValueError):
        xt.AdamW([torch.zeros(4)])
    with pytest.raises(ValueError):
        xt.AdamW([f(4).half()])
    with pytest.raises(ValueError):
        xt.AdamW([f((4, 4)).t()[:, :2]])
    for kw in ({"state_bits": 16}, {"copies": [f(4)]}, {"copies": [f(5).half()]}, {"state": ([f(4)],)}, {"steps": -1},
               {"state": ([f(4)], [f(3)])}, {"state_bits": 8, "state": ([f(4)], [f(4)], [f(1)], [f(1)])}):
        with pytest.raises(ValueError):
            xt.AdamW([f(4)], **kw)
    p = f(8)
    with pytest.raises(xt.XtvxyError):  # overlapping parameters
        xt.AdamW([p, p[4:]])
    opt = xt.AdamW([f(8), f(3)])
    for grads in ([f(8)], [f(8), f(4)], [f(8), f(3).half()], [f(8), f(6)[::2]], [f(8), torch.zeros(3)], [f(8).double()] * 2):
        with pytest.raises(ValueError):
            opt.step(grads)
    with pytest.raises(xt.XtvxyError):  # a gradient inside what the step writes
        opt.step([opt.params[0], f(3)])
    for name, value in (("lr", -1.0), ("lr", float("nan")), ("eps", -1e-8), ("betas", (1.0, 0.9)), ("weight_decay", -0.1)):
        bad = xt.AdamW([f(8), f(3)])
        setattr(bad, name, value)
        with pytest.raises(xt.XtvxyError):
            bad.step([f(8), f(3)])
        assert bad.steps == 0
    xt.AdamW([]).step([])
