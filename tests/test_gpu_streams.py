"""Tensors that a helper makes for a call on another stream come from that stream's memory: a block just given
back on the current stream may still be read there."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
from gpu_util import dev, note

pytestmark = pytest.mark.gpu

M, N = 4096, 2048


def given_back(*bytes_):
    """Addresses of blocks of the current stream that are free again: the next tensors of these sizes there."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.empty(b, dtype=torch.uint8, device=dev()) for b in bytes_]
    return [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]


def apart(blocks, *made):
    for t in made:
        assert all(t.data_ptr() >= end or t.data_ptr() + t.numel() * t.element_size() <= begin for begin, end in blocks)


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev())


def test_layer():
    X, W, G = normal((M, N), 1, torch.bfloat16), normal((N, N), 2, torch.bfloat16), normal((M, N), 3, torch.bfloat16)
    s = torch.cuda.Stream()
    sizes = (M * N * 2, M * N * 2, N * N * 2, 1 << 20, 4 * N)
    blocks = given_back(*sizes)
    note("layer on another stream")
    out, pre = xt.linear(X, W, act="silu", save_pre=True, stream=s)
    apart(blocks, out, pre)
    grads = xt.linear_backward(G, X, W, pre, "silu", stream=s)
    apart(blocks, *grads)
    s.synchronize()
    want = xt.linear(X, W, act="silu", save_pre=True)
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, xt.linear_backward(G, X, W, pre, "silu")))


def test_results_are_kept_for_the_current_stream():
    """A result dropped while the current stream still reads it is not overwritten by the next call."""
    X, W = normal((M, N), 1, torch.bfloat16), normal((N, N), 2, torch.bfloat16)
    others = [normal((M, N), seed, torch.bfloat16) for seed in (5, 6, 7)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    note("result dropped by the current stream")
    out = xt.linear(X, W, stream=s)
    s.synchronize()
    first = out.clone()
    torch.cuda._sleep(50_000_000)  # the current stream is busy for a while
    copy = out.clone()  # and reads the result after that
    del out
    for x in others:
        xt.linear(x, W, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(copy, first)


def test_pattern():
    X, y, v = normal((M, N), 1), normal(N, 2), normal(M, 3)
    s = torch.cuda.Stream()
    blocks = given_back(4 * N, 16 << 20, 4 * M, 4 * M * N)
    note("pattern on another stream")
    out = xt.dense(X, y, v, stream=s)
    apart(blocks, out, xt.dense_transpose(X, stream=s))
    s.synchronize()
    assert torch.equal(out, xt.dense(X, y, v))
    A = torch.relu(X[:, :256] - 1.5).to_sparse_csr()
    rp, ci, vals = A.crow_indices().int(), A.col_indices().int(), A.values()
    y = normal(256, 5)
    blocks = given_back(4 * 256, 16 << 20, 4 * M)
    note("CSR on another stream")
    t = xt.csr_rowdot(rp, ci, vals, 256, y, stream=s)
    u = xt.csr_tmv(rp, ci, vals, 256, v, stream=s)
    whole = xt.csr(rp, ci, vals, 256, y, v, stream=s)
    analysed = xt.CsrAnalysis(rp, ci, 256, stream=s)(vals, y, v, stream=s)
    apart(blocks, t, u, whole, analysed)
    s.synchronize()
    ref = A.double().cpu().to_dense()
    z = ref @ y.double().cpu()
    for got, want in ((t, z), (u, ref.T @ v.double().cpu()), (whole, ref.T @ (v.double().cpu() * z)),
                      (analysed, ref.T @ (v.double().cpu() * z))):
        assert (got.double().cpu() - want).norm() <= 1e-5 * want.norm()


def test_check_on_another_stream_behind_a_busy_one():
    """The flag is cleared on the stream that sets it: a busy current stream does not clear it afterwards."""
    rp = torch.tensor([0, 1], dtype=torch.int32, device=dev())
    ci = torch.tensor([9], dtype=torch.int32, device=dev())  # of 4 columns
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    note("structure check on another stream")
    want = xt.csr_check(rp, ci, 4)
    assert want != 0
    torch.cuda._sleep(50_000_000)
    assert xt.csr_check(rp, ci, 4, stream=s) == want


def test_fresh_optimiser_states_behind_a_busy_stream():
    """Fresh states are zero when the object is there, whatever stream its first step runs on."""
    n = 4096
    g, p = normal(n, 1), normal(n, 2)
    made, used = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    note("fresh states on another stream")
    with torch.cuda.stream(made):
        torch.cuda._sleep(50_000_000)
        opt = xt.AdamW([p], betas=(0.9, 0.99))
    opt.step([g], stream=used)
    torch.cuda.synchronize()
    assert torch.equal(opt.state[0][0], g * torch.tensor(1 - 0.9, device=dev()))
    assert (opt.state[1][0] > 0).all()


def test_calls_on_a_side_stream_of_a_captured_graph():
    X, W, G = normal((300, 520), 1, torch.bfloat16), normal((264, 520), 2, torch.bfloat16), normal((300, 264), 3, torch.bfloat16)
    y, v = normal(520, 4), normal(300, 5)
    side = torch.cuda.Stream()

    def step(stream):
        out, pre = xt.linear(X, W, act="silu", save_pre=True, stream=stream)
        return (out, pre) + xt.linear_backward(G, X, W, pre, "silu", stream=stream) + (xt.dense(X, y, v, stream=stream),)

    note("side stream of a captured graph")
    step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        held = step(side)
        here.wait_stream(side)
    for seed in (10, 20, 30):
        for i, t in enumerate((X, W, G)):
            t.copy_(normal(t.shape, seed + i, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
